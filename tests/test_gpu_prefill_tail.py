"""Prefill over an e4m3 cache where one token holds most of a long row and a flat
tail of hundreds of thousands holds the rest, against a restatement in 64 bits.

Tolerances. A weight is fp16: off by half a step, 2^-11 relative, or where it is
subnormal by the amount msa.h states, whose sum over a row is at most 2^-12 of the
largest weight. Scores are exact here (one product of a query); exponentials are
off by 2^-21. So far at most 2^-10 sum_t p_t |v_t| and 2^-12 p_max. O is added to in fp32 by
the tensor core, which aligns the 16 products of a step with the sum so far and cuts
each where the sum ends, 2^-23 of it: a token's product of less than 2^-23 of the sum
may go by unseen in that dim (as over a bf16 cache), so a dim that holds the large value
loses up to n 2^-23 of it, which is no less than the tail here: such dims (the second half)
are only held to that. In a dim where the large value is 0 the j-th of n equal products is off
by at most 2^-23 of the j before it, all together by n / 2 2^-23 of their sum. l is added to
once for every block, off by 2^-24: n 2^-30 of it. Then one rounding to bf16, half a step:
2^-8 relative."""
import math

import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


@pytest.mark.parametrize("hq", [3, 8])
@pytest.mark.parametrize("blocks,below", [(513, 25.1), (2048, 25.1), (2048, 24.6), (2048, 16.5), (16384, 25.1),
                                          (16384, 24.6), (16384, 17.5)])
def test_one_large_weight_over_a_flat_tail(dev, blocks, below, hq):
    """Half of the dims hold the tail alone (the large weight's value is 0 there)."""
    t, n = 64 * blocks, 2
    k = torch.zeros(1, 1, t, 128, dtype=torch.float8_e4m3fn, device=dev)
    k[0, 0, 0, 0] = 448.0
    sign = 1.0 - 2.0 * (torch.arange(128, device=dev) % 2)
    v = sign.expand(1, 1, t, 128).to(torch.float8_e4m3fn).contiguous()
    v[0, 0, 0, :64], v[0, 0, 0, 64:] = 0.0, 1.0
    ks, vs = torch.ones(1, 1, t, device=dev), torch.full((1, 1, t), 0.75, device=dev)
    ks[0, 0, 0] = below * math.log(2) / (SCALE * 8 * 448)
    lens = torch.tensor([t], dtype=torch.int32, device=dev)
    desc = msa.kv_desc(k, v, lens, k_scale=ks, v_scale=vs)
    q = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device=dev)
    q[..., 0] = 8.0
    out, lse = torch.empty_like(q), torch.empty(n, hq, device=dev)
    ws = msa.Workspace(msa.msa_workspace_size(msa.MSA_OP_DENSE_PREFILL, desc, hq, n, 1), dev)
    msa.msa_dense_gqa_prefill(q, hq, n, t - n, desc, SCALE, out, lse, ws.buf, ws.nbytes)
    torch.cuda.synchronize()
    assert msa.msa_read_device_status(ws.buf) == 0
    s0 = SCALE * 8 * 448 * ks[0, 0, 0].double().item()
    first, rest = v[0, 0, 0].double() * 0.75, v[0, 0, 1].double() * 0.75
    for r in range(n):
        tail = (t - n + r) * math.exp(-s0)  # tokens 1 .. position
        total = 1.0 + tail
        want, size = (first + tail * rest) / total, (first.abs() + tail * rest.abs()) / total
        cut = torch.full((128,), t * 2.0 ** -24, device=dev)
        cut[64:] = t * 2.0 ** -23
        slack = (2.0 ** -10 + t * 2.0 ** -30 + cut) * size + 2.0 ** -12 * 0.75 / total
        tol = 2.0 ** -8 * (want.abs() + slack) + slack
        d = (out[r].double() - want).abs()
        assert bool((d <= tol).all()), f"row {r}: worst {(d / tol).max().item():.3f} of the tolerance"
        ref = s0 + math.log(total)
        dl = (lse[r].double() - ref).abs().max().item()
        assert dl <= 2.0 ** -21 * ref + 2.0 ** -21 + t * 2.0 ** -30
