"""Prefill over an e4m3 cache with V scales of any power of two: up to 2^80 the outputs
are those of a scale of 1, times the power; above, where the sum of a row's weights
would lose its small terms, the device status says so.

Tolerances. With every V scale 2^e a row's reference moves with e, so that weights and their sum are
the same numbers at another exponent; the reference is rounded to fp32 (2^-17 for values below 128),
which moves a weight and the sum alike, and so their ratio only by the exponentials' 2^-21 and the
weights' roundings, 2^-10: below 2^-9 of the largest value together. Then one bf16 rounding each, 2^-8."""
import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


@pytest.mark.parametrize("hq", [2, 8])
@pytest.mark.parametrize("e", [-60, -20, 40, 80, 100, 112, 119])
def test_power_of_two_scales(dev, hq, e):
    n, t = 70, 64 * 9 + 30
    g = torch.Generator(device=dev).manual_seed(5)
    k = torch.randn(1, 1, 640, 128, generator=g, device=dev).to(torch.float8_e4m3fn)
    v = torch.randn(1, 1, 640, 128, generator=g, device=dev).to(torch.float8_e4m3fn)
    ks = torch.rand(1, 1, 640, generator=g, device=dev) * 3
    q = torch.randn(n, hq, 128, generator=g, device=dev).bfloat16()
    lens = torch.tensor([t], dtype=torch.int32, device=dev)
    got = []
    for p in (0, e):
        vs = torch.full((1, 1, 640), 2.0 ** p, device=dev)
        desc = msa.kv_desc(k, v, lens, k_scale=ks, v_scale=vs)
        ws = msa.Workspace(1 << 16, dev)
        out, lse = torch.full_like(q, float("nan")), torch.full((n, hq), float("nan"), device=dev)
        msa.msa_dense_gqa_prefill(q, hq, n, t - n, desc, SCALE, out, lse, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        got.append((out.double() * 2.0 ** -p, lse.double(), msa.msa_read_device_status(ws.buf)))
    assert got[0][2] == 0
    if e > 80:
        assert got[1][2] == msa.MSA_ERR_UNSUPPORTED
        return
    assert got[1][2] == 0
    (o0, l0, _), (o1, l1, _) = got
    tol = 2.0 ** -7 * o0.abs() + 2.0 ** -9 * v.float().abs().max()
    assert bool(((o1 - o0).abs() <= tol).all())
    assert bool(((l1 - l0).abs() <= 2.0 ** -15).all())


def test_one_large_scale_among_small_ones(dev):
    """Reported where the row sees it, not where it lies behind the query."""
    t, hq = 300, 4
    g = torch.Generator(device=dev).manual_seed(6)
    k = torch.randn(1, 1, 320, 128, generator=g, device=dev).to(torch.float8_e4m3fn)
    v = k.clone()
    ks, vs = torch.ones(1, 1, 320, device=dev), torch.ones(1, 1, 320, device=dev)
    q = torch.randn(t, hq, 128, generator=g, device=dev).bfloat16()
    lens = torch.tensor([t], dtype=torch.int32, device=dev)
    vs[0, 0, 290] = 2.0 ** 110
    desc = msa.kv_desc(k, v, lens, k_scale=ks, v_scale=vs)
    for n, want in ((290, 0), (291, msa.MSA_ERR_UNSUPPORTED)):
        ws = msa.Workspace(1 << 16, dev)
        out, lse = torch.full_like(q[:n], float("nan")), torch.full((n, hq), float("nan"), device=dev)
        msa.msa_dense_gqa_prefill(q[:n].contiguous(), hq, n, 0, desc, SCALE, out, lse, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == want
        assert not out[:min(n, 290)].isnan().any()
