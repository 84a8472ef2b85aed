"""A query's result over an e4m3 cache does not depend, to the bit, on the tokens of
its chunk behind it."""
import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE
from tests.test_gpu_e4m3 import Cache, check_chunk, chunk_queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


@pytest.mark.parametrize("hq", [2, 6, 16])
@pytest.mark.parametrize("at", [1, 20, 43, 44, 50, 75, 76, 89])
@pytest.mark.parametrize("scale", [1e4, 1e30])
def test_large_scales_of_later_tokens(dev, hq, at, scale):
    """Keys and values behind position q_start + at get large finite scales and other codes."""
    n, q_start = 90, 64 * 6 + 20  # blocks end after tokens 43 and 107
    c = Cache(dev, [q_start + n], hq, 2, "contiguous", seed=71, spread=2.0)
    q, ws = chunk_queries(c, n, 7), c.workspace()

    def run():
        out, lse = torch.full_like(q, float("nan")), torch.full((n, hq), float("nan"), device=dev)
        msa.msa_dense_gqa_prefill(q, hq, n, q_start, c.desc, SCALE, out, lse, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
        return out, lse
    o0, l0 = run()
    check_chunk(c, 0, q, q_start, o0, l0)
    later = slice(q_start + at, None)
    c.t["k_scale"][..., later] *= scale
    c.t["v_scale"][..., later] *= scale
    c.t["v"].view(torch.uint8)[..., later, :] = 0x7e
    o1, l1 = run()
    assert torch.equal(o0[:at], o1[:at]) and torch.equal(l0[:at], l1[:at])
