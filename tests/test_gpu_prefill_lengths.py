"""A chunk's queries see every token up to their own position, whether the sequence
lengths were raised before the chunk's attention or are raised after it: the
same bits for every cache type and group size."""
import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def cache(dev, dtype, layout, b, hkv, cap, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    shape = (b * cap // 64, hkv, 64, 128) if layout == "paged" else (b, hkv, cap, 128)
    t = {n: torch.randn(shape, generator=g, device=dev).bfloat16() for n in "kv"}
    if dtype == "e4m3":
        t = {n: x.to(torch.float8_e4m3fn) for n, x in t.items()}
        for n in "kv":
            t[n + "_scale"] = torch.rand(shape[:3], generator=g, device=dev) + 0.25
    table = torch.randperm(b * cap // 64, generator=g, device=dev).int().view(b, -1) if layout == "paged" else None
    return t, table


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 16, 2), ("bf16", 6, 2), ("e4m3", 16, 2), ("e4m3", 6, 2)])
@pytest.mark.parametrize("layout", ["paged", "contiguous"])
def test_lengths_raised_before_or_after_the_chunk(dev, dtype, layout, hq, hkv):
    starts, counts = [64 * 5 + 17, 0, 64 * 3], [64 + 30, 100, 64]
    b, cap = 3, 64 * 8
    t, table = cache(dev, dtype, layout, b, hkv, cap, 1)
    q = torch.randn(sum(counts), hq, 128, generator=torch.Generator(device=dev).manual_seed(2), device=dev).bfloat16()
    after = torch.tensor([a + n for a, n in zip(starts, counts)], dtype=torch.int32, device=dev)
    before = torch.tensor(starts, dtype=torch.int32, device=dev)
    tiles = msa.varlen_tiles(counts, starts)
    idx = torch.full((tiles, hkv, 3), -1, dtype=torch.int32, device=dev)
    i = 0
    for a, n in zip(starts, counts):
        for d in range(a // 64, (a + n - 1) // 64 + 1):  # the diagonal block, the first one and the one before
            idx[i, :, 0] = d
            if d > 0:
                idx[i, :, 1] = 0
            if d > 1:
                idx[i, :, 2] = d - 1
            i += 1
    ws = msa.Workspace(1 << 16, dev)
    got = []
    for lens in (after, before, torch.zeros_like(before)):
        d = msa.kv_desc(t["k"], t["v"], lens, table, k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=dev)
        msa.msa_sparse_attn_prefill_varlen(q, hq, starts, counts, d, idx, 3, SCALE, out, lse, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
        got.append((out, lse))
    assert not got[0][0].isnan().any() and bool(got[0][1].isfinite().all())
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("dtype,hq", [("bf16", 8), ("bf16", 4), ("e4m3", 8), ("e4m3", 4)])
def test_dense_chunk_before_its_length_is_raised(dev, dtype, hq):
    t, _ = cache(dev, dtype, "contiguous", 1, 1, 64 * 4, 3)
    q = torch.randn(70, hq, 128, generator=torch.Generator(device=dev).manual_seed(4), device=dev).bfloat16()
    ws = msa.Workspace(1 << 16, dev)
    got = []
    for n in (64 * 2 + 10 + 70, 64 * 2 + 10):
        lens = torch.tensor([n], dtype=torch.int32, device=dev)
        d = msa.kv_desc(t["k"], t["v"], lens, k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=dev)
        msa.msa_dense_gqa_prefill(q, hq, 70, 64 * 2 + 10, d, SCALE, out, lse, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
        got.append((out, lse))
    assert not got[0][0].isnan().any()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
