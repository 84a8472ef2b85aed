"""List lengths: up to 2^30 entries everywhere, longer ones are refused on the host (a
kernel's walk over a list counts in 32 bits)."""
import ctypes

import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

MOST = 1 << 30
P, WS = 0x1000, 1 << 40


def desc(dtype):
    d = msa.KvDesc()
    d.layout, d.dtype, d.batch, d.num_kv_heads, d.head_dim, d.block_size = msa.MSA_KV_PAGED, dtype, 1, 1, 128, 64
    d.k = d.v = d.seq_lens = d.page_table = d.k_scale = d.v_scale = P
    d.max_pages_per_seq, d.num_pages = 16, 16
    return ctypes.byref(d)


def calls(lib, dtype, k):
    d, one = desc(dtype), msa.select_cfg(4)
    tile = msa.select_cfg(4, True, 64)
    starts, counts = (ctypes.c_int64 * 1)(0), (ctypes.c_int32 * 1)(5)
    yield lib.msa_sparse_attn_decode(P, 4, d, P, k, SCALE, P, None, P, WS, None)
    yield lib.msa_sparse_attn_decode_noalloc(P, 4, d, P, k, SCALE, P, None, None)
    yield lib.msa_select_topk_blocks(P, 4, 1, P, d, ctypes.byref(one), P, k, None, P, WS, None)
    yield lib.msa_sparse_decode_step(P, 4, P, d, ctypes.byref(one), P, k, SCALE, P, None, P, WS, None)
    yield lib.msa_sparse_decode_step_pool(P, 4, P, d, ctypes.byref(one), P, k, SCALE, P, None, P, WS, None)
    yield lib.msa_select_topk_blocks_varlen(P, 4, 1, starts, counts, P, d, ctypes.byref(tile), P, k, None, P, WS, None)
    if dtype != msa.MSA_DTYPE_F32:
        yield lib.msa_sparse_attn_prefill(P, 4, 5, 0, d, P, k, SCALE, P, None, P, WS, None)
        yield lib.msa_sparse_attn_prefill_varlen(P, 4, 1, starts, counts, d, P, k, SCALE, P, None, P, WS, None)


@pytest.mark.parametrize("dtype", [msa.MSA_DTYPE_F32, msa.MSA_DTYPE_BF16, msa.MSA_DTYPE_E4M3])
@pytest.mark.parametrize("k", [MOST + 1, 2 ** 31 - 32, 2 ** 31 - 1])
def test_longer_lists_are_refused_before_any_launch(lib, dtype, k):
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up: only where nothing can be launched")
    assert all(st == msa.MSA_ERR_UNSUPPORTED for st in calls(lib, dtype, k))


@pytest.mark.gpu
def test_longest_lists_of_two_heads(lib):
    """2^31 - 2 list entries in all, a handful of them blocks: an e4m3 decode deals them all out."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    k, v = (torch.randn(1, 2, 640, 128, generator=g, device=dev).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.rand(1, 2, 640, generator=g, device=dev) + 0.5 for _ in range(2))
    lens = torch.tensor([640], dtype=torch.int32, device=dev)
    desc = msa.kv_desc(k, v, lens, k_scale=ks, v_scale=vs)
    q = torch.randn(1, 8, 128, generator=g, device=dev).bfloat16()
    n = MOST - 1
    idx = torch.full((1, 2, n), -1, dtype=torch.int32, device=dev)
    at = [0, n // 3, n // 2, n - 2, n - 1]
    blocks = [7, 0, 3, 9, 5]
    for a, b in zip(at, blocks):
        idx[0, :, a] = b
    ws = msa.Workspace(msa.msa_workspace_size(msa.MSA_OP_DECODE, desc, 8, 1, n), dev)
    out, lse = torch.full_like(q, float("nan")), torch.full((1, 8), float("nan"), device=dev)
    msa.msa_sparse_attn_decode(q, 8, desc, idx, n, SCALE, out, lse, ws.buf, ws.nbytes)
    short = torch.tensor([[blocks, blocks]], dtype=torch.int32, device=dev)
    o1, l1 = torch.empty_like(q), torch.empty(1, 8, device=dev)
    msa.msa_sparse_attn_decode(q, 8, desc, short, 5, SCALE, o1, l1, ws.buf, ws.nbytes)
    torch.cuda.synchronize()
    assert msa.msa_read_device_status(ws.buf) == 0
    # the same blocks split differently: weights are fp16 and sums fp32 in both, outputs within two bf16 roundings
    # and the weights' 2^-10 of the largest value
    tol = 2.0 ** -7 * o1.float().abs() + 2.0 ** -9 * (v.float() * vs[..., None]).abs().max()
    assert bool(((out.float() - o1.float()).abs() <= tol).all())
    assert bool(((lse - l1).abs() <= 2.0 ** -18 * (1 + l1.abs())).all())
