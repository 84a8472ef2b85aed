"""Rows of a bf16 cache that lie past a sequence's end in its last block, whatever an
earlier owner of the page left there, do nothing to any result."""
import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf"), 3e38]


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def caches(dev, lens, hkv, layout, seed):
    """Two caches with the same tokens: zeros past the ends, and NaN, infinities and large values there."""
    g = torch.Generator(device=dev).manual_seed(seed)
    b, per = len(lens), [-(-n // 64) for n in lens]
    width = max(max(per), 1)
    if layout == "paged":
        table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
        perm, at = torch.randperm(max(1, sum(per)), generator=g, device=dev).int(), 0
        for s, p in enumerate(per):
            table[s, :p] = perm[at:at + p]
            at += p
        shape = (max(1, sum(per)), hkv, 64, 128)
    else:
        table, shape = None, (b, hkv, width * 64, 128)
    clean = [torch.randn(shape, generator=g, device=dev).bfloat16() for _ in range(2)]
    stale = [x.clone() for x in clean]
    for s, n in enumerate(lens):
        for tok in range(n, per[s] * 64):
            at = (int(table[s, tok // 64]), slice(None), tok % 64) if layout == "paged" else (s, slice(None), tok)
            for x, y in zip(clean, stale):
                x[at] = 0.0
                y[at] = torch.tensor(BAD, device=dev).repeat(32).roll(tok).bfloat16()
    seq = torch.tensor(lens, dtype=torch.int32, device=dev)
    return [(msa.kv_desc(k, v, seq, table), (k, v, seq, table)) for k, v in (clean, stale)]


def same(runs):
    torch.cuda.synchronize()
    first = runs[0]
    for r in runs[1:]:
        for x, y in zip(first, r):
            assert not y.isnan().any()
            assert torch.equal(x, y)


LENS = [1, 17, 63, 64, 65, 64 * 9 + 16, 64 * 9 + 31, 64 * 9 + 33, 64 * 40 + 48, 0]


@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (6, 2), (16, 2)])
def test_decode_and_step(dev, layout, hq, hkv):
    k_scored = 5
    dense, listed, step = [], [], []
    idx0 = None
    for desc, keep in caches(dev, LENS, hkv, layout, 1):
        q = torch.randn(len(LENS), hq, 128, generator=torch.Generator(device=dev).manual_seed(2), device=dev).bfloat16()
        ops = (msa.MSA_OP_SELECT, msa.MSA_OP_DECODE, msa.MSA_OP_DENSE_DECODE, msa.MSA_OP_DECODE_STEP, msa.MSA_OP_POOL)
        ws = msa.Workspace(max(msa.msa_workspace_size(op, desc, hq, 1, k_scored + 1) for op in ops), dev)
        pooled = torch.zeros(msa.pooled_shape(desc), dtype=torch.bfloat16, device=dev)
        msa.msa_pool_block_keys(desc, 0, -1, pooled, ws.buf, ws.nbytes)

        def outputs():
            return torch.zeros_like(q), torch.zeros(q.shape[:2], device=dev)
        out, lse = outputs()
        msa.msa_dense_gqa_decode(q, hq, desc, SCALE, out, lse, ws.buf, ws.nbytes)
        dense.append((out, lse))
        idx = torch.full((len(LENS), hkv, k_scored + 1), -7, dtype=torch.int32, device=dev)
        out, lse = outputs()
        msa.msa_sparse_decode_step(q, hq, pooled, desc, msa.select_cfg(k_scored), idx, k_scored + 1, SCALE, out, lse,
                                   ws.buf, ws.nbytes)
        step.append((out, lse, idx))
        idx0 = idx if idx0 is None else idx0
        out, lse = outputs()
        msa.msa_sparse_attn_decode(q, hq, desc, idx0, k_scored + 1, SCALE, out, lse, ws.buf, ws.nbytes)
        noalloc = outputs()
        msa.msa_sparse_attn_decode_noalloc(q, hq, desc, idx0, k_scored + 1, SCALE, *noalloc)
        listed.append((out, lse, *noalloc))
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
    same(dense)
    same(step)
    same(listed)


@pytest.mark.parametrize("layout", ["paged", "contiguous"])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (5, 1), (16, 2), (8, 2)])
@pytest.mark.parametrize("starts,counts", [([0], [1]), ([0], [63]), ([64 * 3 + 5], [70]), ([64 * 2], [64]),
                                           ([64 * 7 + 60, 0, 64 * 4, 9], [5, 130, 1, 0])])
def test_prefill(dev, layout, hq, hkv, starts, counts):
    """Chunks of several sequences, through lists in which the diagonal block comes first, last or in a pair's middle."""
    lens = [a + n for a, n in zip(starts, counts)]
    tiles = msa.varlen_tiles(counts, starts)
    diag = [d for a, n in zip(starts, counts) if n for d in range(a // 64, (a + n - 1) // 64 + 1)]
    lists = []
    for order in range(3):
        idx = torch.full((tiles, hkv, 4), -1, dtype=torch.int32, device=dev)
        for i, d in enumerate(diag):
            others = [x for x in (0, d - 1, d - 2) if 0 <= x < d]
            others = sorted(set(others))
            at = min(order, len(others))
            row = others[:at] + [d] + others[at:]
            idx[i, :, :len(row)] = torch.tensor(row, dtype=torch.int32, device=dev)
        lists.append(idx)
    runs = [[] for _ in range(4)]
    for desc, keep in caches(dev, lens, hkv, layout, 3):
        q = torch.randn(sum(counts), hq, 128, generator=torch.Generator(device=dev).manual_seed(4),
                        device=dev).bfloat16()
        ws = msa.Workspace(1 << 16, dev)
        for r, idx in zip(runs, lists):
            out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=dev)
            msa.msa_sparse_attn_prefill_varlen(q, hq, starts, counts, desc, idx, 4, SCALE, out, lse, ws.buf, ws.nbytes)
            r.append((out, lse))
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=dev)
        if len(counts) == 1:
            msa.msa_dense_gqa_prefill(q, hq, counts[0], starts[0], desc, SCALE, out, lse, ws.buf, ws.nbytes)
        runs[3].append((out, lse))
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
    for r in runs:
        same(r)


def test_a_page_of_a_finished_request_reaches_nobody(dev):
    """A request overflows to NaN and ends; its pages go to another one, whose results are those of a fresh cache."""
    hq, hkv, pages = 16, 2, 8
    inv = (10000.0 ** -(torch.arange(64, device=dev) / 64)).float()
    cfg = msa.norm_rope_cfg(128)
    results = []
    for spoil in (False, True):
        k, v = (torch.zeros(pages, hkv, 64, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
        lens = torch.zeros(1, dtype=torch.int32, device=dev)
        table = torch.full((1, pages), -1, dtype=torch.int32, device=dev)
        free = torch.arange(pages, dtype=torch.int32, device=dev)
        left = torch.tensor([pages], dtype=torch.int32, device=dev)
        desc = msa.kv_desc(k, v, lens, table)
        ops = (msa.MSA_OP_EXTEND, msa.MSA_OP_TRIM, msa.MSA_OP_APPEND, msa.MSA_OP_DENSE_DECODE)
        ws = msa.Workspace(max(msa.msa_workspace_size(op, desc, hq, 1, 1) for op in ops), dev)

        def append(n, x):
            pos = torch.empty(n, dtype=torch.int32, device=dev)
            slots = torch.empty(n, dtype=torch.int64, device=dev)
            q_off = torch.empty(2, dtype=torch.int32, device=dev)
            cnt = torch.tensor([n], dtype=torch.int32, device=dev)
            msa.msa_extend_sequences(desc, cnt, free, left, n, table, lens, left, q_off, pos, slots, ws.buf, ws.nbytes)
            q = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device=dev)
            msa.msa_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], hq, n, None, None, pos, inv,
                                        slots, desc, cfg, q, ws.buf, ws.nbytes)
            return q
        if spoil:
            append(64 * pages, torch.full((64 * pages, hq + 2 * hkv, 128), float("nan"), device=dev).bfloat16())
            msa.msa_trim_sequences(desc, torch.zeros(1, dtype=torch.int32, device=dev), free, left, lens, left, ws.buf,
                                   ws.nbytes)
        x = torch.randn(200, hq + 2 * hkv, 128, generator=torch.Generator(device=dev).manual_seed(5),
                        device=dev).bfloat16()
        q = append(200, x)
        out, lse = torch.zeros(1, hq, 128, dtype=torch.bfloat16, device=dev), torch.zeros(1, hq, device=dev)
        msa.msa_dense_gqa_decode(q[-1:], hq, desc, SCALE, out, lse, ws.buf, ws.nbytes)
        chunk = torch.zeros_like(q), torch.zeros(200, hq, device=dev)
        msa.msa_dense_gqa_prefill(q, hq, 200, 0, desc, SCALE, *chunk, ws.buf, ws.nbytes)
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws.buf) == 0
        results.append((out, lse, *chunk))
    same(results)
