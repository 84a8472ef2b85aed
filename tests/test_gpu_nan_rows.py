"""A row whose scores hold a NaN is NaN in the output and in the log-sum-exp: -inf
marks a row that attends to nothing, and only that."""
import pytest
import torch

from sparse_attention_step_gb300 import msa
from tests.parity import SCALE

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "f32", "e4m3"]


@pytest.fixture(scope="module")
def dev(lib):
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def make(dev, dtype, lens, hq, hkv, seed, max_pages=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    b, per = len(lens), [-(-n // 64) for n in lens]
    width = max_pages or max(max(per), 1)
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    perm, at = torch.randperm(max(1, sum(per)), generator=g, device=dev).int(), 0
    for s, p in enumerate(per):
        table[s, :p] = perm[at:at + p]
        at += p
    shape = (max(1, sum(per)), hkv, 64, 128)
    k, v = (torch.randn(shape, generator=g, device=dev) for _ in range(2))
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    cache = torch.float8_e4m3fn if dtype == "e4m3" else io
    k, v = k.to(cache), v.to(cache)
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = (torch.rand(shape[:3], generator=g, device=dev) + 0.5 for _ in range(2))
    seq = torch.tensor(lens, dtype=torch.int32, device=dev)
    desc = msa.kv_desc(k, v, seq, table, k_scale=ks, v_scale=vs)
    q = torch.randn(b, hq, 128, generator=g, device=dev).to(io)
    return desc, q, (k, v, ks, vs, seq, table)


def outputs(q):
    return torch.zeros_like(q), torch.zeros(q.shape[:2], device=q.device)


def expect(out, lse, nan_rows, empty_rows):
    """nan_rows, empty_rows: [rows, heads] truth values."""
    torch.cuda.synchronize()
    assert torch.equal(out.isnan().all(-1), nan_rows) and torch.equal(out.isnan().any(-1), nan_rows)
    assert torch.equal(lse.isnan(), nan_rows), "lse of the rows that are NaN"
    assert torch.equal(lse == float("-inf"), empty_rows)
    assert bool((out[empty_rows] == 0).all())


def workspace(desc, hq, k_total, dev):
    ops = (msa.MSA_OP_SELECT, msa.MSA_OP_DECODE, msa.MSA_OP_DENSE_DECODE, msa.MSA_OP_DECODE_STEP, msa.MSA_OP_POOL)
    return msa.Workspace(max(msa.msa_workspace_size(op, desc, hq, 1, k_total) for op in ops), dev)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("where", ["query", "key"])
@pytest.mark.parametrize("lens,max_pages", [([64 * 30 + 5, 0, 70], None), ([3, 64, 0], None), ([700, 0, 90], 16384)])
def test_decode(dev, dtype, where, lens, max_pages):
    hq, hkv, k_total = 8, 2, 4
    desc, q, keep = make(dev, dtype, lens, hq, hkv, 3, max_pages)
    nan = torch.zeros(len(lens), hq, dtype=torch.bool, device=dev)
    empty = (keep[4] == 0)[:, None].expand(-1, hq)
    if where == "query":  # every score of one head
        q[0, 5, 77] = float("nan")
        nan[0, 5] = True
    else:  # one token of the last block, under the heads of one group
        page, row = int(keep[5][0, (lens[0] - 1) // 64]), (lens[0] - 1) % 64
        if dtype == "e4m3":
            keep[2][page, 1, row] = float("nan")
        else:
            keep[0][page, 1, row, 9] = float("nan")
        nan[0, 4:] = True
    ws = workspace(desc, hq, k_total, dev)
    out, lse = outputs(q)
    msa.msa_dense_gqa_decode(q, hq, desc, SCALE, out, lse, ws.buf, ws.nbytes)
    expect(out, lse, nan, empty)
    idx = torch.full((len(lens), hkv, k_total), -1, dtype=torch.int32, device=dev)
    for s, n in enumerate(lens):
        if n:
            idx[s, :, 2] = (n - 1) // 64
            if n > 64:
                idx[s, :, 0] = 0
    out, lse = outputs(q)
    msa.msa_sparse_attn_decode(q, hq, desc, idx, k_total, SCALE, out, lse, ws.buf, ws.nbytes)
    expect(out, lse, nan, empty)
    assert msa.msa_read_device_status(ws.buf) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,k_scored", [([64 * 30 + 5, 0, 70], 3), ([64 * 200 + 1, 0, 70], 40)])
def test_step(dev, dtype, lens, k_scored):
    """The newest block, always attended, holds a key of NaN."""
    hq, hkv = 8, 2
    desc, q, keep = make(dev, dtype, lens, hq, hkv, 4)
    page, row = int(keep[5][0, (lens[0] - 1) // 64]), (lens[0] - 1) % 64
    if dtype == "e4m3":
        keep[2][page, 1, row] = float("nan")
    else:
        keep[0][page, 1, row, 9] = float("nan")
    nan = torch.zeros(len(lens), hq, dtype=torch.bool, device=dev)
    nan[0, 4:] = True
    pooled = torch.zeros(msa.pooled_shape(desc), dtype=q.dtype, device=dev)
    ws = workspace(desc, hq, k_scored + 1, dev)
    msa.msa_pool_block_keys(desc, 0, -1, pooled, ws.buf, ws.nbytes)
    idx = torch.full((len(lens), hkv, k_scored + 1), -7, dtype=torch.int32, device=dev)
    out, lse = outputs(q)
    msa.msa_sparse_decode_step(q, hq, pooled, desc, msa.select_cfg(k_scored), idx, k_scored + 1, SCALE, out, lse,
                               ws.buf, ws.nbytes)
    expect(out, lse, nan, (keep[4] == 0)[:, None].expand(-1, hq))
    assert msa.msa_read_device_status(ws.buf) == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [8, 16])
def test_prefill(dev, dtype, hq):
    hkv, n, q_start = 2, 40, 64 * 5 + 3
    desc, _, keep = make(dev, dtype, [q_start + n], hq, hkv, 5)
    q = torch.randn(n, hq, 128, generator=torch.Generator(device=dev).manual_seed(6), device=dev).bfloat16()
    nan = torch.zeros(n, hq, dtype=torch.bool, device=dev)
    empty = torch.zeros_like(nan)
    ws = msa.Workspace(1 << 16, dev)
    q[7, 2, 100] = float("nan")
    nan[7, 2] = True
    out, lse = outputs(q)
    msa.msa_dense_gqa_prefill(q, hq, n, q_start, desc, SCALE, out, lse, ws.buf, ws.nbytes)
    expect(out, lse, nan, empty)
    idx = torch.full((1, hkv, 2), -1, dtype=torch.int32, device=dev)
    idx[:, 0, 1] = 5  # the second head's list is empty
    nan[:, hq // 2:], empty[:, hq // 2:] = False, True
    out, lse = outputs(q)
    msa.msa_sparse_attn_prefill(q, hq, n, q_start, desc, idx, 2, SCALE, out, lse, ws.buf, ws.nbytes)
    expect(out, lse, nan, empty)
    assert msa.msa_read_device_status(ws.buf) == 0
