"""The rotation's angles at any position for any finite inv_freq, against exact
rational arithmetic.

With x = (1, 0) in every pair the outputs are the cosine and the sine. The angle's
fraction of a turn is off by at most 2^-24 half turns (pi 2^-24 rad, 1.9e-7) and
sincospif by 2 ulp (1.2e-7): below 3.2e-7 < 2^-21."""
from fractions import Fraction

import math

import numpy as np
import pytest
import torch

from sparse_attention_step_gb300 import msa

pytestmark = pytest.mark.gpu

FREQS = [0.0, 1e-45, 1e-30, 1e-18, 2.0 ** -55, 1.7e-13, 2.0 ** -41, 1e-9, 1e-4, 0.99999994, 1.0, 1.0000001, 3.7, 31.99, 32.5,
         100.0, 1000.0, 12345.678, 1e6, 16777216.0, 1e9, 2.0 ** 40, 1e15, 2.0 ** 63, 1e19, 2.0 ** 64, 1e20, 1e25, 1e30,
         1e36, 2.0 ** 127, 3.4028235e38]
POSITIONS = [0, 1, 2, 3, 1000, 65537, 2 ** 20 + 1, 2 ** 24 + 1, 999999937, 2 ** 31 - 1, -1, -(2 ** 31)]


def pi_bits(n):
    """floor(pi 2^n) (Machin's formula)."""
    one = 1 << (n + 32)

    def arctan(x):
        total = term = one // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    return (4 * (4 * arctan(5) - arctan(239))) >> 32


PI = Fraction(pi_bits(400), 1 << 400)


def angle(pos, f):
    """pos f in radians modulo one turn, in (-pi, pi]."""
    x = pos * Fraction(f) / (2 * PI)
    x -= math.floor(x + Fraction(1, 2))
    return float(x * 2 * PI)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_at_any_frequency(lib, inter, sign):
    dev = torch.device("cuda:0")
    freq = np.array([sign * f for f in FREQS], dtype=np.float32)
    half = len(freq)
    assert half == 32
    x = torch.zeros(len(POSITIONS), 1, 128)
    a, b = (2 * np.arange(half), 2 * np.arange(half) + 1) if inter else (np.arange(half), np.arange(half) + half)
    x[..., a] = 1.0
    q = x.to(dev)
    cache = torch.zeros(1, 1, 64, 128, device=dev)
    lens, table = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(1, 1, dtype=torch.int32, device=dev)
    desc = msa.kv_desc(cache, cache.clone(), lens, table)
    ws = msa.Workspace(msa.msa_workspace_size(msa.MSA_OP_APPEND, desc, 1, len(POSITIONS), 1), dev)
    cfg = msa.norm_rope_cfg(2 * half, inter, 1e-6, False, False)
    out = torch.full_like(q, float("nan"))
    pos, inv = torch.tensor(POSITIONS, dtype=torch.int32, device=dev), torch.from_numpy(freq).to(dev)
    msa.msa_qk_norm_rope_append(q, None, None, 1, len(POSITIONS), None, None, pos, inv, None, desc, cfg, out, ws.buf,
                                ws.nbytes)
    torch.cuda.synchronize()
    assert msa.msa_read_device_status(ws.buf) == 0
    got = out[:, 0].double().cpu().numpy()
    bad = []
    for i, p in enumerate(POSITIONS):
        for j, f in enumerate(freq):
            t = angle(p, float(f))
            d = max(abs(got[i, a[j]] - math.cos(t)), abs(got[i, b[j]] - math.sin(t)))
            if not d <= 2.0 ** -21:
                bad.append((p, float(f), d))
    assert not bad, bad
    assert bool((out[:, 0, 2 * half:] == 0).all())
