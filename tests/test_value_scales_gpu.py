"""8-bit caches whose value rows have scales of every size: rows of zeros (stored at the smallest scale, 2^-100) and tiny
rows among large ones. Each key counts in the softmax's sum whatever the scale of its value row.

Tolerance: the usual bound (a probability rounded to 16 bits, relatively), and one term more. What is rounded to fp16 is
the probability times its row's value scale, relative to a reference that is one of these products, so the largest is
1 at least, and what is below fp16's normal numbers is rounded by up to 2^-25 of that. Key j's codes c_j then bring an
error of 2^-25 max_i(p_i s_i) |c_j|, which shows in an element whose code is 0 in the large rows (and is far below
half a step of those). As for the other terms, twice that is allowed."""
import numpy as np
import pytest
import torch

from _kv import UB, Paged, quantise, reference, values
from test_paged_attn_gpu import run

pytestmark = pytest.mark.gpu


def with_rows(case, factor):
    """The case with value rows times `factor` [num_pages, Hkv, page], stored as they would be."""
    x = case.rows["v"] * factor[..., None]
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    case.code["v"], case.scale["v"] = quantise(x, case.cache)
    case.rows["v"] = values(case.code["v"], case.scale["v"], case.cache)
    return case


def fp16_term(case, q, T, scale):
    """2^-25 max_i(p_i s_i) sum_j |c_j| for every element; one key head."""
    q = q.double().numpy()
    out = np.zeros_like(q)
    for n, x in enumerate(case.lens):
        k, v = case.sequence("k", n, 0), case.sequence("v", n, 0)
        s = case.scale["v"][case.table[n, : -(-x // case.page)], 0].reshape(-1)[:x].astype(np.float64)
        c = np.abs(v / s[:, None])
        for t in range(T):
            keys = x - T + t + 1
            if keys <= 0:
                continue
            y = scale * (q[n * T + t] @ k[:keys].T)
            p = np.exp(y - y.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[n * T + t] = 2.0 ** -25 * (p * s[:keys]).max(1)[:, None] * c[:keys].sum(0)
    return out


@pytest.mark.parametrize("cache", ["fp8", "int8"])
@pytest.mark.parametrize("exponent", [0, 12, 30, 60, 100])
@pytest.mark.parametrize("lens,T,G,d,page", [
    ([500, 77], 1, 8, 128, 16), ([500, 77], 1, 8, 256, 64), ([700, 33], 1, 4, 64, 32), ([300, 90], 2, 7, 64, 16),   # few rows
    ([4000], 1, 8, 128, 64), ([3000], 4, 4, 256, 32),                                                              # (split)
    ([500, 77], 40, 8, 128, 16), ([300, 120], 50, 4, 256, 64), ([300, 40], 30, 8, 64, 16), ([4000], 33, 8, 128, 64)])
def test_zeros_and_tiny_rows_among_large_ones(lens, T, G, d, page, exponent, cache):
    """Half of the rows zero, tiny or small, the others 2^exponent times their size: in no order, and in runs as long as
    a tile (so that a part of the work may hold nothing but zeros)."""
    for run_length in (1, 160):
        case = Paged(lens, 1, d, page, cache, "bf16", seed=31)
        r = np.random.RandomState(exponent)
        factor = np.ones(case.scale["v"].shape)
        for n, x in enumerate(lens):
            small = np.repeat(r.rand(x // run_length + 1) < 0.5, run_length)[:x]
            f = np.where(small, r.choice([0.0, 2.0 ** -110, 2.0 ** -60, 2.0 ** -8], x), 2.0 ** exponent)
            for j in range(-(-x // page)):
                rows = f[j * page:(j + 1) * page]
                factor[case.table[n, j], 0, :len(rows)] = rows
        case = with_rows(case, factor)
        q, out = run(case, [T] * len(lens), G)
        ref, mag, _ = reference(case, q, [T] * len(lens), d ** -0.5)
        bound = 2 * (UB * (np.abs(ref) + mag) + fp16_term(case, q, T, d ** -0.5))
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        excess = np.abs(got - ref) - bound
        assert (excess <= 1e-30).all(), f"off by {np.abs(got - ref).max():.3e}, over the bound by {excess.max():.3e}"
