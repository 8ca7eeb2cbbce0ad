"""Values that are not finite, at positions that some of a call's new tokens see and others do not.

By the formula a token's sum runs over the positions up to its own, so an infinity or a NaN further on has no effect
on it, and one that it sees reaches the element it stands in and no other. Against the formula in 64 bits: what is
not finite there has to be the same here (which infinity, or NaN), the rest within the usual bound."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV, DTYPES, U32, UB, Paged, reference

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def put(case, cache, n, pos, h, column, value):
    """`value` into sequence n's value row, in the case's rows and in its cache on the GPU."""
    page, off = case.table[n, pos // case.page], pos % case.page
    case.rows["v"][page, h, off, column] = value
    cache[page, h, off, column] = value


def check(out, want):
    ref, mag, err = want
    got = out.double().cpu().numpy()
    known = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), known), f"{(np.isfinite(got) != known).sum()} elements"
    bad = ~known
    assert np.array_equal(np.isnan(got[bad]), np.isnan(ref[bad]))
    inf = bad & ~np.isnan(ref)
    assert np.array_equal(np.sign(got[inf]), np.sign(ref[inf]))
    bound = 2 * UB * (np.abs(ref) + mag) if out.dtype == torch.bfloat16 else 2 * err[..., None] * mag
    excess = (np.abs(got - ref) - bound)[known]
    assert (excess <= 1e-30).all(), f"over the bound by {excess.max():.3e}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [(100, 64), (3000, 17)])
@pytest.mark.parametrize("T,Hkv,G,d,page", [(2, 2, 3, 128, 16), (8, 1, 1, 64, 16), (2, 2, 4, 256, 32),   # few rows
                                            (5, 2, 8, 256, 64), (16, 1, 7, 128, 16), (40, 2, 1, 64, 32),
                                            (50, 1, 4, 128, 256)])
def test_values_that_are_not_finite(T, Hkv, G, d, page, lens, dtype):
    case = Paged(lens, Hkv, d, page, "same", dtype, seed=21)
    kc, vc, _, _, table, kv_lens = case.tensors()
    x = lens[0]
    put(case, vc, 0, x - 1, 0, 3, INF)                 # the last token's
    put(case, vc, 0, x - 1, Hkv - 1, d - 1, NAN)
    put(case, vc, 0, x - T + T // 2, 0, 9, -INF)       # one in the middle
    put(case, vc, 0, x - 1, 0, 9, INF)                 # (with the last one: NaN)
    put(case, vc, 0, x - T + 1, 0, 40, NAN)            # the second
    put(case, vc, 1, lens[1] - 1, 0, 17, -INF)
    q = torch.randn(2 * T, Hkv * G, d, generator=torch.Generator().manual_seed(3)).to(DTYPES[dtype])
    out = torch.zeros(q.shape, dtype=q.dtype, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, kv_lens, out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    with np.errstate(invalid="ignore"):
        want = reference(case, q, [T, T], d ** -0.5)
        assert np.isfinite(want[0][0]).all() and not np.isfinite(want[0][T - 1]).all()
        check(out, want)


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4)])
@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_a_row_stored_as_nan_in_fp32(cache, T, G):
    """fp32 inputs over an 8-bit cache: a value row with scale NaN makes the tokens that see it NaN, and no others."""
    case = Paged([100, 90], 1, 64, 16, cache, "f32", seed=6)
    kc, vc, ks, vs, table, lens = case.tensors()
    pos = 98
    vs[int(table[0, pos // 16]), 0, pos % 16] = NAN
    q = torch.randn(2 * T, G, 64, generator=torch.Generator().manual_seed(3))
    out = torch.empty(q.shape, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, out, ks, vs)
    assert torch.isnan(out[T - 2:T]).all()
    ref, mag, err = reference(case, q, [T, T], 64 ** -0.5)
    keep = [i for i in range(2 * T) if i < T - 2 or i >= T]
    check(out[keep], (ref[keep], mag[keep], err[keep]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[3], [40], [128, 300]])
def test_tokens_before_and_after_agree_with_fragments(new, dtype):
    """A prompt's fragments whose later tokens hold infinities: the earlier tokens' outputs, bit for bit, are those of
    the same call with finite values there."""
    lens = [400 + 7 * n for n in range(len(new))]
    case = Paged(lens, 2, 128, 64, "same", dtype, seed=5)
    kc, vc, _, _, table, kv_lens = case.tensors()
    q = torch.randn(sum(new), 8, 128, generator=torch.Generator().manual_seed(4)).to(DTYPES[dtype]).to(DEV)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    finite, out = torch.empty_like(q), torch.empty_like(q)
    gdn.gdn_paged_attn(q, kc, vc, table, kv_lens, finite, cu_seqlens=cu)
    first, keep = 0, []
    for n, T in enumerate(new):
        half = T // 2 + 1
        for t in range(half, T):
            pos = lens[n] - T + t
            vc[int(table[n, pos // 64]), :, pos % 64, t % 128] = INF if t % 2 else NAN
        keep += range(first, first + half)
        first += T
    gdn.gdn_paged_attn(q, kc, vc, table, kv_lens, out, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.isfinite(finite).all() and torch.equal(out[keep], finite[keep])
    assert not torch.isfinite(out[first - 1]).all()
