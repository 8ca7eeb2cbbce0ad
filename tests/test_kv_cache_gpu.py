"""Writing tokens into a paged cache and reading them back, on the GPU, against the definition in
64 bits: equal codes, scales and values, and nothing else in the pool touched."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, DTYPES, Paged, cu_of, quantise, values

pytestmark = pytest.mark.gpu

# (kv_lens, new tokens): single tokens, runs over page ends, padding (len < T), nothing new
SHAPES = {
    "decode": ([1, 2, 16, 17, 0, 63, 64, 65, 300], [1] * 9),
    "few": ([3, 5, 6, 64, 69, 2], [5] * 6),
    "packed": ([40, 0, 7, 131, 17, 500], [40, 0, 7, 100, 1, 3]),
    "padded_packed": ([4, 0, 9], [6, 2, 9]),
}


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def make_rows(tokens, Hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, Hkv, d, generator=g) * torch.exp(3 * torch.randn(tokens, Hkv, 1, generator=g))
    if tokens > 2:
        x[0, 0] = 0.0                      # a row of zeros
        x[1, -1] *= 1e-37                  # below the smallest scale
        x[2, 0, 0] = 448.0 * 8             # the largest code exactly
        x[2, 0, 1:] = x[2, 0, 1:].clamp(-3000, 3000)
    return x.to(DTYPES[dtype])


def expected_row(x, cache):
    if cache == "same":
        return None, None, x.double().numpy()
    code, scale = quantise(x.double().numpy(), cache)
    return code, scale, values(code, scale, cache)


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,d,page", [(2, 256, 16), (3, 128, 64), (8, 64, 256), (1, 64, 32), (5, 256, 128)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_write_then_read(shape, Hkv, d, page, dtype, cache):
    lens, new = SHAPES[shape]
    case = Paged(lens, Hkv, d, page, cache, dtype, seed=3)
    kc, vc, ks, vs, table, kv_lens = case.tensors()
    before = [None if t is None else bits(t) for t in (kc, vc, ks, vs)]
    tokens = sum(new)
    k, v = make_rows(tokens, Hkv, d, dtype, 1), make_rows(tokens, Hkv, d, dtype, 2)
    cu = None if len(set(new)) == 1 else cu_of(new)
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), kc, vc, table, kv_lens, ks, vs, cu_seqlens=cu)
    got = torch.full((2, tokens, Hkv, d), float("nan"), dtype=DTYPES[dtype], device=DEV)
    gdn.gdn_kv_read(kc, vc, table, kv_lens, got[0], got[1], ks, vs, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    # the pool as it should be: the new rows at their places, every other byte as before
    first = 0
    want = [b if b is None else b.clone() for b in before]
    rowbytes = d * kc.element_size()
    pools = [w.view(case.num_pages, Hkv, page, -1) if w is not None else None for w in want]
    back = np.zeros((2, tokens, Hkv, d))
    for n, T in enumerate(new):
        for t in range(T):
            pos = lens[n] - T + t
            if pos < 0:
                continue
            pg, off = case.table[n, pos // page], pos % page
            for m, x in enumerate((k, v)):
                row = x[first + t]
                code, scale, val = expected_row(row, cache)
                if cache == "same":
                    pools[m][pg, :, off] = row.contiguous().view(torch.uint8).view(Hkv, rowbytes)
                else:
                    pools[m][pg, :, off] = torch.from_numpy(code)
                    pools[2 + m][pg, :, off] = torch.from_numpy(scale).view(torch.uint8).view(Hkv, 4)
                back[m, first + t] = val
        first += T
    for name, w, t in zip(("k_cache", "v_cache", "k_scale", "v_scale"), want, (kc, vc, ks, vs)):
        if t is not None:
            assert torch.equal(w.view(-1), bits(t).view(-1)), f"{name} differs"
    ref = torch.from_numpy(back).to(DTYPES[dtype])  # one rounding to the I/O type
    assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_rounding_is_to_nearest_even_and_close(cache):
    """Every tie between two codes, and the distance of what is stored from what was written."""
    d = 64
    if cache == "fp8":
        from _kv import E4M3
        pos = E4M3[:127]
        x = np.concatenate([(pos[1:] + pos[:-1]) / 2, pos, [448.0]])
    else:
        x = np.concatenate([np.arange(-127, 127) + 0.5, [127.0]])
    x = np.concatenate([x, np.zeros(-len(x) % (d - 1))]).reshape(-1, d - 1)
    top = 448.0 if cache == "fp8" else 127.0
    rows = torch.from_numpy(np.concatenate([np.full((len(x), 1), top), x], 1).astype(np.float32))[:, None]
    T = len(rows)
    kc = torch.zeros(8, 1, 16, d, dtype=torch.uint8, device=DEV).view(CACHES[cache])
    vc, ks, vs = torch.zeros_like(kc), torch.zeros(8, 1, 16, device=DEV), torch.zeros(8, 1, 16, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    gdn.gdn_kv_write(rows.to(DEV), -rows.to(DEV), kc, vc, table, torch.tensor([T], dtype=torch.int32, device=DEV), ks, vs)
    code, scale = quantise(rows.double().numpy(), cache)
    assert (scale == 1.0).all()
    assert np.array_equal(bits(kc).view(-1, d).numpy()[:T], code[:, 0])
    neg, _ = quantise(-rows.double().numpy(), cache)
    assert np.array_equal(bits(vc).view(-1, d).numpy()[:T], neg[:, 0])
    err = np.abs(values(code, scale, cache) - rows.double().numpy())
    assert (err <= (np.maximum(np.abs(rows.numpy()) / 16, 2.0 ** -10) if cache == "fp8" else 0.5)).all()


@pytest.mark.parametrize("cache", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_reads_back_as_nan(cache, bad):
    kc = torch.zeros(2, 2, 16, 128, dtype=torch.uint8, device=DEV).view(CACHES[cache])
    vc, ks, vs = torch.zeros_like(kc), torch.zeros(2, 2, 16, device=DEV), torch.zeros(2, 2, 16, device=DEV)
    k = torch.randn(3, 2, 128, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    k[1, 0, 77] = bad
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_write(k, v, kc, vc, table, lens, ks, vs)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.gdn_kv_read(kc, vc, table, lens, ko, vo, ks, vs)
    assert torch.isnan(ko[1, 0]).all() and int(bits(kc[1, 0, 1]).sum()) == 0
    ko[1, 0] = 0
    assert not torch.isnan(ko).any() and not torch.isnan(vo).any()


def test_slices_of_a_fused_projection():
    """Token strides: q, k and v as slices of one [tokens, (Hq + 2 Hkv) d] tensor, read back into slices."""
    Hq, Hkv, d, T = 4, 2, 64, 21
    fused = torch.randn(T, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device=DEV)
    k = fused[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    v = fused[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
    kc = torch.zeros(3, Hkv, 16, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_write(k, v, kc, vc, table, lens)
    back = torch.zeros_like(fused)
    gdn.gdn_kv_read(kc, vc, table, lens, back[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)),
                    back[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)))
    assert torch.equal(back[:, Hq * d:], fused[:, Hq * d:]) and not back[:, :Hq * d].any()
    assert torch.equal(kc[2].transpose(0, 1), k[:16])


def test_offsets_past_32_bits():
    """Pages beyond 2^31 elements (and 2^32 bytes) of the pool."""
    Hkv, d, page = 8, 256, 256
    pages = 2 ** 31 // (Hkv * page * d) + 9
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1, 3], [pages - 2, pages - 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([300, 512], dtype=torch.int32, device=DEV)
    k = torch.randn(812, Hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.randn_like(k)
    gdn.gdn_kv_write(k, v, kc, vc, table, lens, cu_seqlens=cu_of([300, 512]))
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    gdn.gdn_kv_read(kc, vc, table, lens, ko, vo, cu_seqlens=cu_of([300, 512]))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.equal(k, ko) and torch.equal(v, vo)
    assert torch.equal(kc[pages - 1].transpose(0, 1), k[:256])


def test_inconsistent_device_data_is_flagged_and_skipped():
    Hkv, d, page = 2, 64, 16
    kc = torch.zeros(4, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.randn(3, Hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.randn_like(k)
    # a page outside of the pool, a length outside of the table, a sound sequence
    table = torch.tensor([[9], [1], [2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 17, 16], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_write(k, v, kc, vc, table, lens)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    ko, vo = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    gdn.gdn_kv_read(kc, vc, table, lens, ko, vo)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.equal(ko[2], k[2]) and torch.equal(vo[2], v[2])
    assert not ko[:2].any() and not vo[:2].any()
    assert torch.equal(kc[2, :, 15], k[2]) and int(torch.count_nonzero(kc)) == int(torch.count_nonzero(k[2]))
    # offsets that do not cover the tokens: the sequences they break are left out
    cu = torch.tensor([0, 2, 1, 3], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_read(kc, vc, table, torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV), ko, vo, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK


def test_another_stream_and_no_tokens():
    Hkv, d, page = 2, 128, 16
    kc = torch.zeros(2, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        k = torch.randn(4, Hkv, d, dtype=torch.bfloat16, device=DEV)
        v = torch.randn_like(k)
        lens = torch.tensor([4], dtype=torch.int32, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    ko, vo = torch.zeros(4, Hkv, d, dtype=torch.bfloat16, device=DEV), torch.zeros(4, Hkv, d, dtype=torch.bfloat16, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_kv_write(k, v, kc, vc, table, lens, stream=s)
    gdn.gdn_kv_read(kc, vc, table, lens, ko, vo, stream=s)
    s.synchronize()
    assert torch.equal(ko, k) and torch.equal(vo, v)
    empty = torch.empty(0, Hkv, d, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_kv_write(empty, empty, kc, vc, table[:0], lens[:0])
    gdn.gdn_kv_read(kc, vc, table, lens, empty, empty, cu_seqlens=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
