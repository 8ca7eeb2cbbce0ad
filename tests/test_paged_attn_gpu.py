"""Attention of new tokens over a paged cache, on the GPU, against the formula in 64 bits.

Every place of the pool that no live position owns holds NaN, and block table entries past a
sequence's last page hold -7, so reading either shows."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, DTYPES, Paged, assert_attention, cu_of, reference

pytestmark = pytest.mark.gpu

# (kv_lens, new tokens)
SHAPES = {
    "decode": ([1, 2, 15, 16, 17, 31, 63, 64, 65, 0, 127, 128, 129, 257, 1000], [1] * 15),
    "few": ([3, 5, 6, 64, 69, 131, 200, 0], [5] * 8),  # the first has more new tokens than positions: padding
    "packed": ([1, 0, 300, 130, 700, 33], [1, 0, 7, 130, 33, 2]),
    "prompt": ([201], [201]),
    "one_long": ([3001], [1]),
    "two_long": ([2500, 1777], [3, 3]),
}


def run(case, new, Hq, scale=None, seed=5, q=None):
    kc, vc, ks, vs, table, lens = case.tensors()
    if q is None:
        g = torch.Generator().manual_seed(seed)
        q = (1.5 * torch.randn(sum(new), Hq, case.d, generator=g)).to(DTYPES[case.dtype])
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    cu = None if len(set(new)) == 1 else cu_of(new)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, out, ks, vs, cu_seqlens=cu, scale=scale)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    return q, out


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G,d,page", [(2, 8, 256, 16), (1, 1, 128, 64), (2, 7, 64, 256), (3, 3, 128, 32),
                                          (1, 5, 256, 128), (2, 4, 64, 16)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_against_the_formula(shape, Hkv, G, d, page, dtype, cache):
    lens, new = SHAPES[shape]
    case = Paged(lens, Hkv, d, page, cache, dtype, seed=7)
    q, out = run(case, new, Hkv * G)
    ref, mag, err = reference(case, q, new, d ** -0.5)
    assert_attention(out, ref, mag, err)
    # padding rows are zeros
    first = 0
    for x, T in zip(lens, new):
        idle = max(0, T - x)
        assert not out[first:first + idle].any()
        first += T


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "fp8"), ("bf16", "int8"), ("f32", "same")])
def test_many_query_heads_to_a_key_head(dtype, cache):
    """64 query heads on one key head, with a few tokens: row tiles of one and two tokens."""
    lens, new = [70, 3, 140], [3, 3, 3]
    case = Paged(lens, 1, 64, 16, cache, dtype, seed=2)
    q, out = run(case, new, 64)
    assert_attention(out, *reference(case, q, new, 64 ** -0.5))


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "fp8"), ("f32", "same")])
def test_scores_of_great_range(dtype, cache):
    """A scale that makes the softmax all but pick one key, and the running maximum grow along the cache."""
    lens, new = [900, 450], [2, 2]
    case = Paged(lens, 2, 128, 64, cache, dtype, seed=11)
    for scale in (2.0, -1.0, 0.0):
        q, out = run(case, new, 4, scale=scale)
        ref, mag, err = reference(case, q, new, scale)
        if scale == 2.0 and dtype == "bf16":
            # scores reach a few hundred: their own fp32 rounding (2 e_s) is no longer covered by the doubling
            mag = mag * (1 + 2 * err[..., None] / (2 * 2.0 ** -9))
        assert_attention(out, ref, mag, err)


@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_values_of_great_range(cache):
    """Value rows whose scales differ by 2^40 within a sequence, and rows of zeros (the smallest scale)."""
    lens, new = [500, 77], [1, 1]
    case = Paged(lens, 1, 128, 16, cache, "bf16", seed=13)
    r = np.random.RandomState(1)
    f = np.exp2(r.randint(-30, 11, case.scale["v"].shape)).astype(np.float32)
    f[r.rand(*f.shape) < 0.1] = 0
    from _kv import values
    tiny = f == 0
    case.scale["v"] = np.where(tiny, np.float32(2.0 ** -100), case.scale["v"] * f).astype(np.float32)
    case.code["v"][tiny] = 0
    case.rows["v"] = values(case.code["v"], case.scale["v"], cache)
    q, out = run(case, new, 8)
    assert_attention(out, *reference(case, q, new, 128 ** -0.5))


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "fp8"), ("bf16", "int8"), ("f32", "int8")])
def test_split_rows_do_not_depend_on_their_company(dtype, cache):
    """One sequence alone (its cache cut between many CTAs) and among others: the same within rounding, and
    the same call twice is the same bit for bit."""
    case = Paged([2900, 1, 40, 800], 2, 128, 64, cache, dtype, seed=4)
    kc, vc, ks, vs, table, lens = case.tensors()
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype]).to(DEV)
    outs = [torch.empty_like(q) for _ in range(2)]
    for o in outs:
        gdn.gdn_paged_attn(q, kc, vc, table, lens, o, ks, vs)
    assert torch.equal(outs[0], outs[1])
    alone = torch.empty_like(q[:1])
    gdn.gdn_paged_attn(q[:1], kc, vc, table[:1].contiguous(), lens[:1].contiguous(), alone, ks, vs)
    ref, mag, err = reference(case, q.cpu(), [1] * 4, 128 ** -0.5)
    assert_attention(alone, ref[:1], mag[:1], err[:1])
    assert_attention(outs[0], ref, mag, err)


def formula64(q, k, v, lens, new, scale):
    """(out, sum_j p_j |v_j|) in fp64 on the GPU, sequence by sequence; k, v: lists of [len, Hkv, d]."""
    out, mag = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    first = 0
    for kk, vv, x, T in zip(k, v, lens, new):
        for a in range(0, T if x else 0, 256):
            b = min(T, a + 256)
            qq = q[first + a:first + b].double().unflatten(1, (kk.shape[1], -1))
            s = torch.einsum("tghd,jgd->tghj", qq, kk.double()) * scale
            hidden = torch.arange(x, device=DEV)[None, :] > (x - T + torch.arange(a, b, device=DEV))[:, None]
            p = s.masked_fill(hidden[:, None, None], -float("inf")).softmax(-1)
            out[first + a:first + b] = torch.einsum("tghj,jgd->tghd", p, vv.double()).flatten(1, 2)
            mag[first + a:first + b] = torch.einsum("tghj,jgd->tghd", p, vv.double().abs()).flatten(1, 2)
        first += T
    return out, mag


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("lens,new,Hkv,G,d,page", [
    ([9001], [700], 2, 8, 256, 64),                       # a fragment: long units, few per CTA
    ([7000, 6500, 8003], [300, 1, 511], 4, 4, 128, 32),   # fragments of several sequences
    ([3000], [3000], 2, 8, 64, 16),                       # a prompt: many units of every length per CTA
    ([1025, 2047, 311, 64], [1025, 2047, 311, 64], 8, 4, 128, 128),
    ([777] * 40, [1] * 40, 8, 4, 128, 16),                # decode with many units per CTA
    ([20000, 15000], [2, 2], 1, 8, 256, 256),             # a few tokens over long caches
    ([5000] * 3, [64] * 3, 1, 1, 64, 16),
])
def test_long_units(lens, new, Hkv, G, d, page, cache):
    """Units of many key tiles and many units per CTA (the small cases above give a CTA a few tiles each)."""
    gen = torch.Generator(device=DEV).manual_seed(len(lens) + d)
    pages = [-(-x // page) for x in lens]
    table = torch.full((len(lens), max(pages)), -7, dtype=torch.int32, device=DEV)
    order = torch.randperm(sum(pages) + 2, generator=gen, device=DEV).to(torch.int32)
    at = 0
    for n, u in enumerate(pages):
        table[n, :u] = order[at:at + u]
        at += u
    kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kind = CACHES[cache] or torch.bfloat16
    pool = (sum(pages) + 2, Hkv, page, d)
    kc, vc = (torch.full(pool, 0x7F, dtype=torch.uint8, device=DEV).view(kind) if cache != "same"
              else torch.full(pool, float("nan"), dtype=kind, device=DEV) for _ in range(2))
    ks, vs = ((torch.full(pool[:-1], float("nan"), device=DEV) if cache != "same" else None) for _ in range(2))
    k, v = (torch.randn(sum(lens), Hkv, d, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    # scores that grow along the cache, so that the running maximum moves in many tiles
    ramp = torch.cat([torch.linspace(0.3, 2.0, x, device=DEV) for x in lens])
    k = (k.float() * ramp[:, None, None]).to(torch.bfloat16)
    gdn.gdn_kv_write(k, v, kc, vc, table, kv_lens, ks, vs, cu_seqlens=cu_of(lens))
    kr, vr = (torch.empty(k.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gdn.gdn_kv_read(kc, vc, table, kv_lens, kr, vr, ks, vs, cu_seqlens=cu_of(lens))
    if cache == "int8":  # values of more than 8 bits: their bf16 rounding is not what the attention sees
        rows = torch.cat([torch.stack([table[n, torch.arange(x, device=DEV) // page].long(),
                                       torch.arange(x, device=DEV) % page], 1) for n, x in enumerate(lens)])
        kr, vr = (c[rows[:, 0], :, rows[:, 1]].double() * s[rows[:, 0], :, rows[:, 1]].double()[..., None]
                  for c, s in ((kc, ks), (vc, vs)))
    q = torch.randn(sum(new), Hkv * G, d, generator=gen, device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, float("nan"))
    cu = None if len(set(new)) == 1 else cu_of(new)
    gdn.gdn_paged_attn(q, kc, vc, table, kv_lens, out, ks, vs, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    cut = lambda x: list(torch.split(x, lens))  # noqa: E731
    ref, mag = formula64(q, cut(kr), cut(vr), lens, new, d ** -0.5)
    bound = 2.0 ** -8 * (ref.abs() + mag)
    excess = ((out.double() - ref).abs() - bound).max().item()
    assert excess <= 0, f"over the bound by {excess:.3e}"
    again = torch.full_like(q, float("nan"))
    gdn.gdn_paged_attn(q, kc, vc, table, kv_lens, again, ks, vs, cu_seqlens=cu)
    assert torch.equal(out, again)


@pytest.mark.parametrize("G,dtype,cache", [(2, "bf16", "same"), (2, "bf16", "int8"), (64, "bf16", "same"), (2, "f32", "same")])
def test_more_sequences_than_threads(G, dtype, cache):
    """1500 sequences, some idle: more than the kernels' threads, so the work is cut in a second pass over them."""
    r = np.random.RandomState(8)
    lens = [int(x) for x in r.randint(0, 60, 1500)]
    lens[700], lens[1499] = 900, 300
    case = Paged(lens, 1, 64, 16, cache, dtype, seed=8)
    q, out = run(case, [1] * 1500, G)
    assert_attention(out, *reference(case, q, [1] * 1500, 64 ** -0.5))


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("lens,new,G", [
    ([1500, 40, 16, 1], [1] * 4, 8),                      # 8 rows, in one tile of 8
    ([1500, 700], [1, 1], 9),                             # 9 rows
    ([900, 33, 5], [4] * 3, 4),                           # 16 rows
    ([700, 650, 20], [5] * 3, 3),                         # 15 rows
    ([77] * 20 + [500], [1] * 20 + [9], 2),               # few rows on average, one sequence with several tiles of them
])
def test_few_rows(lens, new, G, d, page, cache):
    case = Paged(lens, 2, d, page, cache, "bf16", seed=9)
    q, out = run(case, new, 2 * G)
    assert_attention(out, *reference(case, q, new, d ** -0.5))


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "int8"), ("f32", "same")])
@pytest.mark.parametrize("lens,new,G", [([2900], [1], 8), ([2900], [3], 7), ([2900], [5], 8), ([2900], [13], 8),
                                        ([2900], [40], 5), ([600, 590, 610], [70] * 3, 4)])
def test_split_units_of_any_number_of_rows(lens, new, G, dtype, cache):
    """8 to 128 rows of a unit whose keys are shared by many CTAs: each row is put together by 8 warps or fewer."""
    case = Paged(lens, 1, 128, 64, cache, dtype, seed=11)
    q, out = run(case, new, G)
    assert_attention(out, *reference(case, q, new, 128 ** -0.5))


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("T", [1, 3, 50])
def test_output_on_a_16_byte_boundary(T, cache):
    """Whole rows and rows of a piece, with an output that is not on a wider boundary: the same results."""
    case = Paged([700, 90], 2, 128, 16, cache, "bf16", seed=12)
    kc, vc, ks, vs, table, lens = case.tensors()
    q = torch.randn(2 * T, 16, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    aligned = torch.empty_like(q)
    room = torch.zeros(q.numel() + 16, dtype=q.dtype, device=DEV)
    out = room[8:8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16 and aligned.data_ptr() % 32 == 0
    for to in (aligned, out):
        gdn.gdn_paged_attn(q, kc, vc, table, lens, to, ks, vs)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.equal(out, aligned)
    assert not room[:8].any() and not room[8 + q.numel():].any()


@pytest.mark.parametrize("T", [1, 30])
def test_another_stream(T):
    """All on a stream of its own, without a workspace: torch's allocator gives it to that stream."""
    case = Paged([400, 90], 2, 128, 16, "fp8", seed=3)
    q = torch.randn(2 * T, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kc, vc, ks, vs, table, lens = case.tensors()
        qd = q.to(DEV)
        out = torch.full_like(qd, float("nan"))
    gdn.gdn_paged_attn(qd, kc, vc, table, lens, out, ks, vs, stream=s)
    s.synchronize()
    assert_attention(out, *reference(case, q, [T, T], 128 ** -0.5))


def test_fragments_of_a_prompt_equal_the_whole():
    """A prompt stored and attended in fragments gives what the whole prompt gives at once."""
    Hq, Hkv, d, T = 8, 2, 256, 333
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(T, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    table = torch.randperm(25, generator=g)[:21].to(torch.int32)[None].to(DEV)
    whole = torch.empty_like(q)
    parts = torch.empty_like(q)
    for out, cuts in ((whole, [0, T]), (parts, [0, 100, 101, 228, T])):
        kc = torch.full((25, Hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        vc = kc.clone()
        for a, b in zip(cuts, cuts[1:]):
            lens = torch.tensor([b], dtype=torch.int32, device=DEV)
            gdn.gdn_kv_write(k[a:b], v[a:b], kc, vc, table, lens)
            gdn.gdn_paged_attn(q[a:b], kc, vc, table, lens, out[a:b])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    x = torch.einsum("tghd,jgd->tghj", q.view(T, Hkv, -1, d).double(), k.double()) * d ** -0.5
    x = x.masked_fill(torch.ones(T, T, dtype=torch.bool, device=DEV).triu(1)[:, None, None], -float("inf")).softmax(-1)
    ref = torch.einsum("tghj,jgd->tghd", x, v.double()).reshape(T, Hq, d)
    mag = torch.einsum("tghj,jgd->tghd", x, v.double().abs()).reshape(T, Hq, d)
    for o in (whole, parts):
        assert ((o.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag)).all()


def test_q_as_a_slice_of_a_fused_projection():
    case = Paged([50, 90], 2, 128, 32, seed=1)
    kc, vc, ks, vs, table, lens = case.tensors()
    fused = torch.randn(6, (8 + 4) * 128, dtype=torch.bfloat16, device=DEV)
    q = fused[:, :8 * 128].unflatten(1, (8, 128))
    out, flat = torch.empty(6, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(6, 8, 128, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_paged_attn(q, kc, vc, table, lens, out)
    gdn.gdn_paged_attn(q.contiguous(), kc, vc, table, lens, flat)
    assert torch.equal(out, flat)
    assert_attention(out, *reference(case, q.cpu(), [3, 3], 128 ** -0.5))


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "fp8"), ("f32", "same")])
def test_what_a_nan_key_reaches(dtype, cache):
    """A NaN key makes the rows that see it NaN, and no others."""
    case = Paged([100, 100], 1, 64, 16, cache, dtype, seed=6)
    kc, vc, ks, vs, table, lens = case.tensors()
    pos = 97  # of sequence 0: seen by its last three of five new tokens (positions 95 .. 99)
    page, off = int(table[0, pos // 16]), pos % 16
    if cache == "same":
        kc[page, 0, off, 3] = float("nan")
    else:
        ks[page, 0, off] = float("nan")
    q = torch.randn(10, 4, 64, generator=torch.Generator().manual_seed(3)).to(DTYPES[dtype])
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, out, ks, vs)
    assert torch.isnan(out[2:5]).all()
    ref, mag, err = reference(case, q, [5, 5], 64 ** -0.5)
    keep = [0, 1, 5, 6, 7, 8, 9]
    assert_attention(out[keep], ref[keep], mag[keep], err[keep])


@pytest.mark.parametrize("T", [5, 40])
@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_what_a_row_stored_as_nan_reaches(cache, T):
    """A value row that was not finite when it was stored (scale NaN): NaN for the rows that see it, and
    nothing for those before it, although it lies in their key tile."""
    case = Paged([100, 100], 1, 64, 16, cache, "bf16", seed=6)
    kc, vc, ks, vs, table, lens = case.tensors()
    pos = 97
    vs[int(table[0, pos // 16]), 0, pos % 16] = float("nan")
    q = torch.randn(2 * T, 3, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, out, ks, vs)
    assert torch.isnan(out[T - 3:T]).all()
    ref, mag, err = reference(case, q, [T, T], 64 ** -0.5)
    keep = [i for i in range(2 * T) if i < T - 3 or i >= T]
    assert_attention(out[keep], ref[keep], mag[keep], err[keep])


def test_offsets_past_32_bits():
    Hkv, d, page = 8, 256, 256
    pages = 2 ** 31 // (Hkv * page * d) + 9
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1, 3, pages - 4]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([600], dtype=torch.int32, device=DEV)
    for p in table[0].tolist():
        kc[p] = torch.randn(Hkv, page, d, device=DEV)
        vc[p] = torch.randn(Hkv, page, d, device=DEV)
    q = torch.randn(2, 16, d, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    gdn.gdn_paged_attn(q, kc, vc, table, lens, out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    k, v = (c[table[0].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :600].double() for c in (kc, vc))
    x = torch.einsum("tghd,gjd->tghj", q.view(2, Hkv, 2, d).double(), k) / 16
    x[0, :, :, 599] = -float("inf")
    x = x.softmax(-1)
    ref = torch.einsum("tghj,gjd->tghd", x, v).reshape(2, 16, d)
    mag = torch.einsum("tghj,gjd->tghd", x, v.abs()).reshape(2, 16, d)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag)).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f32", "same")])
def test_a_captured_graph_follows_its_lengths(dtype, cache):
    """A graph of one decode step (write, attention), replayed while the lengths grow, on its own stream."""
    Hkv, G, d, page, B = 2, 4, 128, 16, 3
    pages = B * 3
    start = [0, 15, 31]
    kc = torch.full((pages, Hkv, page, d), float("nan"), dtype=DTYPES[dtype], device=DEV)
    vc = kc.clone()
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, 3).to(DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, Hkv * G, d, dtype=DTYPES[dtype], device=DEV)
    k, v = (torch.zeros(B, Hkv, d, dtype=DTYPES[dtype], device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_paged_attn_workspace_size(B, 1, Hkv * G, Hkv, d), dtype=torch.uint8, device=DEV)

    def step():
        gdn.gdn_kv_write(k, v, kc, vc, table, lens)
        gdn.gdn_paged_attn(q, kc, vc, table, lens, out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    r = np.random.RandomState(0)
    K, V = [[np.zeros((0, Hkv, d))] * B, [np.zeros((0, Hkv, d))] * B]
    K, V = list(K), list(V)
    for n in range(B):  # what is cached before the first step
        if start[n]:
            kk, vv = (torch.from_numpy(r.randn(start[n], Hkv, d)).to(DTYPES[dtype]) for _ in range(2))
            gdn.gdn_kv_write(kk.to(DEV), vv.to(DEV), kc, vc, table[n:n + 1].contiguous(),
                             torch.tensor([start[n]], dtype=torch.int32, device=DEV))
            K[n], V[n] = kk.double().numpy(), vv.double().numpy()
    torch.cuda.synchronize()
    for t in range(6):
        qq, kk, vv = (torch.from_numpy(r.randn(*x.shape)).to(DTYPES[dtype]) for x in (q, k, v))
        q.copy_(qq); k.copy_(kk); v.copy_(vv)
        lens.copy_(torch.tensor([x + t + 1 for x in start], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in range(B):
            K[n] = np.concatenate([K[n], kk[n:n + 1].double().numpy()])
            V[n] = np.concatenate([V[n], vv[n:n + 1].double().numpy()])
            for h in range(Hkv):
                sc = qq[n, h * G:(h + 1) * G].double().numpy() @ K[n][:, h].T * d ** -0.5
                p = np.exp(sc - sc.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                ref, mag = p @ V[n][:, h], p @ np.abs(V[n][:, h])
                got = out[n, h * G:(h + 1) * G].double().cpu().numpy()
                tol = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -14
                assert (np.abs(got - ref) <= tol * (np.abs(ref) + mag)).all(), (t, n, h)


def test_inconsistent_device_data_is_flagged():
    case = Paged([40, 50, 20], 2, 64, 16, seed=1)
    kc, vc, ks, vs, table, lens = case.tensors()
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for bad in (-1, case.width * 16 + 1):
        wrong = lens.clone()
        wrong[1] = bad
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
        gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, wrong, out)
        assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
        assert not out[1].any()
        ref, mag, err = reference(case, q, [1, 1, 1], 64 ** -0.5)
        assert_attention(out[[0, 2]], ref[[0, 2]], mag[[0, 2]], err[[0, 2]])
    # a page outside of the pool counts as keys and values of zero
    for bad in (-1, case.num_pages, 2 ** 31 - 1):
        t2 = table.clone()
        t2[1, 1] = bad
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
        gdn.gdn_paged_attn(q.to(DEV), kc, vc, t2, lens, out)
        assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
        zero = Paged([40, 50, 20], 2, 64, 16, seed=1)
        for name in ("k", "v"):
            zero.rows[name][zero.table[1, 1]] = 0
        assert_attention(out, *reference(zero, q, [1, 1, 1], 64 ** -0.5))
    # offsets that go down: those sequences are skipped
    cu = torch.tensor([0, 2, 1, 3], dtype=torch.int32, device=DEV)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, out, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


def test_no_tokens_and_only_idle_rows():
    case = Paged([40, 50], 2, 64, 16, seed=1)
    kc, vc, ks, vs, table, lens = case.tensors()
    q = torch.randn(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, float("nan"))
    gdn.gdn_paged_attn(q[:0], kc, vc, table[:0], lens[:0], out[:0])
    gdn.gdn_paged_attn(q[:0], kc, vc, table, lens, out[:0], cu_seqlens=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert torch.isnan(out).all()
    gdn.gdn_paged_attn(q, kc, vc, table, torch.zeros_like(lens), out)
    assert not out.any()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
