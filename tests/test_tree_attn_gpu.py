"""Attention of trees of drafted tokens over a paged cache, on the GPU, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, DTYPES, Paged, assert_attention, cu_of
from _tree import random_tree, tree_attention

pytestmark = pytest.mark.gpu

# contexts, nodes, kind, padding nodes at the end of each tree
SHAPES = {
    "small": ([0, 1, 15, 16, 60, 63, 64, 127, 128, 300], [4] * 10, "wide", 0),
    "single": ([0, 7, 64, 500], [1] * 4, "wide", 0),
    "packed": ([30, 0, 250, 129, 700], [17, 3, 64, 1, 33], "deep", 1),
    "chain": ([100, 3], [64, 64], "chain", 0),
    "star": ([70], [64], "star", 7),
    "forest": ([0, 200], [23, 23], "forest", 3),
    "long": ([2900, 2000], [5, 5], "wide", 2),
}


def make(shape, Hkv, d, page, cache, dtype, seed=3):
    ctx, nodes, kind, padding = SHAPES[shape]
    r = np.random.RandomState(seed)
    trees = [random_tree(r, T, kind, min(padding, T - 1)) for T in nodes]
    return Paged([c + T for c, T in zip(ctx, nodes)], Hkv, d, page, cache, dtype, seed=seed), trees


def flat(trees):
    return torch.tensor([u for p in trees for u in p], dtype=torch.int32, device=DEV)


def run(case, trees, Hq, scale=None, seed=5, status=gdn.GDN_OK):
    kc, vc, ks, vs, table, lens = case.tensors()
    new = [len(p) for p in trees]
    q = (1.5 * torch.randn(sum(new), Hq, case.d, generator=torch.Generator().manual_seed(seed))).to(DTYPES[case.dtype])
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    cu = None if len(set(new)) == 1 else cu_of(new)
    gdn.gdn_tree_attn(q.to(DEV), kc, vc, table, lens, flat(trees), out, ks, vs, cu_seqlens=cu, scale=scale)
    assert gdn.gdn_get_device_status() == status
    return q, out


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G,d,page", [(2, 8, 256, 16), (1, 1, 128, 64), (2, 7, 64, 256), (3, 3, 128, 32), (2, 4, 64, 16)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_against_the_formula(shape, Hkv, G, d, page, dtype, cache):
    case, trees = make(shape, Hkv, d, page, cache, dtype)
    q, out = run(case, trees, Hkv * G)
    assert_attention(out, *tree_attention(case, q, trees, d ** -0.5))


@pytest.mark.parametrize("dtype,cache,Hkv,G", [("bf16", "same", 1, 64), ("bf16", "fp8", 1, 64), ("f32", "same", 1, 64), ("bf16", "int8", 8, 2)])
def test_many_row_tiles(dtype, cache, Hkv, G):
    """64 query heads to a key head: a tree's rows fill many tiles, each of which sees nodes of earlier ones."""
    case, trees = make("packed", Hkv, 64, 16, cache, dtype)
    q, out = run(case, trees, Hkv * G)
    assert_attention(out, *tree_attention(case, q, trees, 64 ** -0.5))


@pytest.mark.parametrize("dtype,cache,G", [("bf16", "same", 1), ("bf16", "same", 3), ("bf16", "fp8", 2), ("bf16", "int8", 5), ("f32", "fp8", 2)])
def test_one_large_tree_among_single_tokens(dtype, cache, G):
    """Few rows on average, so that the kernel for few rows takes a tree over many row tiles, whose nodes' ancestors are in earlier
    tiles and whose positions lie in several chunks."""
    r = np.random.RandomState(12)
    trees = [[-1]] * 12 + [random_tree(r, 61, "deep", 2)] + [[-1]] * 20
    lens = [int(x) for x in r.randint(1, 300, 12)] + [61 + 37] + [int(x) for x in r.randint(1, 90, 20)]
    case = Paged(lens, 2, 128, 16, cache, dtype, seed=8)
    q, out = run(case, trees, 2 * G)
    assert_attention(out, *tree_attention(case, q, trees, 128 ** -0.5))


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "fp8"), ("f32", "int8"), ("f32", "same")])
def test_a_chain_is_paged_attention(dtype, cache):
    """A tree without branches gives what gdn_paged_attn gives, bit for bit: the same positions are seen."""
    for shape, Hq in (("chain", 4), ("single", 4), ("single", 16)):
        case, trees = make(shape, 2, 128, 32, cache, dtype)
        kc, vc, ks, vs, table, lens = case.tensors()
        q, out = run(case, trees, Hq)
        plain = torch.full_like(out, float("nan"))
        gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, plain, ks, vs)
        assert torch.equal(out, plain)


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "int8"), ("f32", "same")])
def test_padding_sequences_and_nodes(dtype, cache):
    """kv_lens 0 (an idle row) and shorter than the tree: nodes without a position are written as zeros, and nobody sees them."""
    r = np.random.RandomState(9)
    trees = [random_tree(r, 6) for _ in range(4)]
    case = Paged([0, 3, 6, 90], 2, 64, 16, cache, dtype, seed=1)
    q, out = run(case, trees, 4)
    assert not out[:6].any() and not out[6:9].any()
    assert_attention(out, *tree_attention(case, q, trees, 64 ** -0.5))


@pytest.mark.parametrize("dtype,cache,G", [("bf16", "same", 1), ("bf16", "same", 8), ("f32", "same", 2), ("bf16", "fp8", 1), ("bf16", "fp8", 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nodes_off_the_path_have_no_effect(dtype, cache, G, bad):
    """Keys and values that are not finite at some nodes: those that do not see them are as without, those that do are not finite."""
    r = np.random.RandomState(4)
    trees = [random_tree(r, 8, "wide"), random_tree(r, 8, "deep")]
    from _tree import paths
    for ctx in (5, 400):
        case = Paged([ctx + 8] * 2, 2, 64, 16, cache, dtype, seed=6)
        q, clean = run(case, trees, 2 * G)
        kc, vc, ks, vs, table, lens = case.tensors()
        node = 3
        for n in range(2):
            pos = ctx + node
            pg, row = int(case.table[n, pos // 16]), pos % 16
            if cache == "same":
                kc[pg, :, row] = bad
                vc[pg, :, row, ::3] = bad
            else:  # what gdn_kv_write stores of a row that is not finite
                for c, s in ((kc, ks), (vc, vs)):
                    c.view(torch.uint8)[pg, :, row] = 0
                    s[pg, :, row] = float("nan")
        out = torch.full_like(clean, 7.0)
        gdn.gdn_tree_attn(q.to(DEV), kc, vc, table, lens, flat(trees), out, ks, vs)
        assert gdn.gdn_get_device_status() == gdn.GDN_OK
        for n in range(2):
            for t, p in enumerate(paths(trees[n])):
                x, y = out[8 * n + t], clean[8 * n + t]
                if node in p:
                    assert cache == "same" and bad == -float("inf") or not torch.isfinite(x).all()
                else:
                    # (the order of sums may change where the unit is done again: one rounding of the outcome)
                    assert torch.isfinite(x).all()
                    assert ((x.double() - y.double()).abs() <= 2.0 ** -7 * y.double().abs() + 1e-5).all()


@pytest.mark.parametrize("dtype,cache,Hq", [("bf16", "same", 4), ("bf16", "same", 32), ("bf16", "int8", 4), ("f32", "same", 4)])
def test_bad_parents_and_too_many_nodes(dtype, cache, Hq):
    """A parent that does not come before its node is flagged and makes padding; a sequence of 65 nodes is flagged and skipped."""
    case, trees = make("small", 2, 64, 16, cache, dtype)
    trees[2][2] = 2
    trees[4][1] = 900
    q, out = run(case, trees, Hq, status=gdn.GDN_ERR_DEVICE_CHECK)
    assert_attention(out, *tree_attention(case, q, trees, 64 ** -0.5))
    case = Paged([80, 100, 9], 2, 64, 16, cache, dtype, seed=2)
    r = np.random.RandomState(0)
    trees = [random_tree(r, 7), random_tree(r, 65), random_tree(r, 4)]
    q, out = run(case, trees, Hq, status=gdn.GDN_ERR_DEVICE_CHECK)
    assert torch.isnan(out[7:72]).all()
    keep = [i for i in range(76) if not 7 <= i < 72]
    ref, mag, err = tree_attention(case, q, trees, 64 ** -0.5)
    assert_attention(out[keep], ref[keep], mag[keep], err[keep])


def test_slices_streams_and_a_captured_graph():
    """q as a slice of a fused projection, on another stream, and in a graph whose tree and lengths change between replays."""
    case, trees = make("small", 2, 128, 16, "same", "bf16")
    kc, vc, _, _, table, lens = case.tensors()
    T, Hq = 4, 8
    fused = torch.randn(len(trees) * T, Hq + 5, 128, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    q = fused[:, 2:2 + Hq]
    dev = fused.to(DEV)
    out, parents = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV), flat(trees)
    ws = torch.empty(gdn.gdn_paged_attn_workspace_size(len(trees), T, Hq, 2, 128), dtype=torch.uint8, device=DEV)
    call = lambda: gdn.gdn_tree_attn(dev[:, 2:2 + Hq], kc, vc, table, lens, parents, out, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert_attention(out, *tree_attention(case, q, trees, 128 ** -0.5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    r = np.random.RandomState(77)
    for shorter in (0, 3):
        trees = [random_tree(r, T, "forest", 1) for _ in trees]
        case.lens = [max(x - shorter, 0) for x in case.lens]
        parents.copy_(flat(trees))
        lens.copy_(torch.tensor(case.lens, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_attention(out, *tree_attention(case, q, trees, 128 ** -0.5))
        assert gdn.gdn_get_device_status() == gdn.GDN_OK
