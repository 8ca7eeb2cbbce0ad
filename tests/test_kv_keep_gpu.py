"""The cache rows of accepted paths, moved right after their contexts, on the GPU: equal bytes."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, Paged, cu_of
from _tree import paths, random_tree

pytestmark = pytest.mark.gpu


def raw(t):
    return t.view(torch.uint8).cpu() if t is not None else None


def expect(case, pools, nodes, accepted):
    """The pools' bytes after the move, in numpy."""
    out = [None if x is None else raw(x).numpy().copy() for x in pools]
    for x, src in zip(out, pools):
        if x is None:
            continue
        old = x.copy()
        for n, (T, path) in enumerate(zip(nodes, accepted)):
            base = case.lens[n] - T
            if base < 0:
                continue
            wide = x.shape[-1] // src.shape[-1] if x.ndim == 3 else None
            for i, u in enumerate(path):
                (a, r0), (b, r1) = ((int(case.table[n, p // case.page]), p % case.page) for p in (base + u, base + i))
                if x.ndim == 4:
                    x[b, :, r1] = old[a, :, r0]
                else:
                    x[b, :, r1 * wide:(r1 + 1) * wide] = old[a, :, r0 * wide:(r0 + 1) * wide]
    return out


def move(case, nodes, accepted, width=None, status=gdn.GDN_OK, moved=None):
    kc, vc, ks, vs, table, lens = case.tensors()
    pools = [kc, vc, ks, vs]
    want = expect(case, pools, nodes, accepted if moved is None else moved)
    width = max([1] + [len(p) for p in accepted]) if width is None else width
    path = torch.tensor([p + [-1] * (width - len(p)) for p in accepted], dtype=torch.int32, device=DEV)
    counts = torch.tensor([len(p) for p in accepted], dtype=torch.int32, device=DEV)
    same = len(set(nodes)) == 1
    gdn.gdn_kv_keep(kc, vc, table, lens, path, counts, ks, vs, cu_seqlens=None if same else cu_of(nodes), T=nodes[0] if same else None)
    assert gdn.gdn_get_device_status() == status
    for got, ref in zip(pools, want):
        if got is not None:
            assert np.array_equal(raw(got).numpy(), ref)


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,d,page", [(2, 256, 16), (1, 64, 64), (8, 128, 32), (3, 64, 16)])
def test_paths_move_together(Hkv, d, page, dtype, cache):
    r = np.random.RandomState(Hkv + d)
    nodes = [1, 9, 64, 40, 7, 12, 0]
    lens = [1, 9 + 11, 64 + 100, 40 + 57, 0, 5, 30]  # the fifth is idle, the sixth has fewer positions than nodes
    trees = [random_tree(r, T, "deep") for T in nodes]
    accepted = [paths(t)[-1] if t else [] for t in trees]
    case = Paged(lens, Hkv, d, page, cache, dtype, seed=1)
    move(case, nodes, accepted)
    move(case, nodes, accepted, width=64)


@pytest.mark.parametrize("cache", ["same", "int8"])
def test_every_kind_of_path(cache):
    """A path that stays where it is, one that moves by one, the last node alone, long ones over several pages, none."""
    T = 40
    accepted = [list(range(40)), [0] + list(range(2, 40)), [39], list(range(1, 40)), [0, 5, 6, 7, 30, 39], [], [0]]
    case = Paged([T + 13 * n for n in range(len(accepted))], 2, 64, 16, cache, "bf16", seed=2)
    move(case, [T] * len(accepted), accepted)


def test_flagged():
    """Paths that are not increasing or name no node, counts out of range: flagged, nothing of that sequence moves."""
    T = 6
    case = Paged([30] * 6, 2, 64, 16, "fp8", "bf16", seed=3)
    accepted = [[0, 2, 4], [0, 3, 3], [2, 1], [0, 6], [-1, 2], [1, 5]]
    moved = [[0, 2, 4], [], [], [], [], [1, 5]]
    move(case, [T] * 6, accepted, status=gdn.GDN_ERR_DEVICE_CHECK, moved=moved)
    kc, vc, ks, vs, table, lens = case.tensors()
    before = [raw(x) for x in (kc, vc, ks, vs)]
    path = torch.tensor([[1, 2]] * 6, dtype=torch.int32, device=DEV)
    counts = torch.tensor([3, -1, 100, 7, 2 ** 30, -5], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_keep(kc, vc, table, lens, path, counts, ks, vs, T=T)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert all(torch.equal(raw(x), y) for x, y in zip((kc, vc, ks, vs), before))
    # a page outside of the pool: what would come from there or go there is left out, and flagged
    case = Paged([30], 2, 64, 16, "same", "bf16", seed=3)
    kc, vc, ks, vs, table, lens = case.tensors()
    table[0, 1] = 1000
    before = raw(kc)
    gdn.gdn_kv_keep(kc, vc, table, lens, torch.tensor([[1, 2]], dtype=torch.int32, device=DEV),
                    torch.tensor([2], dtype=torch.int32, device=DEV), T=6)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert torch.equal(raw(kc), before)


def test_a_captured_graph_and_another_stream():
    T = 12
    r = np.random.RandomState(5)
    case = Paged([50, 20, 12], 2, 128, 16, "int8", "bf16", seed=4)
    kc, vc, ks, vs, table, lens = case.tensors()
    path = torch.zeros(3, T, dtype=torch.int32, device=DEV)
    counts = torch.zeros(3, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        gdn.gdn_kv_keep(kc, vc, table, lens, path, counts, ks, vs, T=T)
    for _ in range(3):
        accepted = [paths(random_tree(r, T, "deep"))[-1] for _ in range(3)]
        want = expect(case, [kc, vc, ks, vs], [T] * 3, accepted)
        path.copy_(torch.tensor([p + [-1] * (T - len(p)) for p in accepted], dtype=torch.int32))
        counts.copy_(torch.tensor([len(p) for p in accepted], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((kc, vc, ks, vs), want):
            assert np.array_equal(raw(got).numpy(), ref)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
