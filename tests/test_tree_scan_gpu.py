"""The gated delta rule over trees of drafted tokens, and along accepted paths, on the GPU, against the token recurrence in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV, DTYPES, cu_of
from _tree import advance, assert_scan, assert_states, paths, random_tree, tree_scan

pytestmark = pytest.mark.gpu

# nodes of each sequence, kind, padding nodes
TREES = {
    "one": ([1, 1, 1], "wide", 0),
    "few": ([5, 5], "wide", 0),
    "packed": ([17, 1, 64, 33, 8, 0, 16], "deep", 1),
    "wide": ([63], "wide", 2),
    "chain": ([64], "chain", 0),
    "star": ([40], "star", 5),
    "forest": ([24, 24], "forest", 3),
}
DIMS = [(1, 2, 128, 128), (2, 2, 64, 32), (1, 3, 32, 128), (2, 4, 128, 64), (1, 1, 32, 32), (1, 2, 64, 64)]


def flat(trees):
    return torch.tensor([u for p in trees for u in p], dtype=torch.int32, device=DEV)


def inputs(trees, Hk, Hv, dk, dv, dtype, seed=0, gate=1.0):
    gen = torch.Generator().manual_seed(seed)
    N = sum(map(len, trees))
    dt = DTYPES[dtype]
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = -gate * torch.nn.functional.softplus(rand(N, Hv))
    return [rand(N, Hk, dk).to(dt), rand(N, Hk, dk).to(dt), rand(N, Hv, dv).to(dt), g.to(dt), rand(N, Hv).to(dt),
            0.3 * rand(len(trees), Hv, dv, dk)]


def make(name, seed=1):
    nodes, kind, padding = TREES[name]
    r = np.random.RandomState(seed)
    return [random_tree(r, T, kind, min(padding, max(T - 1, 0))) for T in nodes]


def cu(trees):
    new = [len(p) for p in trees]
    return None if len(set(new)) == 1 else cu_of(new)


def scan(x, trees, **kw):
    q, k, v, g, b, S = (t.to(DEV) for t in x)
    before = S.clone()
    out = torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV)
    gdn.gdn_tree_scan(q, k, v, g, b, S, flat(trees), out, cu_seqlens=cu(trees), **kw)
    assert torch.equal(S, before)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", DIMS)
@pytest.mark.parametrize("name", sorted(TREES))
def test_scan(name, Hk, Hv, dk, dv, dtype):
    trees = make(name)
    x = inputs(trees, Hk, Hv, dk, dv, dtype)
    out = scan(x, trees)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert_scan(out, *tree_scan(*x, trees), dk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [1e-3, 6.0])
def test_scan_slow_and_fast_gates(gate, dtype):
    """Gates that forget nothing, and gates whose sum along a path is several hundred."""
    for name in ("chain", "packed"):
        trees = make(name)
        x = inputs(trees, 1, 2, 128, 128, dtype, seed=3, gate=gate)
        assert_scan(scan(x, trees), *tree_scan(*x, trees), 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** 20])
def test_scan_sizes_of_inputs(size, dtype):
    """Small and large keys, values and states (the keys' norm hides their size; 1e-6 is added to its square)."""
    trees = make("few")
    q, k, v, g, b, S = inputs(trees, 2, 4, 128, 128, dtype, seed=4)
    x = [(q * size).to(q.dtype), (k * size).to(k.dtype), (v * size).to(v.dtype), g, b, S * size]
    assert_scan(scan(x, trees), *tree_scan(*x, trees), 128)


def test_scan_of_one_node_is_the_decode_step():
    trees = [[-1]] * 9
    x = inputs(trees, 2, 4, 128, 128, "bf16", seed=5)
    out = scan(x, trees)
    q, k, v, g, b, S = (t.to(DEV) for t in x)
    step = torch.empty_like(out)
    gdn.gdn_decode_step(q, k, v, g, b, S, step)
    # the scan's value a and the step's b differ by at most 2^-13 M before they are rounded (_tree.py: 2^-14 M for a, less for b);
    # each is then rounded to bf16, off by at most 2^-8 of it: |out - step| <= 2^-13 M + 2^-8 |a| + 2^-8 |b|, and |a| <= |b| + 2^-13 M
    # and |b| <= |step| / (1 - 2^-8), so at most 2^-12 M + 2^-7 (1 + 2^-7) |step|
    _, mag, _ = tree_scan(*x, trees)
    diff = (out.double() - step.double()).abs().cpu().numpy()
    assert (diff <= 2.0 ** -12 * mag + 2.0 ** -7 * (1 + 2.0 ** -7) * step.double().abs().cpu().numpy()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", DIMS)
@pytest.mark.parametrize("name", sorted(TREES))
def test_advance(name, Hk, Hv, dk, dv, dtype):
    trees = make(name)
    x = inputs(trees, Hk, Hv, dk, dv, dtype, seed=2)
    r = np.random.RandomState(7)
    ways = [[p for p in paths(t) if p] for t in trees]
    accepted = [w[r.randint(len(w))] if w and n % 4 != 3 else [] for n, w in enumerate(ways)]
    if name == "chain":
        accepted = [ways[0][-1]]
    S = x[5].to(DEV)
    out = torch.full_like(S, float("nan"))
    step(x, trees, accepted, S, out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    ref, mag = advance(*x[1:], [len(t) for t in trees], accepted)
    assert_states(out, ref, mag, accepted, dk)
    for n, p in enumerate(accepted):
        if not p:
            assert torch.equal(out[n], S[n])
    step(x, trees, accepted, S, S)  # in place
    assert torch.equal(S, out)


def tables(accepted, width=None):
    width = max([1] + [len(p) for p in accepted]) if width is None else width
    path = torch.tensor([p + [-1] * (width - len(p)) for p in accepted], dtype=torch.int32, device=DEV)
    return path, torch.tensor([len(p) for p in accepted], dtype=torch.int32, device=DEV)


def step(x, trees, accepted, S, out, **kw):
    _, k, v, g, b, _ = (t.to(DEV) for t in x)
    path, counts = tables(accepted)
    gdn.gdn_tree_advance(k, v, g, b, S, out, path, counts, cu_seqlens=cu(trees), **kw)


def test_pools_and_padding():
    """States in a pool: the entries that sequences name are read and advanced, all others left; a negative slot is an idle row."""
    trees = make("few") * 3
    x = inputs(trees, 2, 4, 128, 128, "bf16", seed=6)
    slots = torch.tensor([7, -1, 0, 3, -5, 9], dtype=torch.int32)
    pool = torch.randn(10, 4, 128, 128, generator=torch.Generator().manual_seed(1))
    q, k, v, g, b, _ = (t.to(DEV) for t in x)
    out = torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV)
    dev = pool.to(DEV)
    gdn.gdn_tree_scan(q, k, v, g, b, dev, flat(trees), out, slots=slots.to(DEV))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK and torch.equal(dev.cpu(), pool)
    states = pool[slots.clamp_min(0).long()]
    ref, mag, length = tree_scan(*x[:5], states, trees)
    out = out.view(6, 5, 4, 128)
    live = [n for n in range(6) if slots[n] >= 0]
    assert not out[[1, 4]].any()
    view = lambda a: a.reshape(6, 5, 4, 128)[live]  # noqa: E731
    assert_scan(out[live].flatten(0, 1), view(ref).reshape(-1, 4, 128), view(mag).reshape(-1, 4, 128),
                length.reshape(6, 5)[live].reshape(-1), 128)
    accepted = [paths(t)[-1] for t in trees]
    step(x, trees, accepted, dev, dev, slots=slots.to(DEV))
    ref, mag = advance(*x[1:5], states, [5] * 6, accepted)
    got = dev.cpu()
    for n in live:
        assert_states(got[slots[n]][None], ref[n:n + 1], mag[n:n + 1], accepted[n:n + 1], 128)
    rest = [i for i in range(10) if i not in slots.tolist()]
    assert torch.equal(got[rest], pool[rest])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_flagged(dtype):
    """A slot outside of the pool, bad parents, counts and nodes, 65 nodes: flagged, and only that sequence is concerned."""
    trees = make("few") * 2
    x = inputs(trees, 2, 4, 128, 128, dtype, seed=8)
    q, k, v, g, b, S = (t.to(DEV) for t in x)
    slots = torch.tensor([0, 4, 2, 3], dtype=torch.int32, device=DEV)
    out = torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV)
    gdn.gdn_tree_scan(q, k, v, g, b, S, flat(trees), out, slots=slots)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert not out[5:10].any() and torch.isfinite(out).all()
    bent = [list(t) for t in trees]
    bent[1][2] = 4
    assert_scan(scan(x, bent), *tree_scan(*x, bent), 128)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    for path, counts in (([[0, 1], [0, 5], [0, -1], [0, 2]], [2, 2, 2, 1]), ([[0, 1]] * 4, [2, 3, -1, 1])):
        out = torch.full_like(S, float("nan"))
        gdn.gdn_tree_advance(k, v, g, b, S, out, torch.tensor(path, dtype=torch.int32, device=DEV),
                             torch.tensor(counts, dtype=torch.int32, device=DEV))
        assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
        good = [path[0][:counts[0]], [], [], path[3][:counts[3]]]
        ref, mag = advance(*x[1:], [5] * 4, good)
        assert_states(out, ref, mag, good, 128)
        assert torch.equal(out[1:3], S[1:3])
    many = [random_tree(np.random.RandomState(1), T) for T in (3, 65, 2)]
    x = inputs(many, 1, 2, 64, 64, dtype)
    out = scan(x, many)
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert torch.isnan(out[3:68]).all() and torch.isfinite(out[:3]).all() and torch.isfinite(out[68:]).all()


def test_values_that_are_not_finite_stay_on_their_paths():
    """Values of a node that are NaN or infinite: no effect on nodes whose path does not hold it."""
    trees = make("wide") + make("packed")
    for dtype in ("bf16", "f32"):
        x = inputs(trees, 1, 2, 128, 128, dtype, seed=9)
        clean = scan(x, trees)
        for bad in (float("nan"), float("inf")):
            v = x[2].clone()
            v[4] = bad
            out = scan([*x[:2], v, *x[3:]], trees)
            off = [i for i in range(v.shape[0]) if i >= 63 or 4 not in paths(trees[0])[i]]
            assert torch.equal(out[off], clean[off])
            on = [i for i in range(63) if i not in off]
            assert not torch.isfinite(out[on]).any()


@pytest.mark.parametrize("which", [0, 1])
def test_keys_and_queries_that_are_not_finite_stay_on_their_paths(which):
    """A key that is not finite concerns the nodes whose path holds it, a query its own node only."""
    trees = make("wide") + make("packed")
    for dtype in ("bf16", "f32"):
        x = inputs(trees, 1, 2, 128, 128, dtype, seed=9)
        clean = scan(x, trees)
        y = x[which].clone()
        y[4, 0, 3:5] = float("nan")
        out = scan([y if i == which else t for i, t in enumerate(x)], trees)
        on = [i for i in range(63) if (4 in paths(trees[0])[i] if which else i == 4)]
        off = [i for i in range(y.shape[0]) if i not in on]
        assert torch.equal(out[off], clean[off])
        assert torch.isnan(out[on]).all()


def test_a_gate_that_is_not_finite_stays_on_its_paths():
    trees = make("wide") + make("packed")
    for dtype in ("bf16", "f32"):
        x = inputs(trees, 1, 2, 128, 128, dtype, seed=9)
        clean = scan(x, trees)
        for which in (3, 4):
            y = x[which].clone()
            y[4] = float("nan")
            out = scan([y if i == which else t for i, t in enumerate(x)], trees)
            on = [i for i in range(63) if 4 in paths(trees[0])[i]]
            off = [i for i in range(y.shape[0]) if i not in on]
            assert torch.equal(out[off], clean[off])
            assert torch.isnan(out[on]).all()


@pytest.mark.parametrize("T", [5, 20, 50])
@pytest.mark.parametrize("cycles", ["1", "3000"])
@pytest.mark.parametrize("dv", [64, 128])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(T, cycles, dv, monkeypatch):
    """GDN_TEST_WAIT_CYCLES shortens the limit of the kernel's waits for its copies."""
    trees = [random_tree(np.random.RandomState(n), T) for n in range(40)]
    x = inputs(trees, 4, 8, 128, dv, "bf16", seed=14)
    q, k, v, g, b, S = (t.to(DEV) for t in x)
    parents, out = flat(trees), torch.empty_like(v)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", cycles)
    torch.zeros(1 << 29, dtype=torch.uint8, device=DEV)  # (larger than L2)
    gdn.gdn_tree_scan(q, k, v, g, b, S, parents, out)
    torch.cuda.synchronize()
    status = gdn.gdn_get_device_status()
    # (a wait sleeps in the hardware between looks at its limit, so 3000 cycles may pass unnoticed)
    assert status == gdn.GDN_ERR_DEVICE_CHECK or (cycles == "3000" and status == gdn.GDN_OK)
    monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
    out.fill_(float("nan"))
    gdn.gdn_tree_scan(q, k, v, g, b, S, parents, out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    first = [t[:T] for t in x[:5]] + [x[5][:1]]
    assert_scan(out[:T], *tree_scan(*first, trees[:1]), 128)
    assert torch.equal(out, scan(x, trees))


def test_a_tree_in_pieces():
    """Scan, advance along a path, and the same path token by token by the decode step: one state."""
    trees = make("few")
    x = inputs(trees, 2, 4, 128, 128, "bf16", seed=10)
    accepted = [paths(t)[-1] for t in trees]
    S = x[5].to(DEV)
    step(x, trees, accepted, S, S)
    q, k, v, g, b, D = (t.to(DEV) for t in x)
    for n, p in enumerate(accepted):
        for u in p:
            o = torch.empty(1, 4, 128, dtype=torch.bfloat16, device=DEV)
            at = slice(5 * n + u, 5 * n + u + 1)
            gdn.gdn_decode_step(*(y[at].clone() for y in (q, k, v, g, b)), D[n:n + 1], o)  # (16-byte boundaries)
    ref, mag = advance(*x[1:], [5, 5], accepted)
    assert_states(S, ref, mag, accepted, 128)
    assert_states(D, ref, mag, accepted, 128)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_empty_pool(dtype, dk, dv):
    """No state at all, and idle rows only: outputs are zeros, nothing is flagged."""
    trees = make("few")
    q, k, v, g, b, _ = (t.to(DEV) for t in inputs(trees, 2, 4, dk, dv, dtype))
    S = torch.empty(0, 4, dv, dk, device=DEV)
    out = torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV)
    slots = torch.tensor([-1, -2], dtype=torch.int32, device=DEV)
    gdn.gdn_tree_scan(q, k, v, g, b, S, flat(trees), out, slots=slots)
    path, counts = tables([[0], [0, 1]])
    gdn.gdn_tree_advance(k, v, g, b, S, S, path, counts, slots=slots)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert not out.any()


def test_calls_at_once():
    """Several calls in flight on streams of their own share nothing."""
    sets = []
    for i in range(4):
        trees = [random_tree(np.random.RandomState(10 * i + n), T) for n, T in enumerate([7, 16, 30, 64][i:] + [5, 64, 33][:i])]
        x = inputs(trees, 4, 8, 128, 128, "bf16", seed=20 + i)
        sets.append((trees, x, [t.to(DEV) for t in x], flat(trees), cu(trees), scan(x, trees)))
    outs = [[torch.empty_like(s[2][2]) for _ in range(10)] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for j in range(10):
        for s, (trees, x, (q, k, v, g, b, S), parents, c, _), o in zip(streams, sets, outs):
            gdn.gdn_tree_scan(q, k, v, g, b, S, parents, o[j], cu_seqlens=c, stream=s)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    for (*_, want), o in zip(sets, outs):
        assert all(torch.equal(y, want) for y in o)


def test_a_captured_graph_and_another_stream():
    trees = make("forest")
    x = inputs(trees, 2, 4, 128, 128, "bf16", seed=11)
    q, k, v, g, b, S = (t.to(DEV) for t in x)
    out, new, parents = torch.empty_like(v), torch.empty_like(S), flat(trees)
    path, counts = tables([paths(t)[0] for t in trees], 24)

    def call():
        gdn.gdn_tree_scan(q, k, v, g, b, S, parents, out)
        gdn.gdn_tree_advance(k, v, g, b, S, new, path, counts)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert_scan(out, *tree_scan(*x, trees), 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    trees = [random_tree(np.random.RandomState(50), 24, "deep", 2) for _ in trees]
    accepted = [max(paths(t), key=len) for t in trees]
    parents.copy_(flat(trees))
    for a, c in zip((path, counts), tables(accepted, 24)):
        a.copy_(c)
    graph.replay()
    torch.cuda.synchronize()
    assert_scan(out, *tree_scan(*x, trees), 128)
    ref, mag = advance(*x[1:], [24] * 2, accepted)
    assert_states(new, ref, mag, accepted, 128)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


def test_many_sequences():
    """More states than CTAs at once, of mixed sizes: each as alone, bit for bit, and the same twice."""
    r = np.random.RandomState(3)
    trees = [random_tree(r, int(T), "wide") for T in r.randint(0, 65, 150)]
    x = inputs(trees, 4, 8, 128, 128, "bf16", seed=12)
    out = scan(x, trees)
    assert torch.equal(out, scan(x, trees))
    first = np.cumsum([0] + [len(t) for t in trees])
    for n in (0, 31, 149):
        at = slice(first[n], first[n + 1])
        if len(trees[n]):
            one = [t[at] for t in x[:5]] + [x[5][n:n + 1]]
            assert_scan(out[at], *tree_scan(*one, trees[n:n + 1]), 128)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("gate", [-float("inf"), "lowest", -1e20, -1e7, -300.0])
def test_gates_that_leave_nothing(gate, dv, dtype):
    """Gates so low that a node's state is what it writes itself: what lies below keeps its own decays."""
    trees = make("wide") + make("packed")
    x = list(inputs(trees, 1, 2, 128, dv, dtype, seed=21))
    g = x[3].clone()
    for node in (1, 4, 9, 70):
        g[node] = torch.finfo(g.dtype).min if gate == "lowest" else gate
    x[3] = g
    out = scan(x, trees)
    assert torch.isfinite(out).all()
    assert_scan(out, *tree_scan(*x, trees), 128)
