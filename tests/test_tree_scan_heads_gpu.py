"""The gated delta rule over trees for many heads of every size: CTAs that take several heads one after another, with idle rows
between them, against the token recurrence in 64 bits; and keys and queries of the largest sizes that the calls take."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV
from _tree import advance, assert_scan, assert_states, paths, random_tree, tree_scan
from test_tree_scan_gpu import flat, inputs, scan, step

pytestmark = pytest.mark.gpu

SIZES = [(32, 32), (32, 64), (32, 128), (64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)]


def some(x, states, trees, n):
    """Sequence n's inputs and state."""
    first = sum(len(t) for t in trees[:n])
    at = slice(first, first + len(trees[n]))
    return at, [t[at] for t in x[:5]] + [states[n:n + 1]]


@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [3, 13, 16, 40, 64])
def test_many_heads(T, dk, dv):
    """1960 heads for at most 456 CTAs, from a pool of states, with idle rows: each sequence as alone, bit for bit."""
    B, Hk, Hv = 245, 4, 8
    r = np.random.RandomState(T + dk + dv)
    trees = [random_tree(r, T, ["wide", "deep", "chain"][n % 3], min(n % 4, T - 1)) for n in range(B)]
    x = inputs(trees, Hk, Hv, dk, dv, "bf16", seed=T)
    slots = torch.from_numpy(r.permutation(B).astype(np.int32))
    slots[::7] = -1
    q, k, v, g, b, pool = (t.to(DEV) for t in x)
    out = [torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV) for _ in range(2)]
    for o in out:
        gdn.gdn_tree_scan(q, k, v, g, b, pool, flat(trees), o, slots=slots.to(DEV))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.equal(out[0], out[1])
    states = x[5][slots.clamp_min(0).long()]
    for n in range(B):
        at, one = some(x, states, trees, n)
        if slots[n] < 0:
            assert not out[0][at].any()
        elif n % 20 == 3 or n > B - 4:
            assert torch.equal(out[0][at], scan(one, trees[n:n + 1]))
            if n % 60 == 3 or n > B - 3:
                assert_scan(out[0][at], *tree_scan(*one, trees[n:n + 1]), dk)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_many_heads_of_packed_trees(dk, dv):
    B, Hk, Hv = 150, 2, 8
    r = np.random.RandomState(dk + dv)
    trees = [random_tree(r, int(T), "deep", 0) for T in r.randint(0, 65, B)]
    trees[-1] = random_tree(r, 64, "chain")
    x = inputs(trees, Hk, Hv, dk, dv, "bf16", seed=5)
    out = scan(x, trees)
    assert torch.equal(out, scan(x, trees))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    for n in (0, 37, 74, 110, 148, 149):
        at, one = some(x, x[5], trees, n)
        if len(trees[n]):
            assert_scan(out[at], *tree_scan(*one, trees[n:n + 1]), dk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (32, 32)])
def test_the_largest_keys_and_queries(dk, dv, dtype):
    """Norms just below 2^60, of one key, and of all."""
    for which in ("all", "some"):
        trees = [random_tree(np.random.RandomState(1), 30, "chain"), random_tree(np.random.RandomState(2), 30, "wide")]
        x = inputs(trees, 2, 4, dk, dv, dtype, seed=17)
        for i in (0, 1):
            size = 0.99 * 2.0 ** 60 / x[i].float().norm(dim=-1, keepdim=True)
            if which == "some":
                size[::3] = 1.0
            x[i] = (x[i].float() * size).to(x[i].dtype)
            assert x[i].double().norm(dim=-1).max() < 2.0 ** 60
        assert_scan(scan(x, trees), *tree_scan(*x, trees), dk)
        accepted = [max(paths(t), key=len) for t in trees]
        S = x[5].to(DEV)
        new = torch.full_like(S, float("nan"))
        step(x, trees, accepted, S, new)
        assert_states(new, *advance(*x[1:], [30, 30], accepted), accepted, dk)
        assert gdn.gdn_get_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("size", [2e19, 1e30, 3e38])
@pytest.mark.parametrize("which", [0, 1])
def test_keys_and_queries_beyond_these_stay_on_their_paths(which, size, dv, dtype):
    """Keys too large for fp32's products concern the nodes whose paths hold them, queries their own nodes."""
    trees = [random_tree(np.random.RandomState(3), 40, "deep"), random_tree(np.random.RandomState(4), 40, "wide")]
    x = inputs(trees, 1, 2, 128, dv, dtype, seed=9)
    clean = scan(x, trees)
    way = max(paths(trees[0]), key=len)
    large = way[2::2]
    y = x[which].clone()
    y[large] = torch.sign(y[large].float()).to(y.dtype) * size
    out = scan([y if i == which else t for i, t in enumerate(x)], trees)
    on = [i for i in range(40) if (set(large) & set(paths(trees[0])[i]) if which else i in large)]
    off = [i for i in range(80) if i not in on]
    assert len(on) >= len(large) and torch.equal(out[off], clean[off])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
