"""Verification of drafted tokens from given random numbers, on the GPU: equal to the definition in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV, cu_of
from _tree import random_tree, verify

pytestmark = pytest.mark.gpu


def case(nodes, V, drafts, kind="wide", seed=0, padding=0, peak=3.0, stride=None):
    """A batch of trees with probabilities, tokens and random numbers (CPU tensors)."""
    r = np.random.RandomState(seed)
    trees = [random_tree(r, T, kind, min(padding, max(T - 1, 0))) for T in nodes]
    N = sum(nodes)
    gen = torch.Generator().manual_seed(seed)
    target = peak * torch.randn(N, V, generator=gen)
    draft = target + torch.randn(N, V, generator=gen)
    first = np.cumsum([0] + nodes)
    up = [first[n] + max(u, 0) for n, t in enumerate(trees) for u in t]
    q = draft.softmax(-1)
    if drafts:
        tokens = torch.multinomial(q[up], 1, generator=gen)[:, 0] if N else torch.zeros(0, dtype=torch.long)
    else:  # distinct among siblings most of the time
        tokens = torch.stack([q[u].topk(min(V, 5)).indices[i % min(V, 5)] for i, u in enumerate(up)]) if N else torch.zeros(0, dtype=torch.long)
    return dict(trees=trees, target=target.softmax(-1), draft=q if drafts else None, tokens=tokens.to(torch.int32),
                r=torch.rand(N, generator=gen), r_last=torch.rand(len(nodes), generator=gen))


def spread(x, stride, shift):
    """x on the GPU with rows `stride` apart."""
    if stride is None:
        return x.to(DEV)
    wide = torch.full((x.shape[0], stride), float("nan"), device=DEV)
    view = wide[:, :x.shape[1]]
    view.copy_(x)
    return view


def run(c, width=None, status=gdn.GDN_OK, strides=(None, None)):
    nodes = [len(t) for t in c["trees"]]
    width = max([1] + nodes) if width is None else width
    path = torch.full((len(nodes), width), 99, dtype=torch.int32, device=DEV)
    counts, token = (torch.full((len(nodes),), 99, dtype=torch.int32, device=DEV) for _ in range(2))
    parents = torch.tensor([u for t in c["trees"] for u in t], dtype=torch.int32, device=DEV)
    gdn.gdn_tree_verify(spread(c["target"], strides[0], 0), None if c["draft"] is None else spread(c["draft"], strides[1], 0),
                        c["tokens"].to(DEV), parents, c["r"].to(DEV), c["r_last"].to(DEV), path, counts, token,
                        cu_seqlens=None if len(set(nodes)) == 1 else cu_of(nodes))
    found = gdn.gdn_get_device_status()
    assert status is None or found == status
    return path.cpu(), counts.cpu(), token.cpu()


def check(c, got, but=()):
    path, counts, token = got
    first, close = 0, 1.0
    for n, parents in enumerate(c["trees"]):
        at = slice(first, first + len(parents))
        first += len(parents)
        if n in but:
            continue
        taken, nxt, near = verify(c["target"][at], None if c["draft"] is None else c["draft"][at], c["tokens"][at], parents,
                                  c["r"][at], c["r_last"][n])
        assert near > 1e-9, "the case is too close to a border to tell"
        assert counts[n] == len(taken) and path[n].tolist() == taken + [-1] * (path.shape[1] - len(taken))
        assert token[n] == nxt, (n, int(token[n]), nxt)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("nodes,kind,padding", [([1, 1], "wide", 0), ([6] * 40, "wide", 0), ([13, 1, 64, 0, 7, 30], "deep", 2),
                                                ([64, 64], "star", 3), ([20, 20], "forest", 0), ([12] * 6, "chain", 0)])
@pytest.mark.parametrize("V", [1, 2, 5, 31, 257, 1000, 4096, 50001])
def test_against_the_definition(V, nodes, kind, padding, drafts):
    c = case(nodes, V, drafts, kind, seed=V + len(nodes), padding=padding)
    check(c, run(c))


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("peak", [0.1, 12.0])
def test_flat_and_peaked_probabilities(peak, drafts):
    """All tokens about as likely, where a draw is one among many partial sums; and nearly one token, where drafts are taken."""
    c = case([40] * 5, 3001, drafts, "deep", seed=7, peak=peak)
    check(c, run(c))
    c = case([40] * 5, 3001, drafts, "deep", seed=8, peak=peak)
    c["r"].zero_()  # whatever the target may say at all is accepted
    check(c, run(c))
    c["r"].fill_(1 - 2.0 ** -24)  # and hardly anything
    c["r_last"].fill_(1 - 2.0 ** -24)
    got = run(c)
    assert (got[1] >= 1).all() and (got[2] >= 0).all()


@pytest.mark.parametrize("strides", [(1004, 1004), (1003, 1001), (1000, 1006), (4001, 1002)])
def test_rows_of_a_wider_tensor(strides):
    """Rows that begin at any element: target and draft rows whose 16-byte boundaries differ."""
    c = case([9] * 7, 1000, True, "wide", seed=5)
    check(c, run(c, strides=strides))
    c = case([9] * 7, 1000, False, "wide", seed=6)
    check(c, run(c, strides=strides, width=64))


@pytest.mark.parametrize("sequences", [2, 9])
@pytest.mark.parametrize("V", [3, 700, 20001, 40001, 70001, 131072])
def test_many_passes_over_a_row(V, sequences):
    """Siblings that are rejected one after another: each asks for the sum of what is left of the same rows."""
    c = case([7] * sequences, V, True, "star", seed=V)
    c["r"] = 0.9 + 0.1 * c["r"]
    c["r"].clamp_(max=1 - 2.0 ** -24)
    check(c, run(c))
    check(c, run(c, strides=(V + 1, V + 2)))


def test_a_large_vocabulary():
    for drafts in (True, False):
        c = case([3, 2], 1 << 20, drafts, seed=3)
        check(c, run(c))


def test_draws_at_the_ends():
    """r_last = 0 gives the first token that has weight, close to 1 the last; rejected tokens are never drawn."""
    V = 700
    p = torch.zeros(4, V)
    p[:, 100:600] = 1 / 500
    trees = [[-1, 0, 0, 0]]
    c = dict(trees=trees, target=p, draft=None, tokens=torch.tensor([0, 100, 599, 101], dtype=torch.int32),
             r=torch.full((4,), 0.999999), r_last=torch.zeros(1))
    path, counts, token = run(c)
    assert counts.item() == 1 and token.item() == 102  # 100 and 101 were rejected
    c["r_last"] = torch.full((1,), 1 - 2.0 ** -24)
    assert run(c)[2].item() == 598
    c["tokens"] = torch.tensor([0, 5, 5, 5], dtype=torch.int32)  # tokens that the target never says
    assert run(c)[2].item() == 599
    c["r"] = torch.zeros(4)
    assert run(c)[1].item() == 1  # 0 is not below 0


def test_nothing_left_of_the_weights():
    """Draft probabilities equal to the target's, and a child whose own probability there is 0, so that it is rejected: the
    draw is then from the target."""
    V = 64
    p = torch.zeros(2, V)
    p[:, 10:20] = 0.1
    c = dict(trees=[[-1, 0]], target=p, draft=p.clone(), tokens=torch.tensor([0, 3], dtype=torch.int32), r=torch.tensor([0.0, 0.5]),
             r_last=torch.tensor([0.349]))
    path, counts, token = run(c)
    assert counts.item() == 1 and token.item() == 13


def test_accepted_and_next_tokens_follow_the_target():
    """The frequencies of the token after the root over 20000 walks, within 5 standard deviations of the target's."""
    V, B = 6, 20000
    gen = torch.Generator().manual_seed(1)
    p, q = torch.rand(V, generator=gen).softmax(0) ** 2, torch.rand(V, generator=gen)
    p, q = p / p.sum(), q / q.sum()
    for drafts in (True, False):
        tree = [-1, 0, 0]
        tokens = torch.zeros(B, 3, dtype=torch.int32)
        if drafts:
            tokens[:, 1:] = torch.multinomial(q, 2 * B, True, generator=gen).view(B, 2).to(torch.int32)
        else:
            tokens[:, 1], tokens[:, 2] = 2, 4
        c = dict(trees=[tree] * B, target=p.expand(3 * B, V), draft=q.expand(3 * B, V) if drafts else None, tokens=tokens.flatten(),
                 r=torch.rand(3 * B, generator=gen), r_last=torch.rand(B, generator=gen))
        path, counts, token = run(c)
        second = torch.where(counts > 1, tokens.gather(1, path[:, 1:2].clamp_min(0).long())[:, 0], token)
        seen = torch.bincount(second, minlength=V).double() / B
        dev = (p.double() * (1 - p.double()) / B).sqrt()
        assert ((seen - p.double()).abs() <= 5 * dev).all(), (seen, p)


def test_flagged():
    """A token outside of the vocabulary, a parent after its node, too many nodes, a row without weight: flagged, that sequence only."""
    c = case([6] * 5, 300, True, seed=2)
    c["tokens"][7] = 300
    c["tokens"][14] = -1
    c["trees"][3][2] = 5
    c["trees"][4][0] = 0
    got = run(c, status=gdn.GDN_ERR_DEVICE_CHECK)
    check(c, got, but=(1, 2, 3, 4))
    assert got[1][4] == 0 and got[2][4] == -1 and (got[0][4] == -1).all()
    for n, node in ((1, 1), (2, 2), (3, 2)):
        assert node not in got[0][n] and got[1][n] >= 1 and got[2][n] >= 0
    c = case([3, 65, 4], 100, True, seed=2)
    got = run(c, status=gdn.GDN_ERR_DEVICE_CHECK, width=70)
    check(c, got, but=(1,))
    assert got[1][1] == 0 and got[2][1] == -1
    for bad in (0.0, float("nan"), float("inf")):
        c = case([2, 2], 100, True, seed=2)
        c["target"][2:] = bad
        c["draft"][2:] = 0.01
        c["r"].fill_(0.5)
        got = run(c, status=gdn.GDN_ERR_DEVICE_CHECK)
        check(c, got, but=(1,))
        assert got[2][1] == -1
    c = case([9, 4], 100, True, seed=2)
    got = run(c, status=gdn.GDN_ERR_DEVICE_CHECK, width=4)  # a path that does not fit
    check(c, got, but=(0,))
    assert got[1][0] == 0


def test_idle_rows():
    c = case([5] * 3, 500, True, seed=4)
    c["trees"][1] = [-2] * 5
    got = run(c)
    check(c, got)
    assert got[1][1] == 0 and got[2][1] == -1


def test_a_captured_graph_and_another_stream():
    c = case([7] * 9, 2000, True, seed=12)
    dev = {n: c[n].to(DEV) for n in ("target", "draft", "tokens", "r", "r_last")}
    parents = torch.tensor([u for t in c["trees"] for u in t], dtype=torch.int32, device=DEV)
    path = torch.zeros(9, 7, dtype=torch.int32, device=DEV)
    counts, token = (torch.zeros(9, dtype=torch.int32, device=DEV) for _ in range(2))
    call = lambda: gdn.gdn_tree_verify(dev["target"], dev["draft"], dev["tokens"], parents, dev["r"], dev["r_last"], path, counts, token)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    check(c, (path.cpu(), counts.cpu(), token.cpu()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c2 = case([7] * 9, 2000, True, seed=13)
    for n in dev:
        dev[n].copy_(c2[n])
    parents.copy_(torch.tensor([u for t in c2["trees"] for u in t], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(c2, (path.cpu(), counts.cpu(), token.cpu()))


@pytest.mark.parametrize("sequences", [1, 20])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(sequences, monkeypatch):
    """GDN_TEST_WAIT_CYCLES shortens the limit of the kernel's waits for what its CTAs send one another."""
    c = case([9] * sequences, 5001, True, "star", seed=3)
    monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", "1")
    path, counts, token = run(c, status=None)
    monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
    assert (counts[counts != 0] > 0).all() and (token >= -1).all()
    check(c, run(c))
