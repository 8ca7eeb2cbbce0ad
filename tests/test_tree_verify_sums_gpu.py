"""Verification of rows whose sum is not 1: equal to the definition, which takes Z = 1 at a node's first child, sums what is left
where there are draft probabilities, and takes rejected children's weights off where there are none."""
import pytest
import torch

from test_tree_verify_gpu import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [0.5, 0.97, 1 + 2.0 ** -12, 1.2])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("kind", ["star", "wide", "chain"])
def test_rows_that_do_not_sum_to_one(kind, drafts, size):
    for sequences in (3, 12):
        c = case([9] * sequences, 3001, drafts, kind, seed=sequences, peak=4.0)
        c["target"] = c["target"] * size
        check(c, run(c))
        if drafts:
            c["draft"] = c["draft"] * (2 - size)
            check(c, run(c))


def test_rows_cut_to_their_likeliest_tokens():
    """Nothing but the 40 likeliest tokens of each row, not normalised; children among them and beside them."""
    c = case([12] * 10, 5000, False, "star", seed=1, peak=3.0)
    top = c["target"].topk(40).indices
    c["target"] = torch.zeros_like(c["target"]).scatter_(1, top, c["target"].gather(1, top))
    check(c, run(c))
    c["r"].fill_(1 - 2.0 ** -24)
    check(c, run(c))


@pytest.mark.parametrize("size", [0.9, 1.1])
def test_children_keep_their_probabilities(size):
    """Frequencies over 20000 walks without draft probabilities, within 5 standard deviations: p(x) of the children's tokens, and
    of the others what is left of 1, in p's proportions."""
    V, B = 6, 20000
    gen = torch.Generator().manual_seed(3)
    p = torch.rand(V, generator=gen).softmax(0) ** 2
    p = p / p.sum() * size
    tokens = torch.zeros(B, 3, dtype=torch.int32)
    tokens[:, 1], tokens[:, 2] = 2, 4
    c = dict(trees=[[-1, 0, 0]] * B, target=p.expand(3 * B, V), draft=None, tokens=tokens.flatten(), r=torch.rand(3 * B, generator=gen),
             r_last=torch.rand(B, generator=gen))
    path, counts, token = run(c)
    second = torch.where(counts > 1, tokens.gather(1, path[:, 1:2].clamp_min(0).long())[:, 0], token)
    want = p.double()
    rest = torch.ones(V, dtype=torch.bool)
    rest[[2, 4]] = False
    want[rest] *= (1 - want[[2, 4]].sum()) / want[rest].sum()
    seen = torch.bincount(second, minlength=V).double() / B
    assert ((seen - want).abs() <= 5 * (want * (1 - want) / B).sqrt()).all(), (seen, want)
