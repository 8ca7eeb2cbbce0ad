"""Verification of drafted tokens where a decision is close to its border: equal to the definition in 64 bits. Random numbers are
fp32, so the closest to a border are up to 2^-25 (3e-8) from it, relative to the sum or the weight that they are compared with; sums
and weights kept to 48 bits (2^-47 a step) tell all of those apart that the reference's own sums (V 2^-53 at most) do."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV

pytestmark = pytest.mark.gpu

NEAR, FAR = 1e-9, 1e-7  # distances of the cases here from their borders


def steps_around(x, r, size):
    """For each border x in (0, 1) a random one of the closest fp32 numbers that are NEAR to FAR from it, in units of size (NaN:
    there is none)."""
    mid, score = x.astype(np.float32), np.zeros(x.shape)
    out = np.full(x.shape, np.nan, np.float32)
    for off in range(-2, 3):
        y = mid.copy()
        for _ in range(abs(off)):
            y = np.nextafter(y, np.float32(2.0 if off > 0 else -1.0))
        d = np.abs(y.astype(np.float64) - x) / size
        s = np.where((d > NEAR) & (d < FAR) & (y >= 0) & (y < 1), r.rand(*x.shape), 0.0)
        out, score = np.where(s > score, y, out), np.maximum(s, score)
    return out


def probabilities(V, peak, seed):
    gen = torch.Generator().manual_seed(seed)
    target = peak * torch.randn(V, generator=gen)
    return target.softmax(-1), (target + torch.randn(V, generator=gen)).softmax(-1)


def rows(p, n):
    return p.to(DEV).expand(n, -1).contiguous()


def verify(p, q, T, tokens, parents, r, r_last):
    B = len(r_last)
    path = torch.full((B, T), 99, dtype=torch.int32, device=DEV)
    counts, token = (torch.full((B,), 99, dtype=torch.int32, device=DEV) for _ in range(2))
    on = lambda x, t: torch.as_tensor(x).to(t).to(DEV).flatten().contiguous()  # noqa: E731
    gdn.gdn_tree_verify(rows(p, B * T), None if q is None else rows(q, B * T), on(tokens, torch.int32), on(parents, torch.int32),
                        on(r, torch.float32), on(r_last, torch.float32), path, counts, token)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    return path.cpu().numpy(), counts.cpu().numpy(), token.cpu().numpy()


@pytest.mark.parametrize("B", [8, 250])
@pytest.mark.parametrize("rejected", [0, 1, 3])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("V,peak", [(4099, 1.0), (200003, 0.3)])
def test_draws(V, peak, drafts, rejected, B):
    """The next token, after a number of rejected children, drawn by numbers next to partial sums of what is left."""
    if rejected == 0 and not drafts:
        V -= 1
    p, q = probabilities(V, peak, seed=V + rejected)
    r = np.random.RandomState(B + rejected)
    p64, q64 = p.double().numpy(), q.double().numpy()
    T = 1 + rejected
    tokens = np.zeros((B, T), np.int64)
    # the same of all sequences: one row of weights is left
    tokens[:, 1:] = r.choice(np.nonzero(q64 > 1.2 * p64)[0] if drafts else V, rejected, replace=False)
    parents = np.array([-1] + [0] * rejected)
    w, Z = p64.copy(), 1.0
    hard = np.float32(1 - 2.0 ** -24)
    for x in tokens[0, 1:]:
        one = np.zeros_like(w)
        one[x] = 1.0
        left = hard * Z * (q64[x] if drafts else 1.0)
        assert left > 1.001 * w[x] or w[x] == 0  # rejected, and not close
        if drafts:
            w = np.maximum(w - Z * q64, 0)
            Z = w.sum()
        else:
            Z, w = Z - w[x], w * (1 - one)
    sums = np.cumsum(w)
    at = r.choice(np.nonzero((w > 0) & (sums / sums[-1] > 0.05) & (sums / sums[-1] < 0.95))[0], 20 * B)
    last = steps_around(sums[at] / sums[-1], r, 1.0)
    last = last[~np.isnan(last)][:B]
    assert len(last) == B
    draw = last.astype(np.float64) * sums[-1]
    want = np.searchsorted(sums, draw, side="right")
    close = np.minimum(np.abs(sums[want] - draw), np.abs(draw - sums[want - 1])) / sums[-1]
    assert close.min() > 0.9 * NEAR and np.median(close) < FAR
    path, counts, token = verify(p, q if drafts else None, T, tokens, np.tile(parents, (B, 1)), np.full((B, T), hard), last)
    assert (counts == 1).all() and (path[:, 0] == 0).all()
    wrong = np.nonzero(token != want)[0]
    assert len(wrong) == 0, f"{len(wrong)} of {B}: {token[wrong[:5]]} for {want[wrong[:5]]}, {close[wrong[:5]]} from the border"


@pytest.mark.parametrize("B", [8, 250])
@pytest.mark.parametrize("rejected", [0, 1, 2])
@pytest.mark.parametrize("drafts", [True, False])
def test_acceptances(drafts, rejected, B):
    """A child after a number of rejected ones, whose random number is next to where it would just be accepted."""
    V = 4001
    p, q = probabilities(V, 1.0, seed=5 + rejected)
    r = np.random.RandomState(B + rejected)
    p64, q64 = p.double().numpy(), q.double().numpy()
    T = 2 + rejected
    hard = np.float32(1 - 2.0 ** -24)
    first = r.choice(np.nonzero(q64 > 1.2 * p64)[0] if drafts else V, rejected, replace=False)
    w, Z = p64.copy(), 1.0
    for x in first:
        assert hard * Z * (q64[x] if drafts else 1.0) > 1.001 * w[x]
        if drafts:
            w = np.maximum(w - Z * q64, 0)
            Z = w.sum()
        else:
            Z -= w[x]
            w[x] = 0
    ratio = w / (Z * (q64 if drafts else 1.0))  # a child is accepted if its number is below
    ok = np.nonzero((ratio > (0.05 if drafts else 1e-5)) & (ratio < 0.95))[0]
    x = r.choice(ok, 20 * B)
    num = steps_around(ratio[x], r, ratio[x])
    x, num = x[~np.isnan(num)][:B], num[~np.isnan(num)][:B]
    assert len(x) == B
    tokens, rn = np.zeros((B, T), np.int64), np.full((B, T), hard)
    tokens[:, 1:-1], tokens[:, -1], rn[:, -1] = first, x, num
    want = num.astype(np.float64) < ratio[x]
    assert 0.1 < want.mean() < 0.9
    path, counts, token = verify(p, q if drafts else None, T, tokens, np.tile([-1] + [0] * (T - 1), (B, 1)), rn, np.full(B, 0.5))
    wrong = np.nonzero((counts == 2) != want)[0]
    assert len(wrong) == 0, f"{len(wrong)} of {B}, {num[wrong[:5]] / ratio[x[wrong[:5]]] - 1} from the border"
    assert (path[want, 1] == T - 1).all()
