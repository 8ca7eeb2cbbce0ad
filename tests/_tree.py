"""Trees of drafted tokens and the formulas on them in 64 bits (numpy and torch on the CPU), apart from the library.

Tolerances, from the number formats (u = 2^-24 for fp32):

* attention: those of _kv.py; a tree only changes which positions a row sees.
* scan, out: with bf16 inputs the states enter the products with 16 bits (relative 2^-17 of each element, at most), and
  the sum over a path, of corrections u and coefficients rounded to 16 bits, at most 3 * 2^-17 of its terms; the fp32
  sums add (dk + 64) u of theirs. All of that is bounded by 2^-14 of the terms' magnitudes,
      M_t = e^{G_t} |S_0| |qh_t| + sum_s e^{G_t-G_s} |kh_s . qh_t| U_s,   U_t = beta_t (|v_t| + e^{G_t} |S_0| |kh_t| + sum ..),
  plus the output's own rounding: bf16 has 8 significant bits, so values in [2^e, 2^(e+1)) are 2^(e-7) apart and a rounding
  is off by at most half of that, 2^(e-8), which is at most 2^-8 of the value. With fp32 inputs everything is fp32: each of
  the sums has at most dk + 64 terms, whose magnitudes are in M_t, and along a path of L nodes the errors of the
  corrections, which M_t multiplies up as they are, add up L times: (dk + 64 + 64) (L + 1) u M_t.
* advance, state: fp32 sums of at most dk + 2 L terms: |S - ref| <= (dk + 64) (L + 1) u of the magnitudes
      e^{G} |S_0| + sum_s e^{G-G_s} U_s |kh_s|.
* verify: whole numbers, equal. (Cases keep every decision further than 1e-9 from its border.)
* keep: bytes, equal.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24


def random_tree(rng, T, kind="wide", padding=0):
    """parents of T nodes; the last `padding` are padding."""
    p = [-1]
    for t in range(1, T):
        if kind == "chain":
            p.append(t - 1)
        elif kind == "star":
            p.append(0)
        elif kind == "forest":  # several roots
            p.append(int(rng.randint(-1, t)))
        else:
            p.append(int(rng.randint(0, t)) if kind == "wide" else int(rng.randint(max(0, t - 3), t)))
    p = p[:T]
    for t in range(max(0, T - padding), T):
        p[t] = -2 - int(rng.randint(0, 3))
    return p


def paths(parents):
    """The nodes from the root to each, none for padding and what descends from it."""
    out = []
    for t, u in enumerate(parents):
        if u == -1:
            out.append([t])
        elif 0 <= u < t and out[u]:
            out.append(out[u] + [t])
        else:
            out.append([])
    return out


def tree_attention(case, q, trees, scale):
    """(out, sum_j p_j |v_j|, e_s), as _kv.reference has them; case: _kv.Paged; trees: parents of every sequence."""
    q = q.double().numpy()
    G = q.shape[1] // case.Hkv
    out, mag, err = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    first = 0
    for n, parents in enumerate(trees):
        T, base = len(parents), case.lens[n] - len(parents)
        for h in range(case.Hkv):
            k, v = case.sequence("k", n, h), case.sequence("v", n, h)
            for t, path in enumerate(paths(parents)):
                if base + t < 0:
                    continue
                seen = list(range(max(base, 0))) + [base + u for u in path if base + u >= 0]
                if not seen:
                    continue
                qq = q[first + t, h * G:(h + 1) * G]
                s = scale * (qq @ k[seen].T)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                at = (first + t, slice(h * G, (h + 1) * G))
                with np.errstate(invalid="ignore"):  # (values that are not finite have their part in what sees them)
                    out[at] = p @ v[seen]
                    mag[at] = p @ np.abs(v[seen])
                a = abs(scale) * (np.abs(qq) @ np.abs(k[seen]).T)
                err[at] = ((case.d + 4) * U32 * a + 8 * U32 * np.abs(s)).max(1) + (16 + np.sqrt(len(seen))) * U32 / 2
        first += T
    return out, mag, err


def _unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)


def chain(S, k, v, g, b, q=None):
    """The recurrence over the given tokens (fp64, one head: S [dv, dk], rows of k, v) token by token. Returns the state,
    its magnitudes, and for a query the output and its magnitudes."""
    S = S.copy()
    M = np.abs(S)
    for kk, vv, gg, bb in zip(k, v, g, b):
        alpha, beta = np.exp(gg), 1 / (1 + np.exp(-bb))
        u = beta * (vv - alpha * (S @ kk))
        U = beta * (np.abs(vv) + alpha * (M @ np.abs(kk)))
        S = alpha * S + np.outer(u, kk)
        M = alpha * M + np.outer(U, np.abs(kk))
    if q is None:
        return S, M
    return S, M, S @ q, M @ np.abs(q)


def tree_scan(q, k, v, g, b, states, trees):
    """(out, magnitudes, path lengths) of every node and head; CPU tensors, states [B, Hv, dv, dk]."""
    q, k, v, g, b, states = (x.double().numpy() for x in (q, k, v, g, b, states))
    q, k = _unit(q), _unit(k)
    r = v.shape[1] // k.shape[1]
    out, mag, length = np.zeros_like(v), np.zeros_like(v), np.zeros(v.shape[0])
    first = 0
    for n, parents in enumerate(trees):
        for t, path in enumerate(paths(parents)):
            at = [first + u for u in path]
            length[first + t] = len(path)
            for h in range(v.shape[1]):
                _, _, o, m = chain(states[n, h], k[at, h // r], v[at, h], g[at, h], b[at, h], q[first + t, h // r])
                out[first + t, h], mag[first + t, h] = o, m
        first += len(parents)
    return out, mag, length


def assert_scan(got, ref, mag, length, dk):
    y = got.double().cpu().numpy()
    assert np.isfinite(y).all()
    if got.dtype == torch.bfloat16:
        bound = 2.0 ** -14 * mag + 2.0 ** -8 * (np.abs(ref) + 2.0 ** -14 * mag)
    else:
        bound = (dk + 128) * (length[:, None, None] + 1) * U32 * mag
    excess = np.abs(y - ref) - bound
    assert (excess <= 1e-30).all(), f"off by {np.abs(y - ref).max():.3e}, over the bound by {excess.max():.3e}"


def advance(k, v, g, b, states, nodes, accepted):
    """(states, magnitudes) after the accepted paths; `nodes`: nodes of every sequence."""
    k, v, g, b, states = (x.double().numpy() for x in (k, v, g, b, states))
    k = _unit(k)
    r = v.shape[1] // k.shape[1]
    out, mag = states.copy(), np.abs(states)
    first = 0
    for n, T in enumerate(nodes):
        at = [first + u for u in accepted[n]]
        for h in range(v.shape[1]):
            out[n, h], mag[n, h] = chain(states[n, h], k[at, h // r], v[at, h], g[at, h], b[at, h])
        first += T
    return out, mag


def assert_states(got, ref, mag, accepted, dk):
    y = got.double().cpu().numpy()
    length = np.array([len(p) for p in accepted], dtype=np.float64)[:, None, None, None]
    excess = np.abs(y - ref) - (dk + 64) * (length + 1) * U32 * mag
    assert (excess <= 1e-30).all(), f"off by {np.abs(y - ref).max():.3e}, over the bound by {excess.max():.3e}"


def verify(target, draft, tokens, parents, r, r_last):
    """(accepted nodes, next token, distance of the closest decision from its border) of one sequence, in fp64."""
    target = target.double().numpy()
    draft = None if draft is None else draft.double().numpy()
    if not parents or parents[0] != -1:
        return [], -1, 1.0
    node, taken, close = 0, [0], 1.0
    while True:
        w, Z, step = target[node].copy(), 1.0, None
        for j in [j for j, u in enumerate(parents) if u == node]:
            x = int(tokens[j])
            if draft is None:
                q = np.zeros_like(w)
                q[x] = 1.0
            else:
                q = draft[node]
            left, right = float(r[j]) * Z * q[x], w[x]
            if max(left, right) > 0:
                close = min(close, abs(left - right) / max(left, right))
            if left < right:
                step = j
                break
            if draft is None:
                Z, w = Z - w[x], w * (1 - q)
            else:
                w = np.maximum(w - Z * q, 0)
                Z = w.sum()
        if step is None:
            break
        node = step
        taken.append(step)
    if not w.sum() > 0:
        w = target[node]
    sums = np.cumsum(w)
    if not (sums[-1] > 0 and np.isfinite(sums[-1])):
        return taken, -1, close
    draw = float(r_last) * sums[-1]
    live = w > 0
    close = min(close, np.abs(sums[live][:-1] - draw).min() / sums[-1] if live.sum() > 1 else 1.0)
    above = np.nonzero(live & (sums > draw))[0]
    return taken, int(above[0] if len(above) else np.nonzero(live)[0][-1]), close
