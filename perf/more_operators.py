"""Measured cases of the operators for trees of drafted tokens: attention of a tree over the paged cache, the
gated delta rule over a tree, the verification of the drafts, and what follows for states and caches.

Sequence n has T_n <= 64 nodes, packed as cu_seqlens says or T each. Node t's parent is parents[t] < t, -1 for
the root; below -1 the node is padding, whose path is empty, as are its descendants'. path(t) are the nodes from
the root to t.

    attn     o_t = softmax over the cached context and path(t) of scale * (q_t . k_j), times v_j; the nodes'
             rows are the last T_n of the kv_lens[n] cached ones (perf/operators.py has the cache's layout)
    scan     S_t = the recurrence  S <- alpha S (I - beta kh kh^T) + beta v kh^T  from the sequence's state over
             path(t); o_t = S_t qh_t; the state is left as it is
    advance  the same recurrence over an accepted path: the sequence's new state
    verify   from node 0 on, with p the node's row of target probabilities and q of draft probabilities (or one at
             the child's token): w = p, Z = 1; its children in order: accepted if r Z q(x) < w(x), else
             w <- max(w - Z q, 0), Z <- sum w. With no child left the next token is the least x whose
             cumulated w is above r times the sum of w (of p, if w has no weight)
    keep     the accepted path's cache rows move to the positions right after the context (here after the nodes
             have been stored, and read back: what a step does with its cache around the attention)

With `own` false, run() evaluates these in elementary torch operations in fp32; in fp64 where a draw is compared
with a sum over the vocabulary.
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"
MIN_SCALE = 2.0 ** -100
WORKSPACE_BYTES = 64 << 20  # scratch for the attention's split rows, kept by the program


def listed():
    def attn(name, B, T, ctx, Hq, Hkv, d, page, cache, dtype="bf16", ragged=False, tree="wide"):
        return dict(name=name, op="attn", B=B, T=T, ctx=ctx, Hq=Hq, Hkv=Hkv, d=d, page=page, cache=cache, dtype=dtype,
                    ragged=ragged, tree=tree)

    def gdn(name, op, B, T, Hk, Hv, dk, dv, dtype="bf16", ragged=False, tree="wide"):
        return dict(name=name, op=op, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, ragged=ragged, tree=tree)

    def verify(name, B, T, V, drafts, ragged=False, tree="wide"):
        return dict(name=name, op="verify", B=B, T=T, V=V, drafts=drafts, ragged=ragged, tree=tree)

    def keep(name, B, T, ctx, Hkv, d, page, cache, dtype="bf16", ragged=False, tree="wide"):
        return dict(name=name, op="keep", B=B, T=T, ctx=ctx, Hkv=Hkv, d=d, page=page, cache=cache, dtype=dtype,
                    ragged=ragged, tree=tree)

    return [
        # one chat session checks a small tree early in its context: latency
        attn("attn_session_bf16", 1, 8, 1000, 16, 2, 256, 16, "same"),
        # a decode batch of long sessions, each with two levels of a few drafts
        attn("attn_batch_fp8", 48, 4, 16384, 32, 8, 128, 64, "fp8", ragged=True),
        # sessions with the largest trees, packed, of mixed sizes
        attn("attn_large_trees_bf16", 32, 64, 8192, 16, 2, 256, 64, "same", ragged=True),
        # one session's tree through a gated delta rule layer: latency
        gdn("scan_session", "scan", 1, 16, 16, 32, 128, 128),
        # a batch of sessions with large trees
        gdn("scan_batch64", "scan", 64, 61, 16, 32, 128, 128),
        # full precision and mixed sizes, small heads
        gdn("scan_f32", "scan", 5, 24, 2, 4, 64, 32, dtype="f32", ragged=True),
        # the accepted tokens of one session, and of a full batch with idle rows
        gdn("advance_session", "advance", 1, 16, 16, 32, 128, 128),
        gdn("advance_batch128", "advance", 128, 16, 16, 32, 128, 128, ragged=True),
        # one session whose drafts are the likeliest tokens
        verify("verify_session", 1, 16, 150001, False),
        # a batch whose drafts were drawn from a draft model
        verify("verify_batch64", 64, 13, 131072, True, ragged=True),
        # what a step does with its cache around the attention: store the nodes, keep the accepted, read; one session in
        # full precision, and a batch
        keep("keep_session_f32", 1, 7, 500, 2, 64, 16, "same", dtype="f32"),
        keep("keep_batch_int8", 64, 32, 2000, 8, 128, 32, "int8", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, bounded by the largest listed costs."""
    while True:
        op = rng.choice(["attn", "attn", "attn", "scan", "scan", "advance", "verify", "verify", "keep"])
        c = dict(op=op, B=_log(rng, 1, 128), T=_log(rng, 1, 64))
        shape = dict(ragged=rng.random() < 0.5, tree=rng.choice(["wide", "wide", "deep", "chain"]))
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        cache = dict(page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["same", "fp8", "int8"]), dtype=dtype)
        if op == "attn":
            d, Hkv, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
            c.update(ctx=_log(rng, 1, 65536) - 1, Hq=Hkv * G, Hkv=Hkv, d=d, **cache, **shape)
            rows = c["B"] * (c["ctx"] + c["T"] + c["page"])
            pairs = c["B"] * c["T"] * c["Hq"] * (c["ctx"] + c["T"])
            if rows * Hkv * d > 4e8 or rows > 2 ** 21 or pairs > 3e8 or (dtype == "f32" and pairs * d > 4e9):
                continue
        elif op in ("scan", "advance"):
            Hk = rng.choice([1, 2, 4, 16])
            c.update(Hk=Hk, Hv=Hk * rng.choice([1, 2, 2, 3]), dk=rng.choice([32, 64, 128, 128]),
                     dv=rng.choice([32, 64, 128, 128]), dtype=dtype, **shape)
            heads = c["B"] * c["Hv"]
            if heads > 4096 or (op == "scan" and heads * c["T"] > 130000):
                continue
        elif op == "verify":
            c.update(V=_log(rng, 500, 200000), drafts=rng.random() < 0.6, **shape)
            if c["B"] * c["T"] * c["V"] > 1.1e8:
                continue
        else:
            c.update(ctx=_log(rng, 1, 8192) - 1, Hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128, 256]), **cache, **shape)
            if c["B"] * (c["ctx"] + c["T"] + c["page"]) * c["Hkv"] * c["d"] > 4e8:
                continue
        return c


# ---- sizes and trees that follow from the case alone --------------------------------------------
def _rng(case, what):
    key = what + " ".join(str(case[k]) for k in sorted(case) if k != "name")
    return np.random.RandomState(zlib.crc32(key.encode()) & 0x7FFFFFFF)


def _nodes(case):
    """Nodes of each sequence."""
    if not case["ragged"]:
        return [case["T"]] * case["B"]
    r = _rng(case, "nodes")
    return [case["T"] if n == 0 else int(r.randint(1, case["T"] + 1)) for n in range(case["B"])]


def _trees(case):
    """parents and path (list of nodes) of every node, of each sequence."""
    r = _rng(case, "tree")
    parents, paths = [], []
    for T in _nodes(case):
        p = [-1]
        for t in range(1, T):
            if case["tree"] == "chain":
                p.append(t - 1)
            elif case["tree"] == "deep":
                p.append(int(r.randint(max(0, t - 2), t)))
            else:  # a few children to a node: about the cube root deep
                p.append(int(r.randint(t // 3, (t + 1) // 2)))
        if case["ragged"]:  # the last nodes of some are padding
            for t in range(T - int(r.randint(0, 1 + T // 4)), T):
                if t > 0:
                    p[t] = -2
        path = []
        for t in range(T):
            path.append([t] if p[t] == -1 else [] if p[t] < -1 or not path[p[t]] else path[p[t]] + [t])
        parents.append(p)
        paths.append(path)
    return parents, paths


def _accepted(case):
    """An accepted path of each sequence (empty: an idle row of the batch)."""
    r = _rng(case, "accepted")
    out = []
    for n, path in enumerate(_trees(case)[1]):
        live = [p for p in path if p]
        out.append([] if case["ragged"] and n % 16 == 15 else live[int(r.randint(0, len(live)))])
    return out


def _lengths(case):
    """Cached tokens of each sequence, its nodes among them."""
    new = _nodes(case)
    if not case["ragged"]:
        return [case["ctx"] + t for t in new]
    r = _rng(case, "lengths")
    hi = case["ctx"]
    lo = max(1, hi // 32)
    ctx = [hi if n == 0 else int(round(math.exp(r.uniform(math.log(lo), math.log(hi + 1))))) for n in range(case["B"])]
    return [0 if n % 16 == 15 else x + t for n, (x, t) in enumerate(zip(ctx, new))]  # an idle row of the batch


def _elem(case):
    return 2 if case["dtype"] == "bf16" else 4


def _row_bytes(case):
    """Bytes of one cached row of one head: codes and scale."""
    return case["d"] * _elem(case) if case["cache"] == "same" else case["d"] + 4


def work(case):
    new, (_, paths) = _nodes(case), _trees(case)
    tokens, B = sum(new), case["B"]
    steps = sum(len(p) for path in paths for p in path)  # of all paths
    if case["op"] == "attn":
        lens = _lengths(case)
        d, Hq, e = case["d"], case["Hq"], _elem(case)
        meta = 4 * (2 * B + 1 + tokens + sum(-(-x // case["page"]) for x in lens))
        data = 2 * tokens * Hq * d * e + sum(lens) * case["Hkv"] * 2 * _row_bytes(case)
        pairs = sum((x - t) * t + sum(map(len, p)) for x, t, p in zip(lens, new, paths) if x)
        return {"bytes": data + meta, "flops": 4 * d * Hq * pairs}
    if case["op"] in ("scan", "advance"):
        Hk, Hv, dk, dv, e = case["Hk"], case["Hv"], case["dk"], case["dv"], _elem(case)
        state = B * Hv * dk * dv * 4
        if case["op"] == "scan":
            return {"bytes": state + tokens * e * (2 * Hk * dk + 2 * Hv * dv + 2 * Hv) + 4 * tokens,
                    "flops": tokens * Hv * 4 * dk * dv + steps * Hv * 4 * (dk + dv)}
        kept = sum(map(len, _accepted(case)))
        return {"bytes": 2 * state + kept * (e * (Hk * dk + Hv * dv + 2 * Hv) + 4) + 4 * B, "flops": kept * Hv * 6 * dk * dv}
    if case["op"] == "verify":  # of each sequence the row of its last accepted node
        rows = B * (2 if case["drafts"] else 1)
        return {"bytes": 4 * rows * case["V"] + tokens * 16 + 12 * B, "flops": rows * case["V"] * 2}
    # keep: the nodes' rows in, codes and scales out; the accepted ones moved; all read back
    e, d, Hkv = _elem(case), case["d"], case["Hkv"]
    live = sum(t for x, t in zip(_lengths(case), new) if x)
    moved = sum(len(p) for x, p in zip(_lengths(case), _accepted(case)) if x)
    return {"bytes": Hkv * 2 * (live * 2 * (d * e + _row_bytes(case)) + 2 * moved * _row_bytes(case)) + 4 * (2 * B + tokens),
            "flops": 4 * live * Hkv * 2 * d}


# ---- inputs -----------------------------------------------------------------------------------------
def _quantise(x, cache):
    """Codes and scales of rows x [..., d] (fp32), in elementary operations."""
    amax = x.abs().amax(-1)
    if cache == "fp8":
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
        k = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-100)
        scale = ((k + 127) << 23).view(torch.float32)  # 2^k by its bits
        return (x / scale[..., None]).to(torch.float8_e4m3fn), scale
    scale = (amax / torch.full_like(amax, 127.0)).clamp_min(MIN_SCALE)  # a true division, not a product with 1 / 127
    return torch.round(x / scale[..., None]).to(torch.int8), scale


def _cache_state(case, s, g):
    """Page pools, block table and lengths; the pools filled with rows."""
    dt, Hkv, d, page = s["dtype"], case["Hkv"], case["d"], case["page"]
    lens = _lengths(case)
    used = [-(-x // page) for x in lens]
    width = max(1, max(used))
    num_pages = sum(used) + 3  # a few pages of the pool belong to nobody
    order = torch.randperm(num_pages - 1, generator=g, device=DEV).to(torch.int32)  # the last page never
    starts = torch.tensor([0] + used[:-1], device=DEV).cumsum(0)
    col = torch.arange(width, device=DEV)
    at = (starts[:, None] + col[None, :]).clamp_max(num_pages - 2)
    table = torch.where(col[None, :] < torch.tensor(used, device=DEV)[:, None], order[at], torch.full_like(order[at], -1))
    s.update(block_table=table.contiguous(), kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), k_scale=None, v_scale=None)

    # a few channels of real keys and values are several times larger than the rest, and so are some tokens
    def rows(*shape):
        chan = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
        tok = torch.exp(0.3 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
        return torch.randn(shape, generator=g, device=DEV) * chan * tok

    for name in ("k", "v"):
        pool = (num_pages, Hkv, page, d)
        if case["cache"] == "same":
            s[name + "_cache"] = rows(*pool).to(dt)
        else:
            s[name + "_cache"], s[name + "_scale"] = _quantise(rows(*pool), case["cache"])
        if case["op"] == "keep":
            s[name] = rows(s["tokens"], Hkv, d).to(dt)


def _drafts(case, s, g):
    """Target and draft probabilities of every node, and the nodes' tokens, which the draft model proposed."""
    V, N = case["V"], s["tokens"]
    first = torch.tensor([0] + _nodes(case)[:-1], device=DEV).cumsum(0)
    own_row = first[s["seq"]]  # the root of each node's sequence
    up = torch.where(s["parents"] >= 0, own_row + s["parents"].clamp_min(0), own_row)  # the parent's row
    # (a language model is sure of many of its tokens, and a good draft model nearly agrees)
    target = 4.5 * torch.randn(N, V, generator=g, device=DEV)
    draft = target + torch.randn(N, V, generator=g, device=DEV)
    tokens = torch.empty(N, dtype=torch.int32, device=DEV)
    if case["drafts"]:
        for a in range(0, N, 256):  # a draw from the parent's draft probabilities: the largest with Gumbel noise
            u = torch.rand(min(256, N - a), V, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
            tokens[a:a + 256] = (draft[up[a:a + 256]] - torch.log(-torch.log(u))).argmax(-1).to(torch.int32)
    else:  # a node's children are its likeliest tokens
        nth = torch.zeros(N, dtype=torch.long)
        seen, rows = {}, up.tolist()
        for t, r in enumerate(rows):
            nth[t] = seen.get(r, 0)
            seen[r] = seen.get(r, 0) + 1
        for a in range(0, N, 256):
            best = draft[up[a:a + 256]].topk(min(V, 64), -1).indices
            tokens[a:a + 256] = best.gather(1, nth[a:a + 256].to(DEV)[:, None]).flatten().to(torch.int32)
    s["tokens_in"] = tokens
    s["target"] = torch.softmax(target, -1)
    s["draft"] = torch.softmax(draft, -1) if case["drafts"] else None
    s["r"] = torch.rand(N, generator=g, device=DEV)
    s["r_last"] = torch.rand(case["B"], generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, B, new = case["op"], case["B"], _nodes(case)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    s = {"case": dict(case), "dtype": dt, "tokens": sum(new), "Tmax": max(new), "cu_seqlens": None}
    s["parents"] = torch.tensor([p for tree in _trees(case)[0] for p in tree], dtype=torch.int32, device=DEV)
    s["seq"] = torch.tensor([n for n, t in enumerate(new) for _ in range(t)], device=DEV)
    if len(set(new)) > 1:
        s["cu_seqlens"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
    if op in ("advance", "keep"):
        acc = _accepted(case)
        s["path"] = torch.tensor([p + [-1] * (max(new) - len(p)) for p in acc], dtype=torch.int32, device=DEV)
        s["counts"] = torch.tensor([len(p) for p in acc], dtype=torch.int32, device=DEV)
    if op in ("attn", "keep"):
        _cache_state(case, s, g)
    if op == "attn":
        s["scale"] = 1.0 / math.sqrt(case["d"])
        s["q"] = (1.5 * torch.randn(s["tokens"], case["Hq"], case["d"], generator=g, device=DEV)).to(dt)
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    elif op in ("scan", "advance"):
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
        s["q"], s["k"] = (rand(s["tokens"], Hk, dk).to(dt) for _ in range(2))
        s["v"] = rand(s["tokens"], Hv, dv).to(dt)
        s["g"] = (-torch.nn.functional.softplus(rand(s["tokens"], Hv))).to(dt)
        s["b"] = rand(s["tokens"], Hv).to(dt)
        s["state"] = 0.1 * rand(B, Hv, dv, dk)
        if op == "advance":
            s["new_state"] = torch.empty_like(s["state"])
    elif op == "verify":
        _drafts(case, s, g)
    return s


# ---- one pass -------------------------------------------------------------------------------------
def _places(s):
    """(sequence, index within it, nodes of it) of every packed node."""
    i, n = torch.arange(s["tokens"], device=DEV), s["seq"]
    if s["cu_seqlens"] is None:
        return n, i % s["Tmax"], torch.full((s["case"]["B"],), s["Tmax"], device=DEV)
    cu = s["cu_seqlens"].long()
    return n, i - cu[n], cu[1:] - cu[:-1]


def _paths(s):
    """[B, Tmax, Tmax] truth values: node t's path holds node u. And the parents, -2 past a sequence's nodes."""
    n, t, _ = _places(s)
    T = s["Tmax"]
    up = torch.full((s["case"]["B"], T), -2, dtype=torch.long, device=DEV)
    up[n, t] = s["parents"].long()
    live = up == -1
    on = torch.zeros(up.shape + (T,), dtype=torch.bool, device=DEV)
    for j in range(T):  # parents come before their children
        above = on.gather(1, up[:, j].clamp_min(0)[:, None, None].expand(-1, 1, T))[:, 0]
        live[:, j] |= (up[:, j] >= 0) & live.gather(1, up[:, j].clamp_min(0)[:, None])[:, 0]
        on[:, j] = above & (up[:, j] >= 0)[:, None]
        on[:, j, j] = True
        on[:, j] &= live[:, j, None]
    return on, up


def _whole(s, name):
    """The cached rows of every sequence, fp32 [B, Hkv, L, d], L a whole number of pages."""
    case, pages, cache = s["case"], s["block_table"].long().clamp_min(0), s[name + "_cache"]
    if case["cache"] == "same":
        x = cache[pages].float()
    else:
        x = cache.view(torch.uint8)[pages].view(cache.dtype).float() * s[name + "_scale"][pages][..., None]
    return x.transpose(1, 2).reshape(pages.shape[0], case["Hkv"], -1, case["d"])


def _plain_attn(s):
    case = s["case"]
    B, Hq, Hkv, d, T = case["B"], case["Hq"], case["Hkv"], case["d"], s["Tmax"]
    n, t, new = _places(s)
    q = torch.zeros(B, T, Hq, d, device=DEV)
    q[n, t] = s["q"].float()
    q = q.view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    k = _whole(s, "k")
    ctx = s["kv_lens"].long() - new
    node = torch.arange(k.shape[2], device=DEV)[None, :] - ctx[:, None]  # of each position; below 0: the context
    on = _paths(s)[0].gather(2, node.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
    seen = torch.where((node < 0)[:, None, :], True, on & (node < new[:, None])[:, None, :])
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, T, Hq // Hkv, -1)
    x = torch.where(seen[:, None, :, None, :], x.mul_(s["scale"]), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    x = x.div_(torch.where(l == 0, 1.0, l)).view(B, Hkv, -1, x.shape[-1])
    o = torch.matmul(x, _whole(s, "v")).view(B, Hkv, T, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    # a node without a position (an idle row) is padding: zeros
    return torch.where((ctx[n] + t >= 0)[:, None, None], o[n, t], 0.0).to(s["dtype"])


def _padded(s, name):
    """A packed input as fp32 [B, Tmax, ...]."""
    n, t, _ = _places(s)
    x = torch.zeros((s["case"]["B"], s["Tmax"]) + s[name].shape[1:], device=DEV)
    x[n, t] = s[name].float()
    return x


def _step_inputs(s):
    """Unit q and k of every value head, v, decay and beta, [B, Tmax, Hv, ..]."""
    r = s["case"]["Hv"] // s["case"]["Hk"]
    unit = lambda x: (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(r, 2)  # noqa: E731
    b = _padded(s, "b")
    return unit(_padded(s, "q")), unit(_padded(s, "k")), _padded(s, "v"), _padded(s, "g").exp(), 1 / (1 + (-b).exp())


def _update(S, k, v, alpha, beta):
    """One step of the recurrence, [B, Hv, ..]."""
    S = S * alpha[..., None, None]
    return S + (beta[..., None] * (v - (S * k[..., None, :]).sum(-1)))[..., None] * k[..., None, :]


def _plain_scan(s):
    q, k, v, alpha, beta = _step_inputs(s)
    n, t, _ = _places(s)
    on, up = _paths(s)
    rows = torch.arange(up.shape[0], device=DEV)
    states = torch.empty((s["Tmax"] + 1,) + s["state"].shape, device=DEV)  # the sequence's own, then the nodes'
    states[0] = s["state"]
    out = torch.empty((up.shape[0], s["Tmax"]) + v.shape[2:], device=DEV)
    for j in range(s["Tmax"]):
        S = _update(states[(up[:, j] + 1).clamp_min(0), rows], k[:, j], v[:, j], alpha[:, j], beta[:, j])
        S = torch.where(on[:, j, j][:, None, None, None], S, states[0])  # padding: an empty path
        states[j + 1] = S
        out[:, j] = (S * q[:, j, :, None, :]).sum(-1)
    return out[n, t].to(s["dtype"])


def _plain_advance(s):
    _, k, v, alpha, beta = _step_inputs({**s, "q": s["k"]})
    rows, S = torch.arange(s["counts"].numel(), device=DEV), s["state"]
    for j in range(s["path"].shape[1]):
        at = s["path"][:, j].long().clamp_min(0)
        new = _update(S, k[rows, at], v[rows, at], alpha[rows, at], beta[rows, at])
        S = torch.where((j < s["counts"])[:, None, None, None], new, S)
    s["new_state"].copy_(S)


def _plain_verify(s):
    B, T, V = s["case"]["B"], s["Tmax"], s["case"]["V"]
    n, t, new = _places(s)
    up = _paths(s)[1]
    first = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), new.cumsum(0)[:-1]])
    tokens = torch.zeros(B, T, dtype=torch.long, device=DEV)
    tokens[n, t] = s["tokens_in"].long()
    r = torch.zeros(B, T, dtype=torch.float64, device=DEV)
    r[n, t] = s["r"].double()
    rows = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    count = torch.ones(B, dtype=torch.long, device=DEV)
    path = torch.full((B, T), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    c, Z = torch.zeros(B, dtype=torch.float64, device=DEV), torch.ones(B, dtype=torch.float64, device=DEV)
    gone = torch.zeros(B, V, dtype=torch.bool, device=DEV)  # without draft probabilities: the rejected tokens

    def weights():
        p = s["target"][first + cur].double()
        if s["draft"] is None:
            return torch.where(gone, 0.0, p)
        return (p - c[:, None] * s["draft"][first + cur].double()).clamp_min(0)

    for j in range(1, T):  # children come after their parents, so one walk over the nodes meets them in turn
        x = tokens[:, j]
        child = up[:, j] == cur
        w = s["target"][first + cur, x].double()
        if s["draft"] is None:
            w = torch.where(gone[rows, x], 0.0, w)
            taken = child & (r[:, j] * Z < w)
            Z = torch.where(child & ~taken, Z - w, Z)
            gone[rows, x] |= child & ~taken
            gone &= ~taken[:, None]
        else:
            qx = s["draft"][first + cur, x].double()
            taken = child & (r[:, j] * Z * qx < (w - c * qx).clamp_min(0))
            c = torch.where(child & ~taken, c + Z, c)
            Z = torch.where(child & ~taken, weights().sum(-1), Z)
            c = torch.where(taken, 0.0, c)
        Z = torch.where(taken, 1.0, Z)
        cur = torch.where(taken, j, cur)
        path[rows, count.clamp_max(T - 1)] = torch.where(taken, j, path[rows, count.clamp_max(T - 1)].long()).to(torch.int32)
        count = count + taken.long()
    w = weights()
    w = torch.where((w.sum(-1) > 0)[:, None], w, s["target"][first + cur].double())
    sums = w.cumsum(-1)
    token = torch.searchsorted(sums, (s["r_last"].double() * sums[:, -1])[:, None], right=True).flatten()
    return {"path": path, "counts": count.to(torch.int32), "next": token.clamp_max(V - 1).to(torch.int32)}


def _cache_places(s):
    """Page and row of every node, and which nodes have a position."""
    n, t, new = _places(s)
    pos = s["kv_lens"].long()[n] - new[n] + t
    page = s["block_table"].long()[n, (pos // s["case"]["page"]).clamp_min(0)]
    page = torch.where(pos >= 0, page, s["k_cache"].shape[0] - 1)  # padding goes to the page that nobody has
    return page, pos.clamp_min(0) % s["case"]["page"], pos >= 0


def _plain_keep(s):
    case, out = s["case"], {}
    page, row, live = _cache_places(s)
    n, t, new = _places(s)
    first = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), new.cumsum(0)[:-1]])
    # what each node's place holds in the end: the path's node, or what it held
    source = torch.where(t < s["counts"].long()[n], s["path"].long()[n, t], t) + first[n]
    for name in ("k", "v"):
        x, cache = s[name].float(), s[name + "_cache"]
        if case["cache"] == "same":
            cache[page, :, row] = x.to(cache.dtype)
            cache[page, :, row] = cache[page[source], :, row[source]]
            y = cache[page, :, row].float()
        else:
            code, scale = _quantise(x, case["cache"])
            raw, scales = cache.view(torch.uint8), s[name + "_scale"]
            raw[page, :, row], scales[page, :, row] = code.view(torch.uint8), scale
            raw[page, :, row], scales[page, :, row] = raw[page[source], :, row[source]], scales[page[source], :, row[source]]
            y = raw[page, :, row].view(cache.dtype).float() * scales[page, :, row][..., None]
        out[name] = torch.where(live[:, None, None], y, 0.0).to(s["dtype"])
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "attn":
            return {"out": _plain_attn(s)}
        if op == "scan":
            return {"out": _plain_scan(s)}
        if op == "advance":
            _plain_advance(s)
            return {"state": s["new_state"]}
        return _plain_verify(s) if op == "verify" else _plain_keep(s)
    import gated_deltanet_linear_delta_gb300 as gdn
    cu = dict(cu_seqlens=s["cu_seqlens"])
    if op == "attn":
        out = torch.empty_like(s["q"])
        gdn.gdn_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["parents"], out,
                          k_scale=s["k_scale"], v_scale=s["v_scale"], scale=s["scale"], workspace=s["workspace"], **cu)
        return {"out": out}
    if op == "scan":
        out = torch.empty_like(s["v"])
        gdn.gdn_tree_scan(s["q"], s["k"], s["v"], s["g"], s["b"], s["state"], s["parents"], out, **cu)
        return {"out": out}
    if op == "advance":
        gdn.gdn_tree_advance(s["k"], s["v"], s["g"], s["b"], s["state"], s["new_state"], s["path"], s["counts"], **cu)
        return {"state": s["new_state"]}
    if op == "verify":
        path = torch.empty(case["B"], s["Tmax"], dtype=torch.int32, device=DEV)
        counts, token = (torch.empty(case["B"], dtype=torch.int32, device=DEV) for _ in range(2))
        gdn.gdn_tree_verify(s["target"], s["draft"], s["tokens_in"], s["parents"], s["r"], s["r_last"], path, counts, token, **cu)
        return {"path": path, "counts": counts, "next": token}
    where = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], **cu)
    gdn.gdn_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], **where)
    gdn.gdn_kv_keep(s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["path"], s["counts"],
                    T=None if s["cu_seqlens"] is not None else s["Tmax"], **where)
    k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    gdn.gdn_kv_read(s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], k, v, **where)
    return {"k": k, "v": v}


# ---- the definition in 64 bits ---------------------------------------------------------------------
def _pow2(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to the even code, in fp64."""
    _, e = torch.frexp(x)
    step = _pow2(e.clamp_min(-5) - 4)  # 4 significant bits, down to 2^-9
    return torch.round(x / step) * step


def _stored(x, cache):
    """What a row of fp64 values reads back as."""
    amax = x.abs().amax(-1, keepdim=True)
    if cache == "fp8":
        _, e = torch.frexp(amax)
        k = e.clamp_min(-90) - 10
        k = torch.where(amax > 448 * _pow2(k), k + 1, k)
        scale = _pow2(torch.where(amax > 448 * _pow2(k), k + 1, k).clamp_min(-100))
        return _e4m3(x / scale) * scale
    scale = (amax / 127).clamp_min(MIN_SCALE)
    return torch.round(x / scale) * scale


def _pool64(s, name, pages):
    cache = s[name + "_cache"]
    if s[name + "_scale"] is None:
        return cache[pages].double()
    return cache.view(torch.uint8)[pages].view(cache.dtype).double() * s[name + "_scale"][pages].double()[..., None]


def _exact_attn(case, s):
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    out = torch.zeros(s["tokens"], Hq, d, dtype=torch.float64, device=DEV)
    G, first = Hq // Hkv, 0
    for i, (x, t) in enumerate(zip(_lengths(case), _nodes(case))):
        hidden = torch.ones(t, x, dtype=torch.bool)
        for j, path in enumerate(_trees(case)[1][i] if x else []):
            hidden[j, :x - t] = False
            hidden[j, [x - t + u for u in path]] = False
        hidden = hidden.to(DEV)
        empty = hidden.all(-1)[:, None, None]
        pages = s["block_table"][i, : -(-x // page)].long()
        for h in range(Hkv if x else 0):
            k, v = ([_pool64(s, n, pages)[:, h].reshape(-1, d)[:x] for n in ("k", "v")])
            y = torch.einsum("tgd,jd->tgj", s["q"][first:first + t, h * G:(h + 1) * G].double(), k) * s["scale"]
            y = torch.softmax(y.masked_fill(hidden[:, None], -math.inf), -1).masked_fill(empty, 0.0)
            out[first:first + t, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", y, v)
        first += t
    return {"out": out}


def _chains64(case, s, paths):
    """For a sequence at a time: its heads' unit keys and queries, values, cumulated gates and the corrections u of the
    listed nodes' paths, by the triangular system that the recurrence along a path amounts to."""
    r, first = case["Hv"] // case["Hk"], 0
    for i, t in enumerate(_nodes(case)):
        at = slice(first, first + t)
        first += t
        unit = lambda x: (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(r, 1).transpose(0, 1)  # noqa: E731
        k, v = unit(s["k"][at].double()), s["v"][at].double().transpose(0, 1)
        on = torch.zeros(t, t, dtype=torch.float64)
        for j, path in enumerate(paths[i]):
            on[j, path] = 1.0
        on = on.to(DEV)
        G = torch.einsum("tu,uh->ht", on, s["g"][at].double())
        beta = torch.sigmoid(s["b"][at].double()).T
        decay = torch.exp((G[:, :, None] - G[:, None, :]).clamp_max(0)) * on
        eye = torch.eye(t, dtype=torch.float64, device=DEV)
        A = eye + beta[:, :, None] * (decay - decay * eye) * (k @ k.transpose(1, 2))
        S = s["state"][i].double()
        rhs = beta[:, :, None] * (v - G.exp()[:, :, None] * (k @ S.transpose(1, 2)))
        u = torch.linalg.solve_triangular(A, rhs, upper=False)
        yield at, S, k, u, G, decay, on, unit


def _exact_scan(case, s):
    out = torch.empty(s["v"].shape, dtype=torch.float64, device=DEV)
    for at, S, k, u, G, decay, on, unit in _chains64(case, s, _trees(case)[1]):
        q = unit(s["q"][at].double())
        o = G.exp()[:, :, None] * (q @ S.transpose(1, 2)) + (decay * (q @ k.transpose(1, 2))) @ u
        out[at] = o.transpose(0, 1)
    return {"out": out}


def _exact_advance(case, s):
    out = torch.empty(s["state"].shape, dtype=torch.float64, device=DEV)
    for i, (chain, last) in enumerate(zip(_chains64(case, s, _trees(case)[1]), _accepted(case))):
        _, S, k, u, G, decay, _, _ = chain
        out[i] = S if not last else \
            G[:, last[-1]].exp()[:, None, None] * S + (u * decay[:, last[-1], :, None]).transpose(1, 2) @ k
    return {"state": out}


def _exact_verify(case, s):
    new, first = _nodes(case), 0
    path, counts, nexts = torch.full((case["B"], s["Tmax"]), -1, dtype=torch.int32), [], []
    tokens, r, r_last = s["tokens_in"].tolist(), s["r"].tolist(), s["r_last"].tolist()
    for i, t in enumerate(new):
        up = _trees(case)[0][i]
        node, taken = 0, [0]
        while True:
            w, Z, step = s["target"][first + node].double(), 1.0, None
            for j in [j for j in range(t) if up[j] == node]:
                x = tokens[first + j]
                if s["draft"] is None:
                    q = torch.zeros_like(w)
                    q[x] = 1.0
                else:
                    q = s["draft"][first + node].double()
                if r[first + j] * Z * q[x].item() < w[x].item():
                    step = j
                    break
                if s["draft"] is None:
                    Z, w = Z - w[x].item(), w * (1 - q)
                else:
                    w = (w - Z * q).clamp_min(0)
                    Z = w.sum().item()
            if step is None:
                break
            node = step
            taken.append(step)
        if not w.sum().item() > 0:
            w = s["target"][first + node].double()
        sums = w.cumsum(0)
        nexts.append(int((sums <= r_last[i] * sums[-1]).sum().clamp_max(case["V"] - 1)))
        path[i, :len(taken)] = torch.tensor(taken, dtype=torch.int32)
        counts.append(len(taken))
        first += t
    return {"path": path.to(DEV), "counts": torch.tensor(counts, dtype=torch.int32, device=DEV),
            "next": torch.tensor(nexts, dtype=torch.int32, device=DEV)}


def _exact_keep(case, s):
    source, live, first = [], [], 0
    for x, t, p in zip(_lengths(case), _nodes(case), _accepted(case)):
        source += [first + j for j in p + list(range(len(p), t))]
        live += [float(x > 0)] * t
        first += t
    live = torch.tensor(live, dtype=torch.float64, device=DEV)[:, None, None]
    stored = {n: s[n].double() if case["cache"] == "same" else _stored(s[n].double(), case["cache"]) for n in ("k", "v")}
    return {n: x[torch.tensor(source, device=DEV)] * live for n, x in stored.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "scan": _exact_scan, "advance": _exact_advance, "verify": _exact_verify,
            "keep": _exact_keep}[case["op"]](case, s)
