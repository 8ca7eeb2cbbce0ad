"""Measured cases of the paged key/value cache operators: writing (and quantising) new tokens into
the cache, reading a cache back, and the attention of new tokens over it.

A hybrid model alternates gated delta rule layers, whose state has a fixed size, with attention
layers, whose keys and values grow by one row per token and head. The caches are pools of pages

    k_cache, v_cache [num_pages][Hkv][page][d]     element type of the inputs, e4m3 or int8
    k_scale, v_scale [num_pages][Hkv][page] fp32   one scale per row of an 8-bit cache

and sequence n's position p sits on page block_table[n][p // page], row p % page. kv_lens[n] counts
the sequence's tokens with this call's T_n new ones among them, so its new token t has position
kv_lens[n] - T_n + t; a negative position is padding. Packed tokens follow cu_seqlens, or are B
sequences of T tokens each.

    write  scale = 2^k, the smallest with amax / scale <= 448 (e4m3), or amax / 127 (int8),
           and at least 2^-100; code = round-to-nearest-even(x / scale)
    read   x = code * scale
    attn   o = sum_j p_j v_j,  p = softmax over j <= position of  scale * (q . k_j)

With `own` false, run() evaluates these in elementary torch operations in fp32.
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
    def case(name, op, B, T, kv, Hq, Hkv, d, page, cache, dtype="bf16", ragged=False, fresh=False):
        return dict(name=name, op=op, B=B, T=T, kv=kv, Hq=Hq, Hkv=Hkv, d=d, page=page, cache=cache,
                    dtype=dtype, ragged=ragged, fresh=fresh)

    return [
        # one chat session's next token early in its context: the call's latency is what counts
        case("attn_session_bf16", "attn", 1, 1, 1000, 16, 2, 256, 16, "same"),
        # one session deep into a long document: one token, few rows, everything along the cache
        case("attn_long_session_fp8", "attn", 1, 1, 131072, 16, 2, 256, 64, "fp8"),
        # a full decode batch of sessions of mixed lengths, some rows idle
        case("attn_decode128_bf16", "attn", 128, 1, 16384, 16, 2, 256, 64, "same", ragged=True),
        # a smaller batch with more key heads and an int8 cache
        case("attn_decode32_int8", "attn", 32, 1, 32768, 32, 8, 128, 32, "int8", ragged=True),
        # checking up to five speculated tokens per session, three query heads to a key head
        case("attn_verify_fp8", "attn", 16, 5, 8191, 12, 4, 64, 16, "fp8", ragged=True),
        # the next fragment of a long prompt over what is cached of it: bound by the products
        case("attn_chunk_bf16", "attn", 1, 2048, 32768, 16, 2, 256, 64, "same"),
        # whole prompts of mixed lengths packed into one call, nothing cached before
        case("attn_prompts_fp8", "attn", 8, 2047, 2047, 32, 8, 128, 128, "fp8", ragged=True, fresh=True),
        # full precision, as for checking a model
        case("attn_chunk_f32", "attn", 2, 100, 1000, 8, 2, 64, 16, "same", dtype="f32"),
        # the decode batch's one new token each, quantised as it is stored
        case("write_decode128_fp8", "write", 128, 1, 16384, 16, 2, 256, 64, "fp8", ragged=True),
        # a long prompt's tokens stored at once
        case("write_prompt_int8", "write", 1, 16384, 16384, 32, 8, 128, 32, "int8", fresh=True),
        # a long session read back, for example to move it to another pool
        case("read_long_session_fp8", "read", 1, 131072, 131072, 16, 2, 256, 64, "fp8", fresh=True),
        # sessions of mixed lengths read back in full precision
        case("read_sessions_int8", "read", 24, 8191, 8191, 32, 8, 128, 16, "int8", dtype="f32", ragged=True, fresh=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, bounded by the largest listed costs."""
    while True:
        op = rng.choice(["attn", "attn", "attn", "write", "read"])
        d = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c = dict(op=op, B=_log(rng, 1, 128), T=_log(rng, 1, 2048), kv=_log(rng, 1, 131072), Hq=Hkv * G, Hkv=Hkv, d=d,
                 page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["same", "fp8", "int8"]), dtype=dtype,
                 ragged=rng.random() < 0.5, fresh=op == "read" or rng.random() < 0.25)
        if rng.random() < 0.4 and not c["fresh"]:
            c["T"] = rng.choice([1, 1, 2, 4, 7])
        if c["fresh"]:
            c["kv"] = c["T"] = min(c["kv"], 16384)
        c["T"] = min(c["T"], c["kv"])
        tokens = c["B"] * (c["kv"] + c["page"])
        if tokens * Hkv * d > 2.2e9 / 4 or tokens > 2 ** 21:
            continue
        if op == "attn":
            flops = 4.0 * c["B"] * c["T"] * c["Hq"] * c["kv"] * d
            if c["B"] * c["Hq"] * c["T"] * c["kv"] > 1.0e9 or flops > (1e12 if dtype == "bf16" else 2e9):
                continue
        elif op == "write" and c["B"] * c["T"] * Hkv * d > 1.7e7:
            continue
        return c


# ---- sizes that follow from the case alone ---------------------------------------------------
def _lengths(case):
    """(kv_lens, new tokens) of each sequence, the same for every seed."""
    B, T, kv = case["B"], case["T"], case["kv"]
    if not case["ragged"]:
        return [kv] * B, [kv if case["fresh"] else T] * B
    r = np.random.RandomState(zlib.crc32(("%d %d %d %d" % (B, T, kv, case["d"])).encode()) & 0x7FFFFFFF)
    lo = max(1, kv // 64)
    lens = [kv if n == 0 else int(round(math.exp(r.uniform(math.log(lo), math.log(kv))))) for n in range(B)]
    lens = [0 if n % 16 == 15 else x for n, x in enumerate(lens)]  # an idle row of the batch
    if case["fresh"]:
        return lens, list(lens)
    new = [T if n == 0 or T == 1 else int(r.randint(1, T + 1)) for n in range(B)]
    return lens, [min(t, x) if x else t for t, x in zip(new, lens)]


def _elem(case):
    return 2 if case["dtype"] == "bf16" else 4


def _row_bytes(case):
    """Bytes of one cached row of one head: codes and scale."""
    return case["d"] * _elem(case) if case["cache"] == "same" else case["d"] + 4


def work(case):
    lens, new = _lengths(case)
    d, Hq, Hkv, e = case["d"], case["Hq"], case["Hkv"], _elem(case)
    live = [(x, t) for x, t in zip(lens, new) if x]
    tokens = sum(new)
    meta = 4 * (2 * len(lens) + 1 + sum(-(-x // case["page"]) for x in lens))
    if case["op"] == "attn":
        # each new token's row of q and out, and every cached row of its sequence once
        data = 2 * tokens * Hq * d * e + sum(x for x, _ in live) * Hkv * 2 * _row_bytes(case)
        pairs = sum(t * (x - t) + t * (t + 1) // 2 for x, t in live)
        return {"bytes": data + meta, "flops": 4 * d * Hq * pairs}
    written = sum(t for _, t in live)
    if case["op"] == "write":  # rows in, codes and scales out; then read back: codes and scales in, rows out
        return {"bytes": written * Hkv * 2 * (d * e + _row_bytes(case)) * 2 + meta, "flops": 4 * written * Hkv * 2 * d}
    return {"bytes": written * Hkv * 2 * (d * e + _row_bytes(case)) + meta, "flops": written * Hkv * 2 * d}


# ---- inputs -------------------------------------------------------------------------------------
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


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, Hq, Hkv, d, page = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    lens, new = _lengths(case)
    used = [-(-x // page) for x in lens]
    width = max(1, -(-case["kv"] // page))
    num_pages = sum(used) + 3  # a few pages of the pool belong to nobody
    order = torch.randperm(num_pages - 1, generator=g, device=DEV).to(torch.int32)  # the last page never
    starts = torch.tensor([0] + used[:-1], device=DEV).cumsum(0)
    col = torch.arange(width, device=DEV)
    counts = torch.tensor(used, device=DEV)
    at = (starts[:, None] + col[None, :]).clamp_max(num_pages - 2)
    table = torch.where(col[None, :] < counts[:, None], order[at], torch.full_like(order[at], -1))
    s = {"case": dict(case), "block_table": table.contiguous(), "cu_seqlens": None,
         "kv_lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "Tmax": max(new), "tokens": sum(new),
         "scale": 1.0 / math.sqrt(d), "dtype": dt, "k_scale": None, "v_scale": None}
    if len(set(new)) > 1:
        s["cu_seqlens"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)

    # a few channels of real keys and values are several times larger than the rest, and so are some tokens
    def rows(*shape):
        chan = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
        tok = torch.exp(0.3 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
        return torch.randn(shape, generator=g, device=DEV) * chan * tok

    for name in ("k", "v"):
        pool = (num_pages, Hkv, page, d)
        if case["op"] == "write":  # what the pool held before does not matter
            kind = {"same": dt, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[case["cache"]]
            s[name + "_cache"] = torch.zeros(pool, dtype=torch.uint8, device=DEV).view(kind) if kind.itemsize == 1 \
                else torch.zeros(pool, dtype=kind, device=DEV)
            s[name + "_scale"] = None if case["cache"] == "same" else torch.zeros(pool[:-1], device=DEV)
            s[name] = rows(s["tokens"], Hkv, d).to(dt)
        elif case["cache"] == "same":
            s[name + "_cache"] = rows(*pool).to(dt)
        else:
            s[name + "_cache"], s[name + "_scale"] = _quantise(rows(*pool), case["cache"])
    if case["op"] == "attn":
        s["q"] = (1.5 * torch.randn(s["tokens"], Hq, d, generator=g, device=DEV)).to(dt)
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------------------------
def _token_places(s):
    """(sequence, index within it, position) of every packed token."""
    B, i = s["kv_lens"].numel(), torch.arange(s["tokens"], device=DEV)
    if s["cu_seqlens"] is None:
        n, t = i // s["Tmax"], i % s["Tmax"]
        new = torch.full((B,), s["Tmax"], device=DEV)
    else:
        cu = s["cu_seqlens"].long()
        n = torch.searchsorted(cu[1:], i, right=True)
        t, new = i - cu[n], cu[1:] - cu[:-1]
    return n, t, s["kv_lens"].long()[n] - new[n] + t, new


def _plain_write(s):
    case = s["case"]
    n, _, pos, _ = _token_places(s)
    page = s["block_table"].long()[n, (pos // case["page"]).clamp_min(0)]
    page = torch.where(pos >= 0, page, s["k_cache"].shape[0] - 1)  # padding goes to the page that nobody has
    row = pos.clamp_min(0) % case["page"]
    for name in ("k", "v"):
        x, cache = s[name].float(), s[name + "_cache"]
        if case["cache"] == "same":
            cache[page, :, row] = x.to(cache.dtype)
        else:
            code, scale = _quantise(x, case["cache"])
            cache.view(torch.uint8)[page, :, row] = code.view(torch.uint8)
            s[name + "_scale"][page, :, row] = scale


def _plain_read(s):
    case = s["case"]
    n, _, pos, _ = _token_places(s)
    page = s["block_table"].long()[n, (pos // case["page"]).clamp_min(0)].clamp_min(0)
    row = pos.clamp_min(0) % case["page"]
    out = []
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        if case["cache"] == "same":
            x = cache[page, :, row].float()
        else:
            x = cache.view(torch.uint8)[page, :, row].view(cache.dtype).float() * s[name + "_scale"][page, :, row][..., None]
        out.append(torch.where((pos >= 0)[:, None, None], x, 0.0).to(s["dtype"]))
    return out


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
    B, Hq, Hkv, d, T = s["kv_lens"].numel(), case["Hq"], case["Hkv"], case["d"], s["Tmax"]
    n, t, pos, new = _token_places(s)
    q = torch.zeros(B, T, Hq, d, device=DEV)
    q[n, t] = s["q"].float()
    q = q.view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    x = torch.matmul(q, _whole(s, "k").transpose(2, 3)).view(B, Hkv, T, Hq // Hkv, -1)
    last = (s["kv_lens"].long() - new)[:, None] + torch.arange(T, device=DEV)  # the last position that each token sees
    seen = torch.arange(x.shape[-1], device=DEV) <= last[:, None, :, None, None]
    x = torch.where(seen, x.mul_(s["scale"]), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    x = x.div_(torch.where(l == 0, 1.0, l)).view(B, Hkv, -1, x.shape[-1])
    o = torch.matmul(x, _whole(s, "v")).view(B, Hkv, T, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    return o[n, t].to(s["dtype"])


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "attn":
            return {"out": _plain_attn(s)}
        if case["op"] == "write":
            _plain_write(s)
        k, v = _plain_read(s)
        return {"k": k, "v": v}
    import gated_deltanet_linear_delta_gb300 as gdn
    where = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], cu_seqlens=s["cu_seqlens"])
    if case["op"] == "attn":
        out = torch.empty_like(s["q"])
        gdn.gdn_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], out,
                           scale=s["scale"], workspace=s["workspace"], **where)
        return {"out": out}
    if case["op"] == "write":
        gdn.gdn_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], **where)
    k = torch.empty(s["tokens"], case["Hkv"], case["d"], dtype=s["dtype"], device=DEV)
    v = torch.empty_like(k)
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


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lengths(case)
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    if case["op"] == "write":
        live = torch.cat([torch.full((t,), float(x > 0), dtype=torch.float64, device=DEV) for x, t in zip(lens, new)])
        return {n: (s[n].double() if case["cache"] == "same" else _stored(s[n].double(), case["cache"])) * live[:, None, None]
                for n in ("k", "v")}
    if case["op"] == "read":
        got = {"k": [], "v": []}
        for i, x in enumerate(lens):
            for n in got:
                rows = _pool64(s, n, s["block_table"][i, : -(-x // page)].long()).transpose(1, 2).reshape(-1, Hkv, d)
                got[n].append(rows[:x])
        return {n: torch.cat(v) for n, v in got.items()}
    out = torch.zeros(s["tokens"], Hq, d, dtype=torch.float64, device=DEV)
    G, first = Hq // Hkv, 0
    for i, (x, t) in enumerate(zip(lens, new)):
        q = s["q"][first:first + t].double()
        pages = s["block_table"][i, : -(-x // page)].long()
        for h in range(Hkv if x else 0):
            k, v = ([_pool64(s, n, pages)[:, h].reshape(-1, d)[:x] for n in ("k", "v")])
            for a in range(0, t, 512):
                b = min(t, a + 512)
                y = torch.einsum("tgd,jd->tgj", q[a:b, h * G:(h + 1) * G], k) * s["scale"]
                hidden = torch.arange(x, device=DEV)[None, :] > (x - t + torch.arange(a, b, device=DEV))[:, None]
                y = torch.softmax(y.masked_fill(hidden[:, None], -math.inf), -1)
                out[first + a:first + b, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", y, v)
        first += t
    return {"out": out}
