"""Paged cache cases and their reference in 64 bits (numpy), apart from the library.

Tolerances, from the number formats (u = 2^-24 for fp32, 2^-9 for one rounding to bf16):

* stored codes and scales: equal. The e4m3 scale is a power of two, so x / s is exact and the code
  is fixed by the definition; the int8 code is defined by two fp32 operations, each correctly rounded.
* attention, bf16 out: the probabilities are rounded to 16 bits (relative 2^-9 at most each, which
  moves the output by at most 2^-9 sum_j p_j |v_j|), the output once more (2^-9 |out|); twice that
  is allowed, which leaves room for the fp32 parts: |out - ref| <= 2^-8 (|ref| + sum_j p_j |v_j|).
* attention, fp32 out: a score's error e_s is at most (d + 4) u scale sum_i |q_i k_ji| (summation)
  plus 8 u |s_j| (scaling, base change, exponential); it moves a probability by a factor e^(2 e_s),
  and the L-term sums add sqrt(L) u: |out - ref| <= (2 e_s + (16 + sqrt(L)) u) sum_j p_j |v_j| with
  the row's largest e_s.
"""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda:0"
U32, UB = 2.0 ** -24, 2.0 ** -9
CACHES = {"same": None, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- codes ---------------------------------------------------------------------------------
def e4m3_values() -> np.ndarray:
    """The value of every e4m3 byte (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f is NaN)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return out


E4M3 = e4m3_values()


def quantise(x: np.ndarray, cache: str):
    """(codes as bytes, scales fp32) of rows x [..., d] (values of fp32 or bf16)."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[..., None], 0.0, x)
    amax = np.abs(y).max(-1)
    if cache == "fp8":
        m, e = np.frexp(amax)
        k = np.maximum(np.where(amax == 0, -100, np.where(m <= 0.875, e - 9, e - 8)), -100)
        scale = np.ldexp(1.0, k)
        pos = E4M3[:127]  # increasing; the even byte is the even mantissa
        r = np.abs(y) / scale[..., None]
        hi = np.clip(np.searchsorted(pos, r), 0, 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = r - pos[lo], pos[hi] - r
        code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        code = np.where((code == 0) & ~np.signbit(y), 0, np.where(np.signbit(y), code | 128, code)).astype(np.uint8)
    else:
        s32 = np.maximum(amax.astype(np.float32) / np.float32(127), np.float32(2.0 ** -100))
        code = np.rint(y.astype(np.float32) / s32[..., None]).astype(np.int8).view(np.uint8)
        scale = s32.astype(np.float64)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code, np.where(bad, np.nan, scale).astype(np.float32)


def values(code: np.ndarray, scale: np.ndarray, cache: str) -> np.ndarray:
    x = E4M3[code] if cache == "fp8" else code.view(np.int8).astype(np.float64)
    return x * scale.astype(np.float64)[..., None]


# ---- cases ----------------------------------------------------------------------------------
class Paged:
    """Sequences with cached rows on randomly ordered pages; every place that no live position owns
    holds NaN (in 8-bit caches: NaN scales, and NaN codes in e4m3)."""

    def __init__(self, lens, Hkv, d, page, cache="same", dtype="bf16", seed=0, spare=2, width=None):
        r = np.random.RandomState(seed)
        self.lens, self.Hkv, self.d, self.page, self.cache, self.dtype = list(lens), Hkv, d, page, cache, dtype
        used = [-(-x // page) for x in lens]
        self.num_pages = max(1, sum(used) + spare)
        self.width = max([1] + used) if width is None else width
        order = r.permutation(self.num_pages)
        self.table = np.full((len(lens), self.width), -7, np.int32)
        at = 0
        for n, u in enumerate(used):
            self.table[n, :u] = order[at:at + u]
            at += u
        shape = (self.num_pages, Hkv, page)
        self.live = np.zeros((self.num_pages, page), bool)
        for n, x in enumerate(lens):
            for j in range(used[n]):
                self.live[self.table[n, j], : min(page, x - j * page)] = True
        self.rows = {}
        self.code, self.scale = {}, {}
        for name in ("k", "v"):
            x = torch.from_numpy(r.randn(*shape, d).astype(np.float32))
            x = (x * torch.from_numpy(np.exp(0.5 * r.randn(d)).astype(np.float32))).to(DTYPES[dtype]).double().numpy()
            if cache == "same":
                self.rows[name] = x
            else:
                self.code[name], self.scale[name] = quantise(x, cache)
                self.rows[name] = values(self.code[name], self.scale[name], cache)

    def tensors(self):
        """k_cache, v_cache, k_scale, v_scale, block_table, kv_lens on the GPU."""
        dead = torch.from_numpy(~self.live)[:, None, :].expand(self.num_pages, self.Hkv, self.page)
        out = []
        for name in ("k", "v"):
            if self.cache == "same":
                t = torch.from_numpy(self.rows[name]).to(DTYPES[self.dtype])
                t[dead] = float("nan")
            else:
                c = torch.from_numpy(self.code[name].copy())
                c[dead] = 0x7F
                t = c.view(CACHES[self.cache])
            out.append(t.to(DEV))
        for name in ("k", "v"):
            if self.cache == "same":
                out.append(None)
            else:
                s = torch.from_numpy(self.scale[name].copy())
                s[dead] = float("nan")
                out.append(s.to(DEV))
        out.append(torch.from_numpy(self.table).to(DEV))
        out.append(torch.tensor(self.lens, dtype=torch.int32, device=DEV))
        return out

    def sequence(self, name, n, h):
        """Cached rows [len, d] of sequence n, head h, in fp64."""
        x = self.lens[n]
        pg = self.table[n, : -(-x // self.page)]
        return self.rows[name][pg, h].reshape(-1, self.d)[:x]


def cu_of(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)


def reference(case: Paged, q: torch.Tensor, new, scale):
    """(out, sum_j p_j |v_j|, e_s) in fp64; q [tokens, Hq, d] on the CPU."""
    q = q.double().numpy()
    G = q.shape[1] // case.Hkv
    out, mag = np.zeros_like(q), np.zeros_like(q)
    err = np.zeros(q.shape[:2])
    first = 0
    for n, T in enumerate(new):
        for h in range(case.Hkv):
            k, v = case.sequence("k", n, h), case.sequence("v", n, h)
            for t in range(T):
                keys = case.lens[n] - T + t + 1
                if keys <= 0:
                    continue
                qq = q[first + t, h * G:(h + 1) * G]
                s = scale * (qq @ k[:keys].T)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[first + t, h * G:(h + 1) * G] = p @ v[:keys]
                mag[first + t, h * G:(h + 1) * G] = p @ np.abs(v[:keys])
                a = abs(scale) * (np.abs(qq) @ np.abs(k[:keys]).T)
                err[first + t, h * G:(h + 1) * G] = ((case.d + 4) * U32 * a + 8 * U32 * np.abs(s)).max(1) + \
                    (16 + np.sqrt(keys)) * U32 / 2
        first += T
    return out, mag, err


def assert_attention(got: torch.Tensor, ref, mag, err):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    if got.dtype == torch.bfloat16:
        bound = 2 * UB * (np.abs(ref) + mag)
    else:
        bound = 2 * err[..., None] * mag
    excess = np.abs(g - ref) - bound
    assert (excess <= 1e-30).all(), f"off by {np.abs(g - ref).max():.3e}, over the bound by {excess.max():.3e}"
