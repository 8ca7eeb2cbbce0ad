"""The calls on trees at the ends of their ranges: 65535 sequences, 2^22 tokens of a vocabulary, no nodes at all."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV, cu_of
from _tree import advance, assert_scan, assert_states, paths, random_tree, tree_scan, verify
from test_tree_scan_gpu import flat, inputs, tables
from test_tree_verify_gpu import case, check, run

pytestmark = pytest.mark.gpu
B_MAX = 65535


def samples(trees):
    """A few sequences and where their nodes are."""
    first = np.cumsum([0] + [len(t) for t in trees])
    return [(n, slice(first[n], first[n + 1])) for n in (0, 1, 4095, 4096, 32768, B_MAX - 2, B_MAX - 1)]


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 32, 32), ("bf16", 128, 128), ("f32", 32, 64)])
def test_65535_sequences_of_states(dtype, dk, dv):
    r = np.random.RandomState(1)
    trees = [random_tree(r, int(T)) for T in r.randint(0, 4, B_MAX)]
    trees[0], trees[-1] = random_tree(r, 20), random_tree(r, 7)
    N, Hk, Hv = sum(map(len, trees)), 1, 2
    gen = torch.Generator(device=DEV).manual_seed(2)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x = [rand(N, Hk, dk).to(dt), rand(N, Hk, dk).to(dt), rand(N, Hv, dv).to(dt),
         (-torch.nn.functional.softplus(rand(N, Hv))).to(dt), rand(N, Hv).to(dt)]
    S = 0.3 * rand(B_MAX, Hv, dv, dk)
    out, new = torch.full_like(x[2], float("nan")), torch.full_like(S, float("nan"))
    cu = cu_of([len(t) for t in trees])
    gdn.gdn_tree_scan(*x, S, flat(trees), out, cu_seqlens=cu)
    accepted = [max(paths(t), key=len) if t else [] for t in trees]
    gdn.gdn_tree_advance(*x[1:], S, new, *tables(accepted), cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert torch.isfinite(out).all() and torch.isfinite(new).all()
    for n, at in samples(trees):
        one = [t[at].cpu() for t in x] + [S[n:n + 1].cpu()]
        if trees[n]:
            assert_scan(out[at], *tree_scan(*one, trees[n:n + 1]), dk)
        assert_states(new[n:n + 1], *advance(*one[1:], [len(trees[n])], accepted[n:n + 1]), accepted[n:n + 1], dk)


@pytest.mark.parametrize("drafts", [True, False])
def test_65535_verifications(drafts):
    c = case([2] * B_MAX, 9, drafts, seed=3)
    path, counts, token = run(c)
    for n, at in samples(c["trees"]):
        one = {k: c[k][at] if c[k] is not None else None for k in ("target", "draft", "tokens", "r")}
        one.update(trees=c["trees"][n:n + 1], r_last=c["r_last"][n:n + 1])
        check(one, (path[n:n + 1], counts[n:n + 1], token[n:n + 1]))
    assert ((counts == 1) | (counts == 2)).all() and ((token >= 0) & (token < 9)).all()


@pytest.mark.parametrize("cache", ["same", "int8"])
def test_65535_sequences_of_a_cache(cache):
    """Trees of two nodes after contexts of 0 to 5 tokens, a page each: attention and the rows that are kept."""
    Hkv, G, d, page = 1, 2, 64, 16
    gen = torch.Generator(device=DEV).manual_seed(4)
    pool = (B_MAX, Hkv, page, d)
    scales = {}
    if cache == "same":
        kc, vc = (torch.randn(pool, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    else:
        kc, vc = (torch.randint(-127, 128, pool, generator=gen, device=DEV, dtype=torch.int8) for _ in range(2))
        scales = {n: 0.01 + 0.01 * torch.rand(pool[:3], generator=gen, device=DEV) for n in ("k_scale", "v_scale")}
    ctx = torch.arange(B_MAX, device=DEV) % 6
    table = torch.randperm(B_MAX, generator=gen, device=DEV).to(torch.int32)[:, None].contiguous()
    lens = (ctx + 2).to(torch.int32)
    q = torch.randn(2 * B_MAX, Hkv * G, d, generator=gen, device=DEV).to(torch.bfloat16)
    parents = torch.tensor([-1, 0, -1, -1], dtype=torch.int32, device=DEV).repeat((B_MAX + 1) // 2)[:2 * B_MAX].contiguous()
    out = torch.full_like(q, float("nan"))
    gdn.gdn_tree_attn(q, kc, vc, table, lens, parents, out, **scales)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    rows = lambda c, n: (c.double() * scales[n][..., None].double() if scales else c.double())[table[:, 0].long(), 0]  # noqa: E731
    k, v = rows(kc, "k_scale"), rows(vc, "v_scale")  # [B, page, d]
    pos = torch.arange(page, device=DEV)
    first = pos[None, :] <= ctx[:, None]
    second = (pos[None, :] < ctx[:, None]) | (pos[None, :] == ctx[:, None] + 1) | (first & (parents[1::2] == 0)[:, None])
    seen = torch.stack([first, second], 1)[:, :, None, :]
    s = torch.einsum("btgd,bpd->btgp", q.view(B_MAX, 2, G, d).double(), k) * d ** -0.5
    p = s.masked_fill(~seen, float("-inf")).softmax(-1)
    ref, mag = torch.einsum("btgp,bpd->btgd", p, v), torch.einsum("btgp,bpd->btgd", p, v.abs())
    assert ((out.view_as(ref).double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag)).all()  # (_kv.py: two roundings to bf16, twice)
    before = [x.clone() for x in (kc, vc, *scales.values())]
    path = torch.tensor([[1]], dtype=torch.int32, device=DEV).repeat(B_MAX, 1)
    gdn.gdn_kv_keep(kc, vc, table, lens, path, torch.ones(B_MAX, dtype=torch.int32, device=DEV), T=2, **scales)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    at = table[:, 0].long()
    for x, old in zip((kc, vc, *scales.values()), before):
        old[at, :, ctx] = old[at, :, ctx + 1]
        assert torch.equal(x, old)


@pytest.mark.parametrize("sequences", [2, 9])
@pytest.mark.parametrize("drafts", [True, False])
def test_the_largest_vocabulary(drafts, sequences):
    c = case([3] * sequences, 1 << 22, drafts, "star", seed=sequences)
    for hard in (False, True):
        if hard:  # children rejected, draws near the end
            c["r"].fill_(1 - 2.0 ** -24)
            c["r_last"] = 0.999 + 0.001 * c["r_last"]
        # (partial sums are 2e-7 apart: one draw in a hundred is closer to one than the reference can tell)
        close = [n for n in range(sequences)
                 if verify(c["target"][3 * n:3 * n + 3], c["draft"][3 * n:3 * n + 3] if drafts else None, c["tokens"][3 * n:3 * n + 3],
                           c["trees"][n], c["r"][3 * n:3 * n + 3], c["r_last"][n])[2] <= 1e-9]
        assert 2 * len(close) < sequences
        check(c, run(c), but=close)


def test_no_nodes():
    """Sequences without a node: nothing accepted, states passed through, nothing moved."""
    B = 3
    e = lambda *s, dtype=torch.bfloat16: torch.empty(0, *s, dtype=dtype, device=DEV)  # noqa: E731
    i = lambda *s: torch.full(s, 99, dtype=torch.int32, device=DEV)  # noqa: E731
    none = torch.zeros(B, dtype=torch.int32, device=DEV)
    for cu in (None, torch.zeros(B + 1, dtype=torch.int32, device=DEV)):
        for drafts in (None, e(50, dtype=torch.float32)):
            path, counts, token = i(B, 4), i(B), i(B)
            gdn.gdn_tree_verify(e(50, dtype=torch.float32), drafts, e(dtype=torch.int32), e(dtype=torch.int32), e(dtype=torch.float32),
                                torch.rand(B, device=DEV), path, counts, token, cu_seqlens=cu)
            assert (path == -1).all() and (counts == 0).all() and (token == -1).all()
        S = torch.randn(B, 4, 64, 128, device=DEV)
        new, out = torch.full_like(S, float("nan")), e(4, 64)
        gdn.gdn_tree_advance(e(2, 128), e(4, 64), e(4), e(4), S, new, i(B, 4), none, cu_seqlens=cu)
        assert torch.equal(new, S)
        gdn.gdn_tree_scan(e(2, 128), e(2, 128), e(4, 64), e(4), e(4), S, e(dtype=torch.int32), out, cu_seqlens=cu)
        kc = torch.randn(4, 2, 16, 64, device=DEV).to(torch.bfloat16)
        vc, table, lens = kc.clone(), torch.arange(3, dtype=torch.int32, device=DEV)[:, None].contiguous(), none + 5
        gdn.gdn_kv_keep(kc, vc, table, lens, i(B, 4), none, cu_seqlens=cu, T=0)
        gdn.gdn_tree_attn(e(4, 64), kc, vc, table, lens, e(dtype=torch.int32), e(4, 64), cu_seqlens=cu)
        assert torch.equal(kc, vc)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    new.fill_(7.0)
    gdn.gdn_tree_advance(e(2, 128), e(4, 64), e(4), e(4), S, new, i(B, 4), none + 1)  # a count without nodes
    assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK and torch.equal(new, S)
