"""What holds for each call on trees: tensors of another device are refused, calls in flight at once share nothing, a call made twice
gives the same bits, and pools and rows of more than 2^31 elements."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, Paged, assert_attention
from _tree import advance, assert_scan, assert_states, paths, random_tree, tree_attention, tree_scan
from test_kv_keep_gpu import expect, raw
from test_tree_scan_gpu import flat, inputs, tables
from test_tree_verify_gpu import case, check

pytestmark = pytest.mark.gpu


def calls():
    b = dict(dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.ones(4, h, 128, **b) for h in (2, 2, 4))
    g, beta = (torch.zeros(4, 4, **b) for _ in range(2))
    state = torch.zeros(2, 4, 128, 128, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    parents, path, counts = i(-1, 0, -1, 0), i([0, 1], [0, 1]), i(2, 2)
    kc, vc = (torch.full((3, 2, 16, 128), 7.0, **b) for _ in range(2))
    table, lens = i([0], [1]), i(2, 2)
    ao, so = torch.full_like(q, 7.0), torch.full_like(v, 7.0)
    new = torch.full_like(state, 7.0)
    probs = torch.full((4, 10), 0.1, device="cuda")
    r, last = torch.zeros(4, device="cuda"), torch.zeros(2, device="cuda")
    po, co, no = i([7, 7], [7, 7]), i(7, 7), i(7, 7)
    return [kc, vc, ao, so, new, po, co, no], {
        "tree_attn": lambda: gdn.gdn_tree_attn(q, kc, vc, table, lens, parents, ao),
        "kv_keep": lambda: gdn.gdn_kv_keep(kc, vc, table, lens, path, counts, T=2),
        "tree_scan": lambda: gdn.gdn_tree_scan(q, k, v, g, beta, state, parents, so),
        "tree_advance": lambda: gdn.gdn_tree_advance(k, v, g, beta, state, new, path, counts),
        "tree_verify": lambda: gdn.gdn_tree_verify(probs, probs, i(0, 1, 0, 1), parents, r, last, po, co, no),
    }


def test_calls_refuse_tensors_of_another_device(monkeypatch):
    kept, by_name = calls()
    monkeypatch.setattr(gdn, "_current_device", lambda: torch.cuda.current_device() + 1, raising=False)
    for call in by_name.values():
        with pytest.raises(ValueError):
            call()
        with torch.cuda.stream(torch.cuda.Stream()), pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in kept)
    monkeypatch.undo()
    for call in by_name.values():  # and the same calls are sound
        call()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


def at_once(jobs):
    """Each job's call 10 times, those of different jobs on streams of their own."""
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(10):
        for s, job in zip(streams, jobs):
            with torch.cuda.stream(s):
                job(i)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK


@pytest.mark.parametrize("drafts", [True, False])
def test_verifications_at_once(drafts):
    cases = [case([13, 1, 40, 7][j:] + [9] * (6 * j), 20001, drafts, "star" if j % 2 else "wide", seed=40 + j) for j in range(4)]
    jobs, outs = [], []
    for c in cases:
        nodes = [len(t) for t in c["trees"]]
        dev = {n: c[n].to(DEV) for n in ("target", "tokens", "r", "r_last")}
        draft, parents = (c["draft"].to(DEV) if drafts else None), flat(c["trees"])
        cu = torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32, device=DEV)
        o = [[torch.full((len(nodes), max(nodes)), 99, dtype=torch.int32, device=DEV)] +
             [torch.full((len(nodes),), 99, dtype=torch.int32, device=DEV) for _ in range(2)] for _ in range(10)]
        outs.append(o)
        jobs.append(lambda i, dev=dev, draft=draft, parents=parents, cu=cu, o=o: gdn.gdn_tree_verify(
            dev["target"], draft, dev["tokens"], parents, dev["r"], dev["r_last"], *o[i], cu_seqlens=cu))
    at_once(jobs)
    for c, o in zip(cases, outs):
        check(c, [t.cpu() for t in o[0]])
        assert all(torch.equal(x, y) for p in o for x, y in zip(p, o[0]))


@pytest.mark.parametrize("cache", sorted(CACHES))
def test_keeps_at_once(cache):
    """Each stream moves rows of caches of its own; a tree's rows, of 10 copies of the caches."""
    jobs, done = [], []
    for j in range(4):
        T = [7, 40, 64, 13][j]
        r = np.random.RandomState(j)
        kept = Paged([T + 30 * n for n in range(1, 9)], 4, 64, 16, cache, "bf16", seed=j)
        kc, vc, ks, vs, table, lens = kept.tensors()
        accepted = [max(paths(random_tree(r, T, "deep")), key=len) for _ in range(8)]
        want = expect(kept, [kc, vc, ks, vs], [T] * 8, accepted)
        copies = [[None if x is None else x.clone() for x in (kc, vc, ks, vs)] for _ in range(10)]
        path, counts = tables(accepted)
        jobs.append(lambda i, p=copies, table=table, lens=lens, path=path, counts=counts, T=T: gdn.gdn_kv_keep(
            p[i][0], p[i][1], table, lens, path, counts, p[i][2], p[i][3], T=T))
        done.append((want, copies))
    at_once(jobs)
    for want, copies in done:
        for pools in copies:
            for got, ref in zip(pools, want):
                assert got is None or np.array_equal(raw(got).numpy(), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attentions_and_advances_at_once(dtype):
    jobs, outs = [], []
    for j in range(4):
        r = np.random.RandomState(j)
        trees = [random_tree(r, [5, 64, 16, 30][j]) for _ in range(4)]
        pages = Paged([len(t) + 200 * n for n, t in enumerate(trees)], 2, 128, 16, "same", dtype, seed=j)
        kc, vc, _, _, table, lens = pages.tensors()
        x = [t.to(DEV) for t in inputs(trees, 2, 4, 128, 128, dtype, seed=j)]
        q = torch.randn(len(x[0]), 8, 128, generator=torch.Generator().manual_seed(j)).to(x[0].dtype).to(DEV)
        path, counts = tables([max(paths(t), key=len) for t in trees])
        a, s = [torch.empty_like(q) for _ in range(10)], [torch.empty_like(x[5]) for _ in range(10)]

        def job(i, q=q, kc=kc, vc=vc, table=table, lens=lens, up=flat(trees), a=a, s=s, x=x, path=path, counts=counts):
            gdn.gdn_tree_attn(q, kc, vc, table, lens, up, a[i])
            gdn.gdn_tree_advance(*x[1:], s[i], path, counts)

        jobs.append(job)
        outs.append((a, s, pages, q, trees))
    at_once(jobs)
    for a, s, pages, q, trees in outs:
        assert_attention(a[0], *tree_attention(pages, q.cpu(), trees, 128 ** -0.5))
        assert all(torch.equal(y, a[0]) for y in a) and all(torch.equal(y, s[0]) for y in s)


@pytest.mark.parametrize("dtype,dv,slots", [("bf16", 128, 33000), ("bf16", 64, 66000), ("f32", 128, 33000)])
def test_a_pool_of_more_states_than_32_bits_count(dtype, dv, slots):
    """Entries at both ends of a pool of more than 2^31 elements, read by the scan and advanced."""
    trees = [random_tree(np.random.RandomState(n), 9) for n in range(4)]
    x = inputs(trees, 2, 4, 128, dv, dtype, seed=3)
    at = torch.tensor([slots - 1, 0, slots - 2, 7], dtype=torch.int32)
    pool = torch.empty(slots, 4, dv, 128, device=DEV)
    assert pool.numel() > 2 ** 31
    pool[at.long()] = x[5].to(DEV)
    q, k, v, g, b, _ = (t.to(DEV) for t in x)
    out = torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV)
    gdn.gdn_tree_scan(q, k, v, g, b, pool, flat(trees), out, slots=at.to(DEV))
    accepted = [max(paths(t), key=len) for t in trees]
    gdn.gdn_tree_advance(k, v, g, b, pool, pool, *tables(accepted), slots=at.to(DEV))
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert_scan(out, *tree_scan(*x, trees), 128)
    assert_states(pool[at.long()], *advance(*x[1:], [9] * 4, accepted), accepted, 128)


@pytest.mark.parametrize("drafts", [True, False])
def test_more_probabilities_than_32_bits_count(drafts):
    """Rows of 2^20 probabilities, more than 2^31 in all: the last sequences' lie beyond."""
    V, B, T = 1 << 20, 700, 3
    c = case([T] * 2, V, drafts, "star", seed=6)
    target = torch.full((B * T, V), 1.0 / V, device=DEV)
    assert target.numel() > 2 ** 31
    target[-6:] = c["target"].to(DEV)
    draft = None
    if drafts:
        draft = torch.full((B * T, V), 1.0 / V, device=DEV)
        draft[-6:] = c["draft"].to(DEV)
    whole = lambda x, n: torch.cat([torch.zeros(n - len(x), dtype=x.dtype), x]).to(DEV)  # noqa: E731
    parents = torch.tensor([-1, 0, 0] * B, dtype=torch.int32, device=DEV)
    c["trees"] = [[-1, 0, 0]] * 2
    path = torch.full((B, T), 99, dtype=torch.int32, device=DEV)
    counts, token = (torch.full((B,), 99, dtype=torch.int32, device=DEV) for _ in range(2))
    gdn.gdn_tree_verify(target, draft, whole(c["tokens"], B * T), parents, whole(c["r"], B * T), whole(c["r_last"], B), path, counts, token)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    check(c, (path[-2:].cpu(), counts[-2:].cpu(), token[-2:].cpu()))


@pytest.mark.parametrize("cache,dtype,Hq", [("same", "bf16", 4), ("same", "bf16", 32), ("int8", "bf16", 4), ("same", "f32", 4)])
def test_a_cache_of_more_elements_than_32_bits_count(cache, dtype, Hq):
    """A small case's pages at the end of a pool of more than 2^31 elements: the same attention, bit for bit, and the same rows moved."""
    trees = [random_tree(np.random.RandomState(n), 12, "deep") for n in range(3)]
    kept = Paged([12 + 40, 12 + 3, 12 + 500], 4, 128, 64, cache, dtype, seed=4)
    kc, vc, ks, vs, table, lens = kept.tensors()
    pages = (1 << 31) // (4 * 128 * 64) + 100
    extra = pages - kept.num_pages

    def far(x):
        if x is None:
            return None
        y = torch.empty((pages,) + x.shape[1:], dtype=x.dtype, device=DEV)
        y.view(torch.uint8)[extra:] = x.view(torch.uint8)
        return y

    big = [far(x) for x in (kc, vc, ks, vs)]
    assert big[0].numel() > 2 ** 31
    there = torch.where(table >= 0, table + extra, table)
    q = torch.randn(36, Hq, 128, generator=torch.Generator().manual_seed(1)).to(torch.float32 if dtype == "f32" else torch.bfloat16).to(DEV)
    out = [torch.full_like(q, float("nan")) for _ in range(2)]
    gdn.gdn_tree_attn(q, kc, vc, table, lens, flat(trees), out[0], ks, vs)
    gdn.gdn_tree_attn(q, big[0], big[1], there, lens, flat(trees), out[1], big[2], big[3])
    assert torch.equal(*out)
    assert_attention(out[0], *tree_attention(kept, q.cpu(), trees, 128 ** -0.5))
    accepted = [max(paths(t), key=len) for t in trees]
    want = expect(kept, [kc, vc, ks, vs], [12] * 3, accepted)
    gdn.gdn_kv_keep(big[0], big[1], there, lens, *tables(accepted), big[2], big[3], T=12)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    for got, ref in zip(big, want):
        assert got is None or np.array_equal(raw(got[extra:]).numpy(), ref)
