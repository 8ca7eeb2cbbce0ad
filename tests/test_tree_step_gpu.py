"""A step by drafts through the calls in turn, eagerly and from a captured graph: nodes stored, checked by attention and by the
gated delta rule, verified, and cache and states moved on along the accepted path; then one plain token after it."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, Paged, assert_attention, reference, values
from _tree import advance, assert_scan, assert_states, random_tree, tree_attention, tree_scan, verify

pytestmark = pytest.mark.gpu
B, T, Hq, Hkv, d, page, Hk, Hv, V = 3, 9, 8, 2, 128, 16, 2, 4, 97


def node_inputs(seed):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    bf = lambda *s: rand(*s).to(torch.bfloat16)  # noqa: E731
    trees = [random_tree(np.random.RandomState(seed + n), T, "deep", n) for n in range(B)]
    first = [T * n for n in range(B) for _ in range(T)]
    up = [f + max(u, 0) for f, u in zip(first, [u for t in trees for u in t])]
    target = 4 * rand(B * T, V)
    drafts = target + 0.7 * rand(B * T, V)
    tokens = torch.multinomial(drafts.softmax(-1)[up], 1, generator=gen)[:, 0].to(torch.int32)
    x = dict(aq=bf(B * T, Hq, d), ak=bf(B * T, Hkv, d), av=bf(B * T, Hkv, d), q=bf(B * T, Hk, 128), k=bf(B * T, Hk, 128),
             v=bf(B * T, Hv, 128), g=(-torch.nn.functional.softplus(rand(B * T, Hv))).to(torch.bfloat16), b=bf(B * T, Hv),
             target=target.softmax(-1), drafts=drafts.softmax(-1), tokens=tokens, r=torch.rand(B * T, generator=gen),
             last=torch.rand(B, generator=gen), parents=torch.tensor([u for t in trees for u in t], dtype=torch.int32))
    return x, trees


@pytest.mark.parametrize("cache", sorted(CACHES))
def test_a_step(cache):
    ctx = [40, 7, 0]
    case = Paged([c + 2 * T + 2 for c in ctx], Hkv, d, page, cache, "bf16", seed=3)  # room for two steps
    kc, vc, ks, vs, table, _ = case.tensors()
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    scales = dict(k_scale=ks, v_scale=vs)
    S = 0.3 * torch.randn(B, Hv, 128, 128, generator=torch.Generator().manual_seed(5))
    dev_S = S.to(DEV)
    ws = torch.empty(gdn.gdn_paged_attn_workspace_size(B, T, Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    x, trees = node_inputs(1)
    dev = {n: t.to(DEV) for n, t in x.items()}
    attn, out = torch.empty_like(dev["aq"]), torch.empty_like(dev["v"])
    path = torch.empty(B, T, dtype=torch.int32, device=DEV)
    counts, token = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))

    def step():
        lens.add_(T)
        gdn.gdn_kv_write(dev["ak"], dev["av"], kc, vc, table, lens, **scales)
        gdn.gdn_tree_attn(dev["aq"], kc, vc, table, lens, dev["parents"], attn, workspace=ws, **scales)
        gdn.gdn_tree_scan(dev["q"], dev["k"], dev["v"], dev["g"], dev["b"], dev_S, dev["parents"], out)
        gdn.gdn_tree_verify(dev["target"], dev["drafts"], dev["tokens"], dev["parents"], dev["r"], dev["last"], path, counts, token)
        gdn.gdn_kv_keep(kc, vc, table, lens, path, counts, T=T, **scales)
        gdn.gdn_tree_advance(dev["k"], dev["v"], dev["g"], dev["b"], dev_S, dev_S, path, counts)
        lens.add_(counts - T)

    def stored(name, n, t):
        """What the cache holds of a node's row."""
        rows = x[name][n * T + t].double().numpy()
        if cache == "same":
            return rows
        from _kv import quantise
        return values(*quantise(rows, cache), cache)

    cached = {n: [[case.sequence(n[-1], s, h)[:ctx[s]] for h in range(Hkv)] for s in range(B)] for n in ("ak", "av")}

    class Seen:  # what tree_attention and reference take of a _kv.Paged
        def __init__(self, extra):
            self.Hkv, self.d, self.lens = Hkv, d, [len(cached["ak"][s][0]) + len(extra[s]) for s in range(B)]
            self.extra = extra

        def sequence(self, name, n, h):
            return np.concatenate([cached["a" + name][n][h]] + [stored("a" + name, n, t)[h][None] for t in self.extra[n]])

    for turn in range(2):
        if turn == 1:  # a second step, other drafts, from a graph
            x, trees = node_inputs(20)
            saved = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), lens, dev_S)]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            for t, y in zip((kc.view(torch.uint8), vc.view(torch.uint8), lens, dev_S), saved):
                assert torch.equal(t, y)  # (capturing runs nothing)
            for n in dev:
                dev[n].copy_(x[n])
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert gdn.gdn_get_device_status() == gdn.GDN_OK
        every = Seen([list(range(T))] * B)
        assert_attention(attn, *tree_attention(every, x["aq"], trees, d ** -0.5))
        assert_scan(out, *tree_scan(x["q"], x["k"], x["v"], x["g"], x["b"], S, trees), 128)
        accepted = []
        for n in range(B):
            at = slice(n * T, n * T + T)
            taken, nxt, near = verify(x["target"][at], x["drafts"][at], x["tokens"][at], trees[n], x["r"][at], x["last"][n])
            assert near > 1e-9
            assert counts[n].item() == len(taken) and path[n, :len(taken)].tolist() == taken and token[n].item() == nxt
            accepted.append(taken)
        ref, mag = advance(x["k"], x["v"], x["g"], x["b"], S, [T] * B, accepted)
        assert_states(dev_S, ref, mag, accepted, 128)
        for name in cached:
            for n in range(B):
                new = [stored(name, n, t) for t in accepted[n]]
                cached[name][n] = [np.concatenate([cached[name][n][h]] + [y[h][None] for y in new]) for h in range(Hkv)]
        assert lens.tolist() == [len(cached["ak"][n][0]) for n in range(B)]
        S = dev_S.cpu()
    # a plain token after it sees the accepted rows and nothing else
    q = torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    x, _ = node_inputs(40)
    one = {n: x[n].view(B, T, Hkv, d)[:, 0].contiguous() for n in ("ak", "av")}
    lens.add_(1)
    gdn.gdn_kv_write(one["ak"].to(DEV), one["av"].to(DEV), kc, vc, table, lens, **scales)
    o = torch.empty_like(q, device=DEV)
    gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, lens, o, **scales)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert_attention(o, *reference(Seen([[0]] * B), q, [1] * B, d ** -0.5))


def test_the_example_runs():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for extra in (["--cache", "int8", "--nodes", "13"], ["--cache", "same", "--nodes", "1", "--sessions", "2"]):
        r = subprocess.run([sys.executable, os.path.join(root, "examples", "hybrid_session.py"), "--prompt", "90", "--tokens", "5", *extra],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "tokens a step" in r.stdout, (r.stdout, r.stderr[-2000:])
