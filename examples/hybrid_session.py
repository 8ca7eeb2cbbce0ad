"""A serving session of a small hybrid stack: gated delta rule layers and attention layers by turns.

Three of four layers are Gated DeltaNet layers, whose state has a fixed size; the fourth is an
attention layer, whose keys and values go to a paged cache (bf16, or quantised to e4m3 or int8 as
they are written). A prompt is taken in fragments, then tokens one at a time, the decode step from a
captured CUDA graph whose lengths live on the device. Then the same tokens again by trees of drafts: all
layers check a tree's nodes at once, the drafts are verified against the model's probabilities, and states
and caches move on along the accepted path. The projections around the layers are plain matrix products
with random weights: the point is how the calls fit together.

    python examples/hybrid_session.py [--cache same|fp8|int8] [--sessions 4] [--prompt 700] [--tokens 16] [--nodes 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_delta_gb300 as gdn  # noqa: E402

DEV = "cuda"


def _linear(x, w):
    return (x @ w).to(torch.bfloat16)


class GdnLayer:
    """x + W_o gdn(x): 2 key heads and 4 value heads of 128."""

    Hk, Hv, d = 2, 4, 128

    def __init__(self, width, sessions, gen):
        w = lambda *s: (torch.randn(*s, generator=gen) / s[0] ** 0.5).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.wq, self.wk, self.wv = w(width, self.Hk * self.d), w(width, self.Hk * self.d), w(width, self.Hv * self.d)
        self.wg, self.wb, self.wo = w(width, self.Hv), w(width, self.Hv), w(self.Hv * self.d, width)
        self.state = torch.zeros(sessions, self.Hv, self.d, self.d, device=DEV)

    def _inputs(self, x):
        heads = lambda y, h: y.view(-1, h, self.d)  # noqa: E731
        g = -torch.nn.functional.softplus(_linear(x, self.wg).float()).to(torch.bfloat16)
        return (heads(_linear(x, self.wq), self.Hk), heads(_linear(x, self.wk), self.Hk),
                heads(_linear(x, self.wv), self.Hv), g, _linear(x, self.wb))

    def prefill(self, x, sessions):
        q, k, v, g, b = self._inputs(x)
        out = torch.empty_like(v)
        gdn.gdn_prefill(q, k, v, g, b, self.state, self.state, out, B=sessions, T=x.shape[0] // sessions)
        return x + _linear(out.flatten(1), self.wo)

    def step(self, x):
        q, k, v, g, b = self._inputs(x)
        out = torch.empty_like(v)
        gdn.gdn_decode_step(q, k, v, g, b, self.state, out)
        return x + _linear(out.flatten(1), self.wo)

    def tree(self, x, parents):
        """Drafted nodes: their outputs, with the state as it is. What `accept` needs of them is kept."""
        q, *self.nodes = self._inputs(x)
        out = torch.empty_like(self.nodes[1])
        gdn.gdn_tree_scan(q, *self.nodes, self.state, parents, out)
        return x + _linear(out.flatten(1), self.wo)

    def accept(self, path, counts):
        gdn.gdn_tree_advance(*self.nodes, self.state, self.state, path, counts)


class AttentionLayer:
    """x + W_o attention(x): 16 query heads and 2 key heads of 256 over a paged cache.

    One projection gives q, k and v, and the calls take them as slices of its output."""

    Hq, Hkv, d, page = 16, 2, 256, 16

    def __init__(self, width, pages, cache, gen):
        cols = (self.Hq + 2 * self.Hkv) * self.d
        self.wqkv = (torch.randn(width, cols, generator=gen) / width ** 0.5).to(torch.bfloat16).to(DEV)
        self.wo = (torch.randn(self.Hq * self.d, width, generator=gen) / (self.Hq * self.d) ** 0.5).to(torch.bfloat16).to(DEV)
        kind = {"same": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[cache]
        pool = (pages, self.Hkv, self.page, self.d)
        self.k_cache, self.v_cache = (torch.empty(pool, dtype=kind, device=DEV) for _ in range(2))
        self.scales = {}
        if cache != "same":
            self.scales = {n: torch.empty(pool[:3], device=DEV) for n in ("k_scale", "v_scale")}

    def __call__(self, x, table, kv_lens, workspace, parents=None):
        """The new tokens of x (B sessions of T each), whose positions end at kv_lens; with parents, nodes of trees."""
        qkv = _linear(x, self.wqkv)
        q, k, v = qkv.unflatten(1, (-1, self.d)).split([self.Hq, self.Hkv, self.Hkv], dim=1)
        gdn.gdn_kv_write(k, v, self.k_cache, self.v_cache, table, kv_lens, **self.scales)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if parents is None:
            gdn.gdn_paged_attn(q, self.k_cache, self.v_cache, table, kv_lens, out, workspace=workspace, **self.scales)
        else:
            gdn.gdn_tree_attn(q, self.k_cache, self.v_cache, table, kv_lens, parents, out, workspace=workspace, **self.scales)
        return x + _linear(out.flatten(1), self.wo)

    def accept(self, table, kv_lens, path, counts, nodes):
        gdn.gdn_kv_keep(self.k_cache, self.v_cache, table, kv_lens, path, counts, T=nodes, **self.scales)


class HybridSession:
    def __init__(self, sessions=4, max_tokens=1024, width=512, cache="fp8", blocks=1, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.B = sessions
        per = -(-max_tokens // AttentionLayer.page)
        self.layers = []
        for _ in range(blocks):
            self.layers += [GdnLayer(width, sessions, gen) for _ in range(3)]
            self.layers.append(AttentionLayer(width, sessions * per, cache, gen))
        # each session's pages, in no particular order; every attention layer uses the same table
        self.table = torch.randperm(sessions * per, generator=gen).to(torch.int32).view(sessions, per).to(DEV)
        self.kv_lens = torch.zeros(sessions, dtype=torch.int32, device=DEV)
        A = AttentionLayer
        need = max(gdn.gdn_paged_attn_workspace_size(sessions, t, A.Hq, A.Hkv, A.d) for t in (1, max_tokens))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=DEV)
        self.graph = None

    def _forward(self, x, step):
        for layer in self.layers:
            if isinstance(layer, AttentionLayer):
                x = layer(x, self.table, self.kv_lens, self.workspace)
            else:
                x = layer.step(x) if step else layer.prefill(x, self.B)
        return x

    def prompt(self, x, fragment):
        """x [B, T, width], taken `fragment` tokens of every session at a time; the last token's output."""
        for a in range(0, x.shape[1], fragment):
            part = x[:, a:a + fragment].contiguous()
            self.kv_lens += part.shape[1]
            y = self._forward(part.flatten(0, 1), step=False).view(part.shape)
        return y[:, -1]

    def check(self, x, parents):
        """Drafted nodes of every session, x [B, T, width], parents [B, T]: the stack's output at each node."""
        self.kv_lens += x.shape[1]
        y = x.flatten(0, 1)
        for layer in self.layers:
            if isinstance(layer, AttentionLayer):
                y = layer(y, self.table, self.kv_lens, self.workspace, parents.flatten())
            else:
                y = layer.tree(y, parents.flatten())
        return y.view(x.shape)

    def accept(self, path, counts, nodes):
        """After `check`: the sessions go on from their accepted paths, path [B, P] and counts [B]."""
        for layer in self.layers:
            if isinstance(layer, AttentionLayer):
                layer.accept(self.table, self.kv_lens, path, counts, nodes)
            else:
                layer.accept(path, counts)
        self.kv_lens += counts - nodes

    def decode(self, x):
        """One token of every session, x [B, width], from a graph captured at the first call."""
        if self.graph is None:
            self.x = x.clone()
            # a warm-up step on copies of what a step changes (states; the cache row past the end is free to write)
            saved = [(layer, layer.state.clone()) for layer in self.layers if isinstance(layer, GdnLayer)]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.kv_lens += 1
                self._forward(self.x, step=True)
                self.kv_lens -= 1
            torch.cuda.current_stream().wait_stream(s)
            for layer, state in saved:
                layer.state.copy_(state)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.kv_lens += 1
                self.y = self._forward(self.x, step=True)
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def speculate(s, embed, token, nodes, rng):
    """One step by drafts: a draft model that guesses proposes a tree under each session's last token, the stack checks
    it, and the sessions move on by what stands. Returns the accepted tokens' number and the next tokens, both [B]."""
    B, V = s.B, embed.shape[0]
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device=DEV).div(2, rounding_mode="floor").repeat(B, 1)
    parents[:, 0] = -1  # (0 and its children 1, 2; 1 and its children 3, 4; ..)
    drafts = torch.full((B * nodes, V), 1.0 / V, device=DEV)
    tokens = torch.randint(V, (B, nodes), generator=rng, device=DEV).to(torch.int32)
    tokens[:, 0] = token
    y = s.check(embed[tokens.long()], parents)
    target = torch.softmax(torch.nn.functional.rms_norm(y, y.shape[-1:]).flatten(0, 1).float() @ embed.float().T, -1)
    path = torch.empty(B, nodes, dtype=torch.int32, device=DEV)
    counts, token = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))
    r, last = (torch.rand(n, generator=rng, device=DEV) for n in (B * nodes, B))
    gdn.gdn_tree_verify(target, drafts, tokens.flatten(), parents.flatten(), r, last, path, counts, token)
    s.accept(path, counts, nodes)
    return counts, token


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=("same", "fp8", "int8"), default="fp8")
    ap.add_argument("--sessions", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--nodes", type=int, default=8)
    a = ap.parse_args()
    width = 512
    s = HybridSession(a.sessions, a.prompt + a.tokens + a.tokens * a.nodes, width, a.cache)
    x = torch.randn(a.sessions, a.prompt, width, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    y = s.prompt(x, fragment=256)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    y = s.decode(torch.nn.functional.rms_norm(y, (width,)))  # (captures the graph)
    start.record()
    for _ in range(a.tokens - 1):
        y = s.decode(torch.nn.functional.rms_norm(y, (width,)))
    end.record()
    torch.cuda.synchronize()
    if gdn.gdn_get_device_status() != gdn.GDN_OK:
        raise RuntimeError("the device status reports inconsistent data")
    print(f"{a.sessions} sessions, cache {a.cache}: {a.prompt} prompt tokens, then {a.tokens} tokens at "
          f"{start.elapsed_time(end) / max(1, a.tokens - 1) * 1e3:.1f} us a step; lengths {s.kv_lens.tolist()}")
    rng = torch.Generator(device=DEV).manual_seed(2)
    embed = torch.randn(32, width, generator=rng, device=DEV).to(torch.bfloat16)
    token, steps, taken = torch.zeros(a.sessions, dtype=torch.int32, device=DEV), 0, torch.zeros(a.sessions, device=DEV)
    while steps < a.tokens and taken.min() < a.tokens:
        counts, token = speculate(s, embed, token, a.nodes, rng)
        taken += counts
        steps += 1
    if gdn.gdn_get_device_status() != gdn.GDN_OK:
        raise RuntimeError("the device status reports inconsistent data")
    print(f"drafts, trees of {a.nodes}: {steps} steps, {taken.mean().item() / steps:.2f} tokens a step; lengths {s.kv_lens.tolist()}")


if __name__ == "__main__":
    main()
