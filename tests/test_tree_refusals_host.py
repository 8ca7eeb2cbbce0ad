"""Host-side checks of the calls on trees: bad arguments are refused with the documented status before any device work.
These calls launch nothing; they run without a GPU."""
import math
import os
import subprocess
import sys

import pytest
import torch

from test_kv_abi_host import A, SHARED, lib, p, pytestmark  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = dict(k=A, v=A, kc=A, vc=A, ks=A, vs=A, table=A, lens=A, cu=None, parents=A, path=A, counts=A, width_path=8, B=2, T=3,
            Hq=4, Hkv=2, d=128, pages=8, page=16, width=4, stride=None, scale=1.0, dtype=0, cache=0, ws=A, ws_bytes=1 << 30,
            q=A, g=A, b=A, state=A, state2=A, slots=None, num_slots=0, Hk=2, Hv=4, dk=128, dv=128, out=A,
            target=A, draft=A, tokens=A, r=A, last=A, nxt=A, V=1000, ts=None, ds=None)


def attn(lib, **kw):
    a = {**BASE, **kw}
    st = a["Hq"] * a["d"] if a["stride"] is None else a["stride"]
    return lib.gdn_tree_attn(p(a["k"]), p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["table"]), p(a["lens"]), p(a["cu"]),
                             p(a["parents"]), p(a["v"]), a["B"], a["T"], a["Hq"], a["Hkv"], a["d"], a["pages"], a["page"],
                             a["width"], st, a["scale"], a["dtype"], a["cache"], p(a["ws"]), a["ws_bytes"], None)


def keep(lib, **kw):
    a = {**BASE, **kw}
    return lib.gdn_kv_keep(p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["table"]), p(a["lens"]), p(a["cu"]), p(a["path"]),
                           p(a["counts"]), a["B"], a["T"], a["width_path"], a["Hkv"], a["d"], a["pages"], a["page"], a["width"],
                           a["cache"], None)


def scan(lib, **kw):
    a = {**BASE, **kw}
    return lib.gdn_tree_scan(p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), p(a["b"]), p(a["state"]), p(a["slots"]), p(a["parents"]),
                             p(a["cu"]), p(a["out"]), a["B"], a["T"], a["num_slots"], a["Hk"], a["Hv"], a["dk"], a["dv"], a["dtype"], None)


def advance(lib, **kw):
    a = {**BASE, **kw}
    return lib.gdn_tree_advance(p(a["k"]), p(a["v"]), p(a["g"]), p(a["b"]), p(a["state"]), p(a["state2"]), p(a["slots"]), p(a["path"]),
                                p(a["counts"]), p(a["cu"]), a["B"], a["T"], a["width_path"], a["num_slots"], a["Hk"], a["Hv"],
                                a["dk"], a["dv"], a["dtype"], None)


def verify(lib, **kw):
    a = {**BASE, **kw}
    ts, ds = (a["V"] if a[n] is None else a[n] for n in ("ts", "ds"))
    return lib.gdn_tree_verify(p(a["target"]), p(a["draft"]), p(a["tokens"]), p(a["parents"]), p(a["r"]), p(a["last"]), p(a["cu"]),
                               p(a["path"]), p(a["counts"]), p(a["nxt"]), a["B"], a["T"], a["V"], ts, ds, a["width_path"], None)


@pytest.fixture(scope="module", autouse=True)
def _types(lib):  # noqa: F811
    for f in (lib.gdn_tree_attn, lib.gdn_kv_keep, lib.gdn_tree_scan, lib.gdn_tree_advance, lib.gdn_tree_verify):
        assert f.argtypes is not None


@pytest.mark.parametrize("kw,code", SHARED)
def test_attention_refuses_what_paged_attention_does(lib, kw, code):  # noqa: F811
    if kw.get("T") == 1 << 30:
        code = -2  # more than 64 nodes
    assert attn(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), -1), (dict(Hq=130), -2), (dict(ws=None), -1), (dict(ws=A + 128), -1), (dict(ws_bytes=1000), -1), (dict(pages=0), -1),
    (dict(width=0), -1), (dict(parents=None), -1), (dict(parents=A + 2), -1), (dict(T=65), -2), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(cu=A + 4), -1)])
def test_attention_refuses(lib, kw, code):  # noqa: F811
    assert attn(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -2), (dict(page=48), -2), (dict(cache=4), -2), (dict(cache=-1), -2), (dict(Hkv=0, Hq=1), -1), (dict(B=-1), -1), (dict(T=-1), -1),
    (dict(B=70000), -1), (dict(T=65), -2), (dict(pages=-1), -1), (dict(kc=None), -1), (dict(vc=A + 4), -1), (dict(table=None), -1),
    (dict(table=A + 2), -1), (dict(lens=None), -1), (dict(lens=A + 1), -1), (dict(cache=2, ks=None), -1), (dict(cache=3, vs=A + 4), -1),
    (dict(path=None), -1), (dict(path=A + 2), -1), (dict(counts=None), -1), (dict(counts=A + 3), -1), (dict(width_path=-1), -1),
    (dict(cu=A + 8), -1), (dict(pages=1 << 30, Hkv=4), -1), (dict(width=1 << 28), -1)])
def test_keep_refuses(lib, kw, code):  # noqa: F811
    assert keep(lib, **kw) == code


STATES = [(dict(Hk=0), -1), (dict(Hv=3), -1), (dict(Hv=70000, Hk=1), -1), (dict(dk=96), -2), (dict(dv=256), -2), (dict(dtype=2), -2), (dict(dtype=-1), -2),
          (dict(B=-1), -1), (dict(T=-1), -1), (dict(T=65), -2), (dict(B=65536), -1), (dict(k=None), -1), (dict(k=A + 8), -1), (dict(v=None), -1),
          (dict(g=None), -1), (dict(b=A + 2), -1), (dict(state=None), -1), (dict(state=A + 4), -1), (dict(slots=A, num_slots=-1), -1),
          (dict(slots=A + 1, num_slots=4), -1), (dict(slots=A, num_slots=1 << 30), -1), (dict(cu=A + 4), -1)]


@pytest.mark.parametrize("kw,code", STATES + [(dict(q=None), -1), (dict(q=A + 2), -1), (dict(out=None), -1), (dict(out=A + 4), -1),
                                              (dict(parents=None), -1), (dict(parents=A + 2), -1)])
def test_scan_refuses(lib, kw, code):  # noqa: F811
    assert scan(lib, **kw) == code


@pytest.mark.parametrize("kw,code", STATES + [(dict(state2=None), -1), (dict(state2=A + 8), -1), (dict(path=None), -1), (dict(path=A + 1), -1),
                                              (dict(counts=None), -1), (dict(counts=A + 2), -1), (dict(width_path=-1), -1)])
def test_advance_refuses(lib, kw, code):  # noqa: F811
    assert advance(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(V=0), -1), (dict(V=-4), -1), (dict(V=(1 << 22) + 1, ts=1 << 23, ds=1 << 23), -2), (dict(ts=999), -1), (dict(ds=0), -1),
    (dict(ts=1 << 41), -1), (dict(width_path=2), -1), (dict(width_path=-1, cu=A), -1), (dict(width_path=(1 << 20) + 1), -1), (dict(T=65), -2),
    (dict(B=-1), -1), (dict(B=65536), -1), (dict(T=-1), -1), (dict(target=None), -1), (dict(target=A + 4), -1), (dict(draft=A + 8), -1),
    (dict(tokens=None), -1), (dict(tokens=A + 2), -1), (dict(parents=None), -1), (dict(r=None), -1), (dict(r=A + 1), -1), (dict(last=None), -1),
    (dict(last=A + 2), -1), (dict(path=None), -1), (dict(path=A + 2), -1), (dict(counts=None), -1), (dict(nxt=None), -1), (dict(nxt=A + 2), -1),
    (dict(cu=A + 4), -1)])
def test_verify_refuses(lib, kw, code):  # noqa: F811
    assert verify(lib, **kw) == code


def test_nothing_to_do_is_ok(lib):  # noqa: F811
    none = {n: None for n in ("k", "v", "kc", "vc", "table", "lens", "parents", "path", "counts", "ws", "q", "g", "b", "state", "state2", "out",
                              "target", "draft", "tokens", "r", "last", "nxt")}
    for call in (attn, keep, scan, advance, verify):
        assert call(lib, **{**none, "B": 0}) == 0
    for call in (attn, keep, scan):
        assert call(lib, **{**none, "T": 0}) == 0


def test_a_sound_call_without_a_gpu_reports_cuda_error(lib):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (attn, keep, scan, advance, verify):
        assert call(lib) == -3
    assert verify(lib, draft=None) == -3 and scan(lib, slots=A, num_slots=5) == -3


# every tensor of every call by turns replaced by what does not fit; the call has to raise in Python
ODD = """
import sys, torch
import gated_deltanet_linear_delta_gb300 as gdn
kind = sys.argv[1]
i, f, b = torch.int32, torch.float32, torch.bfloat16
rows, cache = (6, 2, 64), (3, 2, 16, 64)
z = lambda *s, dtype=b: torch.ones(*s, dtype=dtype)
kv = dict(k_cache=z(*cache), v_cache=z(*cache), block_table=z(2, 1, dtype=i), kv_lens=z(2, dtype=i))
calls = {
  gdn.gdn_tree_attn: (dict(q=z(6, 4, 64), **kv, parents=z(6, dtype=i), out=z(6, 4, 64)), {}),
  gdn.gdn_kv_keep: (dict(**kv, path=z(2, 3, dtype=i), counts=z(2, dtype=i)), dict(T=3)),
  gdn.gdn_tree_scan: (dict(q=z(*rows), k=z(*rows), v=z(6, 4, 32), g=z(6, 4), b=z(6, 4), state=z(2, 4, 32, 64, dtype=f),
                           parents=z(6, dtype=i), out=z(6, 4, 32)), {}),
  gdn.gdn_tree_advance: (dict(k=z(*rows), v=z(6, 4, 32), g=z(6, 4), b=z(6, 4), state_in=z(2, 4, 32, 64, dtype=f),
                              state_out=z(2, 4, 32, 64, dtype=f), path=z(2, 3, dtype=i), counts=z(2, dtype=i)), {}),
  gdn.gdn_tree_verify: (dict(target_probs=z(6, 50, dtype=f), draft_probs=z(6, 50, dtype=f), tokens=z(6, dtype=i), parents=z(6, dtype=i),
                             r=z(6, dtype=f), r_last=z(2, dtype=f), path=z(2, 3, dtype=i), counts=z(2, dtype=i), next=z(2, dtype=i)), {}),
}
def odd(x):
    if kind == "sparse": return x.to_sparse()
    if kind == "nested": return torch.nested.nested_tensor([x[j] for j in range(x.shape[0])], dtype=x.dtype) if x.dim() > 1 else x.to_sparse()
    if kind == "dtype": return x.double()
    if kind == "shape": return x[:-1] if x.dim() == 1 else x.narrow(x.dim() - 1, 0, x.shape[-1] - 1).contiguous() if x.shape[-1] > 1 else x[:1]
    if kind == "dims": return x[None]
    if kind == "number": return 3
    if kind == "cpu": return x
for call, (args, more) in calls.items():
    for name in args:
        a = dict(args)
        a[name] = odd(a[name])
        if kind == "cpu" and name != next(iter(args)): continue
        try:
            call(**a, **more)
        except (TypeError, ValueError, RuntimeError, AttributeError):
            continue
        sys.exit(f"{call.__name__}, {name}: no exception")
    for extra in (dict(cu_seqlens=z(3, dtype=f)), dict(cu_seqlens=z(3, 1, dtype=i)), dict(T=5), dict(T=-1)):
        if call is gdn.gdn_kv_keep and extra == dict(T=5): continue
        try:
            call(**args, **{**more, **extra})
        except (TypeError, ValueError, RuntimeError):
            continue
        sys.exit(f"{call.__name__}, {extra}: no exception")
print("all refused")
"""


@pytest.mark.parametrize("kind", ["sparse", "nested", "dtype", "shape", "dims", "number", "cpu"])
def test_tensors_that_do_not_fit(lib, kind):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", ODD, kind], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "all refused" in r.stdout, (r.returncode, r.stdout[-500:], r.stderr[-2000:])
