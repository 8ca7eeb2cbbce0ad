"""Host-side checks of the paged cache calls: bad arguments are refused with the documented status
before any device work. These calls launch nothing; they run without a GPU."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc is needed to build the library")

A = 4096  # an aligned fake address: the checks never read it
BASE = dict(k=A, v=A, kc=A, vc=A, ks=A, vs=A, table=A, lens=A, cu=None, B=2, T=3, Hq=4, Hkv=2, d=128, pages=8,
            page=16, width=4, stride=None, scale=1.0, dtype=0, cache=0, ws=A, ws_bytes=1 << 30)


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_delta_gb300 import _build
    import gated_deltanet_linear_delta_gb300 as gdn
    _build.build()
    return gdn.library()


def p(x):
    return None if x is None else ctypes.c_void_p(x)


def write(lib, **kw):
    a = {**BASE, **kw}
    st = a["Hkv"] * a["d"] if a["stride"] is None else a["stride"]
    return lib.gdn_kv_write(p(a["k"]), p(a["v"]), p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["table"]),
                            p(a["lens"]), p(a["cu"]), a["B"], a["T"], a["Hkv"], a["d"], a["pages"], a["page"],
                            a["width"], st, st, a["dtype"], a["cache"], None)


def read(lib, **kw):
    a = {**BASE, **kw}
    st = a["Hkv"] * a["d"] if a["stride"] is None else a["stride"]
    return lib.gdn_kv_read(p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["table"]), p(a["lens"]), p(a["cu"]),
                           p(a["k"]), p(a["v"]), a["B"], a["T"], a["Hkv"], a["d"], a["pages"], a["page"], a["width"],
                           st, st, a["dtype"], a["cache"], None)


def attn(lib, **kw):
    a = {**BASE, **kw}
    st = a["Hq"] * a["d"] if a["stride"] is None else a["stride"]
    return lib.gdn_paged_attn(p(a["k"]), p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["table"]), p(a["lens"]),
                              p(a["cu"]), p(a["v"]), a["B"], a["T"], a["Hq"], a["Hkv"], a["d"], a["pages"], a["page"],
                              a["width"], st, a["scale"], a["dtype"], a["cache"], p(a["ws"]), a["ws_bytes"], None)


SHARED = [
    (dict(d=96), -2), (dict(d=32), -2), (dict(d=512), -2), (dict(page=8), -2), (dict(page=48), -2), (dict(page=512), -2),
    (dict(page=0), -2), (dict(dtype=2), -2), (dict(dtype=0, cache=1), -2), (dict(dtype=1, cache=0), -2),
    (dict(cache=4), -2), (dict(cache=-1), -2), (dict(Hkv=0), -1), (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=70000), -1),
    (dict(pages=-1), -1), (dict(width=-1), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(k=A + 2), -1),
    (dict(v=A + 8), -1), (dict(kc=None), -1), (dict(vc=A + 4), -1), (dict(table=None), -1), (dict(table=A + 2), -1),
    (dict(lens=None), -1), (dict(lens=A + 2), -1), (dict(cu=A + 8), -1), (dict(cache=2, ks=None), -1),
    (dict(cache=3, vs=None), -1), (dict(cache=2, ks=A + 4), -1), (dict(stride=8), -1), (dict(stride=516), -1),
    (dict(dtype=1, cache=1, stride=514), -1), (dict(T=1 << 30, B=4), -1), (dict(pages=1 << 30, Hkv=4, Hq=4), -1),
    (dict(width=1 << 28), -1),
]


@pytest.mark.parametrize("call", [write, read, attn], ids=["write", "read", "attn"])
@pytest.mark.parametrize("kw,code", SHARED)
def test_rejects(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), -1), (dict(Hq=0), -1), (dict(Hq=130), -2), (dict(ws=None), -1), (dict(ws=A + 128), -1),
    (dict(ws_bytes=1000), -1), (dict(pages=0), -1), (dict(width=0), -1),
])
def test_attention_rejects(lib, kw, code):
    assert attn(lib, **kw) == code


@pytest.mark.parametrize("call", [write, read, attn], ids=["write", "read", "attn"])
@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0)])
def test_nothing_to_do_is_ok(lib, call, kw):
    assert call(lib, k=None, v=None, kc=None, table=None, lens=None, ws=None, **kw) == 0


def test_a_sound_call_without_a_gpu_reports_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert write(lib) == -3 and read(lib) == -3 and attn(lib) == -3


def test_workspace_size(lib):
    f = lib.gdn_paged_attn_workspace_size
    assert f(1, 1, 0, 16, 2, 96) == 0 and f(1, 1, 0, 15, 2, 128) == 0 and f(0, 1, 0, 16, 2, 128) == 0
    assert f(1, 0, 0, 16, 2, 128) == 0
    one, many = f(1, 1, 0, 16, 2, 256), f(64, 1, 0, 16, 2, 256)
    assert one == many > 0  # two parts of 8 rows per SM, whatever the batch
    assert one >= 152 * 2 * 8 * 256 * 4
    assert f(1, 4096, 0, 16, 2, 256) == f(8, 4096, 1, 16, 2, 256) <= 48 << 20
    assert attn(lib, B=1, T=1, Hq=16, d=256, ws_bytes=one - 1) == -1


def test_binding_refuses_what_it_cannot_pass_on():
    import gated_deltanet_linear_delta_gb300 as gdn
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    for bad in (dict(v=k[:, :1]), dict(v=k.float()), dict(vc=kc[:2]), dict(vc=kc.float()), dict(kc=kc[..., :32], vc=kc[..., :32]),
                dict(table=table[:2]), dict(lens=lens[:3]), dict(T=3), dict(kc=kc[:, :1], vc=kc[:, :1])):
        a = {**dict(v=k, kc=kc, vc=kc, table=table, lens=lens, T=None), **bad}
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_kv_write(k, a["v"], a["kc"], a["vc"], a["table"], a["lens"], T=a["T"])
    for bad in (dict(table=table.long()), dict(lens=lens.long()), dict(kc=kc.half(), vc=kc.half()),
                dict(kc=kc.to(torch.int8), vc=kc.to(torch.int8))):  # an 8-bit cache without scales
        a = {**dict(kc=kc, vc=kc, table=table, lens=lens), **bad}
        with pytest.raises(TypeError):
            gdn.gdn_kv_write(k, k, a["kc"], a["vc"], a["table"], a["lens"])
    with pytest.raises(ValueError):  # CPU tensors
        gdn.gdn_kv_write(k, k, kc, kc, table, lens)
    with pytest.raises(ValueError):
        gdn.gdn_paged_attn(k, kc, kc, table, lens, torch.zeros(4, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):  # heads not contiguous
        gdn.gdn_kv_write(k.transpose(0, 1).contiguous().transpose(0, 1), k, kc, kc, table, lens)
