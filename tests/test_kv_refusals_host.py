"""More of what the paged cache calls refuse on the host, before any device work. These run without a GPU."""
import math
import os
import subprocess
import sys

import pytest

from test_kv_abi_host import attn, lib, pytestmark  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype,cache", [(0, 0), (0, 2), (0, 3), (1, 1), (1, 3)])
@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite(lib, scale, dtype, cache):  # noqa: F811
    assert attn(lib, scale=scale, dtype=dtype, cache=cache) == -1


ODD = """
import sys, torch
import gated_deltanet_linear_delta_gb300 as gdn
kind = sys.argv[1]
def odd(shape, dtype):
    if kind == "sparse":
        return torch.ones(shape, dtype=dtype).to_sparse()
    if kind == "nested" and len(shape) > 1:
        return torch.nested.nested_tensor([torch.ones(shape[1:], dtype=dtype) for _ in range(shape[0])], dtype=dtype)
    if kind == "ragged" and len(shape) > 2:
        return torch.nested.nested_tensor([torch.ones((1 + i % 2,) + tuple(shape[2:]), dtype=dtype) for i in range(shape[0])], dtype=dtype)
    return None
rows, cache, b, i = (4, 2, 64), (3, 2, 16, 64), torch.bfloat16, torch.int32
good = dict(k=torch.ones(rows, dtype=b), v=torch.ones(rows, dtype=b), k_cache=torch.ones(cache, dtype=b),
            v_cache=torch.ones(cache, dtype=b), block_table=torch.zeros(2, 1, dtype=i), kv_lens=torch.ones(2, dtype=i),
            k_scale=torch.ones(cache[:3]), v_scale=torch.ones(cache[:3]), cu_seqlens=torch.zeros(3, dtype=i))
for name, x in good.items():
    y = odd(tuple(x.shape), x.dtype)
    if y is None:
        continue
    for scales in (False, True):
        a = dict(good)
        if scales:
            a["k_cache"], a["v_cache"] = (torch.ones(cache, dtype=torch.int8) for _ in range(2))
        a[name] = odd(tuple(x.shape), a[name].dtype)
        q, out = a.pop("k"), a.pop("v")
        where = (a.pop("k_cache"), a.pop("v_cache"), a.pop("block_table"), a.pop("kv_lens"))
        for call in (lambda: gdn.gdn_kv_write(q, out, *where, **a), lambda: gdn.gdn_kv_read(*where, q, out, **a),
                     lambda: gdn.gdn_paged_attn(q, *where, out, **a)):
            try:
                call()
            except (TypeError, ValueError, RuntimeError):
                continue
            sys.exit(f"{name}: no exception")
print("all refused")
"""


@pytest.mark.parametrize("kind", ["sparse", "nested", "ragged"])
def test_tensors_without_a_plain_layout(lib, kind):  # noqa: F811
    """Sparse and nested tensors raise in Python; an exception that left the module would end the process."""
    r = subprocess.run([sys.executable, "-c", ODD, kind], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "all refused" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_tensors_of_another_device(monkeypatch):
    """The stream of every call is asked for with one of its tensors, which has to be on the current device."""
    import gated_deltanet_linear_delta_gb300 as gdn

    class Elsewhere:
        def get_device(self):
            return 1

    monkeypatch.setattr(gdn, "_current_device", lambda: 0, raising=False)
    for stream in (None, 0, 1234):
        with pytest.raises(ValueError):
            gdn._stream(stream, Elsewhere())
    monkeypatch.setattr(gdn, "_current_device", lambda: 1)
    assert gdn._stream(1234, Elsewhere()) == 1234
