"""The hybrid session example: states, paged caches and lengths carried through fragments and a graph.

A session's outputs depend on its tokens alone, not on how they were cut into fragments and steps. Each
layer rounds its outputs to bf16 (2^-9 relative each, 8 roundings along the four layers and their residual
sums), and cut differently the same sums are taken in another order before they are rounded, so two
cuts may differ by single bf16 roundings that later layers carry on: 8 roundings of 2^-9, doubled for
both sides, is 3.2e-2 of the norm. An e4m3 cache rounds keys and values to 2^-4 relative, where such
a difference can move a code by one step, of one row in a sum of many: the same bound holds with room."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("cache", ["same", "fp8", "int8"])
def test_cuts_of_a_session_agree(cache):
    from hybrid_session import HybridSession
    import gated_deltanet_linear_delta_gb300 as gdn
    B, T, width = 3, 150, 256
    x = torch.randn(B, T, width, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to("cuda")
    whole = HybridSession(B, T, width, cache).prompt(x, fragment=T)
    parts = HybridSession(B, T, width, cache).prompt(x, fragment=64)
    steps = HybridSession(B, T, width, cache)
    steps.prompt(x[:, :140], fragment=100)
    for t in range(140, T):
        last = steps.decode(x[:, t])
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert steps.kv_lens.tolist() == [T] * B
    ref = whole.double()
    for y in (parts, last):
        assert ((y.double() - ref).norm() / ref.norm()).item() <= 3.2e-2


@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_a_quantised_cache_stays_close(cache):
    """8-bit keys and values against bf16 ones: e4m3 rounds to 2^-4 of each element at most, int8 to 1/254
    of a row's largest. The attention layer is one of four that add to the residual stream."""
    from hybrid_session import HybridSession
    B, T, width = 2, 200, 256
    x = torch.randn(B, T, width, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to("cuda")
    ref = HybridSession(B, T, width, "same").prompt(x, fragment=128).double()
    y = HybridSession(B, T, width, cache).prompt(x, fragment=128).double()
    assert ((y - ref).norm() / ref.norm()).item() <= 2.0 ** -4
