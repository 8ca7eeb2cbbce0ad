"""The attention kernels' give-up paths, exercised without any fault.

Every wait of the kernels is bounded; when one runs out, its warp raises the device status word and
leaves, the others follow as their own waits run out, copies and products in flight are waited for, and
the launch ends. GDN_TEST_WAIT_CYCLES shortens the limit (a test hook read at each call). Such a call
must report GDN_ERR_DEVICE_CHECK, and the next one with the normal limit must be right, with the same
workspace."""
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, Paged, assert_attention, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cycles", ["1", "2000"])
@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("T,G,d,longest", [(1, 8, 128, 160000), (40, 8, 256, 600), (64, 4, 64, 600)])
def test_wait_give_up_is_reported_and_next_call_passes(T, G, d, longest, cache, cycles, monkeypatch):
    # (one token: long enough for every warp to have more chunks than its ring, and read from memory rather than L2,
    # so that some copies are still on their way when a warp first looks)
    lens = [longest, 333, 70]
    case = Paged(lens, 2, d, 32, cache, "bf16", seed=3)
    kc, vc, ks, vs, table, kv_lens = case.tensors()
    q = torch.randn(3 * T, 2 * G, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    ws = torch.empty(gdn.gdn_paged_attn_workspace_size(3, T, 2 * G, 2, d), dtype=torch.uint8, device=DEV)
    call = lambda: gdn.gdn_paged_attn(q.to(DEV), kc, vc, table, kv_lens, out, ks, vs, workspace=ws)  # noqa: E731
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", cycles)
    torch.zeros(1 << 29, dtype=torch.uint8, device=DEV)  # (larger than L2)
    call()
    torch.cuda.synchronize()
    status = gdn.gdn_get_device_status()
    # (a wait sleeps in the hardware between looks at its limit, so 2000 cycles may pass unnoticed)
    assert status == gdn.GDN_ERR_DEVICE_CHECK or (cycles == "2000" and status == gdn.GDN_OK)
    monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
    out.fill_(float("nan"))
    call()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert_attention(out, *reference(case, q, [T] * 3, d ** -0.5))
