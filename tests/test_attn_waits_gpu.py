"""Waits of the 128-row attention kernel that run out at different places.

A limit of a few cycles makes the first wait of every warp run out; longer ones let a warp or two get further, so
that others run out of time waiting for them: among these the wait of the warp that copies Q for the other warps to
have read what the stage held. Whatever runs out, the launch ends; the status word tells, and a call that it does not
name is right."""
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import CACHES, DEV, Paged, assert_attention, reference

pytestmark = pytest.mark.gpu


def setting(T, G, d, cache, lens=(600, 333, 70)):
    case = Paged(lens, 2, d, 32, cache, "bf16", seed=3)
    kc, vc, ks, vs, table, kv_lens = case.tensors()
    q = torch.randn(len(lens) * T, 2 * G, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    qd = q.to(DEV)
    ws = torch.empty(gdn.gdn_paged_attn_workspace_size(len(lens), T, 2 * G, 2, d), dtype=torch.uint8, device=DEV)

    def call(out):
        gdn.gdn_paged_attn(qd, kc, vc, table, kv_lens, out, ks, vs, workspace=ws)

    return call, torch.empty_like(qd), reference(case, q, [T] * len(lens), d ** -0.5)


@pytest.mark.parametrize("cycles", [1, 200, 700, 1500, 4000, 12000])
@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("T,G,d", [(40, 8, 256), (100, 8, 128), (64, 4, 64)])
def test_any_wait_may_run_out(T, G, d, cache, cycles, monkeypatch):
    call, out, want = setting(T, G, d, cache)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    for _ in range(3):
        monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", str(cycles))
        call(out)
        torch.cuda.synchronize()
        monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
        status = gdn.gdn_get_device_status()
        assert status in (gdn.GDN_OK, gdn.GDN_ERR_DEVICE_CHECK)
        if status == gdn.GDN_OK:
            assert_attention(out, *want)
    out.fill_(float("nan"))
    call(out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    assert_attention(out, *want)


@pytest.mark.parametrize("cache", sorted(CACHES))
@pytest.mark.parametrize("T,G,d", [(40, 8, 256), (100, 8, 128), (64, 4, 64)])
def test_a_call_queued_behind_one_that_gives_up(T, G, d, cache, monkeypatch):
    """Copies of a call that gives up land before its blocks leave: the call right behind it uses the same shared
    memory, and its results are right."""
    call, out, want = setting(T, G, d, cache)
    lost = torch.empty_like(out)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    for _ in range(4):
        torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)  # (larger than L2: copies come from memory)
        monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", "1")
        call(lost)
        monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
        call(out)
        assert gdn.gdn_get_device_status() == gdn.GDN_ERR_DEVICE_CHECK
        assert_attention(out, *want)
