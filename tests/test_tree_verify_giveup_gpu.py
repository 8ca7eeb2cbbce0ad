"""Verification with a limit on the kernel's waits so short that they run out (GDN_TEST_WAIT_CYCLES): the CTAs of a sequence agree
on its outcome, which is the definition's or an idle row's and a flag, and the next call is right."""
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

from _kv import DEV
from test_tree_verify_gpu import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cycles", [1, 400, 1000, 1800, 2600, 4000, 8000])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("sequences", [1, 8, 20, 200])
def test_waits_that_run_out(sequences, drafts, cycles, monkeypatch):
    """Walks of several passes (rejected siblings), whose CTAs are not done at the same time."""
    c = case([9] * sequences, 20001 if sequences < 100 else 5001, drafts, "star", seed=sequences + cycles)
    c["r"] = 0.9 + 0.1 * c["r"]
    c["r"].clamp_(max=1 - 2.0 ** -24)
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
    other = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)  # (larger than L2)
    for _ in range(3):
        other.zero_()
        monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", str(cycles))
        path, counts, token = run(c, status=None)
        monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
        gave_up = [n for n in range(sequences) if counts[n] == 0]
        for n in gave_up:
            assert (path[n] == -1).all() and token[n] == -1
        check(c, (path, counts, token), but=gave_up)
        if cycles == 1:  # no sum comes from another CTA in one cycle
            assert gave_up
        got = run(c)
        check(c, got)


@pytest.mark.parametrize("cycles", [1, 1500])
def test_the_flag_tells(cycles, monkeypatch):
    """Flagged if and only if a sequence gave up."""
    c = case([5] * 40, 5001, True, "star", seed=2)
    for _ in range(10):
        assert gdn.gdn_get_device_status() == gdn.GDN_OK
        dev = {n: c[n].to(DEV) for n in ("target", "draft", "tokens", "r", "r_last")}
        parents = torch.tensor([u for t in c["trees"] for u in t], dtype=torch.int32, device=DEV)
        path = torch.full((40, 5), 99, dtype=torch.int32, device=DEV)
        counts, token = (torch.full((40,), 99, dtype=torch.int32, device=DEV) for _ in range(2))
        monkeypatch.setenv("GDN_TEST_WAIT_CYCLES", str(cycles))
        gdn.gdn_tree_verify(dev["target"], dev["draft"], dev["tokens"], parents, dev["r"], dev["r_last"], path, counts, token)
        monkeypatch.delenv("GDN_TEST_WAIT_CYCLES")
        status = gdn.gdn_get_device_status()
        assert status == (gdn.GDN_ERR_DEVICE_CHECK if (counts == 0).any() else gdn.GDN_OK)
        assert cycles > 1 or status == gdn.GDN_ERR_DEVICE_CHECK
