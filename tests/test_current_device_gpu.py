"""Every call refuses tensors that are not on the current device, and launches nothing: seen from the host, by a current
device that is not the tensors' (the GPU's own stays as it is)."""
import pytest
import torch

import gated_deltanet_linear_delta_gb300 as gdn

pytestmark = pytest.mark.gpu


def calls():
    b = dict(dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.ones(2, h, 128, **b) for h in (2, 2, 4))
    g, beta = (torch.zeros(2, 4, **b) for _ in range(2))
    state = torch.zeros(2, 4, 128, 128, device="cuda")
    out = torch.full_like(v, 7.0)
    f = [torch.full((2, h), 7.0, device="cuda") for h in (2, 2, 4, 4)]
    kc, vc = (torch.full((3, 2, 16, 128), 7.0, **b) for _ in range(2))
    table, lens = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    ko, vo, ao = (torch.full((2, 2, 128), 7.0, **b) for _ in range(3))
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    kept = [out, *f, kc, vc, ko, vo, ao]
    return kept, {
        "prefill": lambda: gdn.gdn_prefill(q, k, v, g, beta, None, state, out, B=2, T=1),
        "prefill_static": lambda: gdn.gdn_prefill_static(q, k, v, g, beta, None, state, out, B=2, T=1),
        "prefill_ws": lambda: gdn.gdn_prefill_ws(q, k, v, g, beta, None, state, out, None, B=2, T=1),
        "decode_step": lambda: gdn.gdn_decode_step(q, k, v, g, beta, state, out),
        "decode_step_slots": lambda: gdn.gdn_decode_step_slots(q, k, v, g, beta, state, slots, out),
        "prepass": lambda: gdn.gdn_prepass(q, k, g, beta, *f, B=2, T=1),
        "kv_write": lambda: gdn.gdn_kv_write(k, k, kc, vc, table, lens),
        "kv_read": lambda: gdn.gdn_kv_read(kc, vc, table, lens, ko, vo),
        "paged_attn": lambda: gdn.gdn_paged_attn(q, kc, vc, table, lens, ao),
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
    assert all((t == 7.0).all() for t in kept)
    monkeypatch.undo()
    for call in by_name.values():  # and the same calls are sound
        call()
    assert gdn.gdn_get_device_status() == gdn.GDN_OK
