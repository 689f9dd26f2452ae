"""What Slots keeps alive of the sources of base loads, on the CPU with the library's calls
replaced: everything that may still be read, and no more than a bound of it."""
import gc
import weakref

import pytest
import torch

from lora_adapter_application_amd import binding


@pytest.fixture
def slots(monkeypatch):
    calls = []
    monkeypatch.setattr(binding, "lora_slots_create", lambda *a: 1)
    monkeypatch.setattr(binding, "lora_slots_destroy", lambda ctx: None)
    monkeypatch.setattr(binding, "lora_base_load", lambda ctx, module, *a: calls.append(("load", module)))
    monkeypatch.setattr(binding, "lora_sync_loads", lambda ctx: calls.append(("sync",)))
    S = binding.Slots(1, 1, [(16384, 65536)], "bf16", 1)
    S.calls = calls
    yield S
    S.ctx = None


def sources(d_in=16384, d_out=65536, group=128):
    """Half a GiB of q, without memory behind it."""
    q = torch.empty(d_out, d_in // 2, dtype=torch.uint8, device="meta")
    s = torch.empty(d_out, d_in // group, device="meta")
    return q, s


def test_sources_stay_until_sync_loads(slots):
    q, s = sources()
    alive = weakref.ref(q)
    slots.load_base(0, q, s)
    del q, s
    gc.collect()
    assert alive() is not None
    slots.sync_loads()
    gc.collect()
    assert alive() is None


def test_a_program_that_never_syncs_holds_a_bounded_amount(slots):
    """Forty loads of half a GiB each: before the sources held pass the bound the loads are
    waited for and the sources let go."""
    alive = []
    for _ in range(40):
        q, s = sources()
        alive.append(weakref.ref(q))
        slots.load_base(0, q, s)
        del q, s
        gc.collect()
        held = [r for r in alive if r() is not None]
        assert alive[-1]() is not None
        assert len(held) <= 2              # 1 GiB, or the one load that is larger
    # nothing was let go without a wait before it
    assert slots.calls.count(("sync",)) >= 19 and slots.calls.count(("load", 0)) == 40


def test_small_loads_are_not_waited_for(slots):
    slots.modules = [(256, 64)]
    for _ in range(100):
        slots.load_base(0, *sources(256, 64))
    assert ("sync",) not in slots.calls
