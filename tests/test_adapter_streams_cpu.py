"""adapter_plan on a stream of the caller's, without a GPU: what it asks of the
streams and the allocator, and in which order."""
import pytest
import torch

import expert_ffn_router_b200 as M


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")


class Plan:
    def __init__(self, log):
        self.log = log

    def record_stream(self, s):
        self.log.append(f"plan is used on {s.name}")


@pytest.fixture
def calls(monkeypatch):
    log = []
    here, side = Stream("current", log), Stream("side", log)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: log.append("current allocates") or Plan(log))
    monkeypatch.setattr(M, "moe_adapter_plan", lambda n, of, plan, stream=None: log.append(f"{(stream or here).name} fills"))
    return log, here, side


def test_plan_on_another_stream_waits_for_the_one_it_is_allocated_on(calls):
    """Its memory may be a plan's that calls on the current stream still read;
    and the allocator must not hand it out again before the other stream's
    work is done."""
    log, here, side = calls
    M.adapter_plan(3, torch.zeros(4, dtype=torch.int32), stream=side)
    assert log.index("current allocates") < log.index("side waits for current") < log.index("side fills")
    assert "plan is used on side" in log


def test_plan_on_the_current_stream_needs_neither(calls):
    log, here, side = calls
    for s in (None, here):
        log.clear()
        M.adapter_plan(3, torch.zeros(4, dtype=torch.int32), stream=s)
        assert log == ["current allocates", "current fills"]
