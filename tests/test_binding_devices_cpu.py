"""The binding refuses tensors on another device than the current one, whichever
argument it is, without a GPU: tensors and library are stand-ins."""
import pytest
import torch

import expert_ffn_router_b200 as M


class T:
    """A CUDA tensor as far as the binding looks."""

    def __init__(self, *shape, dtype=torch.float32, dev=0):
        self.shape, self.dtype, self.dev, self.is_cuda = shape, dtype, dev, True
        self.device = torch.device("cuda", dev)

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(torch.empty(self.shape, device="meta").stride())

    def data_ptr(self):
        return 1 << 20


class Lib:
    """Takes every call."""

    def __getattr__(self, name):
        return lambda *a: M.MOE_OK


@pytest.fixture
def launched(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "lib", Lib())
    monkeypatch.setattr(M, "_stream", lambda s: 0)
    monkeypatch.setattr(M, "_stream_on", lambda s, d: 0)


I32, U8, BF = torch.int32, torch.uint8, torch.bfloat16
C = M.config(128, 64, 24, 5)
R = M.gate_rule()


def gate(a):
    M.moe_gate(C, R, a("logits", 4, 24), a("bias", 24), a("topk_idx", 4, 5, dtype=I32), a("topk_w", 4, 5))


def route_gated(a):
    M.moe_route_gated(C, R, a("x", 4, 128), a("w_router", 24, 128), a("bias", 24), a("topk_idx", 4, 5, dtype=I32),
                      a("topk_w", 4, 5), a("ws", 1000, dtype=U8))


def layer_routed(a):
    pool = M.make_pool(a("pool.w", 100, dtype=U8), a("pool.s", 100), a("pool.slot_of", 25, dtype=I32), 3)
    M.moe_layer_routed(C, pool, a("topk_idx", 4, 5, dtype=I32), a("topk_w", 4, 5), a("x", 4, 128), a("out", 4, 128),
                       a("ws", 1000, dtype=U8))


def plan(a):
    M.moe_adapter_plan(3, a("adapter_of", 4, dtype=I32), a("plan", 1000, dtype=U8))


def adapter(a):
    ad = M.make_adapters(a("adapters.a", 3, 16, 128, dtype=BF), a("adapters.b", 3, 64, 16, dtype=BF),
                         a("adapters.rank", 3, dtype=I32), a("adapters.scale", 3))
    M.moe_adapter(ad, a("plan", 1000, dtype=U8), a("x", 4, 128, dtype=torch.int8), a("y", 4, 64), base=a("base", 4, 64),
                  sx=a("sx", 4))


NAMES = {gate: ["logits", "bias", "topk_idx", "topk_w"],
         route_gated: ["x", "w_router", "bias", "topk_idx", "topk_w", "ws"],
         layer_routed: ["pool.w", "pool.s", "pool.slot_of", "topk_idx", "topk_w", "x", "out", "ws"],
         plan: ["adapter_of", "plan"],
         adapter: ["adapters.a", "adapters.b", "adapters.rank", "adapters.scale", "plan", "x", "y", "base", "sx"]}


@pytest.mark.parametrize("call", list(NAMES))
def test_all_on_the_current_device(launched, call):
    call(lambda name, *shape, dtype=torch.float32: T(*shape, dtype=dtype))


@pytest.mark.parametrize("call,name", [(c, n) for c in NAMES for n in NAMES[c]])
def test_one_on_another_device(launched, call, name):
    with pytest.raises(ValueError, match="device"):
        call(lambda n, *shape, dtype=torch.float32: T(*shape, dtype=dtype, dev=int(n == name)))


@pytest.mark.parametrize("call", [layer_routed, adapter])
def test_tables_all_on_another_device(launched, call):
    """A pool or a set of adapters that agrees with itself, but not with the call."""
    with pytest.raises(ValueError, match="device"):
        call(lambda n, *shape, dtype=torch.float32: T(*shape, dtype=dtype, dev=int("." in n)))
