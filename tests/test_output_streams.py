"""CPU check of where the Python front end takes the memory of a call's
outputs: from the stream that the call runs on, recorded on the current one.
The library, the streams and the allocations are stand-ins that note what is
asked of them; tests/test_gpu_output_streams.py holds the effect."""
import contextlib

import pytest
import torch

import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import api, experts

CURRENT, SIDE = 7, 9


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Noted(torch.Tensor):
    """A CPU tensor that notes the streams it is recorded on."""

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


class Library:
    def __getattr__(self, name):
        def call(*a):
            if name == "mgs_moe_rows":
                a[-1]._obj.value = 160
            elif name == "mgs_moe_workspace_bytes":
                a[-1]._obj.value = 512
            return mgs.MGS_OK
        return call


@pytest.fixture
def taken(monkeypatch):
    """The tensors that a call allocates, with the stream each was taken on."""
    now, out = [CURRENT], []

    @contextlib.contextmanager
    def on(s):
        now.append(s.cuda_stream)
        yield
        now.pop()
    real = torch.empty

    def empty(*a, **kw):
        t = real(*a, **kw).as_subclass(Noted)
        t.taken_on, t.recorded = now[-1], []
        out.append(t)
        return t
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(api, "_raw_stream", lambda device: now[-1])
    for module in (api, experts):
        monkeypatch.setattr(module, "_need", lambda *a, **kw: None)
        monkeypatch.setattr(module, "lib", Library)
    experts._order_sizes.cache_clear()
    yield out
    experts._order_sizes.cache_clear()


X = torch.zeros((32, 64), dtype=torch.bfloat16)
U8, F32 = torch.zeros((32, 64), dtype=torch.uint8), torch.zeros((32, 1))
IDS, OFF = torch.zeros((32, 2), dtype=torch.int32), torch.tensor([32], dtype=torch.int32)
CALLS = {
    "mgs_moe_sort": (lambda **kw: mgs.mgs_moe_sort(IDS, 4, **kw), 4),
    "mgs_moe_dispatch": (lambda **kw: mgs.mgs_moe_dispatch(X, IDS, 4, permuted=True, **kw), 7),
    "mgs_moe_combine": (lambda **kw: mgs.mgs_moe_combine(X, IDS, **kw), 1),
    "mgs_moe_combine_grad": (lambda **kw: mgs.mgs_moe_combine_grad(X, X, IDS, IDS[:, 0], IDS.float(), **kw), 2),
    "mgs_quant_rows128": (lambda **kw: mgs.mgs_quant_rows128(X, **kw), 2),
    "mgs_quant_blocks128": (lambda **kw: mgs.mgs_quant_blocks128(X[None], **kw), 4),
    "mgs_mm_block128": (lambda **kw: mgs.mgs_mm_block128(U8, F32, U8[None], F32[None, :1], OFF, **kw), 1),
    "mgs_mm_wgrad": (lambda **kw: mgs.mgs_mm_wgrad(U8, F32, U8, F32, OFF, **kw), 1),
    "mgs_quant_groups_dim0": (lambda **kw: mgs.mgs_quant_groups_dim0(X, OFF, **kw), 2),
    "mgs_quant_groups_dim0_noalloc": (lambda **kw: mgs.mgs_quant_groups_dim0_noalloc(X, OFF, **kw), 2),
    "mgs_quant_groups_dim0_t": (lambda **kw: mgs.mgs_quant_groups_dim0_t(X, OFF, **kw), 2),
    "mgs_quant_experts_dim1": (lambda **kw: mgs.mgs_quant_experts_dim1(X[None], **kw), 2),
    "mgs_quant_groups_dim1": (lambda **kw: mgs.mgs_quant_groups_dim1(X, OFF, **kw), 2),
    "mgs_mx_quant_dim0": (lambda **kw: mgs.mgs_mx_quant_dim0(X, **kw), 2),
    "mgs_mx_quant_dim1": (lambda **kw: mgs.mgs_mx_quant_dim1(X, **kw), 2),
    "mgs_mx_dequant_dim0": (lambda **kw: mgs.mgs_mx_dequant_dim0(U8, U8[:, :2], **kw), 1),
    "mgs_cast_e4m3": (lambda **kw: mgs.mgs_cast_e4m3(F32, **kw), 1),
}


def test_every_call_that_takes_a_stream_is_here():
    import inspect
    names = {n for n, f in vars(mgs).items() if inspect.isfunction(f) and "stream" in inspect.signature(f).parameters}
    assert names == set(CALLS) | {"mgs_copy"}        # mgs_copy allocates nothing


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("as_int", [False, True])
def test_memory_of_another_stream(taken, name, as_int):
    call, outputs = CALLS[name]
    call(stream=SIDE if as_int else Stream(SIDE))
    assert [t.taken_on for t in taken] == [SIDE] * outputs
    assert [t.recorded for t in taken] == [[CURRENT]] * outputs


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, CURRENT])
def test_memory_of_the_current_stream(taken, name, stream):
    call, outputs = CALLS[name]
    call(stream=stream)
    assert [t.taken_on for t in taken] == [CURRENT] * outputs
    assert [t.recorded for t in taken] == [[]] * outputs
