"""What the Python layer of the 8-bit floating point experts does on the host, against a library
that only writes down its calls: error checks of both workspaces, and the device and stream that
every call is made on."""
import contextlib
import ctypes
import types

import pytest
import torch

import routing_dispatch_expert_warp_b200 as M
from routing_dispatch_expert_warp_b200 import _abi, fp8

INVALID, CUDA, TIMEOUT, DATA = 1, 4, 5, 6
TEXT = {TIMEOUT: b"a device wait ran out", DATA: b"fp8 product: bucket 3", CUDA: b"cuda"}


class FakeLibrary:
    """Records calls.  A workspace's status is what `status` holds for its address; reading it
    clears it, as the library does."""

    def __init__(self):
        self.status, self.calls, self.last = {}, [], b""
        self.device = 0  # the current device, as torch.cuda.device sets it
        self.streams = [1000, 1001]  # each device's current stream
        self.split_bytes = 4096

    def moe_check_device_error(self, ws, n, stream):
        self.calls.append(("check", ws, self.device, stream))
        code = self.status.pop(ws, 0)
        self.last = TEXT.get(code, b"")
        return code

    def moe_fp8_workspace_init(self, ws, n, stream):
        self.calls.append(("init", ws, self.device, stream))
        self.last = b"init"
        return self.status.get("init", 0)

    def moe_last_error(self):
        return self.last

    def moe_router_split_size(self, cfg, n):
        ctypes.cast(n, ctypes.POINTER(ctypes.c_size_t))[0] = self.split_bytes
        return 0

    def moe_router_split(self, cfg, w, out, n, stream):
        self.calls.append(("split", out, self.device, stream))
        return 0

    def moe_pick_rank_counts(self, cfg, idx, row, group, routed, kept, differs, ws, n, stream):
        self.calls.append(("counts", ws, self.device, stream))
        return 0

    def moe_fp8_quantize_weights(self, dtype, E, N, K, w, q, scale, stream):
        self.calls.append(("quantize", w, self.device, stream))
        return 0

    def moe_fp8_workspace_size(self, n):
        ctypes.cast(n, ctypes.POINTER(ctypes.c_size_t))[0] = 4096
        return 0


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream, self.device = handle, device


class FakeTensor:
    """A tensor of the fake library's devices: what the Python layer asks of one."""

    def __init__(self, shape, dtype, device, at):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.at = at  # (device, stream) whose memory it was given
        self.address = id(self)

    def data_ptr(self):
        return self.address

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLibrary()
    monkeypatch.setattr(_abi, "lib", lambda: fake)
    monkeypatch.setattr(fp8, "_current_device", lambda: fake.device)
    monkeypatch.setattr(fp8, "_raw_stream", lambda index: fake.streams[index])
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(
        handle, torch.device("cuda", fake.device) if device is None else torch.device(device)))
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: FakeStream(fake.streams[fake.device]))

    def empty(*shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        at = torch.device(device).index
        return FakeTensor(shape, dtype, device, (at, fake.streams[at]))

    monkeypatch.setattr(torch, "empty", empty)

    @contextlib.contextmanager
    def stream(s):
        if s is None:
            yield
            return
        device, fake.device = fake.device, s.device.index
        before, fake.streams[s.device.index] = fake.streams[s.device.index], s.cuda_stream
        try:
            yield
        finally:
            fake.streams[s.device.index], fake.device = before, device

    monkeypatch.setattr(torch.cuda, "stream", stream)

    @contextlib.contextmanager
    def device(d):
        before, fake.device = fake.device, d if isinstance(d, int) else torch.device(d).index
        try:
            yield
        finally:
            fake.device = before

    monkeypatch.setattr(torch.cuda, "device", device)
    return fake


def workspace(address, index=0):
    return types.SimpleNamespace(device=torch.device("cuda", index), data_ptr=lambda: address,
                                 numel=lambda: 4096)


def bare_layer(index=0):
    """A layer without its constructor: what the methods under test read of it."""
    layer = object.__new__(M.MoELayerFp8)
    layer.ws, layer.fp8_ws = workspace(0x100, index), workspace(0x200, index)
    layer.ws.is_contiguous = lambda: True
    layer.cfg = M.make_config(64, 256, 128, 8, 2)

    def on_device(dtype, *shape):
        return FakeTensor(shape, dtype, f"cuda:{index}", None)

    layer.w_router = on_device(torch.float32, 256, 8)
    layer.experts = types.SimpleNamespace(w_gate=on_device(fp8.E4M3, 8, 128, 256))
    layer.bufs = types.SimpleNamespace(topk_idx=on_device(torch.int32, 64, 2),
                                       assign_row=on_device(torch.int32, 64, 2))
    return layer


# ------------------------------------------------------------------ errors
def checked(layer, lib, **kw):
    lib.calls.clear()
    try:
        layer.check_device_error(**kw)
        return None
    except M.MoEError as e:
        return e


def test_check_of_a_clean_layer_reads_both_workspaces(lib):
    assert checked(bare_layer(), lib) is None
    assert [c[:2] for c in lib.calls] == [("check", 0x100), ("check", 0x200)]


def test_check_reads_and_restores_the_products_workspace_when_the_layers_has_an_error_too(lib):
    """A dispatch whose wait ran out leaves bad offsets, which the products then report: both
    statuses are set.  The counters that cut tiles leave behind must not outlive the check."""
    layer = bare_layer()
    lib.status = {0x100: TIMEOUT, 0x200: DATA}
    e = checked(layer, lib)
    assert e.status == TIMEOUT and "wait" in str(e)  # the first stage's error
    assert [c[:2] for c in lib.calls] == [("check", 0x100), ("check", 0x200), ("init", 0x200)]
    assert checked(layer, lib) is None  # both were read and cleared


def test_check_with_an_error_of_the_layers_workspace_alone(lib):
    layer = bare_layer()
    lib.status = {0x100: DATA}
    assert checked(layer, lib).status == DATA
    assert [c[:2] for c in lib.calls] == [("check", 0x100), ("check", 0x200)]


@pytest.mark.parametrize("code", [TIMEOUT, DATA])
def test_check_restores_the_products_workspace_after_any_error(lib, code):
    """The status keeps the first error alone: a bad bucket may hide a wait that ran out later."""
    layer = bare_layer()
    lib.status = {0x200: code}
    assert checked(layer, lib).status == code
    assert [c[:2] for c in lib.calls] == [("check", 0x100), ("check", 0x200), ("init", 0x200)]


def test_check_reports_the_first_error_when_the_workspace_cannot_be_restored(lib):
    layer = bare_layer()
    lib.status = {0x100: CUDA, 0x200: CUDA, "init": INVALID}
    assert checked(layer, lib).status == CUDA


def test_check_on_the_layers_device_and_stream(lib):
    layer = bare_layer(1)
    lib.status = {0x200: TIMEOUT}
    checked(layer, lib)
    assert [c[2:] for c in lib.calls] == [(1, 1001)] * 3
    lib.status = {0x200: TIMEOUT}
    checked(layer, lib, stream=77)
    assert [c[2:] for c in lib.calls] == [(1, 77)] * 3
    assert lib.device == 0


# ------------------------------------------------------------------ devices and streams
@pytest.mark.parametrize("stream,runs_on", [(None, 1001), (77, 77),
                                            (FakeStream(88, torch.device("cuda", 1)), 88)],
                         ids=["current", "handle", "stream"])
def test_a_layers_calls_run_on_its_device(lib, stream, runs_on):
    """The layer's device is not the current one; what a call allocates belongs to its stream."""
    layer = bare_layer(1)
    layer.resplit_router(stream)
    counts = layer.pick_rank_counts(stream=stream)
    assert [(c[0], *c[2:]) for c in lib.calls] == [("split", 1, runs_on), ("counts", 1, runs_on)]
    for t in (layer.w_router_split, *counts):
        assert t.at == (1, runs_on)
    assert lib.device == 0 and lib.streams == [1000, 1001]


def test_a_layer_refuses_a_stream_of_another_device(lib):
    layer = bare_layer(1)
    for call in (layer.resplit_router, layer.check_device_error,
                 lambda s: layer.pick_rank_counts(stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(FakeStream(88, torch.device("cuda", 0)))
    assert lib.calls == []


@pytest.mark.parametrize("stream,runs_on", [(None, 1001), (77, 77)], ids=["current", "handle"])
def test_new_tensors_belong_to_the_stream_on_their_own_device(lib, stream, runs_on):
    """A stream's handle does not say its device: it is the tensors' one."""
    w = [FakeTensor(s, torch.bfloat16, "cuda:1", None)
         for s in ((2, 128, 256), (2, 128, 256), (2, 256, 128))]
    ex = M.Fp8Experts.quantize(*w, stream)
    ws = M.alloc_fp8_workspace("cuda:1", stream)
    for t in (ex.w_gate, ex.gate_scale, ex.w_up, ex.up_scale, ex.w_down, ex.down_scale, ws):
        assert t.at == (1, runs_on)
    assert [(c[0], *c[2:]) for c in lib.calls] == [("quantize", 1, runs_on)] * 3 + [
        ("init", 1, runs_on)]
    assert lib.device == 0


def test_weights_on_the_host_are_refused():
    w = torch.zeros(1, 16, 16)
    with pytest.raises(ValueError):
        M.Fp8Experts.quantize(w, w, w)


def test_a_router_weight_is_split_again_where_it_was(lib):
    """A captured forward reads the split router weight at the address it had then."""
    layer = bare_layer(1)
    layer.resplit_router()
    first = layer.w_router_split
    layer.resplit_router()
    layer.resplit_router(77)
    assert layer.w_router_split is first
    assert lib.calls == [("split", first.address, 1, 1001)] * 2 + [("split", first.address, 1, 77)]
    layer.cfg.d_model, lib.split_bytes = 512, 8192  # another layer's router weight: another buffer
    layer.resplit_router()
    assert layer.w_router_split.numel() == 8192
