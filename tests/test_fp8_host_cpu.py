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


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLibrary()
    monkeypatch.setattr(_abi, "lib", lambda: fake)
    monkeypatch.setattr(fp8, "_current_device", lambda: fake.device)
    monkeypatch.setattr(fp8, "_raw_stream", lambda index: 1000 + index)

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
