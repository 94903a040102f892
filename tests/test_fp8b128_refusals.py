"""Refusals of the fp8b128 calls on made-up addresses, safe on any machine: each call made here is
one that is refused (or has nothing to do) and ends before the library's first HIP call. Without a
GPU a call that gets past the checks returns TQ_EHIP; with one it would run a kernel on the
addresses. Two tests of test_fp8b128_args.py make such calls beside the ones they check, so they
are skipped on a machine with a GPU, and their cases are here call by call."""

import ctypes
import inspect

import pytest

import conftest
import test_fp8b128_args as args

tq = pytest.importorskip("trellis_quantized_moe_amd")
from trellis_quantized_moe_amd import _lib  # noqa: E402

P, BIG = args.P, args.BIG
OUT, IN = 256, 512


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def call(lib, name, L, T=3, xq=P, xs=P, y=P, dx=P, dw=P, ws=P, ws_bytes=BIG, flags=0):
    """The one call `name` (y: the output, or the output's gradient)."""
    r = ctypes.byref(L)
    if name == "gemm":
        return lib.fp8b128_gemm(r, xq, xs, T, y, flags, None)
    if name == "gated":
        return lib.fp8b128_gated(r, xq, xs, T, y, None)
    return getattr(lib, "fp8b128_" + name)(r, xq, xs, T, y, dx, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("flags", [1, 2, 4, 16, 64, 33])
def test_flags(lib, flags):
    assert call(lib, "gemm", args.layer(), flags=flags) == _lib.TQ_EINVAL


@pytest.mark.parametrize("name", ["gated", "gated_backward"])
def test_half_of_the_outputs_is_a_multiple_of_16(lib, name):
    for T in (0, 3):
        assert call(lib, name, args.layer(out=48), T=T, dw=0) == _lib.TQ_EINVAL


def test_a_product_of_48_outputs_has_no_halves(lib):
    odd = args.layer(out=48)
    assert call(lib, "gemm", odd, T=0, xq=0, xs=0, y=0) == _lib.TQ_OK
    assert call(lib, "gemm_backward", odd, T=0, xq=0, xs=0, y=0, dw=0, ws=0) == _lib.TQ_OK


@pytest.mark.parametrize("name", ["gemm_backward", "gated_backward"])
@pytest.mark.parametrize("kw,code", [
    ({"dx": 0, "dw": 0}, _lib.TQ_EINVAL), ({"dx": P + 8}, _lib.TQ_EALIGN), ({"dw": P + 4}, _lib.TQ_EALIGN),
    ({"ws": 0}, _lib.TQ_EWORKSPACE), ({"ws": P + 64}, _lib.TQ_EALIGN), ({"ws_bytes": None}, _lib.TQ_EWORKSPACE),
])
def test_backward(lib, name, kw, code):
    if "ws_bytes" in kw:
        kw = {"ws_bytes": lib.tq_fp8b128_workspace_bytes(3, OUT, IN) - 1}
    assert call(lib, name, args.layer(out=OUT, inp=IN), **kw) == code


@pytest.mark.skipif(conftest.device_present(), reason="looks for calls that would run on a GPU")
def test_the_skipped_tests_are_those_that_get_past_the_checks(lib, monkeypatch):
    past = set()

    class Watched:
        def __getattr__(self, name):
            fn = getattr(lib, name)

            def watched(*a):
                rc = fn(*a)
                if rc == _lib.TQ_EHIP:
                    past.add(test)
                return rc
            return watched

    watched_lib = Watched()
    for test, fn in vars(args).items():
        if not test.startswith("test_") or "lib" not in inspect.signature(fn).parameters:
            continue
        marks = [m.args[1] for m in getattr(fn, "pytestmark", []) if m.name == "parametrize"]
        for values in (marks[0] if marks else [()]):
            fn(watched_lib, *values)
    assert past == conftest.REACH_THE_DEVICE["test_fp8b128_args.py"]


def test_they_are_skipped_where_a_device_is_present(monkeypatch):
    class Item:
        def __init__(self, name, file="test_fp8b128_args.py"):
            self.originalname, self.path, self.marks = name, conftest.pathlib.Path("tests") / file, []

        def add_marker(self, mark):
            self.marks.append(mark.name)

    def marked(present):
        monkeypatch.setattr(conftest, "device_present", lambda: present)
        items = [Item("test_backward_arguments"), Item("test_bad_layers"),
                 Item("test_bad_flags_and_shapes"), Item("test_backward_arguments", "test_abi.py")]
        conftest.pytest_collection_modifyitems(items)
        return [i.marks for i in items]

    assert marked(False) == [[], [], [], []]
    assert marked(True) == [["skip"], [], ["skip"], []]
