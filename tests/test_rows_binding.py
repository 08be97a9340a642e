"""The binding's handling of work buffers, and the row operators' compiled calls, without a GPU: stand-ins for tensors
and for the library's functions record what would be launched with which buffer."""
import ctypes
import os
import subprocess
import sys
import sysconfig

import pytest

from sorting_lsd_radix_gb300 import build as gbuild
from sorting_lsd_radix_gb300 import gbsort

torch = pytest.importorskip("torch")
A = 1 << 40  # an address, never followed
_empty = torch.empty


class Stand:
    """A tensor's outside: what the binding asks of one."""

    def __init__(self, *shape, dtype=torch.uint8, stride=None, device=0):
        self.shape, self.dtype, self.device = shape, dtype, device
        self.strides = stride or tuple(_empty(shape, device="meta").stride())

    def stride(self):
        return self.strides

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return self.strides == tuple(_empty(self.shape, device="meta").stride())

    def get_device(self):
        return self.device

    def data_ptr(self):
        return A if self.numel() else 0


NEED = 4096


@pytest.fixture
def entry(monkeypatch):
    """An entry point with the work-buffer protocol that lists the buffers it was run with."""
    ran = []

    def fn(d_temp, size, *args):
        size = ctypes.cast(size, ctypes.POINTER(ctypes.c_size_t))
        if not (d_temp.value if isinstance(d_temp, ctypes.c_void_p) else d_temp):
            size[0] = NEED
            return gbsort.GBS_OK
        if size[0] < NEED:
            return gbsort.GBS_ERR_TEMP_TOO_SMALL
        ran.append(size[0])
        return gbsort.GBS_OK

    monkeypatch.setattr(gbsort, "_current_device", lambda: 0)
    monkeypatch.setattr(gbsort.torch, "empty", lambda n, **kw: Stand(n))
    fn.ran = ran
    return fn


GOOD = [Stand(NEED), Stand(2, NEED), Stand(NEED // 2, 2)]
# too little memory behind them for their elements, or memory that the GPU does not have
BAD = [Stand(2 * NEED, stride=(0,)), Stand(NEED, stride=(2,)), Stand(NEED, 2, stride=(1, NEED)), Stand(NEED, device=-1),
       Stand(NEED, device=1)]


@pytest.mark.parametrize("temp", GOOD)
def test_work_buffers_taken(entry, temp):
    assert gbsort._run(entry, (), temp, "entry") is temp and entry.ran == [temp.numel()]


@pytest.mark.parametrize("temp", BAD)
def test_work_buffers_refused(entry, temp):
    with pytest.raises(ValueError, match="temp"):
        gbsort._run(entry, (), temp, "entry")
    assert entry.ran == []


@pytest.mark.parametrize("temp", [None, Stand(0), Stand(NEED - 1)])
def test_work_buffers_made(entry, temp):
    """A call without a buffer, with an empty one or with one that is too small is still done."""
    made = gbsort._run(entry, (), temp, "entry")
    assert made.numel() == NEED and entry.ran == [NEED]


@pytest.fixture
def compiled():
    """The compiled calls with stand-ins behind them, and the list of calls that got through."""
    gbuild.build()
    lib = gbsort.load()
    if gbsort._fast is None:
        pytest.skip("the compiled calls are not built")
    calls = []
    sort = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t))(
        lambda temp, size: calls.append((temp, size[0])) or 0)
    at = ctypes.cast(sort, ctypes.c_void_p).value
    gbsort._fast.setup((torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64), lambda dev: 0, lambda: 0,
                       (at,) * 7)
    yield gbsort._fast, calls
    gbsort._load_fast(lib)


def _sorted_with(temp):
    plan = tuple(Stand(*s, dtype=torch.int32) for s in ((12,), (6, 2), (5,), (4,)))
    return Stand(6, 2, dtype=torch.int64), 4, 0, 1, plan, temp


@pytest.mark.parametrize("temp", GOOD)
def test_compiled_calls_take_work_buffers(compiled, temp):
    fast, calls = compiled
    assert fast.sort(*_sorted_with(temp)) == 0 and calls == [(A, temp.numel())]


@pytest.mark.parametrize("temp", BAD + [Stand(0)])
def test_compiled_calls_leave_other_buffers_alone(compiled, temp):
    fast, calls = compiled
    assert fast.sort(*_sorted_with(temp)) == -1 and calls == []


def test_compiled_calls_belong_to_this_interpreter():
    """Their file carries the interpreter's tag, so that no other version of Python loads it."""
    gbuild.build()
    gbsort.load()
    if gbsort._fast is None:
        pytest.skip("the compiled calls are not built")
    assert gbuild.ROWS_PY.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.samefile(gbsort._fast.__file__, gbuild.ROWS_PY)


def test_a_build_without_a_c_compiler(monkeypatch, tmp_path):
    """The compiled calls are left out then, as without Python's headers; one that fails on them still says so."""
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("Python's headers are not installed")
    made = tmp_path / "_rows.so"
    monkeypatch.setattr(gbuild, "ROWS_PY", str(made))
    monkeypatch.setenv("CC", str(tmp_path / "no-compiler"))
    gbuild._build_rows_py()
    assert not made.exists()
    broken = tmp_path / "broken"
    broken.write_text("#!/bin/sh\nexit 3\n")
    broken.chmod(0o755)
    monkeypatch.setenv("CC", str(broken))
    with pytest.raises(RuntimeError, match="rows_py.c"):
        gbuild._build_rows_py()


def test_import_on_a_torch_without_cuda():
    """The binding imports, loads the library and refuses tensors where torch has no CUDA functions at all."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from sorting_lsd_radix_gb300 import gbsort
assert gbsort.gbs_version()
ids = torch.zeros(6, 2, dtype=torch.int64)
for call in (lambda: gbsort.gbs_expert_sort(ids, 4), lambda: gbsort.gbs_embedding_lookup(torch.zeros(6, 8), ids),
             lambda: gbsort.gbs_embedding_lookup(torch.zeros(6, 8), ids[:, 0].contiguous(), out=torch.zeros(6, 8))):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("not refused")
"""
    gbuild.build()
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=gbuild.ROOT)
    assert r.returncode == 0, r.stderr


def test_integers_past_64_bits_are_refused(monkeypatch):
    """They were cut to their low 64 bits."""
    ran = []
    entry = lambda *args: ran.append(args) or 0
    lib = type("Library", (), {name: staticmethod(entry) for name in gbsort.EXPORTS})
    monkeypatch.setattr(gbsort, "load", lambda: lib)
    monkeypatch.setattr(gbsort, "_fast", None)
    monkeypatch.setattr(gbsort, "_current_device", lambda: 0)
    monkeypatch.setattr(gbsort, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(Stand, "dim", lambda self: len(self.shape), raising=False)
    monkeypatch.setattr(Stand, "size", lambda self, i: self.shape[i], raising=False)
    monkeypatch.setattr(Stand, "stride", lambda self, *i: self.strides[i[0]] if i else self.strides)
    ids, words = Stand(6, 2, dtype=torch.int64), Stand(6, dtype=torch.int64)
    plan = tuple(Stand(*s, dtype=torch.int32) for s in ((12,), (6, 2), (5,), (4,)))
    x, table, temp = Stand(6, 8, dtype=torch.float32), Stand(9, 8, dtype=torch.float32), Stand(4096)
    rows = Stand(12, 8, dtype=torch.float32)
    calls = [lambda first: gbsort.gbs_expert_sort(ids, 4, first, plan_out=plan, temp=temp),
             lambda first: gbsort.gbs_expert_dispatch(x, ids, 4, first, rows_out=rows, plan_out=plan, temp=temp),
             lambda first: gbsort.gbs_embedding_lookup(table, words, first_id=first, out=x),
             lambda first: gbsort.gbs_embedding_grad(x, words, table, first_id=first, temp=temp),
             lambda first: gbsort.gbs_embedding_grad(x, words, table, padding_id=first, temp=temp)]
    for call in calls:
        for good in (0, 2 ** 63 - 1, -2 ** 63):
            call(good)
            assert ran.pop() and not ran
        for bad in (2 ** 63, -2 ** 63 - 1, 2 ** 64 + 3):
            with pytest.raises(ValueError, match="64 bits"):
                call(bad)
    for bad in (dict(num_experts=2 ** 64 + 4), dict(num_experts=4, row_align=2 ** 64 + 1)):
        with pytest.raises(ValueError, match="64 bits"):
            gbsort.gbs_expert_sort(ids, **bad)
    assert ran == []
