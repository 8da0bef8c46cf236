"""The binding's calls in C, without a GPU: on stand-ins for tensors, and with C functions of the
host in the library's place."""

import subprocess
import sys

from conftest import ROOT

PRELUDE = """
import ctypes, importlib.util, os, sys, threading, time
sys.path.insert(0, %r)
import __graft_entry__
build = __graft_entry__._library_builder()
build.build()


def load():
    spec = importlib.util.spec_from_file_location("fast_calls", build.FAST)
    fast = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fast)
    return fast


class Tensor:
    def __init__(self, shape, dtype="i32", at=64):
        self.shape, self.dtype, self.at = shape, dtype, at

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.at

    def stride(self):
        out = [1]
        for n in self.shape[:0:-1]:
            out.insert(0, out[0] * n)
        return tuple(out)


def address(name):
    return ctypes.cast(getattr(ctypes.CDLL(None), name), ctypes.c_void_p).value
""" % ROOT


def run(text):
    r = subprocess.run([sys.executable, "-c", PRELUDE + text], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_other_threads_run_during_a_call():
    """The host's sleep in the place of each call (its first argument, here an array's address of
    1, is the seconds): another thread counts meanwhile."""
    out = run("""
fast = load()

types = tuple(sys.intern(x) for x in ("bf16", "f16", "f32", "i32", "u8"))
fast.setup((address("sleep"),) * 7, types, lambda dev: 0, lambda: 0)
one = lambda *shape, dtype="i32": Tensor(shape, sys.intern(dtype), 1)
rows, four = one(3, 2, 128, dtype="bf16"), one(3, 2, 2, 128, dtype="bf16")
g, state, ws = one(2, dtype="f32"), one(1, 2, 128, 128, dtype="f32"), one(9, dtype="u8")
many = one(3, 2, 128, 128, dtype="f32")
table, refs, lens, count = one(3, 4), one(8), one(3), one(1)
calls = {
    "lin_prefill": (rows, rows, rows, g, rows, state, None, None, None, 1.0, ws),
    "lin_decode": (four, four, four, g, four, many, None, (), 1.0),
    "rope": (rows, None, lens, one(64, dtype="f32"), None, None, None, False, 1.0),
    "resize": (table, lens, refs, 64, ws),
    "fork": (table, lens, refs, lens, None, None, None, lens, lens, count, 64, ws),
    "compact": (table, refs, None, None, one(4), one(4), count, ws),
}
for name, args in calls.items():
    seen, stop = [], threading.Event()

    def watch():
        while not stop.is_set():
            seen.append(time.monotonic())
            time.sleep(0.02)

    thread = threading.Thread(target=watch)
    thread.start()
    time.sleep(0.1)
    start = time.monotonic()
    status = getattr(fast, name)(*args)
    end = time.monotonic()
    stop.set()
    thread.join()
    assert status == 0, (name, status)
    assert end - start > 0.9, (name, end - start)
    during = sum(start + 0.1 < x < end - 0.1 for x in seen)
    print(name, during > 5)
""")
    assert out.split() == [x for name in ("lin_prefill", "lin_decode", "rope", "resize", "fork",
                                          "compact") for x in (name, "True")]


def test_the_package_without_the_extension(tmp_path):
    """A copy of the package that lacks it: imported, and the calls take their forms in Python."""
    out = run("""
import shutil
here, there = os.path.dirname(build.__file__), os.path.join(%r, "gated_delta_rule_prepare_gb300")
shutil.copytree(here, there, ignore=shutil.ignore_patterns("fast_calls*", "*.o", "__pycache__"))
sys.path.insert(0, %r)
import torch
import gated_delta_rule_prepare_gb300 as K
assert K.__file__.startswith(there) and not os.path.exists(K._build.FAST)
x = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
assert K._fast.rope(x, None, None, None, None, None, None, False, 1.0) == -1
i = torch.zeros(3, dtype=torch.int32)
for call in (lambda: K.kda_attn_rope(x, None, i, torch.zeros(64)),
             lambda: K.kda_lin_prefill(x, x, x, torch.zeros(2), x),
             lambda: K.kda_lin_decode(x, x, x, torch.zeros(2), x),
             lambda: K.kda_attn_kv4_resize(i[None], i, i),
             lambda: K.kda_attn_kv4_fork(i[None], i, i, i),
             lambda: K.kda_attn_kv4_compact(i[None], i),
             lambda: K.kda_attn_kv4_copy([x], i, i, i)):
    try:
        call()
    except TypeError as e:
        assert "CUDA" in str(e), e
    else:
        assert False
print("fine")
""" % (str(tmp_path), str(tmp_path)))
    assert out.strip() == "fine"


def test_a_build_without_pythons_headers(tmp_path):
    """The extension is left out, with a warning, and the library is built all the same."""
    out = run("""
import shutil, warnings
there = os.path.join(%r, "package")
shutil.copytree(os.path.dirname(build.__file__), there,
                ignore=shutil.ignore_patterns("__pycache__", "*.o"))
shutil.copytree(build.INCLUDE, os.path.join(%r, "include"))
spec = importlib.util.spec_from_file_location("there", os.path.join(there, "build.py"))
copy = importlib.util.module_from_spec(spec)
spec.loader.exec_module(copy)
assert copy.FAST.startswith(there) and os.path.exists(copy.FAST)
os.utime(copy.LIB)
paths = copy.sysconfig.get_paths
copy.sysconfig.get_paths = lambda: dict(paths(), include=there)
os.utime(os.path.join(copy.CSRC, "fast_calls.c"))
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    assert copy.build() == copy.LIB
assert len(seen) == 1 and "Python.h" in str(seen[0].message)
assert not os.path.exists(copy.FAST) and not copy.up_to_date()
copy.sysconfig.get_paths = paths
assert copy.build() == copy.LIB and copy.up_to_date()
print("fine", sys.implementation.cache_tag in copy.FAST)
""" % (str(tmp_path), str(tmp_path)))
    assert out.split() == ["fine", "True"]
