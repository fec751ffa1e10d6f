"""Calls on an 8-bit cache while another device than its own is current."""
import ctypes as C
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_with_another_device_current(tmp_path):
    """The C calls' host side, linked with a runtime that only counts (no device is needed)."""
    from bit_kv_cache_ott_gb300 import build
    build.build()
    obj, exe = os.path.join(build.OUT_DIR, "ott_byte.o"), str(tmp_path / "host")
    if not os.path.exists(obj):   # the library came without what it was linked of
        build.build(force=True)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    inc = [f"-I{d}" for d in (os.path.join(ROOT, "include"), os.path.join(cuda, "include")) if os.path.isdir(d)]
    r = subprocess.run(["g++", "-std=c++17", *inc, os.path.join(ROOT, "tests", "byte_device_host.cpp"), obj, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


class _Fake:
    """Two devices, and a library that notes which one was current in its calls."""

    def __init__(self, monkeypatch):
        import bit_kv_cache_ott_gb300 as pkg
        self.current, self.seen = 1, []
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "set_device", lambda d: setattr(self, "current", d))
        self.cache = c = object.__new__(pkg.ByteCache)
        c._L, c._h, c._dev = self, C.c_void_p(), 0

    def ott_byte_check(self, handle):
        self.seen.append(self.current)
        return 0


def test_check_device_goes_to_the_cache_s_device(monkeypatch):
    f = _Fake(monkeypatch)
    f.cache.check_device()
    assert f.seen == [0] and f.current == 1
