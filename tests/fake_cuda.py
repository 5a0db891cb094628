"""libspkv.so over a CUDA runtime that runs nothing (fake_cudart.cpp), in a child process: what the
library launches and refuses, on any machine."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
PKG = os.path.join(ROOT, "sparse_paged_kv_score_gb300")


def build(out_dir: str) -> str:
    """Compiles the fake runtime."""
    out = os.path.join(out_dir, "fake_cudart.so")
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(home, "include"),
                    os.path.join(HERE, "fake_cudart.cpp"), "-o", out], check=True)
    return out


def run(fake: str, program: str) -> str:
    """Output of a child's `program`, which begins with `import fake_cuda` done and the fake loaded as `f`."""
    head = f"import sys; sys.path.insert(0, {HERE!r}); import fake_cuda; f = fake_cuda.Library({fake!r})\n"
    r = subprocess.run([sys.executable, "-X", "faulthandler", "-c", head + program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"status {r.returncode}\n{r.stderr}"
    return r.stdout


class Library:
    """The library on the fake runtime; pointers are numbers that nothing reads."""

    def __init__(self, fake: str):
        self.rt = ctypes.CDLL(fake, mode=ctypes.RTLD_GLOBAL)
        self.rt.fake_event.restype = ctypes.c_char_p
        spec = importlib.util.spec_from_file_location("spkv_abi", os.path.join(PKG, "_abi.py"))
        self.abi = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(self.abi)   # without the package, which loads torch and its CUDA runtime
        self.lib = self.abi.load()

    def events(self):
        """What was asked of the runtime since the last look."""
        got = [self.rt.fake_event(i).decode() for i in range(self.rt.fake_events())]
        self.rt.fake_clear()
        return got

    def handle(self, q4: bool, Hk: int, n_phys: int = 8, sums: bool = True, max_units: int = 4096):
        s = 4096 if sums else None
        if q4:
            d = self.abi.SpkvDescQ4(Hk, 128, 64, 16, n_phys, 4096, 4096, 4096, s, s, max_units, 0)
        else:
            d = self.abi.SpkvDesc(Hk, 128, 64, 16, n_phys, 4096, 4096, s, s, max_units, 0)
        h = ctypes.c_void_p()
        create = self.lib.paged_kv_create_q4 if q4 else self.lib.paged_kv_create
        assert create(ctypes.byref(d), None, ctypes.byref(h)) == 0
        return h
