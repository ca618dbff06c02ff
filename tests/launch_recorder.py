"""Records the library's kernel launches on a machine without a GPU.

A child process loads a small C library in front of the HIP runtime: its
hipLaunchKernel writes down the calling thread, the grid and the kernel's
first argument (a structure by value) and returns; nothing runs.  It sleeps a
little in every launch, so that calls from several threads meet between their
launches.
"""
from __future__ import annotations

import json
import subprocess
import sys
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]

SOURCE = r"""
#define _GNU_SOURCE
#include <stdint.h>
#include <string.h>
#include <unistd.h>
#include <sys/syscall.h>

typedef struct { uint32_t x, y, z; } dim3;
enum { MOST = 4096, WORDS = 32 };
struct { uint64_t thread, x, y, z, arg[WORDS]; } launches[MOST];
int count;
int pause_us;

static __thread struct { dim3 grid, block; size_t lds; void *stream; } config;

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream)
{
    config.grid = grid;
    config.block = block;
    config.lds = lds;
    config.stream = stream;
    return 0;
}

int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream)
{
    *grid = config.grid;
    *block = config.block;
    *lds = config.lds;
    *stream = config.stream;
    return 0;
}

int hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream)
{
    int i = __atomic_fetch_add(&count, 1, __ATOMIC_SEQ_CST);
    if (i < MOST) {
        launches[i].thread = (uint64_t)syscall(SYS_gettid);
        launches[i].x = grid.x;
        launches[i].y = grid.y;
        launches[i].z = grid.z;
        memcpy(launches[i].arg, args[0], sizeof launches[i].arg);
    }
    if (pause_us)
        usleep(pause_us);
    return 0;
}

int hipGetLastError(void) { return 0; }
"""

PRELUDE = """
import ctypes, json, sys, threading
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from dense_gemm_18_amd import binding

class Launch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("thread", "x", "y", "z")] + [
        ("arg", ctypes.c_uint64 * 32)]

count = ctypes.c_int.in_dll(shim, "count")
pause_us = ctypes.c_int.in_dll(shim, "pause_us")

def launches():
    all = (Launch * 4096).in_dll(shim, "launches")
    return [{"thread": x.thread, "grid": [x.x, x.y, x.z], "arg": list(x.arg)}
            for x in all[:count.value]]

def weights(router=0x100000000, w13=0x1100000000, w2=0x2200000000, experts=8, hidden=256, inner=64,
            **kw):
    return binding.moe_nt_weights(router, w13, kw.get("s13"), None, w2, kw.get("s2"), None,
                                  experts, hidden, inner, kw.get("group", 0), 0)
"""


def run(tmp_path: Path, code: str):
    """What ``code`` (after PRELUDE) leaves in ``result``."""
    src, so = tmp_path / "recorder.c", tmp_path / "recorder.so"
    src.write_text(SOURCE)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", str(src), "-o", str(so)], check=True)
    res = subprocess.run([sys.executable, "-c", PRELUDE + code + "\nprint(json.dumps(result))",
                          str(so)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    return json.loads(res.stdout.splitlines()[-1])
