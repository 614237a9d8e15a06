"""The FP4 linear's choice of schedule, asked of its own source (compiled for the host)."""
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

from mtp_speculative_draft_head_gb300 import build

SHIM = """
#include "linear_fp4_sched.h"
extern "C" void schedule(int R, int N, int kp, int sms, int* out) {
  const mtp::LinearSched c = mtp::make_sched(R, N, kp, sms);
  out[0] = c.nt, out[1] = c.mt, out[2] = c.tiles, out[3] = c.nkb, out[4] = c.splits, out[5] = c.group;
}
"""


@functools.cache
def _lib():
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        raise RuntimeError("no host C++ compiler")
    d = tempfile.mkdtemp()
    try:
        src, so = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", so], check=True)
        return ctypes.CDLL(so)
    finally:
        shutil.rmtree(d, ignore_errors=True)


def schedule(R: int, N: int, K: int, sms: int = 152) -> dict:
    """nt (rows a tile), mt (weight tiles), tiles, nkb (stages), splits (CTAs a tile), group, and per_cta, the most
    tiles that a CTA takes."""
    out = (ctypes.c_int * 6)()
    _lib().schedule(R, N, -(-K // 256) * 256, sms, out)
    s = dict(zip(("nt", "mt", "tiles", "nkb", "splits", "group"), out))
    s["per_cta"] = 1 if s["splits"] > 1 else -(-s["tiles"] // sms)
    return s
