"""The launches of gdn_replay_advance's chunked form (csrc/advance_plan.h), compiled for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decode_recurrent_gb300", "csrc")
UNIT = {64: 3 * 8192 + 3 * 8192 + 512, 128: 3 * 16384 + 3 * 8192 + 512}     # bytes of a chunk of a head: E, M P, gamma

CODE = r"""
#include "advance_plan.h"
extern "C" int plan(int B, int T, int H, int dv, long long unit, int sms, long long *out, int *sizes, int n) {
    const gdn::AdvancePlan p = gdn::advance_plan(B, T, H, dv, unit, sms);
    const long long x[] = {p.all, p.seqs, p.most, p.first_room(), p.room(), p.workspace()};
    for (int i = 0; i < 6; ++i) out[i] = x[i];
    int launches = 0;
    for (int i = 0, rest = p.all, size = 0; rest > 0; ++i, rest -= size, ++launches) {
        size = p.next(i, size, rest);
        if (launches < n) sizes[launches] = size;
    }
    return launches;
}
"""


@functools.lru_cache(None)
def _load():
    with tempfile.TemporaryDirectory() as d:
        cpp, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(cpp, "w") as f:
            f.write(CODE)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", SRC, cpp, "-o", so])
        lib = ctypes.CDLL(so)
    lib.plan.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]
    return lib


def plan(B, T, H, dk, dv, sms=152):
    """Chunks of T tokens, sequences of a launch, the most chunks of a launch, the first workspace's chunks, both workspaces',
    their bytes; and the chunks of each launch of a group of sequences."""
    out, sizes = (ctypes.c_longlong * 6)(), (ctypes.c_int * (1 << 15))()
    n = _load().plan(B, T, H, dv, UNIT[dk], sms, out, sizes, len(sizes))
    return dict(zip(("all", "seqs", "most", "first_room", "room", "bytes"), out), sizes=list(sizes[:n]))
