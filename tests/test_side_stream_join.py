"""Calls that fork work onto the library's side stream and then fail (no GPU):
the C ABI's own object files, linked with stand-ins for every launcher and CUDA
call, one launcher of which reports an error. Whatever a call returns, later
work on the caller's stream follows what the call put on the side stream."""
import ctypes
import os
import shutil
import subprocess

import pytest

from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build

CC = shutil.which("gcc") or shutil.which("cc")
pytestmark = pytest.mark.skipif(CC is None, reason="no C compiler")
P = 1 << 20      # a well-aligned address, never dereferenced
CALLER = 1 << 8  # the caller's stream

FAKES = r"""
#include <stdio.h>
#include <string.h>
static char text[1 << 16];
static int launches, fail_at;
static long handles;
static void note(const char *fmt, const char *what, long a, long b) {
  const size_t n = strlen(text);
  snprintf(text + n, sizeof text - n, fmt, what, a, b);
}
void fake_reset(int at) { text[0] = 0; launches = 0; fail_at = at; }
const char *fake_log(void) { return text; }
static long hit(const char *name) {
  if (strstr(name, "launch_")) {
    note("launch %s\n", name, 0, 0);
    return ++launches == fail_at;
  }
  return strstr(name, "supported") || strstr(name, "xtd_splits") || strstr(name, "blocks");
}
static int make(long *h) { *h = 0x1000 + 16 * ++handles; return 0; }
int cudaStreamCreateWithFlags(long *h, unsigned f) { (void)f; return make(h); }
int cudaEventCreateWithFlags(long *h, unsigned f) { (void)f; return make(h); }
int cudaEventRecord(long e, long s) { note("%s %ld %ld\n", "record", e, s); return 0; }
int cudaStreamWaitEvent(long s, long e, unsigned f) {
  (void)f;
  note("%s %ld %ld\n", "wait", s, e);
  return 0;
}
"""
MADE = {"cudaStreamCreateWithFlags", "cudaEventCreateWithFlags", "cudaEventRecord",
        "cudaStreamWaitEvent"}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    moe_build.build()
    objs = [os.path.join(moe_build.BUILD_DIR, o) for o in ("moe_api.o", "gated_api.o")]

    def symbols(flag):
        out = subprocess.run(["nm", flag, *objs], capture_output=True, text=True, check=True).stdout
        return {f[-1] for f in map(str.split, out.splitlines()) if f and not f[-1].endswith(":")}
    names = sorted(n for n in symbols("--undefined-only") - symbols("--defined-only") - MADE
                   if n.startswith(("_ZN3moe", "cuda", "__cuda")))
    src = FAKES + "".join(
        f'long fake{i}(void) __asm__("{n}");\nlong fake{i}(void) {{ return hit("{n}"); }}\n'
        for i, n in enumerate(names))
    d = tmp_path_factory.mktemp("fakes")
    (d / "fakes.c").write_text(src)
    out = str(d / "libfakes.so")
    subprocess.run([CC, "-shared", "-fPIC", "-Wl,-Bsymbolic", "-o", out, str(d / "fakes.c"), *objs,
                    "-lstdc++", "-ldl", "-lm", "-lpthread"], check=True)
    L = ctypes.CDLL(out)
    for n in B.EXPORTS:
        if hasattr(L, n):
            getattr(L, n).argtypes = getattr(B.lib(), n).argtypes
    L.fake_log.restype = ctypes.c_char_p
    return L


def gated(d, F, act):
    cfg = B.config(300, d, 6, F, 2, 2.0, act_dtype=act)
    return "moe_experts_gated_backward", cfg, [B.MOE_ACT_SILU] + [P] * 19 + [CALLER]


def plain(act):
    cfg = B.config(300, 64, 6, 128, 2, 2.0, act_dtype=act)
    return "moe_backward", cfg, [P] * 12 + [0.1, 0.1, 0.1] + [P] * 11 + [CALLER]


def checkpoint(act):
    cfg = B.config(300, 64, 6, 128, 2, 2.0, act_dtype=act)
    return "moe_backward_checkpoint", cfg, [P] * 13 + [0.1, 0.1, 0.1] + [P] * 11 + [CALLER]


def forward():
    cfg = B.config(300, 64, 6, 128, 2, 2.0)
    return "moe_forward", cfg, [P] * 16 + [CALLER]


CALLS = dict(gated_bf16=gated(64, 128, B.MOE_BF16), gated_f32=gated(33, 65, B.MOE_F32),
             backward_bf16=plain(B.MOE_BF16), backward_f32=plain(B.MOE_F32),
             checkpoint_bf16=checkpoint(B.MOE_BF16), checkpoint_f32=checkpoint(B.MOE_F32),
             forward=forward())


def run(L, what, fail_at):
    name, cfg, args = CALLS[what]
    L.fake_reset(fail_at)
    status = getattr(L, name)(ctypes.byref(cfg), *args)
    log = [line.split() for line in L.fake_log().decode().splitlines()]
    return status, log


def joined(log):
    """Whether the caller's stream waits for an event that the side stream
    recorded after the last time work was forked onto it (or none was)."""
    forks = [i for i, l in enumerate(log) if l[0] == "wait" and int(l[1]) != CALLER]
    if not forks:
        return True
    side = log[forks[-1]][1]
    rest = log[forks[-1] + 1:]
    for i, l in enumerate(rest):
        if l[0] == "record" and l[2] == side:
            if any(w[0] == "wait" and int(w[1]) == CALLER and w[2] == l[1] for w in rest[i + 1:]):
                return True
    return False


@pytest.mark.parametrize("what", sorted(CALLS))
def test_joined_however_the_call_ends(lib, what):
    status, log = run(lib, what, 0)
    n = sum(l[0] == "launch" for l in log)
    assert status == 0 and n > 3
    assert any(l[0] == "wait" and int(l[1]) != CALLER for l in log), "nothing was forked"
    assert joined(log)
    for at in range(1, n + 1):
        status, log = run(lib, what, at)
        assert status == 3, at
        assert sum(l[0] == "launch" for l in log) == at
        assert joined(log), (at, log[-3:])
