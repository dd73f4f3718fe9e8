"""The quick binding and other Python threads: the interpreter's lock is free while the library's call runs."""
import ctypes
import shutil
import subprocess
import threading

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import paged
from paged_q8_helpers import q8_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"

# A library whose calls wait (2 s at most) for another thread to say "go", and refuse where none does.
WAITS = r"""
#include <stddef.h>
#include <time.h>
static volatile int entered, go;
int is_entered(void) { return entered; }
void say_go(void) { go = 1; }
static int wait_for_go(void) {
    entered = 1;
    for (int i = 0; i < 2000 && !go; ++i) {
        struct timespec t = {0, 1000000};
        nanosleep(&t, 0);
    }
    const int went = go;
    entered = go = 0;
    return went ? 0 : 7;
}
#define CALL(name) int name(void *a, void *b, size_t c, void *d) { return wait_for_go(); }
CALL(attn_paged_append) CALL(attn_paged_append_q8) CALL(attn_paged_read_q8) CALL(attn_paged_fwd) CALL(attn_paged_fwd_q8)
CALL(attn_paged_prefix_fwd)
#define SIZE(name) size_t name(void *a) { return 0; }
SIZE(attn_paged_fwd_workspace_bytes) SIZE(attn_paged_fwd_q8_workspace_bytes) SIZE(attn_paged_prefix_fwd_workspace_bytes)
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("name", ["append", "append_q8", "read_q8", "fwd", "fwd_q8", "prefix_fwd"])
def test_other_threads_run_meanwhile(name, tmp_path):
    src, so = tmp_path / "waits.c", tmp_path / "libwaits.so"
    src.write_text(WAITS)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    waits = ctypes.CDLL(str(so))
    s = q8_inputs([1], [20], 2, 1, 64, 16, poison=False)
    bf = [torch.zeros(s["kp"].shape, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    kv = [torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    c8, sc, t = (s["kp"], s["vp"]), (s["ks"], s["vs"]), (s["bt"], s["lens"])
    calls = {"append": lambda: ofa.attn_paged_append(s["q"], *kv, *bf, *t),
             "append_q8": lambda: ofa.attn_paged_append_q8(s["q"], *kv, *c8, *sc, *t),
             "read_q8": lambda: ofa.attn_paged_read_q8(*c8, *sc, *t, 1),
             "fwd": lambda: ofa.attn_paged_fwd(s["q"], *bf, *t),
             "fwd_q8": lambda: ofa.attn_paged_fwd_q8(s["q"], *c8, *sc, *t),
             "prefix_fwd": lambda: ofa.attn_paged_prefix_fwd(s["q"], *bf, *t, *t)}
    calls[name]()  # the real library, and whatever a first call sets up
    stop = threading.Event()

    def other():
        while not stop.is_set():
            if waits.is_entered():
                waits.say_go()
            stop.wait(0.005)

    thread = threading.Thread(target=other)
    quick = paged._binding()
    quick.open(str(so))
    thread.start()
    try:
        calls[name]()  # (a call that nobody lets go on is refused: AttnError)
    finally:
        quick.open(ofa.library_path())
        stop.set()
        thread.join()
    calls[name]()
    assert ofa.device_error_flags() == 0
