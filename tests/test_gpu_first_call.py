"""Calls from threads that have made none before: one thread after the other,
and many at once as the first calls of a process."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BF = torch.bfloat16


def attend_slots():
    cache = latent.LatentCache(torch.ones(2, 64, latent.RECORD, dtype=BF, device="cuda"))
    args = (torch.ones(1, 16, 512, dtype=BF, device="cuda"), torch.ones(1, 16, 64, dtype=BF, device="cuda"),
            torch.arange(64, device="cuda")[None].contiguous(), 0.1, torch.zeros(1, 16, 512, dtype=BF, device="cuda"),
            dsaidx.new_workspace(latent.workspace_bytes(1, 16, 64)))
    return lambda: latent.latent_attend_slots(cache, *args), args[4]


def attend_paged():
    cache = latent.LatentCache(torch.ones(2, 64, latent.RECORD, dtype=BF, device="cuda"))
    one = torch.ones(1, 1, dtype=torch.int32, device="cuda")
    args = (torch.ones(1, 16, 512, dtype=BF, device="cuda"), torch.ones(1, 16, 64, dtype=BF, device="cuda"), one, one[0], 64,
            0.1, torch.zeros(1, 16, 512, dtype=BF, device="cuda"), dsaidx.new_workspace(latent.workspace_bytes(1, 16, 64)))
    return lambda: latent.latent_attend_paged(cache, *args), args[6]


def attend_expanded():
    q, k = torch.ones(4, 2, 192, dtype=BF, device="cuda"), torch.ones(4, 2, 128, dtype=BF, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    args = (q, k, k[:, 0, :64], k, cu, cu, 0.1, torch.zeros(4, 2, 128, dtype=BF, device="cuda"))
    return lambda: latent.latent_attend_expanded(*args), args[-1]


def append():
    cache = latent.LatentCache(torch.zeros(2, 64, latent.RECORD, dtype=BF, device="cuda"))
    args = (torch.ones(128, 512, dtype=BF, device="cuda"), torch.ones(128, 64, dtype=BF, device="cuda"), None,
            torch.arange(128, device="cuda"), None)
    return lambda: latent.latent_append(cache, *args), cache.pool


def rope():
    x, out = torch.ones(4, 2, 64, dtype=BF, device="cuda"), torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    plan, pos = latent.rope_plan(64), torch.zeros(4, dtype=torch.int64, device="cuda")
    return lambda: latent.rope(x, pos, plan, out=out), out


def index_cache():
    pool = torch.zeros(4 * dsaidx.block_bytes(dsaidx.FP8, 64), dtype=torch.uint8, device="cuda")
    done = torch.zeros(1)

    def create():
        handle = ctypes.c_void_p()
        dsaidx._check(dsaidx.load().idx_cache_create(ctypes.byref(handle), pool.data_ptr(), 4, 64, 128, dsaidx.FP8), "create")
        dsaidx.load().idx_cache_destroy(handle)
        done.fill_(1.0)
    return create, done


@pytest.mark.parametrize("make", [attend_slots, attend_paged, attend_expanded, append, rope, index_cache])
def test_call_in_a_new_thread(make):
    """A new thread has no current context; the library has to do without one made by an earlier call.  All inputs are ones, so
    are the results: the average of equal records, a copy, a turn by position 0."""
    call, out = make()
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            call()
        except Exception as e:
            failed.append(str(e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    stream.synchronize()
    torch.cuda.synchronize()
    assert not failed, failed
    assert bool((out == 1).all())


# Native threads that spin on one flag, so that they enter the call within a
# fraction of a microsecond of each other (Python's are started one by one).
HELPER = r"""
#include <pthread.h>
#include <stdatomic.h>
#include <stddef.h>
#include <stdint.h>
typedef int (*create_fn)(void**, void*, int64_t, int, int, int);
typedef int (*init_fn)(void*, size_t, void*);
struct job { create_fn create; init_fn init; char* pool; int key_dtype; int code; void* handle; };
static atomic_int ready, go;
static void* run(void* p) {
    struct job* j = p;
    j->code = j->init(j->pool, 256, 0);      // the thread's start-up in the runtime
    atomic_fetch_add(&ready, 1);
    while (!atomic_load(&go)) { }
    if (j->code == 0) j->code = j->create(&j->handle, j->pool, 4, 64, 128, j->key_dtype);
    return 0;
}
int together(create_fn create, init_fn init, void* pool, int key_dtype, int n, int* codes, void** handles) {
    pthread_t t[64];
    struct job j[64];
    if (n > 64) return 1;
    for (int i = 0; i < n; ++i) {
        j[i] = (struct job){create, init, pool, key_dtype, -1, 0};
        if (pthread_create(&t[i], 0, run, &j[i])) return 1;
    }
    while (atomic_load(&ready) < n) { }
    atomic_store(&go, 1);
    for (int i = 0; i < n; ++i) {
        pthread_join(t[i], 0);
        codes[i] = j[i].code;
        handles[i] = j[i].handle;
    }
    return 0;
}
"""

CHILD = """
import ctypes, sys
import torch
from sparse_attention_top_idx_gb300 import dsaidx
H, L, n = ctypes.CDLL(sys.argv[1]), dsaidx.load(), 12
pool = torch.zeros(4 * dsaidx.block_bytes(dsaidx.FP8, 64), dtype=torch.uint8, device="cuda")
codes, handles = (ctypes.c_int * n)(), (ctypes.c_void_p * n)()
H.together.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
create, init = (ctypes.cast(f, ctypes.c_void_p) for f in (L.idx_cache_create, L.idx_workspace_init))
assert H.together(create, init, pool.data_ptr(), dsaidx.FP8, n, codes, handles) == 0
for h in handles:
    if h: L.idx_cache_destroy(h)
print(list(codes))
"""


@pytest.mark.parametrize("again", range(6))
def test_many_threads_first_thing_in_a_process(again, tmp_path):
    """What the library looks up once must be there for every thread that asks at the same time: index caches and the
    attention calls share the tensor-map encoder."""
    src, lib = tmp_path / "together.c", tmp_path / "libtogether.so"
    src.write_text(HELPER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(src), "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == str([0] * 12)
