"""Calls from threads that have made none before: one thread after the other."""
import ctypes
import threading

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent

pytestmark = pytest.mark.gpu

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
