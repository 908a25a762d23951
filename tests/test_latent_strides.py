"""Rotary calls whose results would share elements: each shared element would be
written by several threads, in place turned several times.  Refused on the host."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest
import torch

import sparse_attention_top_idx_gb300 as pkg
from sparse_attention_top_idx_gb300 import build, latent

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")
INVALID = 1
A = 1 << 20   # an aligned address that is never read: the calls are refused


@pytest.fixture(scope="module")
def rows_apart(tmp_path_factory):
    """The host function alone, built for this machine."""
    d = tmp_path_factory.mktemp("strides")
    src, lib = d / "s.cpp", d / "libs.so"
    src.write_text('#include "strides.h"\nextern "C" int apart(int64_t t, int64_t h, int64_t w, int64_t ts, int64_t hs)'
                   '{ return dsaidx::rows_apart(t, h, w, ts, hs); }\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).apart
    f.argtypes = [ctypes.c_int64] * 5
    return lambda *a: bool(f(*a))


def brute(t, h, w, ts, hs):
    seen = set()
    for i, j in itertools.product(range(t), range(h)):
        at = i * ts + j * hs
        row = range(at, at + w)
        if not seen.isdisjoint(row):
            return False
        seen.update(row)
    return True


def test_rows_apart_against_enumeration(rows_apart):
    r, yes = random.Random(2), 0
    for _ in range(20000):
        c = (r.randint(1, 7), r.randint(1, 7), r.randint(1, 5), r.randint(-24, 24), r.randint(-24, 24))
        assert rows_apart(*c) == brute(*c), c
        yes += brute(*c)
    assert 2000 < yes < 18000


def test_rows_apart_of_large_arguments(rows_apart):
    big = (1 << 63) - 1
    assert rows_apart(1 << 9, 1 << 24, 1024, big, 1024) and not rows_apart(1 << 9, 1 << 24, 1024, big, 1023)
    assert rows_apart(1 << 33, 1, 64, 64, 0) and rows_apart(1, 1 << 24, 2, 0, -2)
    assert not rows_apart(90000, 90000, 2, 90001, 90000)       # rows (b, 0) and (b - 1, 1) one apart
    assert rows_apart(90000, 90000, 1, 90001, 90000)           # interleaved, no two the same


BAD = [  # T, H, D, rot, offset, token stride, head stride
    (3, 4, 64, 64, 0, 64, 0), (3, 4, 64, 64, 0, 0, 64), (3, 1, 64, 64, 0, 0, 64), (1, 2, 64, 64, 0, 64, 63),
    (3, 4, 64, 64, 0, 128, 64), (2, 2, 64, 64, 0, 64, 64), (2, 8, 128, 64, 64, 256, 63), (2, 2, 64, 64, 0, -64, 64)]


@pytest.mark.parametrize("T,H,D,rot,offset,ts,hs", BAD)
def test_shared_elements_are_refused(T, H, D, rot, offset, ts, hs):
    build.build()
    L = latent.load()
    here = [0, T, H, D, A, A, rot, offset, 1.0, 0, None]
    assert L.idx_rope(A, ts, hs, A, ts, hs, *here) == INVALID                                   # in place
    assert L.idx_rope(A, H * D, D, A + (1 << 16), ts, hs, *here) == INVALID                     # as the result


def test_whole_heads_are_written_out_of_place():
    build.build()
    # the turned halves are apart, the copied ones are not
    assert latent.load().idx_rope(A, 512, 128, A + (1 << 16), 512, 64, 0, 3, 4, 128, A, A, 64, 0, 1.0, 0, None) == INVALID


@pytest.mark.gpu
def test_expanded_tensors_are_refused_by_the_binding():
    k = torch.ones(5, 64, dtype=torch.bfloat16, device="cuda")
    pos, plan = torch.arange(5, device="cuda"), latent.rope_plan(64)
    shared = k[:, None].expand(5, 3, 64)
    with pytest.raises(latent.IdxError) as e:
        latent.rope(shared, pos, plan)
    assert e.value.code == INVALID
    with pytest.raises(latent.IdxError) as e:
        latent.rope(torch.ones(5, 3, 64, dtype=torch.bfloat16, device="cuda"), pos, plan, out=shared)
    assert e.value.code == INVALID
    torch.cuda.synchronize()
    assert bool((k == 1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("half", [False, True])
def test_turned_parts_that_interleave_in_place(half):
    """Heads 32 elements apart of which 16 are turned: their other elements are shared, and left alone."""
    layout = latent.HALF if half else latent.INTERLEAVED
    g = torch.Generator(device="cuda").manual_seed(1)
    flat = torch.randn(7 * 5 * 32 + 32, generator=g, device="cuda")
    x, before = flat.as_strided((7, 5, 64), (160, 32, 1)), flat.clone()
    pos, plan = torch.arange(7, device="cuda") * 100, latent.rope_plan(16)
    want = torch.empty(7, 5, 64, device="cuda")
    latent.rope(x, pos, plan, layout=layout, offset=8, out=want)
    latent.rope(x, pos, plan, layout=layout, offset=8)
    assert torch.equal(x[:, :, 8:24], want[:, :, 8:24])
    rest = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    rest.as_strided((7, 5, 16), (160, 32, 1), 8).fill_(False)
    assert torch.equal(flat[rest], before[rest])
