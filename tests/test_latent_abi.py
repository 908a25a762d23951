"""The latent-attention calls of include/dsaidx_latent.h: exports, rotary
steps on the host, and every host-side refusal (answered before any CUDA call,
so no GPU is needed: pointers are made-up addresses that are never read)."""
import ctypes
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import build, latent

OK, INVALID, TOO_SMALL = 0, 1, 4
A = 1 << 20   # an aligned address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return latent.load()


def pool(data=A, blocks=4, bs=64):
    return ctypes.byref(latent._Pool(data, blocks, bs))


def test_exports_every_declared_function(lib):
    names = latent.header_functions()
    assert len(names) == 7, names
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("dim", [2, 64, 96, 1024])
def test_steps_are_fractions_of_a_turn(dim):
    steps, amp = latent.rope_steps(dim, 10000.0)
    assert amp == 1.0 and steps.numel() == dim // 2
    for i, s in enumerate(steps.tolist()):
        f = 10000.0 ** (-2.0 * i / dim)
        # the double f carries half a step (2^-53), pow and the division a few more
        assert abs((s & (2 ** 64 - 1)) / 2.0 ** 64 * 2 * math.pi - f) <= 8 * 2.0 ** -53 * f + 2.0 ** -60


def test_linear_and_yarn_steps():
    plain, _ = latent.rope_steps(64, 10000.0)
    lin, amp = latent.rope_steps(64, 10000.0, "linear", 4.0)
    assert amp == 1.0
    assert all(abs(a - 4 * b) <= 8 + abs(a) * 2.0 ** -50 for a, b in zip(plain.tolist(), lin.tolist()))
    yarn, amp = latent.rope_steps(64, 10000.0, "yarn", 40.0, 4096, 32.0, 1.0)
    assert amp == ctypes.c_float(0.1 * math.log(40.0) + 1.0).value
    turns = lambda b: 64 * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = math.floor(turns(32.0)), math.ceil(turns(1.0))
    for i, (a, b) in enumerate(zip(plain.tolist(), yarn.tolist())):
        r = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert abs(b - a * (1 - r + r / 40.0)) <= 64 + abs(a) * 2.0 ** -49, i


def test_steps_refusals(lib):
    buf, amp = (ctypes.c_uint64 * 512)(), ctypes.c_float()
    p, a = ctypes.cast(buf, ctypes.c_void_p), ctypes.byref(amp)
    good = [64, 10000.0, 2, 40.0, 4096.0, 32.0, 1.0]
    assert lib.idx_rope_steps(*good, p, a) == OK
    nan, inf = math.nan, math.inf
    for i, bad in [(0, 0), (0, 63), (0, 1026), (0, -2), (1, 1.0), (1, nan), (1, inf), (2, 3), (2, -1), (3, 0.5), (3, nan),
                   (3, inf), (4, 0.0), (4, inf), (5, 0.5), (5, inf), (6, 0.0), (6, nan)]:
        args = list(good)
        args[i] = bad
        assert lib.idx_rope_steps(*args, p, a) == INVALID, (i, bad)
    assert lib.idx_rope_steps(*good, None, a) == INVALID
    assert lib.idx_rope_steps(*good, p, None) == INVALID
    with pytest.raises(ValueError):
        latent.rope_steps(64, scaling="cubic")


def test_rope_refusals(lib):
    #        x  xt   xh  y      yt   yh  dt T  H  D   pos steps rot off amp flags stream
    good = [A, 128, 64, A + 2, 128, 64, 0, 0, 2, 64, A, A, 64, 0, 1.0, 0, None]
    assert lib.idx_rope(*good) == OK                      # no tokens: nothing to do
    for i, bad in [(6, 3), (6, -1), (7, -1), (7, 2 ** 32), (8, 0), (8, 2 ** 24 + 1), (9, 0), (9, 1025), (12, 0), (12, 63), (12, 66), (13, 1),
                   (13, -1), (15, 4)]:
        args = list(good)
        args[i] = bad
        assert lib.idx_rope(*args) == INVALID, (i, bad)
    some = list(good)
    some[7] = 3
    for i, bad in [(0, None), (3, None), (10, None), (11, None), (0, A + 1), (3, A + 1), (10, A + 4), (11, A + 4)]:
        args = list(some)
        args[i] = bad
        assert lib.idx_rope(*args) == INVALID, (i, bad)
    args = list(some)
    args[3], args[4] = A, 256                             # in place with other strides
    assert lib.idx_rope(*args) == INVALID
    args = list(some)
    args[6], args[0] = 2, A + 2                           # fp32 off its size
    assert lib.idx_rope(*args) == INVALID


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=A + 64), dict(blocks=0), dict(blocks=2 ** 31), dict(bs=0),
                                 dict(bs=65537), dict(blocks=2 ** 27, bs=64)])
def test_pool_refusals(lib, bad):
    assert lib.idx_latent_append(pool(**bad), A, 512, A, 64, A, A, 1, A, 1.0, 0, None, None) == INVALID
    assert lib.idx_latent_attend_slots(pool(**bad), A, 512, 512, A, 64, 64, A, 8, 1, 1, 8, 1.0, A, None, A, 1 << 40,
                                       None) == INVALID
    assert lib.idx_latent_attend_paged(pool(**bad), A, 512, 512, A, 64, 64, A, 1, A, 1, 8, 1, 1.0, A, None, A, 1 << 40,
                                       None) == INVALID


def test_append_refusals(lib):
    #        latent stride pe stride pos slots n steps amp flags status stream
    good = [A, 512, A, 64, A, A, 0, A, 1.0, 0, None, None]
    assert lib.idx_latent_append(pool(), *good) == OK
    assert lib.idx_latent_append(None, *good) == INVALID
    good[6] = 2
    for i, bad in [(0, None), (0, A + 8), (1, 516), (2, None), (2, A + 2), (3, 66), (4, None), (4, A + 4), (5, None),
                   (5, A + 4), (6, -1), (7, A + 4), (9, 2), (9, 4)]:
        args = list(good)
        args[i] = bad
        assert lib.idx_latent_append(pool(), *args) == INVALID, (i, bad)


def test_attend_refusals(lib):
    ws = latent.workspace_bytes(2, 16, 8)
    assert ws >= 256 and latent.workspace_bytes(-1, 16, 8) == 0 and latent.workspace_bytes(2, 0, 8) == 0
    assert latent.workspace_bytes(2, 1025, 8) == 0 and latent.workspace_bytes(2, 16, -1) == 0
    #        ql row  head qp row head slots stride rows heads topk scale out lse ws bytes stream
    slots = [A, 8192, 512, A, 1024, 64, A, 8, 2, 16, 8, 1.0, A, None, A, ws, None]
    #        ql row  head qp row head table mbps lens batch max heads scale out lse ws bytes stream
    paged = [A, 8192, 512, A, 1024, 64, A, 4, A, 2, 8, 16, 1.0, A, None, A, ws, None]
    assert lib.idx_latent_attend_slots(None, *slots) == INVALID
    assert lib.idx_latent_attend_paged(None, *paged) == INVALID
    for i, bad, want in [(0, None, INVALID), (0, A + 8, INVALID), (1, 8196, INVALID), (2, 4, INVALID), (3, None, INVALID),
                         (3, A + 2, INVALID), (4, 1028, INVALID), (5, 66, INVALID), (6, None, INVALID), (6, A + 4, INVALID),
                         (8, -1, INVALID), (8, 2 ** 31, INVALID), (9, 0, INVALID), (9, 1025, INVALID), (10, -1, INVALID),
                         (10, 2 ** 24 + 1, INVALID), (11, math.nan, INVALID), (11, math.inf, INVALID), (12, None, INVALID),
                         (1, 0, INVALID), (2, 0, INVALID), (4, -1024, INVALID), (5, 0, INVALID), (1, 2 ** 40, INVALID),
                         (12, A + 8, INVALID), (14, None, INVALID), (14, A + 128, INVALID), (15, ws - 1, TOO_SMALL)]:
        args = list(slots)
        args[i] = bad
        assert lib.idx_latent_attend_slots(pool(), *args) == want, (i, bad)
    for i, bad, want in [(0, None, INVALID), (3, None, INVALID), (6, None, INVALID), (6, A + 2, INVALID), (7, 0, INVALID),
                         (8, None, INVALID), (9, -1, INVALID), (10, -1, INVALID), (11, 0, INVALID), (12, math.nan, INVALID),
                         (13, None, INVALID), (15, None, INVALID), (16, ws - 1, TOO_SMALL)]:
        args = list(paged)
        args[i] = bad
        assert lib.idx_latent_attend_paged(pool(), *args) == want, (i, bad)
    slots[8] = 0
    paged[9] = 0
    assert lib.idx_latent_attend_slots(pool(), *slots) == OK       # no rows: nothing to do
    assert lib.idx_latent_attend_paged(pool(), *paged) == OK


def test_expanded_refusals(lib):
    #        q row  head kn row  head kp row v row  head cuq cuk batch T S heads scale out lse status stream
    good = [A, 1536, 192, A, 1024, 128, A, 64, A, 1024, 128, A, A, 1, 0, 0, 8, 1.0, A, None, None, None]
    assert lib.idx_latent_attend_expanded(*good) == OK
    good[14], good[15] = 4, 4
    for i, bad in [(0, None), (0, A + 8), (1, 1540), (2, 2 ** 31), (3, None), (3, A + 8), (4, -8), (5, 132), (6, None),
                   (7, 68), (8, None), (9, 12), (10, 4), (11, None), (11, A + 2), (12, None), (13, -1), (13, 4097),
                   (1, 0), (2, 0), (4, 0), (7, 0), (9, 0), (14, -1), (14, 2 ** 31), (15, -1), (15, 2 ** 31), (16, 0), (16, 1025), (17, math.nan), (18, None),
                   (18, A + 8)]:
        args = list(good)
        args[i] = bad
        assert lib.idx_latent_attend_expanded(*args) == INVALID, (i, bad)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int64)
    plan = latent.rope_plan(64, device="cpu")
    with pytest.raises(TypeError):
        latent.rope(x, pos, plan)
    with pytest.raises(TypeError):
        latent.rope(x.double(), pos, plan)
    with pytest.raises(TypeError):
        latent.LatentCache(torch.zeros(2, 64, 576, dtype=torch.bfloat16))
