"""The pages' calls of include/dsaidx_pages.h and the 8-bit latent cache's of
include/dsaidx_qlatent.h: exports, sizes, and every host-side refusal (answered
before any CUDA call, so no GPU is needed: pointers are made-up addresses that
are never read)."""
import ctypes
import math
import random

import pytest
import torch

from sparse_attention_top_idx_gb300 import build, dsaidx, latent, pages
from tests.test_latent_devices import On, on

OK, INVALID, TOO_SMALL = 0, 1, 4
A, B, C, D, E, F, G = (k << 20 for k in range(1, 8))   # aligned addresses, far apart


@pytest.fixture(scope="module")
def lib():
    build.build()
    latent.load()
    return pages.load()


def refused(call, good, cases):
    for i, bad, *want in cases:
        args = list(good)
        args[i] = bad
        assert call(*args) == (want[0] if want else INVALID), (i, bad)


def test_exports_every_declared_function(lib):
    for header, n in ((latent.QUANT_HEADER, 5), (pages.HEADER, 6)):
        names = latent.header_functions(header)
        assert len(names) == n, names
        for name in names:
            assert hasattr(lib, name), name


def test_sizes(lib):
    assert [latent.quant_block_bytes(b) for b in (0, -1, 65537)] == [0, 0, 0]
    for bs in (1, 7, 32, 64, 65536):
        assert latent.quant_block_bytes(bs) == (644 * bs + 127) // 128 * 128
    assert [pages.workspace_bytes(*a) for a in ((0, 1), (1 << 29, 1), (1, -1), (1, 65537))] == [0] * 4
    sizes = [pages.workspace_bytes(n, r) for n, r in ((1, 0), (1, 1), (1000, 1), (1000, 65536))]
    assert sizes == sorted(sizes) and sizes[0] >= 260


def pool(data=A, blocks=4, bs=64):
    return ctypes.byref(latent._Pool(data, blocks, bs))


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=A + 64), dict(blocks=0), dict(blocks=2 ** 31), dict(bs=0),
                                 dict(bs=65537), dict(blocks=2 ** 27, bs=64), dict(blocks=1 << 24, bs=64)])
def test_pool_refusals(lib, bad):
    assert lib.idx_qlatent_append(pool(**bad), A, 512, A, 64, A, A, 1, A, 1.0, 0, None, None) == INVALID
    assert lib.idx_qlatent_read(pool(**bad), A, 1, A, 576, None, None) == INVALID
    assert lib.idx_qlatent_attend_slots(pool(**bad), A, 512, 512, A, 64, 64, A, 8, 1, 1, 8, 1.0, A, None, A, 1 << 40,
                                        None) == INVALID
    assert lib.idx_qlatent_attend_paged(pool(**bad), A, 512, 512, A, 64, 64, A, 1, A, 1, 8, 1, 1.0, A, None, A, 1 << 40,
                                        None) == INVALID


def test_append_and_read_refusals(lib):
    #        latent stride pe stride pos slots n steps amp flags status stream
    good = [A, 512, A, 64, A, A, 0, A, 1.0, 0, None, None]
    assert lib.idx_qlatent_append(pool(), *good) == OK
    assert lib.idx_qlatent_append(None, *good) == INVALID
    good[6] = 2
    refused(lambda *a: lib.idx_qlatent_append(pool(), *a), good,
            [(0, None), (0, A + 8), (1, 516), (2, None), (2, A + 2), (3, 66), (4, None), (4, A + 4), (5, None), (5, A + 4),
             (6, -1), (6, 1 << 34), (7, A + 4), (9, 2), (9, 4), (10, A + 2)])
    #       slots n out stride status stream
    good = [A, 0, A, 576, None, None]
    assert lib.idx_qlatent_read(pool(), *good) == OK
    assert lib.idx_qlatent_read(None, *good) == INVALID
    good[1] = 2
    refused(lambda *a: lib.idx_qlatent_read(pool(), *a), good,
            [(0, None), (0, A + 4), (1, -1), (1, 1 << 34), (2, None), (2, A + 8), (3, 575), (3, 580), (3, 0), (4, A + 1)])


def test_attend_refusals(lib):
    ws = 256
    #        ql row  head qp row head slots stride rows heads topk scale out lse ws bytes stream
    slots = [A, 8192, 512, A, 1024, 64, A, 8, 2, 16, 8, 1.0, A, None, A, ws, None]
    #        ql row  head qp row head table mbps lens batch max heads scale out lse ws bytes stream
    paged = [A, 8192, 512, A, 1024, 64, A, 4, A, 2, 8, 16, 1.0, A, None, A, ws, None]
    assert lib.idx_qlatent_attend_slots(None, *slots) == INVALID
    assert lib.idx_qlatent_attend_paged(None, *paged) == INVALID
    refused(lambda *a: lib.idx_qlatent_attend_slots(pool(), *a), slots,
            [(0, None), (0, A + 8), (1, 8196), (2, 4), (3, None), (3, A + 2), (4, 1028), (5, 66), (6, None), (6, A + 4),
             (8, -1), (8, 2 ** 31), (9, 0), (9, 1025), (10, -1), (10, 2 ** 24 + 1), (11, math.nan), (11, math.inf),
             (12, None), (1, 0), (2, 0), (4, -1024), (5, 0), (1, 2 ** 40), (12, A + 8), (13, A + 2), (14, None),
             (14, A + 128), (15, ws - 1, TOO_SMALL)])
    refused(lambda *a: lib.idx_qlatent_attend_paged(pool(), *a), paged,
            [(0, None), (3, None), (6, None), (6, A + 2), (7, 0), (8, None), (9, -1), (10, -1), (11, 0), (12, math.nan),
             (13, None), (14, A + 1), (15, None), (16, ws - 1, TOO_SMALL)])
    slots[8] = 0
    paged[9] = 0
    assert lib.idx_qlatent_attend_slots(pool(), *slots) == OK
    assert lib.idx_qlatent_attend_paged(pool(), *paged) == OK


def ws_answers(lib, rows, heads, keys, size):
    """What calls without slots or a table answer, which is looked at behind the workspace's size."""
    head = [A, 512 * heads, 512, A, 64 * heads, 64]
    return (lib.idx_qlatent_attend_slots(pool(), *head, None, keys, rows, heads, keys, 1.0, A, None, A, size, None),
            lib.idx_qlatent_attend_paged(pool(), *head, None, 1, A, rows, keys, heads, 1.0, A, None, A, size, None))


def test_a_workspace_of_the_largest_call_serves_every_smaller_one(lib):
    r = random.Random(3)
    sizes = [(rows, heads, keys) for rows in (1, 7, 14, 18, 19, 37, 38, 75, 76, 77, 152, 153, 300, 4096)
             for heads in (1, 16, 17, 32, 33, 64, 65, 128, 1024) for keys in (1, 128, 640, 641, 1024, 1025, 4096, 131072, 1 << 24)]
    sizes += [(r.randint(1, 700), r.randint(1, 300), int(2 ** r.uniform(0, 18))) for _ in range(3000)]
    for c in sizes:
        size = latent.workspace_bytes(*c)
        assert ws_answers(lib, *c, size) == (INVALID, INVALID), c
        smaller = [r.randint(1, x) for x in c]
        assert ws_answers(lib, *smaller, size) == (INVALID, INVALID), (smaller, c)
    # a cut one needs room, and says so (32 rows of selected slots lie over clusters, which need none)
    assert ws_answers(lib, 32, 16, 10000, 256) == (INVALID, TOO_SMALL)
    assert ws_answers(lib, 160, 16, 1024, 256) == (TOO_SMALL, TOO_SMALL)


def test_fork_refusals(lib):
    #       refs blocks bs table old mbps lens parents rows new mbps lens pairs ws bytes stream
    good = [A, 100, 64, B, 2, 8, C, D, 0, E, 8, F, G, 8 << 20, 1 << 20, None]
    assert lib.idx_pages_fork(*good) == OK
    good[8] = 3
    refused(lib.idx_pages_fork, good,
            [(0, None), (0, A + 4), (1, 0), (1, 1 << 29), (2, 0), (2, 65537), (3, None), (3, B + 2), (4, -1), (4, 65537),
             (5, 0), (5, 1 << 30), (6, None), (7, None), (7, D + 1), (8, -1), (8, 65537), (9, None), (10, 0), (10, 1 << 29),
             (11, None), (12, None), (12, G + 3), (13, None), (13, (8 << 20) + 128), (14, 255, TOO_SMALL),
             (9, B), (9, B + 32), (9, A + 396), (11, C), (11, C + 4), (12, D), (11, E + 4), (12, E), (0, G)])


def test_extend_refusals(lib):
    #       refs blocks bs table rows mbps lens longer ws bytes stream
    good = [A, 100, 64, B, 0, 8, C, D, G, 1 << 20, None]
    assert lib.idx_pages_extend(*good) == OK
    good[4] = 3
    refused(lib.idx_pages_extend, good,
            [(0, None), (0, A + 8), (1, 0), (2, 0), (3, None), (4, -1), (5, 0), (6, None), (7, None), (7, D + 2), (8, None),
             (8, G + 4), (9, 400, TOO_SMALL), (6, B + 8), (7, C), (7, A), (3, A + 4), (6, A + 396)])


def test_free_refusals(lib):
    #       refs blocks table rows mbps lens which n status stream
    good = [A, 100, B, 4, 8, C, None, 0, None, None]
    assert lib.idx_pages_free(*good) == OK
    good[7] = 4
    refused(lib.idx_pages_free, good,
            [(0, None), (1, 0), (2, None), (2, B + 1), (3, -1), (4, 0), (5, None), (6, D + 2), (7, -1), (7, 5), (7, 65537),
             (8, G + 2)])
    good[6], good[7] = D, 65537
    assert lib.idx_pages_free(*good) == INVALID


def test_compact_refusals(lib):
    #       refs blocks table rows mbps new_refs new_table map pairs count ws bytes stream
    good = [A, 100, B, 4, 8, C, D, E, F, G, 8 << 20, 256, None]
    refused(lib.idx_pages_compact, good,
            [(0, None), (0, A + 4), (1, 0), (2, None), (3, -1), (4, 0), (5, None), (6, None), (7, None), (8, None), (8, F + 4),
             (9, None), (10, None), (10, (8 << 20) + 4), (11, 255, TOO_SMALL), (5, A + 4), (6, B + 4), (7, A), (8, E), (9, A),
             (9, C + 8), (7, D), (5, B), (6, A)])


def test_copy_refusals(lib):
    two = (pages._PagePool * 2)(pages._PagePool(A, 64), pages._PagePool(B, 41216))
    #       pools n blocks pairs n count status stream
    good = [two, 2, 100, C, 0, None, None, None]
    assert lib.idx_pages_copy(*good) == OK
    good[4] = 3
    refused(lib.idx_pages_copy, good, [(0, None), (1, -1), (1, 129), (2, 0), (3, None), (3, C + 4), (4, -1), (5, D + 2), (6, D + 1)])
    for data, nbytes in ((None, 64), (A + 8, 64), (A, 0), (A, 24), (A, -16), (A, 1 << 33)):
        one = (pages._PagePool * 1)(pages._PagePool(data, nbytes))
        assert lib.idx_pages_copy(one, 1, 100, C, 3, None, None, None) == INVALID, (data, nbytes)


# ---------------------------------------------------------------------------
# the binding: CPU tensors that claim a device, and a library that notes its calls
# ---------------------------------------------------------------------------
I32, I64, U8 = torch.int32, torch.int64, torch.uint8


class Library:
    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        if name == "idx_qlatent_block_bytes":
            return lambda bs: (644 * bs + 127) // 128 * 128
        return lambda *args: self.made.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(dsaidx, "_lib", fake)
    monkeypatch.setattr(latent, "_bound", fake)
    monkeypatch.setattr(pages, "_bound", fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return fake


def cache(d):
    return latent.QuantLatentCache(on(d, 2, 41216, dtype=U8), 64)


def page_set(d):
    return pages.PageSet(on(d, 10, dtype=I32), 64, [on(d, 10, 16, dtype=U8), on(d, 10, 3, 8)])


def ints(*shape):
    return lambda d: on(d, *shape, dtype=I32)


WS = lambda d: on(d, 1024, dtype=U8)  # noqa: E731
CALLS = {
    "append": (lambda cache, c, pe, slots, status: latent.latent_append(cache, c, pe, None, slots, None, status=status),
               dict(cache=cache, c=lambda d: on(d, 3, 512), pe=lambda d: on(d, 3, 64), slots=lambda d: on(d, 3, dtype=I64),
                    status=ints(1)), "idx_qlatent_append"),
    "read": (lambda cache, slots, out, status: latent.latent_read(cache, slots, out, status=status),
             dict(cache=cache, slots=lambda d: on(d, 3, dtype=I64), out=lambda d: on(d, 3, 576), status=ints(1)), "idx_qlatent_read"),
    "slots": (lambda cache, ql, qp, slots, out, ws: latent.latent_attend_slots(cache, ql, qp, slots, 0.1, out, ws),
              dict(cache=cache, ql=lambda d: on(d, 3, 16, 512), qp=lambda d: on(d, 3, 16, 64),
                   slots=lambda d: on(d, 3, 8, dtype=I64), out=lambda d: on(d, 3, 16, 512), ws=WS), "idx_qlatent_attend_slots"),
    "paged": (lambda cache, ql, qp, table, lens, out, ws: latent.latent_attend_paged(cache, ql, qp, table, lens, 8, 0.1, out, ws),
              dict(cache=cache, ql=lambda d: on(d, 3, 16, 512), qp=lambda d: on(d, 3, 16, 64), table=ints(3, 1), lens=ints(3),
                   out=lambda d: on(d, 3, 16, 512), ws=WS), "idx_qlatent_attend_paged"),
    "fork": (lambda ps, table, lens, parents, t2, l2, pairs, ws: pages.fork(ps, table, lens, parents, t2, l2, pairs, ws),
             dict(ps=page_set, table=ints(4, 5), lens=ints(4), parents=ints(3), t2=ints(3, 6), l2=ints(3), pairs=ints(3, 2), ws=WS),
             "idx_pages_fork"),
    "extend": (lambda ps, table, lens, longer, ws: pages.extend(ps, table, lens, longer, ws),
               dict(ps=page_set, table=ints(4, 5), lens=ints(4), longer=ints(4), ws=WS), "idx_pages_extend"),
    "free": (lambda ps, table, lens, which, status: pages.free(ps, table, lens, which, status=status),
             dict(ps=page_set, table=ints(4, 5), lens=ints(4), which=ints(2), status=ints(1)), "idx_pages_free"),
    "compact": (lambda ps, table, r2, t2, page_map, pairs, count, ws: pages.compact(ps, table, r2, t2, page_map, pairs, count, ws),
                dict(ps=page_set, table=ints(4, 5), r2=ints(10), t2=ints(4, 5), page_map=ints(10), pairs=ints(5, 2), count=ints(1),
                     ws=WS), "idx_pages_compact"),
    "copy": (lambda ps, pairs, count, status: pages.copy(ps, pairs, count=count, status=status),
             dict(ps=page_set, pairs=ints(3, 2), count=ints(1), status=ints(1)), "idx_pages_copy"),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_the_current_device_are_made(name, library):
    call, args, want = CALLS[name]
    call(**{k: make(0) for k, make in args.items()})
    assert library.made == [want]


@pytest.mark.parametrize("name,other", [(n, a) for n, (_, args, _) in CALLS.items() for a in args])
def test_one_argument_elsewhere_is_refused(name, other, library):
    call, args, _ = CALLS[name]
    for here, there in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="cuda:"):
            call(**{k: make(there if k == other else here) for k, make in args.items()})
    assert not library.made


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_a_device_that_is_not_current_are_refused(name, library):
    call, args, _ = CALLS[name]
    with pytest.raises(ValueError, match="current"):
        call(**{k: make(1) for k, make in args.items()})
    assert not library.made


@pytest.mark.parametrize("name,other", [(n, a) for n, (_, args, _) in CALLS.items() for a in args if a not in ("cache", "ps")])
def test_tensors_of_another_kind_are_refused(name, other, library):
    """On the CPU, of another type, of another shape."""
    call, args, _ = CALLS[name]

    def with_other(change):
        made = {k: make(0) for k, make in args.items()}
        made[other] = change(made[other])
        return made

    with pytest.raises(TypeError):
        call(**with_other(lambda t: t.as_subclass(torch.Tensor)))
    with pytest.raises(TypeError):
        call(**with_other(lambda t: on(0, *t.shape, dtype=torch.float64)))
    if other not in ("status", "ws", "which", "cuq"):
        with pytest.raises(ValueError):
            call(**with_other(lambda t: on(0, *[n + 1 for n in t.shape], 2, dtype=t.dtype)))
    assert not library.made


def test_handles_refuse(library):
    with pytest.raises(ValueError):
        latent.QuantLatentCache(on(0, 2, 41215, dtype=U8), 64)
    with pytest.raises(ValueError):
        latent.QuantLatentCache(on(0, 2 * 41216, dtype=U8), 64)
    with pytest.raises(TypeError):
        latent.QuantLatentCache(on(0, 2, 41216, dtype=torch.int8), 64)
    with pytest.raises(TypeError):
        latent.latent_read(latent.LatentCache(on(0, 2, 64, 576)), on(0, 3, dtype=I64), on(0, 3, 576))
    with pytest.raises(ValueError):
        pages.PageSet(on(0, 10, dtype=I32), 64, [on(0, 10, 12, dtype=U8)])
    with pytest.raises(ValueError):
        pages.PageSet(on(0, 10, dtype=I32), 64, [on(0, 11, 16, dtype=U8)])
    with pytest.raises(ValueError):
        pages.PageSet(on(0, 10, dtype=I32), 64, [on(1, 10, 16, dtype=U8)])
    with pytest.raises(ValueError):
        pages.PageSet(on(0, 0, dtype=I32), 64)
    with pytest.raises(TypeError):
        pages.PageSet(on(0, 10, dtype=I64), 64)
    with pytest.raises(ValueError):
        pages.PageSet(on(0, 10, dtype=I32), 64, [on(0, 10, 16, dtype=U8)] * 129)
    assert isinstance(on(0, 1), On) and not library.made
