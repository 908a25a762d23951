"""One workspace of the largest batch serves every smaller absorbed attention call."""
import itertools
import random

import pytest
import torch

from sparse_attention_top_idx_gb300 import build, dsaidx, latent
from tests.test_gpu_latent import check_attend, normal, gen, paged_inputs, queries, want_paged, want_slots, LAT, BF, SCALE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_sizes_never_fall():
    rows = sorted({0, 1, 2, 7, 18, 19, 37, 38, 63, 64, 75, 76, 77, 128, 151, 152, 153, 160, 256, 300, 303, 304, 305, 1000, 4096, 100000})
    heads = [1, 16, 17, 32, 33, 64, 65, 128, 129, 1024]
    keys = [0, 1, 64, 512, 576, 640, 641, 704, 705, 768, 832, 833, 1024, 1025, 2048, 4096, 10000, 22000, 131072, 1 << 24]
    size = {c: latent.workspace_bytes(*c) for c in itertools.product(rows, heads, keys)}
    for axis, values in enumerate((rows, heads, keys)):
        for c, s in size.items():
            at = values.index(c[axis])
            if at:
                less = list(c)
                less[axis] = values[at - 1]
                assert size[tuple(less)] <= s, (less, c)
    assert min(size.values()) == 256 and max(size.values()) <= 40100000


def test_sizes_never_fall_at_random():
    r = random.Random(1)
    for _ in range(20000):
        c = [r.randint(0, 700), r.randint(1, 300), int(2 ** r.uniform(0, 18))]
        d = [r.randint(0, c[0]), r.randint(1, c[1]), r.randint(0, c[2])]
        assert latent.workspace_bytes(*d) <= latent.workspace_bytes(*c), (c, d)


def test_sizes_of_calls_that_are_refused():
    assert latent.workspace_bytes(1 << 31, 1, 8) == 0 and latent.workspace_bytes(1 << 62, 1024, 8) == 0
    assert latent.workspace_bytes((1 << 31) - 1, 64, 8) > 0 and latent.workspace_bytes(1 << 30, 65, 8) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("large,small,H,most", [(152, 151, 16, 131072), (76, 75, 128, 131072), (300, 128, 16, 22000),
                                                (40, 3, 20, 10000), (200, 1, 64, 4096)])
def test_paged_calls_in_the_workspace_of_a_larger_one(large, small, H, most):
    g = gen(large + H)
    lens = [int(x) for x in torch.randint(0, 200, (small,), generator=g, device="cuda").tolist()]
    lens[-1] = min(1500, most)
    pool, table, sl, slots = paged_inputs(g, lens, 64)
    ql, qp = queries(g, small, H)
    out = torch.full((small, H, LAT), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((small, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(large, H, most))
    latent.latent_attend_paged(latent.LatentCache(pool), ql, qp, table, sl, most, SCALE, out, ws, lse=lse)
    assert dsaidx.read_device_status(ws) == 0
    check_attend(out, lse, want_paged(pool, ql, qp, slots))


@pytest.mark.gpu
@pytest.mark.parametrize("large,small,H,topk", [(300, 160, 16, 1024), (300, 2, 16, 2048), (152, 100, 64, 2048)])
def test_slot_calls_in_the_workspace_of_a_larger_one(large, small, H, topk):
    g = gen(large + H + topk)
    pool = normal(g, 40, 64, latent.RECORD)
    ql, qp = queries(g, small, H)
    slots = torch.randint(0, 40 * 64, (small, topk), generator=g, device="cuda")
    out = torch.full((small, H, LAT), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((small, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(large, H, topk))
    latent.latent_attend_slots(latent.LatentCache(pool), ql, qp, slots, SCALE, out, ws, lse=lse)
    assert dsaidx.read_device_status(ws) == 0
    check_attend(out, lse, want_slots(pool, ql, qp, slots))
