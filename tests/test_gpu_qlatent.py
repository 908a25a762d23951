"""GPU numerics of the 8-bit latent cache: the append against the format's
definition byte by byte, the read-back, and the absorbed attention against plain
64-bit formulas (tolerances: qrecords.attend64)."""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent
from tests import qrecords as qr
from tests.qrecords import LAT, PE, REC, SCALE, filled, want_paged, want_slots
from tests.test_gpu_latent import BF, check_attend, check_turned, gen, normal, paged_call, queries, slots_call, turned

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
def latents(g, n):
    """Tokens whose largest latents lie all over the type's range, at and beside the scale's steps."""
    c = normal(g, n, LAT + 8)[:, :LAT]
    size = [1.0, 1e-30, 3e37, 448.0, 450.0, 0.0, 2.0 ** -41, 2.0 ** -60, 1e-40, 7.0, 7.03125, 2.0 ** 20]
    for i in range(n):
        k = size[i % len(size)]
        if i % 12 >= 3:
            c[i] *= k / 8.0 if k else 0.0
            c[i, i % LAT] = k * (-1) ** i
        else:
            c[i] *= k
    return c


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,bs", [(1, 64), (7, 32), (333, 48), (50, 1), (20, 7)])
def test_append(half, n, bs):
    g = gen(n)
    c, pe = latents(g, n), normal(g, n, 2 * PE)[:, PE:]
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda")
    nb = n // bs + 2
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:n].contiguous()
    slots[3::5] = -1
    pool = torch.full((nb, qr.block_bytes(bs)), 0xA5, dtype=torch.uint8, device="cuda")
    cache = latent.QuantLatentCache(pool, bs)
    latent.latent_append(cache, c, pe, pos, slots, latent.rope_plan(PE), layout=latent.HALF if half else latent.INTERLEAVED)
    ok = slots >= 0
    at = slots[ok]
    codes, p, s = qr.take(pool, bs, at)
    want_c, _, want_s = qr.encode(c[ok], pe[ok])
    assert torch.equal(s, want_s) and torch.equal(codes, want_c)
    want, mag = turned(pe[:, None], pos, PE, 0, half)
    # the turned key in bf16, divided by a power of two: where that leaves the normal range, rounded once more
    got = p.double() * s.double()[:, None]
    err = (got - want[ok, 0]).abs()
    tol = want[ok, 0].abs() * 2.0 ** -8 + mag[ok, 0] * 2.0 ** -21 + 2.0 ** -133 * s.double()[:, None] + 2.0 ** -126
    assert bool((err <= tol).all())
    # nothing else was written
    rest = torch.full_like(pool, 0xA5)
    qr.put(rest, bs, at, codes, p, s)
    assert torch.equal(pool, rest)
    latent.latent_append(cache, c, pe, None, slots, None)
    for a, b in zip(qr.take(pool, bs, at), qr.encode(c[ok], pe[ok])):
        assert torch.equal(a, b)


def test_append_agrees_with_the_bf16_cache():
    """The same turned key, element by element."""
    g = gen(2)
    kv, pos = normal(g, 100, REC), torch.randint(0, 1 << 20, (100,), generator=g, device="cuda")
    slots, plan = torch.randperm(128, generator=g, device="cuda")[:100], latent.rope_plan(PE, amplitude=1.3)
    a, b = latent.LatentCache.allocate(2, 64), latent.QuantLatentCache.allocate(2, 64)
    for layout in (latent.INTERLEAVED, latent.HALF):
        for c in (a, b):
            latent.latent_append(c, kv[:, :LAT], kv[:, LAT:], pos, slots, plan, layout=layout)
        out = torch.empty(100, REC, dtype=BF, device="cuda")
        latent.latent_read(b, slots, out)
        assert torch.equal(out[:, LAT:], a.pool.view(-1, REC)[slots][:, LAT:])


def test_append_rounds_every_bf16_number():
    """Every finite bf16 number under each of its possible scales' neighbours: the nearest code, ties to even."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    x = bits.view(BF)
    x = x[x.isfinite()]
    x = torch.cat([x, x.new_zeros(-x.numel() % (LAT - 1))]).view(-1, LAT - 1)
    g = gen(3)
    for top in (1.0, 448.0, 0.01, 1.75, 1.7578125):
        c = torch.cat([x.abs().clamp_max(top) * torch.sign(x.float()).to(BF), torch.full_like(x[:, :1], top)], 1)
        n = c.shape[0]
        cache = latent.QuantLatentCache.allocate((n + 63) // 64, 64)
        slots = torch.randperm(cache.num_blocks * 64, generator=g, device="cuda")[:n]
        latent.latent_append(cache, c, torch.zeros(n, PE, dtype=BF, device="cuda"), None, slots, None)
        codes, _, s = qr.take(cache.pool, 64, slots)
        want, _, ws = qr.encode(c, torch.zeros(n, PE, dtype=BF, device="cuda"))
        assert torch.equal(s, ws)
        # a zero's sign is kept by the format and lost by the sign function above
        assert torch.equal(torch.where(codes == 128, 0, codes), torch.where(want == 128, 0, want))


def test_append_not_finite_and_status():
    g = gen(4)
    kv = normal(g, 6, REC)
    kv[1, 7], kv[2, 9], kv[3, :LAT], kv[4, LAT + 3] = math.inf, math.nan, -math.inf, -math.inf
    cache = latent.QuantLatentCache.allocate(2, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 70, 9, 127, 64, 128], device="cuda")
    latent.latent_append(cache, kv[:, :LAT], kv[:, LAT:], None, slots, None, status=status)
    assert int(status) == 5
    codes, p, s = qr.take(cache.pool, 64, slots[:5])
    wc, wp, ws = qr.encode(kv[:5, :LAT], kv[:5, LAT:])
    assert torch.equal(codes & 127, wc & 127) and torch.equal(s, ws)
    assert torch.equal(p.isnan(), wp.isnan()) and torch.equal(p[~p.isnan()], wp[~wp.isnan()])
    out = torch.empty(5, REC, dtype=BF, device="cuda")
    latent.latent_read(cache, slots[:5].contiguous(), out)
    bad = ~kv[:5].isfinite()
    assert bool(out[:, :LAT][bad[:, :LAT]].isnan().all()) and float(out[4, LAT + 3]) == -math.inf
    assert bool(out[~bad].isfinite().all())


@pytest.mark.parametrize("n,bs", [(1, 64), (5, 32), (1000, 48), (77, 3)])
def test_read(n, bs):
    g = gen(n)
    cache = filled(g, 20 if bs > 3 else 100, bs, spread=3.0)
    slots = torch.randint(0, cache.num_blocks * bs, (n,), generator=g, device="cuda")
    slots[2::7] = -5
    wide = torch.full((n, REC + 24), 7.0, dtype=BF, device="cuda")
    out = wide[:, 8:8 + REC]
    assert latent.latent_read(cache, slots, out) is out
    rec, _ = qr.records(cache.pool, bs, slots.clamp_min(0))
    want = torch.where((slots >= 0)[:, None], rec, 0.0)
    assert torch.equal(out.double(), want)                       # exact: codes and bf16 under powers of two
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + REC:] == 7).all())


def test_read_status():
    cache = filled(gen(5), 2, 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((4, REC), 3.0, dtype=BF, device="cuda")
    latent.latent_read(cache, torch.tensor([1, 64, -1, 1 << 40], device="cuda"), out, status=status)
    assert int(status) == 5 and bool((out[1:] == 0).all())
    assert torch.equal(out[0].double(), qr.records(cache.pool, 32, torch.tensor([1], device="cuda"))[0][0])


# ---------------------------------------------------------------------------
# absorbed attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,H,topk,kind", [(1, 1, 1, 0), (1, 128, 64, 0), (3, 16, 63, 1), (2, 64, 65, 0), (5, 20, 1000, 1),
                                           (32, 128, 512, 1), (2, 130, 129, 0), (700, 17, 40, 1), (160, 64, 128, 0),
                                           (4, 33, 2048, 0), (1, 16, 4096, 0), (620, 100, 192, 0), (64, 16, 129, 0),
                                           (64, 30, 300, 1), (30, 128, 577, 0), (16, 64, 512, 0), (8, 5, 1024, 0),
                                           (3, 32, 700, 1), (70, 40, 128, 0), (200, 24, 1024, 0)])
def test_attend_slots(T, H, topk, kind):
    g = gen(T * 7 + H)
    cache = filled(g, 40, 64)
    ql, qp = queries(g, T, H, kind)
    slots = torch.randint(0, 40 * 64, (T, topk), generator=g, device="cuda")
    check_attend(*slots_call(cache, ql, qp, slots), want_slots(cache, ql, qp, slots))


@pytest.mark.parametrize("H", [5, 24, 64, 128])
def test_attend_slots_masks(H):
    """Rows with no key, one key, keys only at the front, at the end, between, a whole tile masked; NaN in every
    record, and scales that are no numbers, that no row lists; slots in a wider buffer."""
    g = gen(H)
    cache = filled(g, 10, 64)
    every = torch.arange(640, device="cuda")
    codes, p, s = qr.take(cache.pool, 64, every)
    codes[::2] = 127
    s[1::8] = math.inf
    s[3::8] = math.nan
    p[5::8] = math.inf
    qr.put(cache.pool, 64, every, codes, p, s)
    good = every[every % 8 == 7]
    T, topk = 9, 300
    wide = torch.full((T, topk + 3), -1, dtype=torch.int64, device="cuda")
    slots = wide[:, :topk]
    pick = lambda *n: good[torch.randint(0, good.numel(), n, generator=g, device="cuda")]  # noqa: E731
    slots[1, 0] = good[0]
    slots[2, topk - 1] = good[1]
    slots[3, :70] = pick(70)
    slots[4, 200:] = pick(100)
    slots[5, ::3] = pick(100)
    slots[6] = pick(topk)
    slots[6, 64:128] = -1
    slots[7, 128:256] = pick(128)
    ql, qp = queries(g, T, H)
    check_attend(*slots_call(cache, ql, qp, slots), want_slots(cache, ql, qp, slots))


def test_attend_slots_no_topk_and_bad_slots():
    g = gen(11)
    cache = filled(g, 3, 32)
    ql, qp = queries(g, 4, 16)
    out, lse = slots_call(cache, ql, qp, torch.empty(4, 0, dtype=torch.int64, device="cuda"))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    slots = torch.randint(0, 96, (4, 70), generator=g, device="cuda")
    slots[1, 5] = 96
    slots[2, 69] = 1 << 40
    check_attend(*slots_call(cache, ql, qp, slots, expect=5), want_slots(cache, ql, qp, slots))


@pytest.mark.parametrize("order", [1.0, -1.0])
@pytest.mark.parametrize("H", [16, 32, 128])
def test_attend_slots_scores_rise_and_fall(order, H):
    """Scores spread over hundreds, rising or falling along the list, so that the running maximum moves all the time."""
    g = gen(12)
    cache = filled(g, 8, 64)
    ql, qp = queries(g, 2, H)
    rec, _ = qr.records(cache.pool, 64, torch.arange(512, device="cuda"))
    by = (rec @ torch.cat([ql[0, 0], qp[0, 0]]).double()).argsort()
    slots = (by if order > 0 else by.flip(0))[None].repeat(2, 1).contiguous()
    for scale in (2.0, -2.0, 0.0):
        got = slots_call(cache, ql, qp, slots, scale=scale)
        check_attend(*got, want_slots(cache, ql, qp, slots, scale=scale))


@pytest.mark.parametrize("order", [1, -1, 0])
@pytest.mark.parametrize("T,H,n", [(2, 16, 512), (170, 64, 512), (1, 32, 3000)])
def test_attend_scales_far_apart(T, H, n, order):
    """Records whose scales lie 2^40 apart, rising, falling and mixed along the list; some of zeros, some never written."""
    g = gen(13)
    cache = latent.QuantLatentCache.allocate(n // 64 + 1, 64)
    c = normal(g, n, LAT)
    size = torch.linspace(-20, 20, n, device="cuda")
    if order == 0:
        size = size[torch.randperm(n, generator=g, device="cuda")]
    c *= torch.exp2((size * (order or 1))[:, None]).to(BF)
    c[5::50] = 0.0
    p = normal(g, n, PE)
    at = torch.arange(n, device="cuda")
    keep = at % 37 != 3
    qr.put(cache.pool, 64, at[keep], *qr.encode(c[keep], p[keep]))
    ql, qp = queries(g, T, H)
    ql *= 2.0 ** -22                                     # scores of the largest records stay in the hundreds
    slots = at[None].repeat(T, 1).contiguous()
    check_attend(*slots_call(cache, ql, qp, slots), want_slots(cache, ql, qp, slots))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("gap", [4.0, 12.0, 30.0])
def test_attend_one_key_above_many(H, gap):
    """One key `gap` above 20000 others that are nearly alike: their small weights add up to as much as its own or more."""
    g = gen(14)
    n = 20000
    cache = latent.QuantLatentCache.allocate(n // 64 + 1, 64)
    c, p = normal(g, n, LAT), torch.zeros(n, PE, dtype=BF, device="cuda")
    c[:, 0] += 1.0                                       # what the many share
    p[123, 0] = gap
    at = torch.arange(n, device="cuda")
    qr.put(cache.pool, 64, at, *qr.encode(c, p))
    ql, qp = queries(g, 1, H)
    ql *= 2.0 ** -6
    qp[:] = 0.0
    qp[:, :, 0] = 1.0
    table = torch.arange(cache.num_blocks, dtype=torch.int32, device="cuda")[None].contiguous()
    out = torch.full((1, H, LAT), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((1, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(1, H, n))
    latent.latent_attend_paged(cache, ql, qp, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, 1.0, out, ws, lse=lse)
    check_attend(out, lse, want_paged(cache, ql, qp, [at], scale=1.0))


@pytest.mark.parametrize("size", [1e-30, 1e-4, 30.0, 1e30])
def test_attend_queries_of_any_size(size):
    """Heads whose queries are far apart, a latent part of zeros, a few outliers; and one that is not finite."""
    g = gen(15)
    cache = filled(g, 5, 64)
    T, H = 3, 20
    ql, qp = queries(g, T, H)
    ql[:, ::2] *= size
    ql[0, 3], ql[1, 4, 100] = 0.0, 50.0
    qp[2, 5] = 0.0
    slots = torch.randint(0, 320, (T, 200), generator=g, device="cuda")
    scale = SCALE / max(size, 1.0)
    want = want_slots(cache, ql, qp, slots, scale=scale)
    got = slots_call(cache, ql, qp, slots, scale=scale)
    check_attend(*got, want)
    ql[1, 7, 3], ql[1, 9, 0] = math.nan, math.inf
    out, lse = slots_call(cache, ql, qp, slots, scale=scale)
    left = torch.tensor([h for h in range(H) if h not in (7, 9)], device="cuda")
    for t in range(T):
        heads = left if t == 1 else torch.arange(H, device="cuda")
        check_attend(out[t:t + 1, heads], lse[t:t + 1, heads], [tuple(x[heads] for x in want[t])])
    assert bool(out[1, [7, 9]].isnan().all()) and bool(lse[1, [7, 9]].isnan().all())


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("T,n", [(2, 300), (170, 520)])
@pytest.mark.parametrize("size", [1e-9, 1e12, 1e34])
def test_attend_records_of_any_size(size, T, n, H):
    """Queries as small as the records are large: scales from the least to 2^106, a first tile of small ones included."""
    g = gen(44)
    pool = torch.zeros(12, qr.block_bytes(64), dtype=torch.uint8, device="cuda")
    at = torch.arange(768, device="cuda")
    c = torch.randn(768, LAT, generator=g, device="cuda") * size
    c[:100] *= 2.0 ** -20
    qr.put(pool, 64, at, *qr.encode(c.to(BF), (torch.randn(768, PE, generator=g, device="cuda") * size).to(BF)))
    cache = latent.QuantLatentCache(pool, 64)
    ql, qp = queries(g, T, H)
    ql, qp = (ql.float() / size).to(BF), (qp.float() / size).to(BF)
    slots = torch.randint(100, 768, (T, n), generator=g, device="cuda")
    slots[::2, :140] %= 100
    got = slots_call(cache, ql, qp, slots)
    rows = sorted({0, 1, T - 1})
    check_attend(got[0][rows], got[1][rows], want_slots(cache, ql[rows], qp[rows], slots[rows]))


@pytest.mark.parametrize("T,H,topk,spread", [(50, 128, 64, 0.4), (20, 64, 512, 0.4), (9, 16, 2048, 0.0), (3, 20, 700, 1.0)])
def test_attend_errors_of_a_head_together(T, H, topk, spread):
    """A head's 512 results together: independent errors of at most 2^-9 (results), 2^-8 / sqrt(3) (weights) and 2^-9
    (small weights, whose steps are chosen for it) of sum p |c|, less than 2^-7 of it."""
    g = gen(16)
    cache = filled(g, 60, 64, spread=spread)
    ql, qp = queries(g, T, H)
    slots = torch.randint(0, 3840, (T, topk), generator=g, device="cuda")
    out, _ = slots_call(cache, ql, qp, slots)
    for t in range(T):
        rec, _ = qr.records(cache.pool, 64, slots[t])
        p = torch.softmax(torch.cat([ql[t], qp[t]], 1).double() @ rec.T * SCALE, 1)
        err = (out[t].double() - p @ rec[:, :LAT]).norm(dim=1)
        assert bool((err <= 2.0 ** -7 * (p @ rec[:, :LAT].abs()).norm(dim=1)).all())


def paged_inputs(g, lens, bs, extra=3):
    """As test_gpu_latent's: blocks at random, NaN everywhere but in the sequences' own records."""
    nblk = [(n + bs - 1) // bs for n in lens]
    perm = torch.randperm(sum(nblk) + extra, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(nblk), 1) + 1), -1, dtype=torch.int32, device="cuda")
    pool = torch.full((sum(nblk) + extra, qr.block_bytes(bs)), 0xFF, dtype=torch.uint8, device="cuda")
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
        i = torch.arange(n, device="cuda")
        slots.append(table[b].long()[i // bs] * bs + i % bs)
    every = torch.cat(slots)
    for some in every.split(65536):
        n = len(some)
        c = normal(g, n, LAT) * torch.exp(0.4 * torch.randn(n, 1, generator=g, device="cuda")).to(BF)
        qr.put(pool, bs, some, *qr.encode(c, normal(g, n, PE)))
    return latent.QuantLatentCache(pool, bs), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), slots


@pytest.mark.parametrize("lens,bs,H", [([1], 64, 16), ([0, 1, 63, 64, 65], 32, 20), ([4500, 10000, 0, 7], 64, 16),
                                       ([129, 257, 2000], 48, 128), ([30000], 64, 64), ([20000, 3], 1, 8),
                                       ([33] * 300, 32, 16), ([50, 1000] * 400, 64, 4), ([0, 1000, 64, 1], 64, 64),
                                       ([0, 0, 900], 16, 33), ([129] * 20, 64, 128), ([0], 64, 16), ([9000, 100], 64, 30)])
def test_attend_paged(lens, bs, H):
    g = gen(sum(lens) + bs)
    cache, table, sl, slots = paged_inputs(g, lens, bs)
    ql, qp = queries(g, len(lens), H, 1)
    check_attend(*paged_call(cache, ql, qp, table, sl, max(lens)), want_paged(cache, ql, qp, slots))


def test_attend_paged_device_checks():
    g = gen(21)
    lens = [100, 200, 64, 90]
    cache, table, sl, slots = paged_inputs(g, lens, 64)
    ql, qp = queries(g, 4, 16)
    bad = sl.clone()
    slots[1] = slots[1][:0]
    for n in (100000, -1):                           # longer than allowed, negative: an empty row
        bad[1] = n
        check_attend(*paged_call(cache, ql, qp, table, bad, 200, expect=5), want_paged(cache, ql, qp, slots))
    bad[1] = 0
    tb = table.clone()
    tb[0, 0] = cache.num_blocks                      # its 64 keys are skipped
    tb[3, 1] = -7
    slots[0], slots[3] = slots[0][64:], slots[3][:64]
    check_attend(*paged_call(cache, ql, qp, tb, bad, 200, expect=5), want_paged(cache, ql, qp, slots))


def test_far_into_a_large_pool():
    """Records beyond 2^32 bytes into the pool: appended, read and attended to."""
    bs = 64
    nb = (1 << 32) // qr.block_bytes(bs) + 50
    cache = latent.QuantLatentCache(torch.empty(nb, qr.block_bytes(bs), dtype=torch.uint8, device="cuda"), bs)
    g = gen(22)
    n = 20 * bs - 5
    at = torch.arange(n, device="cuda") + (nb - 20) * bs
    kv = normal(g, n, REC)
    latent.latent_append(cache, kv[:, :LAT], kv[:, LAT:], None, at, None)
    for a, b in zip(qr.take(cache.pool, bs, at), qr.encode(kv[:, :LAT], kv[:, LAT:])):
        assert torch.equal(a, b)
    out = torch.empty(n, REC, dtype=BF, device="cuda")
    latent.latent_read(cache, at, out)
    assert torch.equal(out.double(), qr.records(cache.pool, bs, at)[0])
    table = torch.arange(nb - 20, nb, dtype=torch.int32, device="cuda")[None].contiguous()
    ql, qp = queries(g, 1, 16)
    got = paged_call(cache, ql, qp, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    check_attend(*got, want_paged(cache, ql, qp, [at]))
    slots = at[torch.randperm(n, generator=g, device="cuda")[:100]][None].contiguous()
    check_attend(*slots_call(cache, ql, qp, slots), want_slots(cache, ql, qp, slots))


@pytest.mark.parametrize("T,H,topk", [(3, 128, 2048), (400, 128, 512), (5, 16, 700), (200, 24, 1024)])
def test_attend_repeats_bit_for_bit(T, H, topk):
    """Cold and warm: nothing may depend on when a copy lands."""
    g = gen(36)
    cache = filled(g, 100, 64)
    ql, qp = queries(g, T, H)
    slots = torch.randint(0, 6400, (T, topk), generator=g, device="cuda")
    first = slots_call(cache, ql, qp, slots)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(12):
        if i % 2:
            flush.zero_()
        out, lse = slots_call(cache, ql, qp, slots)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_results_without_lse():
    g = gen(37)
    cache = filled(g, 10, 64)
    ql, qp = queries(g, 6, 24)
    slots = torch.randint(0, 640, (6, 200), generator=g, device="cuda")
    want = slots_call(cache, ql, qp, slots)[0]
    out = torch.empty_like(want)
    latent.latent_attend_slots(cache, ql, qp, slots, SCALE, out, dsaidx.new_workspace(latent.workspace_bytes(6, 24, 200)))
    assert torch.equal(out, want)


def test_empty_calls_write_nothing():
    g = gen(39)
    cache = filled(g, 2, 64)
    before = cache.pool.clone()
    ws = dsaidx.new_workspace(latent.workspace_bytes(1, 16, 8))
    none, no_slots = torch.empty(0, 16, LAT, dtype=BF, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    latent.latent_attend_slots(cache, none, torch.empty(0, 16, PE, dtype=BF, device="cuda"),
                               torch.empty(0, 8, dtype=torch.int64, device="cuda"), SCALE, none, ws)
    latent.latent_append(cache, normal(g, 0, LAT), normal(g, 0, PE), None, no_slots, None)
    latent.latent_read(cache, no_slots, torch.empty(0, REC, dtype=BF, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(cache.pool, before)
