"""GPU numerics of the latent attention against plain 64-bit formulas.

Tolerances are derived, element by element:
* a rounding to a type is off by at most eps / 2 relative (bf16 2^-8);
* an angle is off by at most pi 2^-25 (its fp32 form), its sine and cosine by
  two fp32 steps, a turned value by three more products and sums: 2^-21 of
  |a| + |b| together, before the last rounding;
* a score sums 576 (192) exact products in fp32: at most terms * 2^-23 of the
  sum of magnitudes, delta, changes a weight by the factor exp(delta); weights
  may be rounded to bf16 before the value product: 2^-8 of sum p |v|; the sum
  over keys in fp32 adds less than that again by 2^-12 for 2^11 keys a
  running sum, covered by doubling delta.
"""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent

pytestmark = pytest.mark.gpu

REC, LAT, PE = latent.RECORD, latent.LATENT_DIM, latent.PE_DIM
H8 = 2.0 ** -8
SCALE = 1.0 / math.sqrt(192)
BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def turned(x, pos, rot, offset, half, base=10000.0, amp=1.0, back=False, freqs=None):
    """(result in 64 bits, |a| + |b| of every element's pair) of the definition."""
    x = x.double()
    n = rot // 2
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(n)], dtype=torch.float64) if freqs is None else freqs
    ang = pos.double()[:, None] * f.to(pos.device)
    c, s = (ang.cos() * amp)[:, None], (ang.sin() * amp)[:, None] * (-1 if back else 1)
    ia = torch.arange(n, device=x.device) * (1 if half else 2) + offset
    ib = ia + (n if half else 1)
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    mag[..., ia] = mag[..., ib] = (x[..., ia].abs() + x[..., ib].abs()) * amp
    return y, mag


def check_turned(got, want, mag):
    tol = want.abs() * (torch.finfo(got.dtype).eps / 2) + mag * 2.0 ** -21 + torch.finfo(got.dtype).smallest_normal
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,D,rot,offset", [(1, 1, 2, 2, 0), (5, 3, 192, 64, 128), (33, 7, 80, 48, 16), (9, 2, 77, 30, 3),
                                              (257, 1, 64, 64, 0), (3, 130, 128, 64, 64), (2, 2, 1024, 1024, 0),
                                              (70, 1, 18, 10, 6)])
def test_rope(dtype, half, T, H, D, rot, offset):
    g = gen(T * 1000 + D)
    x = normal(g, T, H, D, dtype=dtype)
    pos = torch.randint(-100, 1 << 20, (T,), generator=g, device="cuda")
    plan = latent.rope_plan(rot)
    out = torch.full_like(x, float("nan"))
    layout = latent.HALF if half else latent.INTERLEAVED
    latent.rope(x, pos, plan, layout=layout, offset=offset, out=out)
    want, mag = turned(x, pos, rot, offset, half)
    check_turned(out, want, mag)
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[offset:offset + rot] = False
    assert torch.equal(out[..., keep], x[..., keep])
    same = x.clone()
    latent.rope(same, pos, plan, layout=layout, offset=offset)   # in place: the same numbers
    assert torch.equal(same, out)


@pytest.mark.parametrize("half", [False, True])
def test_rope_strides(half):
    g = gen(3)
    T, H, D = 19, 6, 64
    wide = normal(g, T, H, 3 * D + 2)
    pos = torch.arange(T, device="cuda") * 77
    plan = latent.rope_plan(D)
    layout = latent.HALF if half else latent.INTERLEAVED
    for view in (wide[:, :, D:2 * D], wide[:, :, 1:D + 1], wide.transpose(0, 1)[:, :, 2:D + 2].transpose(0, 1),
                 wide[:, :1, :D].expand(T, H, D)):
        out = torch.full((H, T, D), float("nan"), dtype=BF, device="cuda").transpose(0, 1)
        latent.rope(view, pos, plan, layout=layout, out=out)
        want, mag = turned(view, pos, D, 0, half)
        check_turned(out, want, mag)


def test_rope_yarn_far_positions():
    T, D, factor = 64, 64, 40.0
    g = gen(4)
    x = normal(g, T, 2, D, dtype=torch.float32)
    pos = torch.randint((1 << 20) - 1000, 1 << 20, (T,), generator=g, device="cuda")
    plan = latent.rope_plan(D, 160000.0, "yarn", factor, 4096)
    f = torch.tensor([160000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64)
    turns = lambda b: D * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(160000.0))  # noqa: E731
    lo, hi = math.floor(turns(32.0)), math.ceil(turns(1.0))
    r = ((torch.arange(D // 2, dtype=torch.float64) - lo) / (hi - lo)).clamp(0, 1)
    amp = 0.1 * math.log(factor) + 1
    out = torch.empty_like(x)
    latent.rope(x, pos, plan, out=out)
    want, mag = turned(x, pos, D, 0, False, amp=amp, freqs=f * (1 - r) + f / factor * r)
    check_turned(out, want, mag)


@pytest.mark.parametrize("half", [False, True])
def test_rope_gradient(half):
    """transpose=True is the gradient: against the formula's by autograd in 64
    bits, and against differences of the forward call."""
    T, H, D, rot, offset = 6, 2, 40, 24, 8
    g = gen(5)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda")
    plan = latent.rope_plan(rot, amplitude=1.25)
    layout = latent.HALF if half else latent.INTERLEAVED
    dy = normal(g, T, H, D, dtype=torch.float32)
    dx = torch.empty_like(dy)
    latent.rope(dy, pos, plan, layout=layout, offset=offset, out=dx, transpose=True)
    x = normal(g, T, H, D, dtype=torch.float32)
    xd = x.double().requires_grad_()
    (turned(xd, pos, rot, offset, half, amp=1.25)[0] * dy.double()).sum().backward()
    _, mag = turned(dy, pos, rot, offset, half, amp=1.25)
    check_turned(dx, xd.grad, mag)
    # the map is linear: a difference along any direction is the map itself
    d = normal(g, T, H, D, dtype=torch.float32)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    latent.rope(x, pos, plan, layout=layout, offset=offset, out=y0)
    latent.rope(x + d, pos, plan, layout=layout, offset=offset, out=y1)
    num = ((y1.double() - y0.double()) * dy.double()).sum()
    ana = (dx.double() * d.double()).sum()
    # both sums have T H D terms of magnitude about 1.25 (|x| + |d|), each off by 2^-20
    assert abs(float(num - ana)) <= T * H * D * 8 * 1.25 * 2.0 ** -20


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,bs", [(1, 64), (7, 32), (333, 48)])
def test_append(half, n, bs):
    g = gen(n)
    kv = normal(g, n, REC + 8)
    lat, pe = kv[:, :LAT], kv[:, LAT:REC]
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda")
    nb = n // bs + 2
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:n].contiguous()
    slots[3::5] = -1
    pool = torch.full((nb, bs, REC), float("nan"), dtype=BF, device="cuda")
    cache = latent.LatentCache(pool)
    layout = latent.HALF if half else latent.INTERLEAVED
    latent.latent_append(cache, lat, pe, pos, slots, latent.rope_plan(PE), layout=layout)
    flat, ok = pool.view(-1, REC), slots >= 0
    assert torch.equal(flat[slots[ok], :LAT], lat[ok])
    want, mag = turned(pe[:, None], pos, PE, 0, half)
    check_turned(flat[slots[ok], LAT:], want[ok, 0], mag[ok, 0])
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[slots[ok]] = False
    assert bool(flat[rest].isnan().all())           # nothing else was written
    latent.latent_append(cache, lat, pe, None, slots, None)
    assert torch.equal(flat[slots[ok], LAT:], pe[ok])


def test_append_status():
    cache = latent.LatentCache.allocate(2, 64)
    kv = normal(gen(1), 3, REC)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 128, -3], device="cuda")
    latent.latent_append(cache, kv[:, :LAT], kv[:, LAT:], None, slots, None, status=status)
    assert int(status) == 5
    assert torch.equal(cache.pool[0, 5], kv[0]) and int((cache.pool != 0).any(-1).sum()) == 1


# ---------------------------------------------------------------------------
# absorbed attention
# ---------------------------------------------------------------------------
def attend64(q, k, v, scale):
    """q [H, d], k [n, d], v [n, e] in 64 bits: out, lse and their tolerances."""
    H = q.shape[0]
    if k.shape[0] == 0:
        z = q.new_zeros(H, v.shape[1])
        return z, q.new_full((H,), -math.inf), z, q.new_zeros(H)
    s = q @ k.T * scale
    delta = (q.abs() @ k.abs().T).amax(1) * abs(scale) * q.shape[1] * 2.0 ** -23
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    o = p @ v
    tol = (H8 + 2 * (delta * 2).expm1())[:, None] * (p @ v.abs()) + H8 * o.abs() + 1e-30
    return o, lse, tol, delta + lse.abs() * 2.0 ** -22 + 2.0 ** -19


def check_attend(out, lse, want):
    o, l, to, tl = (torch.stack(x) for x in zip(*want))
    err = (out.double() - o).abs()
    assert bool((err <= to).all()), "out %g over" % float((err - to).max())
    empty = l == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    el = (lse.double() - l).abs()
    assert bool((el[~empty] <= tl[~empty]).all()), "lse %g over" % float((el - tl)[~empty].max())


def queries(g, T, H, kind=0):
    if kind == 1:   # heads outermost, as a batched product per head leaves them
        return normal(g, H, T, LAT).transpose(0, 1), normal(g, T, H, 192)[:, :, 128:]
    return normal(g, T, H, LAT), normal(g, T, H, PE)


def slots_call(cache, ql, qp, slots, scale=SCALE, expect=0, ws=None, stream=None):
    T, H = ql.shape[:2]
    out = torch.full((T, H, LAT), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(T, H, slots.shape[1])) if ws is None else ws
    latent.latent_attend_slots(cache, ql, qp, slots, scale, out, ws, lse=lse, stream=stream)
    assert dsaidx.read_device_status(ws) == expect
    return out, lse


def want_slots(pool, ql, qp, slots, scale=SCALE):
    flat = pool.view(-1, REC)
    res = []
    for t in range(ql.shape[0]):
        at = slots[t][(slots[t] >= 0) & (slots[t] < flat.shape[0])]
        rec = flat[at].double()
        res.append(attend64(torch.cat([ql[t], qp[t]], 1).double(), rec, rec[:, :LAT], scale))
    return res


@pytest.mark.parametrize("T,H,topk,kind", [(1, 1, 1, 0), (1, 128, 64, 0), (3, 16, 63, 1), (2, 64, 65, 0), (5, 20, 1000, 1),
                                           (32, 128, 512, 1), (2, 130, 129, 0), (700, 17, 40, 1), (160, 64, 128, 0),
                                           (4, 33, 2048, 0), (1, 16, 4096, 0), (620, 100, 192, 0), (64, 16, 129, 0),
                                           (64, 30, 300, 1), (30, 128, 577, 0), (16, 64, 512, 0), (8, 5, 1024, 0),
                                           (3, 32, 700, 1), (70, 40, 128, 0)])
def test_attend_slots(T, H, topk, kind):
    g = gen(T * 7 + H)
    pool = normal(g, 40, 64, REC)
    ql, qp = queries(g, T, H, kind)
    slots = torch.randint(0, 40 * 64, (T, topk), generator=g, device="cuda")
    got = slots_call(latent.LatentCache(pool), ql, qp, slots)
    check_attend(*got, want_slots(pool, ql, qp, slots))


@pytest.mark.parametrize("H", [5, 64, 128])
def test_attend_slots_masks(H):
    """Rows with no key, one key, keys only at the front, at the end, between, a whole tile masked; NaN and infinities
    in every record that no row lists; slots in a wider buffer."""
    g = gen(H)
    pool = normal(g, 10, 64, REC)
    flat = pool.view(-1, REC)
    flat[::2] = float("nan")
    flat[1::8] = float("inf")
    good = torch.arange(640, device="cuda")
    good = good[(good % 2 == 1) & (good % 8 != 1)]
    T, topk = 9, 300
    wide = torch.full((T, topk + 3), -1, dtype=torch.int64, device="cuda")
    slots = wide[:, :topk]
    pick = lambda *s: good[torch.randint(0, good.numel(), s, generator=g, device="cuda")]  # noqa: E731
    slots[1, 0] = good[0]
    slots[2, topk - 1] = good[1]
    slots[3, :70] = pick(70)
    slots[4, 200:] = pick(100)
    slots[5, ::3] = pick(100)
    slots[6] = pick(topk)
    slots[6, 64:128] = -1
    slots[7, 128:256] = pick(128)
    ql, qp = queries(g, T, H)
    got = slots_call(latent.LatentCache(pool), ql, qp, slots)
    check_attend(*got, want_slots(pool, ql, qp, slots))


def test_attend_slots_no_topk_and_bad_slots():
    g = gen(11)
    pool = normal(g, 3, 32, REC)
    ql, qp = queries(g, 4, 16)
    out, lse = slots_call(latent.LatentCache(pool), ql, qp, torch.empty(4, 0, dtype=torch.int64, device="cuda"))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    slots = torch.randint(0, 96, (4, 70), generator=g, device="cuda")
    slots[1, 5] = 96
    slots[2, 69] = 1 << 40
    got = slots_call(latent.LatentCache(pool), ql, qp, slots, expect=5)
    check_attend(*got, want_slots(pool, ql, qp, slots))


@pytest.mark.parametrize("order", [1.0, -1.0])
@pytest.mark.parametrize("H", [16, 128])
def test_attend_slots_scores_rise_and_fall(order, H):
    """Scores spread over hundreds, rising or falling along the list, so that the running maximum moves all the time."""
    g = gen(12)
    pool = normal(g, 8, 64, REC)
    ql, qp = queries(g, 2, H)
    rec = pool.view(-1, REC)
    by = (rec.double() @ torch.cat([ql[0, 0], qp[0, 0]]).double()).argsort()
    slots = (by if order > 0 else by.flip(0))[None].repeat(2, 1).contiguous()
    got = slots_call(latent.LatentCache(pool), ql, qp, slots, scale=2.0)
    check_attend(*got, want_slots(pool, ql, qp, slots, scale=2.0))
    got = slots_call(latent.LatentCache(pool), ql, qp, slots, scale=-2.0)
    check_attend(*got, want_slots(pool, ql, qp, slots, scale=-2.0))


def test_attend_repeats_bit_for_bit():
    g = gen(13)
    pool = normal(g, 100, 64, REC)
    ql, qp = queries(g, 3, 128)
    slots = torch.randint(0, 6400, (3, 2048), generator=g, device="cuda")
    cache = latent.LatentCache(pool)
    ws = dsaidx.new_workspace(latent.workspace_bytes(3, 128, 2048))
    a, b = slots_call(cache, ql, qp, slots, ws=ws), slots_call(cache, ql, qp, slots, ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def paged_inputs(g, lens, bs, extra=3):
    nblk = [(n + bs - 1) // bs for n in lens]
    perm = torch.randperm(sum(nblk) + extra, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(nblk), 1) + 1), -1, dtype=torch.int32, device="cuda")
    pool = torch.full((sum(nblk) + extra, bs, REC), float("nan"), dtype=BF, device="cuda")
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
        i = torch.arange(n, device="cuda")
        s = table[b].long()[i // bs] * bs + i % bs
        pool.view(-1, REC)[s] = normal(g, n, REC)   # the rest of the last block stays NaN
        slots.append(s)
    return pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), slots


def paged_call(cache, ql, qp, table, lens, mx, expect=0, stream=None):
    B, H = ql.shape[:2]
    out = torch.full((B, H, LAT), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(B, H, mx), stream=stream)
    latent.latent_attend_paged(cache, ql, qp, table, lens, mx, SCALE, out, ws, lse=lse, stream=stream)
    assert dsaidx.read_device_status(ws, stream=stream) == expect
    return out, lse


def want_paged(pool, ql, qp, slots):
    flat = pool.view(-1, REC)
    return [attend64(torch.cat([ql[b], qp[b]], 1).double(), flat[s].double(), flat[s][:, :LAT].double(), SCALE)
            for b, s in enumerate(slots)]


@pytest.mark.parametrize("lens,bs,H", [([1], 64, 16), ([0, 1, 63, 64, 65], 32, 20), ([4500, 10000, 0, 7], 64, 16),
                                       ([129, 257, 2000], 48, 128), ([30000], 64, 64), ([20000, 3], 1, 8),
                                       ([33] * 300, 32, 16), ([50, 1000] * 400, 64, 4), ([0, 1000, 64, 1], 64, 64),
                                       ([0, 0, 900], 16, 33), ([129] * 20, 64, 128), ([0], 64, 16)])
def test_attend_paged(lens, bs, H):
    g = gen(sum(lens) + bs)
    pool, table, sl, slots = paged_inputs(g, lens, bs)
    ql, qp = queries(g, len(lens), H, 1)
    got = paged_call(latent.LatentCache(pool), ql, qp, table, sl, max(lens))
    check_attend(*got, want_paged(pool, ql, qp, slots))


def test_attend_paged_device_checks():
    g = gen(21)
    lens = [100, 200, 64, 90]
    pool, table, sl, slots = paged_inputs(g, lens, 64)
    ql, qp = queries(g, 4, 16)
    cache = latent.LatentCache(pool)
    bad = sl.clone()
    bad[1] = 100000                                  # longer than allowed: an empty row
    slots[1] = slots[1][:0]
    got = paged_call(cache, ql, qp, table, bad, 200, expect=5)
    check_attend(*got, want_paged(pool, ql, qp, slots))
    bad[1] = -1
    got = paged_call(cache, ql, qp, table, bad, 200, expect=5)
    check_attend(*got, want_paged(pool, ql, qp, slots))
    bad[1] = 0
    tb = table.clone()
    tb[0, 0] = pool.shape[0]                         # its 64 keys are skipped
    tb[3, 1] = -7
    slots[0], slots[3] = slots[0][64:], slots[3][:64]
    got = paged_call(cache, ql, qp, tb, bad, 200, expect=5)
    check_attend(*got, want_paged(pool, ql, qp, slots))


def test_attend_far_into_a_large_pool():
    """Records beyond 2^31 elements and 2^32 bytes into the pool."""
    bs = 64
    nb = (1 << 32) // (bs * REC) + 50
    pool = torch.empty(nb, bs, REC, dtype=BF, device="cuda")
    g = gen(22)
    pool[-20:] = normal(g, 20, bs, REC)
    lens = [20 * bs - 5]
    table = torch.arange(nb - 20, nb, dtype=torch.int32, device="cuda")[None].contiguous()
    ql, qp = queries(g, 1, 16)
    i = torch.arange(lens[0], device="cuda") + (nb - 20) * bs
    got = paged_call(latent.LatentCache(pool), ql, qp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), lens[0])
    check_attend(*got, want_paged(pool, ql, qp, [i]))
    slots = i[torch.randperm(lens[0], generator=g, device="cuda")[:100]][None].contiguous()
    got = slots_call(latent.LatentCache(pool), ql, qp, slots)
    check_attend(*got, want_slots(pool, ql, qp, slots))


def test_other_stream_and_graph():
    g = gen(23)
    lens = [3000, 17]
    pool, table, sl, slots = paged_inputs(g, lens, 64)
    ql, qp = queries(g, 2, 16)
    cache = latent.LatentCache(pool)
    want = want_paged(pool, ql, qp, slots)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    check_attend(*paged_call(cache, ql, qp, table, sl, 3000, stream=side), want)
    out = torch.zeros(2, 16, LAT, dtype=BF, device="cuda")
    lse = torch.zeros(2, 16, device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(2, 16, 3000))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        latent.latent_attend_paged(cache, ql, qp, table, sl, 3000, SCALE, out, ws, lse=lse)
    q2 = normal(g, 2, 16, LAT)
    ql.copy_(q2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    check_attend(out, lse, want_paged(pool, ql, qp, slots))


# ---------------------------------------------------------------------------
# expanded attention
# ---------------------------------------------------------------------------
def expanded_inputs(g, nq, nk, H, split=True):
    T, S = sum(nq), sum(nk)
    q = normal(g, T, H, 192)
    kv = normal(g, S, H, 256)
    k, v = (kv[:, :, :128], kv[:, :, 128:]) if split else (kv[:, :, :128].contiguous(), kv[:, :, 128:].contiguous())
    cu = lambda n: torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
    return q, k, normal(g, S, PE), v, cu(nq), cu(nk)


def expanded_call(q, k, pe, v, cuq, cuk, scale=SCALE, expect=0, stream=None):
    T, H = q.shape[:2]
    out = torch.full((T, H, 128), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()
    latent.latent_attend_expanded(q, k, pe, v, cuq, cuk, scale, out, lse=lse, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status) == expect
    return out, lse


def check_expanded(out, lse, q, k, pe, v, nq, nk, scale=SCALE):
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        i = torch.arange(n, device="cuda")
        see = torch.arange(m, device="cuda")[None] <= (m - n + i)[:, None]
        for h in range(q.shape[1]):
            qd = q[q0:q0 + n, h].double()
            kd = torch.cat([k[k0:k0 + m, h], pe[k0:k0 + m]], 1).double()
            vd = v[k0:k0 + m, h].double()
            s = (qd @ kd.T * scale).masked_fill(~see, -math.inf)
            l = torch.logsumexp(s, 1)
            empty = ~see.any(1)
            p = torch.exp(s - l.masked_fill(empty, 0.0)[:, None])
            o = p @ vd
            mag = (qd.abs() @ kd.abs().T).masked_fill(~see, 0.0)
            delta = (mag.amax(1) if m else torch.zeros(n, device="cuda").double()) * abs(scale) * 192 * 2.0 ** -23
            tol = (H8 + 2 * (2 * delta).expm1())[:, None] * (p @ vd.abs()) + H8 * o.abs() + 1e-30
            err = (out[q0:q0 + n, h].double() - o).abs()
            assert bool((err <= tol).all()), "out %g over" % float((err - tol).max())
            lg = lse[q0:q0 + n, h].double()
            assert torch.equal(lg == -math.inf, empty)
            el = (lg - l).abs()[~empty]
            assert bool((el <= (delta + l.abs() * 2.0 ** -22 + 2.0 ** -19)[~empty]).all()), float(el.max())
        q0, k0 = q0 + n, k0 + m


@pytest.mark.parametrize("nq,nk,H", [([1], [1], 1), ([5], [5], 3), ([128], [128], 2), ([129], [129], 1), ([127], [300], 2),
                                     ([1, 0, 64, 200], [1, 7, 64, 500], 2), ([300], [290], 2), ([4], [0], 1),
                                     ([256, 256], [256, 400], 4), ([1000], [1000], 2), ([1] * 40, list(range(1, 41)), 3),
                                     ([513], [2049], 1), ([700, 3, 385], [1400, 3, 385], 8)])
def test_expanded(nq, nk, H):
    g = gen(sum(nq) + 13 * sum(nk))
    q, k, pe, v, cuq, cuk = expanded_inputs(g, nq, nk, H)
    got = expanded_call(q, k, pe, v, cuq, cuk)
    check_expanded(*got, q, k, pe, v, nq, nk)


def test_expanded_large_scores_and_layouts():
    g = gen(31)
    nq, nk, H = [200, 77], [450, 77], 2
    q, k, pe, v, cuq, cuk = expanded_inputs(g, nq, nk, H, split=False)
    k = k.transpose(0, 1).contiguous().transpose(0, 1)      # heads outermost
    for scale in (3.0, -3.0, 0.0):
        got = expanded_call(q, k, pe, v, cuq, cuk, scale=scale)
        check_expanded(*got, q, k, pe, v, nq, nk, scale=scale)


def test_expanded_masked_places_do_not_matter():
    """NaN and infinities in keys and values behind every query's horizon, and in a neighbour sequence."""
    g = gen(32)
    nq, nk, H = [100, 60], [100, 200], 2
    q, k, pe, v, cuq, cuk = expanded_inputs(g, nq, nk, H)
    kv = [x.clone() for x in (k, pe, v)]
    for x in kv:
        x[100:] = float("nan")
    out, lse = expanded_call(q[:100], *kv, cuq[:2].contiguous(), cuk[:2].contiguous())
    check_expanded(out, lse, q[:100], k[:100], pe[:100], v[:100], [100], [100])
    for x in kv:
        x[:100] = float("inf")
        x[100:] = float("nan")
    kv[0][100:], kv[1][100:], kv[2][100:] = k[100:], pe[100:], v[100:]
    out, lse = expanded_call(q, *kv, cuq, cuk)
    check_expanded(out[100:], lse[100:], q[100:], k[100:], pe[100:], v[100:], [60], [200])


def test_expanded_future_keys_do_not_matter():
    """Keys behind the horizon that are not finite, and values there of the largest finite magnitude."""
    g = gen(33)
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [300], [300], 1)
    a = expanded_call(q, k, pe, v, cuq, cuk)
    k2, pe2, v2 = k.clone(), pe.clone(), v.clone()
    k2[150:], pe2[200:], v2[150:] = float("nan"), float("inf"), torch.finfo(BF).max
    b = expanded_call(q, k2, pe2, v2, cuq, cuk)
    assert torch.equal(a[0][:150], b[0][:150]) and torch.equal(a[1][:150], b[1][:150])


def test_expanded_status_and_stream():
    g = gen(34)
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [50, 60], [50, 60], 2)
    got = expanded_call(q, k, pe, v, cuq, cuk, stream=torch.cuda.Stream())
    check_expanded(*got, q, k, pe, v, [50, 60], [50, 60])
    bad = cuk.clone()
    bad[2] = 1000                                       # beyond the keys: the second sequence is skipped
    out, lse = expanded_call(q, k, pe, v, cuq, bad, expect=5)
    check_expanded(out[:50], lse[:50], q[:50], k[:50], pe[:50], v[:50], [50], [50])
    assert bool(out[50:].isnan().all())


def test_expanded_repeats_bit_for_bit():
    """Many CTAs at once, cold and warm: nothing may depend on when a copy lands."""
    g = gen(35)
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [1500, 300], [9000, 300], 16)
    first = expanded_call(q, k, pe, v, cuq, cuk)
    assert bool(first[0].isfinite().all()) and bool(first[1].isfinite().all())
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        if i % 2:
            flush.zero_()
        out, lse = expanded_call(q, k, pe, v, cuq, cuk)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_attend_repeats_bit_for_bit_cold():
    g = gen(36)
    pool = normal(g, 300, 64, REC)
    ql, qp = queries(g, 400, 128)
    slots = torch.randint(0, 300 * 64, (400, 512), generator=g, device="cuda")
    cache = latent.LatentCache(pool)
    first = slots_call(cache, ql, qp, slots)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        if i % 2:
            flush.zero_()
        out, lse = slots_call(cache, ql, qp, slots)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_results_without_lse_and_status():
    g = gen(37)
    pool = normal(g, 10, 64, REC)
    ql, qp = queries(g, 6, 24)
    slots = torch.randint(0, 640, (6, 200), generator=g, device="cuda")
    cache = latent.LatentCache(pool)
    want = slots_call(cache, ql, qp, slots)[0]
    out = torch.empty_like(want)
    latent.latent_attend_slots(cache, ql, qp, slots, SCALE, out, dsaidx.new_workspace(latent.workspace_bytes(6, 24, 200)))
    assert torch.equal(out, want)
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [70, 3], [90, 3], 2)
    want = expanded_call(q, k, pe, v, cuq, cuk)[0]
    out = torch.empty_like(want)
    latent.latent_attend_expanded(q, k, pe, v, cuq, cuk, SCALE, out)
    assert torch.equal(out, want)


def test_expanded_keys_and_values_shared_by_the_heads():
    """Head stride 0: one key and value head for all."""
    g = gen(38)
    nq, nk, H = [150, 20], [200, 40], 6
    q, k, pe, v, cuq, cuk = expanded_inputs(g, nq, nk, H)
    k1, v1 = k[:, :1].expand(-1, H, -1), v[:, :1].expand(-1, H, -1)
    got = expanded_call(q, k1, pe, v1, cuq, cuk)
    check_expanded(*got, q, k1, pe, v1, nq, nk)
    wide = normal(g, 240, 3 * PE)                       # a strided shared key part
    got = expanded_call(q, k1, wide[:, PE:2 * PE], v, cuq, cuk)
    check_expanded(*got, q, k1, wide[:, PE:2 * PE], v, nq, nk)


def test_empty_calls_write_nothing():
    g = gen(39)
    cache = latent.LatentCache(normal(g, 2, 64, REC))
    ws = dsaidx.new_workspace(latent.workspace_bytes(1, 16, 8))
    none = torch.empty(0, 16, LAT, dtype=BF, device="cuda")
    latent.latent_attend_slots(cache, none, torch.empty(0, 16, PE, dtype=BF, device="cuda"),
                               torch.empty(0, 8, dtype=torch.int64, device="cuda"), SCALE, none, ws)
    before = cache.pool.clone()
    latent.latent_append(cache, normal(g, 0, LAT), normal(g, 0, PE), None, torch.empty(0, dtype=torch.int64, device="cuda"), None)
    assert torch.equal(cache.pool, before)
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [0, 0], [0, 5], 2)
    expanded_call(q, k, pe, v, cuq, cuk)
