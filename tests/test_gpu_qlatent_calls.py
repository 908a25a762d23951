"""How the 8-bit latent cache's calls are issued: captured into graphs, on other
streams, two at once, with padded strides, in a larger call's workspace, and with
scores that are not finite.  Formulas and tolerances are qrecords'."""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent
from tests import qrecords as qr
from tests import test_gpu_latent_calls as bf16_calls
from tests.qrecords import LAT, PE, REC, SCALE, filled, want_paged, want_slots
from tests.test_gpu_latent import BF, check_attend, check_turned, gen, normal, queries, slots_call, turned
from tests.test_gpu_qlatent import paged_inputs

pytestmark = pytest.mark.gpu


class Call(bf16_calls.Call):
    """New inputs go into the same pool, too."""

    def refill(self):
        cache = self.cache
        super().refill()
        assert self.cache is cache and self.pool.data_ptr() == cache.pool.data_ptr()


class Append(Call):
    def fill(self):
        self.kv = normal(self.g, 77, REC)
        self.pos = torch.randint(0, 1 << 20, (77,), generator=self.g, device="cuda")
        self.slots = torch.randperm(192, generator=self.g, device="cuda")[:77].contiguous()
        self.plan = latent.rope_plan(PE)
        self.cache = latent.QuantLatentCache.allocate(3, 64)
        self.pool = self.cache.pool

    def __call__(self, stream=None):
        latent.latent_append(self.cache, self.kv[:, :LAT], self.kv[:, LAT:], self.pos, self.slots, self.plan, stream=stream)

    def check(self):
        codes, p, s = qr.take(self.pool, 64, self.slots)
        want = qr.encode(self.kv[:, :LAT], self.kv[:, LAT:])
        assert torch.equal(codes, want[0]) and torch.equal(s, want[2])
        at, mag = turned(self.kv[:, None, LAT:], self.pos, PE, 0, False)
        check_turned((p.double() * s.double()[:, None]).bfloat16(), at[:, 0], mag[:, 0])


class Read(Call):
    def fill(self):
        self.cache = filled(self.g, 5, 32)
        self.pool = self.cache.pool
        self.slots = torch.randint(0, 160, (99,), generator=self.g, device="cuda")
        self.out = torch.full((99, REC), float("nan"), dtype=BF, device="cuda")

    def __call__(self, stream=None):
        latent.latent_read(self.cache, self.slots, self.out, stream=stream)

    def check(self):
        assert torch.equal(self.out, qr.records(self.pool, 32, self.slots)[0].bfloat16())


class Slots(Call):
    T, H, topk = 160, 64, 128
    fresh = bf16_calls.Slots

    def fill(self):
        self.fresh.fill(self)
        self.cache = filled(self.g, 30, 64)
        self.pool = self.cache.pool

    def __call__(self, stream=None):
        latent.latent_attend_slots(self.cache, self.ql, self.qp, self.slots, SCALE, self.out, self.ws, lse=self.lse, stream=stream)

    def check(self):
        assert dsaidx.read_device_status(self.ws) == 0
        check_attend(self.out, self.lse, want_slots(self.cache, self.ql, self.qp, self.slots))


class SlotsCluster(Slots):
    T, H, topk = 3, 16, 512


class SlotsCut(Slots):
    T, H, topk = 160, 16, 1024


class SlotsCutWide(Slots):
    T, H, topk = 39, 64, 2048


class SlotsWide(Slots):
    T, H, topk = 20, 128, 1024


class Paged(Call):
    lens = [0, 900, 64, 1]

    def fill(self):
        self.cache, self.table, self.sl, self.at = paged_inputs(self.g, self.lens, 64)
        self.pool = self.cache.pool
        self.ql, self.qp = queries(self.g, len(self.lens), 20)
        self.ws = dsaidx.new_workspace(latent.workspace_bytes(len(self.lens), 20, max(self.lens)))
        self.out = torch.full((len(self.lens), 20, LAT), float("nan"), dtype=BF, device="cuda")
        self.lse = torch.full((len(self.lens), 20), float("nan"), device="cuda")

    def __call__(self, stream=None):
        latent.latent_attend_paged(self.cache, self.ql, self.qp, self.table, self.sl, max(self.lens), SCALE, self.out, self.ws,
                                   lse=self.lse, stream=stream)

    def check(self):
        assert dsaidx.read_device_status(self.ws) == 0
        bs = 64
        at = [self.table[b].long()[i // bs] * bs + i % bs for b, n in enumerate(self.lens)
              for i in [torch.arange(n, device="cuda")]]
        check_attend(self.out, self.lse, want_paged(self.cache, self.ql, self.qp, at))


class PagedCut(Paged):
    lens = [4000, 17, 9000]


CALLS = [Append, Read, Slots, SlotsCluster, SlotsCut, SlotsCutWide, SlotsWide, Paged, PagedCut]


@pytest.mark.parametrize("make", CALLS)
def test_captured_into_a_graph(make):
    bf16_calls.test_captured_into_a_graph(make)


@pytest.mark.parametrize("make", CALLS)
def test_on_another_stream(make):
    bf16_calls.test_on_another_stream(make)


@pytest.mark.parametrize("first,second", [(Slots, PagedCut), (SlotsCut, SlotsCluster), (SlotsWide, SlotsWide)])
def test_two_calls_at_once(first, second):
    """On two streams, each with a workspace of its own."""
    a, b = first(2), second(3)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a(stream=one)
        b(stream=two)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_two_graphs_that_share_a_workspace():
    """Replayed one behind the other, in either order."""
    a, b = SlotsCut(4), PagedCut(5)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    torch.cuda.synchronize()
    graphs = []
    for c in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for order in ((0, 1), (1, 0), (1, 1, 0, 0)):
        for c in (a, b):
            c.out.fill_(float("nan"))
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        a.check()
        b.check()


@pytest.mark.parametrize("rows,heads", [(8, 0), (24, 16), (0, 8), (520, 136)])
@pytest.mark.parametrize("T,H", [(5, 20), (200, 70)])
def test_row_strides_that_are_no_multiple_of_the_head_stride(T, H, rows, heads):
    g = gen(60 + rows)
    cache = filled(g, 12, 64)
    ql, qp = queries(g, T, H)
    slots = torch.full((T, 150), -1, dtype=torch.int64, device="cuda")[:, :133]
    slots.copy_(torch.randint(0, 12 * 64, (T, 133), generator=g, device="cuda"))
    want = slots_call(cache, ql, qp, slots.contiguous())
    got = slots_call(cache, bf16_calls.padded(ql, rows, heads), bf16_calls.padded(qp, rows + 8, heads), slots)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attend(*got, want_slots(cache, ql, qp, slots))


def first_position_element(c, values):
    """Records of the whole pool with this first position element (times its scale)."""
    at = torch.arange(c.cache.num_blocks * 64, device="cuda")
    codes, p, s = qr.take(c.pool, 64, at)
    p[:, 0] = values
    qr.put(c.pool, 64, at, codes, p, s)
    return at.numel()


@pytest.mark.parametrize("make", [Slots, SlotsCluster, SlotsCut, SlotsCutWide, SlotsWide])
def test_infinite_scores_of_selected_keys(make):
    """A score of -inf is a weight of 0, a row of them alone an empty one; +inf leaves no finite softmax: NaN.  Heads beside
    it are not touched."""
    c = make()
    n = c.cache.num_blocks * 64
    first_position_element(c, (torch.arange(n, device="cuda") % 2 == 0).to(BF))
    c.qp[:, :, 0] = 0.0
    c.slots.copy_(torch.randint(0, n, c.slots.shape, generator=c.g, device="cuda"))
    c.slots[1] = c.slots[1] // 2 * 2           # every key has it
    c.slots[2] = c.slots[2] // 2 * 2 + 1       # none has
    c()
    torch.cuda.synchronize()
    c.check()
    plain = c.out.clone(), c.lse.clone()
    want = want_slots(c.cache, c.ql, c.qp, c.slots)[1]
    c.qp[1, 3, 0] = -math.inf                  # row 1, head 3: every key at -inf
    c.qp[1, 4, 0] = math.inf                   # row 1, head 4: every key at +inf
    c()
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(c.ws) == 0
    assert bool((c.out[1, 3] == 0).all()) and float(c.lse[1, 3]) == -math.inf
    assert bool(c.out[1, 4].isnan().all()) and not math.isfinite(float(c.lse[1, 4]))
    rows = torch.arange(c.T, device="cuda") != 1
    assert torch.equal(c.out[rows], plain[0][rows]) and torch.equal(c.lse[rows], plain[1][rows])
    heads = torch.tensor([h for h in range(c.H) if h not in (3, 4)], device="cuda")
    check_attend(c.out[1:2, heads], c.lse[1:2, heads], [tuple(x[heads] for x in want)])


@pytest.mark.parametrize("make", [Slots, SlotsCluster, SlotsCut, SlotsCutWide, SlotsWide])
def test_some_keys_at_minus_infinity(make):
    """Records with -inf in an element that every query weighs positively: their weights are 0, the others' as without them."""
    c = make()
    n = c.cache.num_blocks * 64
    c.qp[:, :, 0] = 1.0
    at = torch.arange(n, device="cuda")
    p = qr.take(c.pool, 64, at)[1]
    first_position_element(c, torch.where(at % 3 == 0, torch.tensor(-math.inf, dtype=BF, device="cuda"), p[:, 0]))
    c.slots.copy_(torch.randint(0, n, c.slots.shape, generator=c.g, device="cuda"))
    c.slots[0] = c.slots[0] // 3 * 3            # all of row 0
    c()
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(c.ws) == 0
    left = torch.where(c.slots % 3 == 0, -1, c.slots)
    check_attend(c.out, c.lse, want_slots(c.cache, c.ql, c.qp, left))
    assert bool((c.out[0] == 0).all())


@pytest.mark.parametrize("make", [Slots, SlotsCluster, SlotsCut, SlotsCutWide, SlotsWide])
def test_keys_and_queries_that_are_no_numbers(make):
    """A NaN latent makes every result of the rows that select it NaN and of no other; one in a query that of its head."""
    c = make()
    at = torch.arange(c.cache.num_blocks * 64, device="cuda")
    codes, p, s = qr.take(c.pool, 64, at)
    codes[5] = 127
    qr.put(c.pool, 64, at, codes, p, s)
    c.slots.copy_(torch.randint(6, at.numel(), c.slots.shape, generator=c.g, device="cuda"))
    c()
    torch.cuda.synchronize()
    c.check()
    plain = c.out.clone(), c.lse.clone()
    c.slots[1, c.topk // 2] = 5
    c.ql[2, 7, 100] = math.nan
    c()
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(c.ws) == 0
    assert bool(c.out[1].isnan().all()) and bool(c.lse[1].isnan().all())
    assert bool(c.out[2, 7].isnan().all()) and bool(c.lse[2, 7].isnan())
    rows = torch.tensor([t for t in range(c.T) if t not in (1, 2)], device="cuda")
    assert torch.equal(c.out[rows], plain[0][rows]) and torch.equal(c.lse[rows], plain[1][rows])
    heads = torch.tensor([h for h in range(c.H) if h != 7], device="cuda")
    want = want_slots(c.cache, c.ql[2:3], c.qp[2:3], c.slots[2:3])[0]
    check_attend(c.out[2:3, heads], c.lse[2:3, heads], [tuple(x[heads] for x in want)])


@pytest.mark.parametrize("B,H,most", [(152, 16, 131072), (151, 16, 131072), (150, 20, 10000), (76, 100, 4096), (300, 5, 1024)])
def test_ragged_batches_around_whole_waves(B, H, most):
    """Batches at and beside a whole number of rows a CTA, one sequence far longer than the others, bounds far above."""
    g = gen(B + H)
    lens = torch.randint(0, 130, (B,), generator=g, device="cuda").tolist()
    lens[B // 3] = min(most, 3000)
    lens[B // 2] = 0
    cache, table, sl, at = paged_inputs(g, lens, 64)
    ql, qp = queries(g, B, H, 1)
    out, lse = torch.full((B, H, LAT), float("nan"), dtype=BF, device="cuda"), torch.full((B, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(B, H, most))
    latent.latent_attend_paged(cache, ql, qp, table, sl, most, SCALE, out, ws, lse=lse)
    assert dsaidx.read_device_status(ws) == 0
    check_attend(out, lse, want_paged(cache, ql, qp, at))


@pytest.mark.parametrize("large,small,H,most", [(152, 151, 16, 131072), (76, 75, 128, 131072), (300, 128, 16, 22000),
                                                (40, 3, 20, 10000), (200, 1, 64, 4096)])
def test_paged_calls_in_the_workspace_of_a_larger_one(large, small, H, most):
    """What stands behind a call's own rows stays as it was."""
    g = gen(large + H)
    lens = [int(x) for x in torch.randint(0, 200, (small,), generator=g, device="cuda").tolist()]
    lens[-1] = min(1500, most)
    cache, table, sl, slots = paged_inputs(g, lens, 64)
    ql, qp = queries(g, small, H)
    out = torch.full((large, H, LAT), 7.0, dtype=BF, device="cuda")
    lse = torch.full((large, H), 7.0, device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(large, H, most))
    latent.latent_attend_paged(cache, ql, qp, table, sl, most, SCALE, out[:small], ws, lse=lse[:small])
    assert dsaidx.read_device_status(ws) == 0
    check_attend(out[:small], lse[:small], want_paged(cache, ql, qp, slots))
    assert bool((out[small:] == 7.0).all()) and bool((lse[small:] == 7.0).all())


def test_the_same_row_and_key_many_times():
    """One slot in every place of a row: its record is the result; equal rows give equal results."""
    g = gen(80)
    cache = filled(g, 4, 64)
    ql, qp = queries(g, 1, 64)
    slots = torch.full((300, 700), 77, dtype=torch.int64, device="cuda")
    out, lse = slots_call(cache, ql.expand(300, -1, -1).contiguous(), qp.expand(300, -1, -1).contiguous(), slots)
    check_attend(out[:1], lse[:1], want_slots(cache, ql, qp, slots[:1]))
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
