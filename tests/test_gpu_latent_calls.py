"""How the latent attention's calls are issued: captured into graphs, on other
streams, with padded strides, and with scores that are not finite.  Formulas and
tolerances are those of test_gpu_latent."""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent
from tests.test_gpu_latent import (BF, LAT, PE, REC, SCALE, attend64, check_attend, check_expanded, check_turned, expanded_inputs,
                                   gen, normal, paged_inputs, queries, slots_call, turned, want_paged, want_slots)

pytestmark = pytest.mark.gpu


class Call:
    """A call, what it changes (by new inputs) and the check of its result."""

    def __init__(self, seed=0):
        self.g = gen(50 + seed)
        self.fill()

    def refill(self):
        """Other values in the same buffers."""
        old = dict(self.__dict__)
        self.fill()
        for k, v in old.items():
            if isinstance(v, torch.Tensor) and k not in ("out", "lse"):
                v.copy_(self.__dict__[k])
                self.__dict__[k] = v
            elif k in ("out", "lse", "ws", "cache", "plan"):
                self.__dict__[k] = v


class Rope(Call):
    half = False

    def fill(self):
        self.x = normal(self.g, 33, 5, 80)
        self.pos = torch.randint(0, 1 << 20, (33,), generator=self.g, device="cuda")
        self.plan = latent.rope_plan(48)
        self.out = torch.full_like(self.x, float("nan"))

    def __call__(self, stream=None):
        latent.rope(self.x, self.pos, self.plan, layout=latent.HALF if self.half else latent.INTERLEAVED, offset=16,
                    out=self.out, stream=stream)

    def check(self):
        check_turned(self.out, *turned(self.x, self.pos, 48, 16, self.half))


class RopeHalf(Rope):
    half = True


class Append(Call):
    def fill(self):
        self.kv = normal(self.g, 77, REC)
        self.pos = torch.randint(0, 1 << 20, (77,), generator=self.g, device="cuda")
        self.slots = torch.randperm(192, generator=self.g, device="cuda")[:77].contiguous()
        self.plan = latent.rope_plan(PE)
        self.cache = latent.LatentCache.allocate(3, 64)

    def __call__(self, stream=None):
        latent.latent_append(self.cache, self.kv[:, :LAT], self.kv[:, LAT:], self.pos, self.slots, self.plan, stream=stream)

    def check(self):
        got = self.cache.pool.view(-1, REC)[self.slots]
        assert torch.equal(got[:, :LAT], self.kv[:, :LAT])
        want, mag = turned(self.kv[:, None, LAT:], self.pos, PE, 0, False)
        check_turned(got[:, LAT:], want[:, 0], mag[:, 0])


class Slots(Call):
    """Rows, heads and keys of each of a call's three shapes: whole rows, a row over a cluster, cut rows."""
    T, H, topk = 160, 64, 128

    def fill(self):
        self.pool = normal(self.g, 30, 64, REC)
        self.ql, self.qp = queries(self.g, self.T, self.H)
        self.slots = torch.randint(-1, 30 * 64, (self.T, self.topk), generator=self.g, device="cuda")
        self.cache = latent.LatentCache(self.pool)
        self.ws = dsaidx.new_workspace(latent.workspace_bytes(self.T, self.H, self.topk))
        self.out = torch.full((self.T, self.H, LAT), float("nan"), dtype=BF, device="cuda")
        self.lse = torch.full((self.T, self.H), float("nan"), device="cuda")

    def __call__(self, stream=None):
        latent.latent_attend_slots(self.cache, self.ql, self.qp, self.slots, SCALE, self.out, self.ws, lse=self.lse, stream=stream)

    def check(self):
        assert dsaidx.read_device_status(self.ws) == 0
        check_attend(self.out, self.lse, want_slots(self.pool, self.ql, self.qp, self.slots))


class SlotsCluster(Slots):
    T, H, topk = 3, 16, 512


class SlotsCut(Slots):
    T, H, topk = 200, 16, 1024


class Paged(Call):
    lens = [0, 900, 64, 1]

    def fill(self):
        self.pool, self.table, self.sl, self.at = paged_inputs(self.g, self.lens, 64)
        self.ql, self.qp = queries(self.g, len(self.lens), 20)
        self.cache = latent.LatentCache(self.pool)
        self.ws = dsaidx.new_workspace(latent.workspace_bytes(len(self.lens), 20, max(self.lens)))
        self.out = torch.full((len(self.lens), 20, LAT), float("nan"), dtype=BF, device="cuda")
        self.lse = torch.full((len(self.lens), 20), float("nan"), device="cuda")

    def __call__(self, stream=None):
        latent.latent_attend_paged(self.cache, self.ql, self.qp, self.table, self.sl, max(self.lens), SCALE, self.out, self.ws,
                                   lse=self.lse, stream=stream)

    def check(self):
        assert dsaidx.read_device_status(self.ws) == 0
        check_attend(self.out, self.lse, want_paged(self.pool, self.ql, self.qp, self.at))


class PagedCut(Paged):
    lens = [4000, 17, 9000]


class Expanded(Call):
    nq, nk = [130, 1, 300], [200, 1, 300]

    def fill(self):
        self.q, self.k, self.pe, self.v, self.cuq, self.cuk = expanded_inputs(self.g, self.nq, self.nk, 3)
        self.out = torch.full((sum(self.nq), 3, 128), float("nan"), dtype=BF, device="cuda")
        self.lse = torch.full((sum(self.nq), 3), float("nan"), device="cuda")

    def __call__(self, stream=None):
        latent.latent_attend_expanded(self.q, self.k, self.pe, self.v, self.cuq, self.cuk, SCALE, self.out, lse=self.lse,
                                      stream=stream)

    def check(self):
        check_expanded(self.out, self.lse, self.q, self.k, self.pe, self.v, self.nq, self.nk)


CALLS = [Rope, RopeHalf, Append, Slots, SlotsCluster, SlotsCut, Paged, PagedCut, Expanded]


@pytest.mark.parametrize("make", CALLS)
def test_captured_into_a_graph(make):
    """Replays read what the buffers hold then."""
    call = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    call.check()
    call.refill()
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    call.check()


@pytest.mark.parametrize("make", CALLS)
def test_on_another_stream(make):
    """Behind work of that stream, while another one has the library's kernels too."""
    call, other = make(), make(1)
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
        call.refill()
        for _ in range(3):
            call(stream=side)
            other(stream=third)
    torch.cuda.synchronize()
    call.check()
    other.check()


def padded(t, rows, heads):
    """The same values with `heads` unused elements behind each head and `rows` behind each row."""
    T, H, D = t.shape
    flat = torch.full((T * (H * (D + heads) + rows),), float("nan"), dtype=t.dtype, device="cuda")
    v = flat.as_strided((T, H, D), (H * (D + heads) + rows, D + heads, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("rows,heads", [(8, 0), (24, 16), (0, 8), (520, 136)])
@pytest.mark.parametrize("T,H", [(5, 20), (200, 70)])
def test_row_strides_that_are_no_multiple_of_the_head_stride(T, H, rows, heads):
    g = gen(60 + rows)
    pool = normal(g, 12, 64, REC)
    ql, qp = queries(g, T, H)
    wide = torch.full((T, 150), -1, dtype=torch.int64, device="cuda")
    slots = wide[:, :133]
    slots.copy_(torch.randint(0, 12 * 64, (T, 133), generator=g, device="cuda"))
    want = slots_call(latent.LatentCache(pool), ql, qp, slots.contiguous())
    got = slots_call(latent.LatentCache(pool), padded(ql, rows, heads), padded(qp, rows + 8, heads), slots)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attend(*got, want_slots(pool, ql, qp, slots))
    # expanded: queries, keys and values padded alike, the shared key part by rows
    nq, nk = [T, 3], [T + 40, 3]
    q, k, pe, v, cuq, cuk = expanded_inputs(g, nq, nk, 3)
    pe_wide = torch.full((pe.shape[0], PE + 8 + rows), float("nan"), dtype=BF, device="cuda")[:, 8:8 + PE]
    pe_wide.copy_(pe)
    out, lse = torch.empty(T + 3, 3, 128, dtype=BF, device="cuda"), torch.empty(T + 3, 3, device="cuda")
    latent.latent_attend_expanded(padded(q, rows, heads), padded(k, rows + 16, heads), pe_wide, padded(v, rows, heads + 8), cuq,
                                  cuk, SCALE, out, lse=lse)
    check_expanded(out, lse, q, k, pe, v, nq, nk)


@pytest.mark.parametrize("make", [Slots, SlotsCluster, SlotsCut])
def test_infinite_scores_of_selected_keys(make):
    """A score of -inf is a weight of 0, a row of them alone an empty one; +inf leaves no finite softmax: NaN.  Heads beside
    it are not touched."""
    c = make()
    flat = c.pool.view(-1, REC)
    flat[:, LAT] = 0.0                         # the first position element decides
    flat[::2, LAT] = 1.0
    c.qp[:, :, 0] = 0.0
    c.slots.copy_(torch.randint(0, flat.shape[0], c.slots.shape, generator=c.g, device="cuda"))
    c.slots[1] = c.slots[1] // 2 * 2           # every key has it
    c.slots[2] = c.slots[2] // 2 * 2 + 1       # none has
    c()
    torch.cuda.synchronize()
    c.check()
    plain = c.out.clone(), c.lse.clone()
    want = want_slots(c.pool, c.ql, c.qp, c.slots)[1]
    c.qp[1, 3, 0] = -math.inf                  # row 1, head 3: every key at -inf
    c.qp[1, 4, 0] = math.inf                   # row 1, head 4: every key at +inf
    c()
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(c.ws) == 0
    assert bool((c.out[1, 3] == 0).all()) and float(c.lse[1, 3]) == -math.inf
    assert bool(c.out[1, 4].isnan().all()) and not math.isfinite(float(c.lse[1, 4]))
    rows = torch.arange(c.T, device="cuda") != 1
    assert torch.equal(c.out[rows], plain[0][rows]) and torch.equal(c.lse[rows], plain[1][rows])
    # the row's other heads: their running maximum may have moved at other tiles
    heads = torch.tensor([h for h in range(c.H) if h not in (3, 4)], device="cuda")
    check_attend(c.out[1:2, heads], c.lse[1:2, heads], [tuple(x[heads] for x in want)])


@pytest.mark.parametrize("make", [Slots, SlotsCluster, SlotsCut])
def test_some_keys_at_minus_infinity(make):
    """Records with -inf in an element that every query weighs positively: their weights are 0, the others' as without them."""
    c = make()
    flat = c.pool.view(-1, REC)
    c.qp[:, :, 0] = 1.0
    flat[::3, LAT] = -math.inf
    c.slots.copy_(torch.randint(0, flat.shape[0], c.slots.shape, generator=c.g, device="cuda"))
    c.slots[0] = c.slots[0] // 3 * 3            # all of row 0
    c()
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(c.ws) == 0
    left = torch.where(c.slots % 3 == 0, -1, c.slots)
    check_attend(c.out, c.lse, want_slots(c.pool, c.ql, c.qp, left))
    assert bool((c.out[0] == 0).all())


def test_infinite_scores_expanded():
    """Keys at -inf have no weight; a query whose visible keys are all at -inf is an empty row; +inf gives NaN from there on."""
    g = gen(70)
    n, H = 300, 2
    q, k, pe, v, cuq, cuk = expanded_inputs(g, [n], [n], H)
    q[:, :, 128] = 1.0
    pe[:, 0] = 0.0
    pe[:40, 0] = -math.inf                      # the first 40 queries see nothing else
    pe[100:260:3, 0] = -math.inf
    out, lse = torch.full((n, H, 128), float("nan"), dtype=BF, device="cuda"), torch.full((n, H), float("nan"), device="cuda")
    latent.latent_attend_expanded(q, k, pe, v, cuq, cuk, SCALE, out, lse=lse)
    torch.cuda.synchronize()
    dead = torch.isinf(pe[:, 0])
    assert bool((out[:40] == 0).all()) and bool((lse[:40] == -math.inf).all())
    # the definition without the dead keys

    def check(out, lse, queries):
        for h in range(H):
            for i in queries:
                at = (~dead[:i + 1]).nonzero()[:, 0]
                kd = torch.cat([k[at, h], pe[at]], 1).double()
                o, l, to, tl = attend64(q[i, h][None].double(), kd, v[at, h].double(), SCALE)
                assert bool(((out[i, h].double() - o[0]).abs() <= to[0]).all())
                assert abs(float(lse[i, h]) - float(l)) <= float(tl)

    check(out, lse, range(40, n, 13))
    pe[150, 0] = math.inf
    again, l2 = torch.empty_like(out), torch.empty_like(lse)
    latent.latent_attend_expanded(q, k, pe, v, cuq, cuk, SCALE, again, lse=l2)
    torch.cuda.synchronize()
    assert torch.equal(again[:128], out[:128]) and torch.equal(l2[:128], lse[:128])
    check(again, l2, range(128, 150))           # these share a warp with queries that see it
    assert bool(again[150:].isnan().all()) and not bool(l2[150:].isfinite().any())


@pytest.mark.parametrize("B,H,most", [(152, 16, 131072), (151, 16, 131072), (150, 20, 10000), (76, 100, 4096), (300, 5, 1024)])
def test_ragged_batches_around_whole_waves(B, H, most):
    """Batches at and beside a whole number of rows a CTA, one sequence far longer than the others, bounds far above."""
    g = gen(B + H)
    lens = torch.randint(0, 130, (B,), generator=g, device="cuda").tolist()
    lens[B // 3] = min(most, 3000)
    lens[B // 2] = 0
    pool, table, sl, at = paged_inputs(g, lens, 64)
    ql, qp = queries(g, B, H, 1)
    out, lse = torch.full((B, H, LAT), float("nan"), dtype=BF, device="cuda"), torch.full((B, H), float("nan"), device="cuda")
    ws = dsaidx.new_workspace(latent.workspace_bytes(B, H, most))
    latent.latent_attend_paged(latent.LatentCache(pool), ql, qp, table, sl, most, SCALE, out, ws, lse=lse)
    assert dsaidx.read_device_status(ws) == 0
    check_attend(out, lse, want_paged(pool, ql, qp, at))
