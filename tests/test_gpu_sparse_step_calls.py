"""What the calls of a sparse layer do to their arguments, and the temperature of its softmax."""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import latent, sparse_step
from tests import qrecords as qr
from tests.test_gpu_latent import attend64, check_attend, check_expanded, check_turned, turned

pytestmark = pytest.mark.gpu


def prompt_inputs(lens=(70, 1, 200), heads=3):
    layer, _, kv, positions = sparse_step.demo_layer(list(lens), 512, 4, seed=9)
    g = torch.Generator(device="cuda").manual_seed(10)
    q = torch.randn(sum(lens), heads, 192, generator=g, device="cuda").bfloat16()
    up = (torch.randn(2, heads, 512, 128, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    cu = torch.tensor([0] + list(lens), device="cuda").cumsum(0).to(torch.int32)
    return layer, q, (up[0], up[1], kv[:, :512], kv[:, 512:], positions, cu), kv


def test_prompt_that_leaves_its_queries():
    layer, q, rest, kv = prompt_inputs()
    before, keys = q.clone(), kv.clone()
    first = sparse_step.prompt(layer, q, *rest, in_place=False)
    again = sparse_step.prompt(layer, q, *rest, in_place=False)
    assert torch.equal(q, before) and torch.equal(kv, keys)
    assert torch.equal(first, again)
    # a strided q is copied with its values
    wide = torch.zeros(q.shape[0], q.shape[1], 256, dtype=q.dtype, device="cuda")
    wide[:, :, :192] = q
    assert torch.equal(sparse_step.prompt(layer, wide[:, :, :192], *rest, in_place=False), first)
    assert torch.equal(wide[:, :, :192], before)
    # in place: the same result, and only the last 64 elements change
    assert torch.equal(sparse_step.prompt(layer, q, *rest), first)
    assert torch.equal(q[:, :, :128], before[:, :, :128]) and not torch.equal(q[:, :, 128:], before[:, :, 128:])


def test_prompt_says_that_it_turns_its_queries():
    assert "must not be passed again" in sparse_step.prompt.__doc__


YARN = dict(base=160000.0, scaling="yarn", factor=40.0, original_max_pos=4096)


def freqs():
    """The layer's steps as radians a position."""
    return torch.tensor([(s & (2 ** 64 - 1)) / 2.0 ** 64 * 2 * math.pi for s in latent.rope_steps(64, **YARN)[0].tolist()],
                        dtype=torch.float64)


def test_a_layer_tempers_the_whole_logit():
    """softmax(t q . k / sqrt(192)) with t = (0.1 ln 40 + 1)^2, every element of q and k of the length it had."""
    t = (0.1 * math.log(40.0) + 1.0) ** 2
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    layer = sparse_step.SparseLayer.allocate(1, 64, table, 64)
    assert layer.plan.amplitude == 1.0 and abs(layer.scale - t / math.sqrt(192)) <= 2.0 ** -22
    lens, heads = [200, 31, 500], 20
    layer, step, kv, positions = sparse_step.demo_layer(lens, 128, heads, seed=11, temperature="logit")
    assert layer.plan.amplitude == 1.0
    out, lse, idx, slots = layer.decode(**step)
    q, start, want = step["q_pe"], 0, []
    tq = latent.rope(q, step["positions"], layer.plan, out=torch.empty(3, heads, 64, dtype=q.dtype, device="cuda"))
    check_turned(tq, *turned(q, step["positions"], 64, 0, False, freqs=freqs()))
    kp, mag = turned(kv[:, None, 512:], positions, 64, 0, False, freqs=freqs())
    flat = layer.records.pool.view(-1, 576)
    for b, n in enumerate(lens):
        sel = idx[b][idx[b] >= 0].long()
        rec = flat[slots[b][:sel.numel()]]
        check_turned(rec[:, 512:], kp[start + sel, 0], mag[start + sel, 0])
        want.append(attend64(torch.cat([step["q_latent"][b], tq[b]], 1).double(), rec.double(), rec[:, :512].double(),
                             t / math.sqrt(192)))
        start += n
    check_attend(out, lse, want)
    dense, dense_lse = layer.decode_dense(step["q_latent"], tq, step["seq_lens"], 500)
    # nothing is left out of the second sequence: the same sums in another order
    assert bool(((dense_lse[1] - lse[1]).abs() <= 2.0 ** -17).all())


def test_a_prompt_tempers_the_whole_logit():
    layer, q, rest, kv = prompt_inputs()
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    layer = sparse_step.SparseLayer.allocate(1, 64, table, 512)
    out = sparse_step.prompt(layer, q, *rest, in_place=False)
    k_up, v_up, c, k_pe, positions, cu = rest
    tq, kp = q.clone(), torch.empty(q.shape[0], 1, 64, dtype=q.dtype, device="cuda")
    latent.rope(tq[:, :, 128:], positions, layer.plan)
    latent.rope(k_pe[:, None], positions, layer.plan, out=kp)
    check_turned(kp, *turned(k_pe[:, None], positions, 64, 0, False, freqs=freqs()))
    k, v = (torch.einsum("tc,hcd->thd", c, u) for u in (k_up, v_up))
    scale = (0.1 * math.log(40.0) + 1.0) ** 2 / math.sqrt(192)
    o, lse = torch.empty_like(out), torch.empty(out.shape[:2], device="cuda")
    latent.latent_attend_expanded(tq, k, kp[:, 0], v, cu, cu, layer.scale, o, lse=lse)
    assert torch.equal(o, out)
    check_expanded(out, lse, tq, k, kp[:, 0], v, [70, 1, 200], [70, 1, 200], scale=scale)


def test_temperatures():
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    layer = sparse_step.SparseLayer.allocate(1, 64, table, 64, temperature="turn")
    assert layer.scale == sparse_step.SCALE and abs(layer.plan.amplitude - (0.1 * math.log(40.0) + 1.0)) <= 2.0 ** -23
    with pytest.raises(ValueError):
        sparse_step.SparseLayer.allocate(1, 64, table, 64, temperature="none")


def same_records(layer, step):
    """A layer's decode against the definition over the records its own slots name."""
    out, lse, idx, slots = layer.decode(**step)
    B, H = step["q_latent"].shape[:2]
    tq = latent.rope(step["q_pe"], step["positions"], layer.plan, out=torch.empty(B, H, 64, dtype=torch.bfloat16, device="cuda"))
    check_attend(out, lse, qr.want_slots(layer.records, step["q_latent"], tq, slots, layer.scale))
    dense, dense_lse = layer.decode_dense(step["q_latent"], tq, step["seq_lens"], step["max_seq_len"])
    bs = layer.records.block_size
    at = [layer.block_table[b].long()[i // bs] * bs + i % bs for b, n in enumerate(step["seq_lens"].tolist())
          for i in [torch.arange(n, device="cuda")]]
    check_attend(dense, dense_lse, qr.want_paged(layer.records, step["q_latent"], tq, at, layer.scale))
    return out, lse, idx, slots


@pytest.mark.parametrize("heads", [16, 128])
def test_records_in_8_bits(heads):
    lens = [300, 31, 2000, 1]
    layer, step, kv, positions = sparse_step.demo_layer(lens, 256, heads, seed=12, temperature="logit", records="fp8")
    other = sparse_step.demo_layer(lens, 256, heads, seed=12, temperature="logit")[0]
    out, lse, idx, slots = same_records(layer, step)
    two = other.decode(**step)
    assert torch.equal(idx, two[2]) and torch.equal(slots, two[3])      # the index keys are the same
    # e4m3 records: each element off by 2^-4 of itself at most, at random: of a result's norm far less
    assert float((out.double() - two[0].double()).norm() / two[0].double().norm()) < 2.0 ** -4
    with pytest.raises(ValueError):
        sparse_step.SparseLayer.allocate(1, 64, layer.block_table, 64, records="int8")


@pytest.mark.parametrize("records", ["bf16", "fp8"])
def test_a_chunk_behind_cached_keys(records):
    """The second part of a prompt attends to the first through its records."""
    lens, news, heads = [200, 90], [70, 90], 3
    layer, _, kv, positions = sparse_step.demo_layer(lens, 512, 4, seed=13, temperature="logit", records=records)
    g = torch.Generator(device="cuda").manual_seed(14)
    q = torch.randn(sum(news), heads, 192, generator=g, device="cuda").bfloat16()
    up = (torch.randn(2, heads, 512, 128, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    cuk = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    cuq = torch.tensor([0] + news, device="cuda").cumsum(0).to(torch.int32)
    bs = layer.records.block_size
    slots = torch.cat([layer.block_table[b].long()[i // bs] * bs + i % bs for b, n in enumerate(lens)
                       for i in [torch.arange(n, device="cuda")]])
    at = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, news)])
    tq = q.clone()
    out = sparse_step.chunk(layer, q, up[0], up[1], at, slots, cuq, cuk)
    latent.rope(tq[:, :, 128:], at, layer.plan)
    assert torch.equal(q, tq)
    if records == "fp8":
        rec = qr.records(layer.records.pool, bs, slots)[0].bfloat16()
    else:
        rec = layer.records.pool.view(-1, 576)[slots]
    c, kp = layer.cached(slots)
    assert torch.equal(torch.cat([c, kp], 1), rec)
    k, v = (torch.einsum("tc,hcd->thd", rec[:, :512], u) for u in up)
    lse = torch.empty(sum(news), heads, device="cuda")
    o = torch.empty_like(out)
    latent.latent_attend_expanded(tq, k, rec[:, 512:], v, cuq, cuk, layer.scale, o, lse=lse)
    assert torch.equal(o, out)
    check_expanded(out, lse, tq, k, rec[:, 512:].contiguous(), v, news, lens, scale=layer.scale)


def rows_of(layer, lens):
    """What each row's keys and records are, by position."""
    bs, nb = layer.records.block_size, layer.records.num_blocks
    index = layer.index.pool.view(nb, -1)
    res = []
    for b, n in enumerate(lens.tolist()):
        i = torch.arange(n, device="cuda")
        blocks = layer.block_table[b].long()[i // bs]
        slots = blocks * bs + i % bs
        keys = index[:, :bs * 128].view(nb, bs, 128)[blocks, i % bs]
        steps = index[:, bs * 128:bs * 132].view(nb, bs, 4)[blocks, i % bs]
        if isinstance(layer.records, latent.QuantLatentCache):
            codes, p, s = qr.take(layer.records.pool, bs, slots)
            rec = torch.cat([codes, p.contiguous().view(torch.uint8), s[:, None].contiguous().view(torch.uint8)], 1)
        else:
            rec = layer.records.pool.view(-1, 576)[slots].view(torch.uint8)
        res.append(torch.cat([keys, steps, rec], 1))
    return res


@pytest.mark.parametrize("records", ["bf16", "fp8"])
def test_rows_forked_grown_ended_and_compacted(records):
    """Generation from shared prompts: every row holds its own prompt and its own continuation throughout, decodes give the
    definition's results, and no page is lost."""
    lens, topk, heads = [130, 64, 500, 1], 128, 16
    layer, step, _, _ = sparse_step.demo_layer(lens, topk, heads, seed=15, temperature="logit", records=records)
    # room: the same pages in pools of three times as many, some in front of them
    nb, more = layer.records.num_blocks, 2 * layer.records.num_blocks + 24
    big = sparse_step.SparseLayer.allocate(nb + more, 64, torch.where(layer.block_table >= 0, layer.block_table + 9, -1), topk,
                                           records=records)
    for a, b in ((big.index.pool, layer.index.pool), (big.records.pool, layer.records.pool)):
        a.view(nb + more, -1)[9:9 + nb] = b.view(nb, -1)
    layer = big
    layer.track_pages(max_rows=7)
    before = rows_of(layer, step["seq_lens"])
    held = int((layer.page_set.refs > 0).sum())
    assert held == sum((n + 63) // 64 for n in lens)

    parents = torch.tensor([2, 0, 2, -1, 1, 0, 2], dtype=torch.int32, device="cuda")
    rows, now = layer.fork(step["seq_lens"], parents, max_blocks_per_seq=12)
    assert now.tolist() == [lens[p] if p >= 0 else 0 for p in parents.tolist()]
    want = [before[p] if p >= 0 else before[0][:0] for p in parents.tolist()]
    assert all(torch.equal(a, b) for a, b in zip(rows_of(rows, now), want))
    assert int((layer.page_set.refs > 0).sum()) == held + 5       # 500 and 130 end inside a page
    layer.end(step["seq_lens"])
    assert step["seq_lens"].tolist() == [0] * 4 and bool((layer.block_table == -1).all())

    g = torch.Generator(device="cuda").manual_seed(16)

    def grown(rows, now, add):
        """add[i] new tokens to row i."""
        was = now.tolist()
        rows.grow(now, now + torch.tensor(add, dtype=torch.int32, device="cuda"))
        pos = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(was, add)])
        row = torch.repeat_interleave(torch.arange(len(add), device="cuda"), torch.tensor(add, device="cuda"))
        slots = rows.block_table[row, pos // 64].long() * 64 + pos % 64
        assert bool((slots >= 0).all()) and slots.unique().numel() == slots.numel()
        kv = torch.randn(len(pos), 704, generator=g, device="cuda").bfloat16()
        rows.append(kv[:, :128].contiguous(), kv[:, 128:640], kv[:, 640:], pos, slots)

    def decoded(rows, now):
        B = len(now)
        q = torch.randn(B, heads, 576, generator=g, device="cuda").bfloat16()
        index_q = torch.randn(B, 64, 128, generator=g, device="cuda").bfloat16()
        s = dict(index_q=index_q, index_w=torch.rand(B, 64, generator=g, device="cuda"),
                 q_latent=q[:, :, :512], q_pe=q[:, :, 512:], seq_lens=now, positions=(now.long() - 1).clamp_min(0),
                 max_seq_len=int(now.max()))
        if records == "fp8":
            same_records(rows, s)
        return s, rows.decode(**s)

    prompts = want
    for add in ([1] * 7, [100, 3, 64, 10, 0, 70, 1], [1, 0, 1, 1, 1, 0, 1]):
        was = rows_of(rows, now)
        grown(rows, now, add)
        assert all(torch.equal(a[:len(b)], b) for a, b in zip(rows_of(rows, now), was))
        decoded(rows, now)
    assert all(torch.equal(a[:len(b)], b) for a, b in zip(rows_of(rows, now), prompts))

    rows.end(now, torch.tensor([0, 4, 0], dtype=torch.int32, device="cuda"))
    s, first = decoded(rows, now)
    was, refs = rows_of(rows, now), rows.page_set.refs.clone()
    page_map = rows.compact()
    live = int((refs > 0).sum())
    assert bool((rows.page_set.refs[:live] > 0).all()) and bool((rows.page_set.refs[live:] == 0).all())
    assert torch.equal(rows.page_set.refs[page_map[refs > 0].long()], refs[refs > 0])
    assert all(torch.equal(a, b) for a, b in zip(rows_of(rows, now), was))
    second = rows.decode(**s)
    assert all(torch.equal(a, b) for a, b in zip(first[:3], second[:3]))
    assert rows.page_status() == 0
    rows.end(now)
    assert bool((rows.page_set.refs == 0).all())


def test_pages_that_run_out():
    """Rows for which none are left keep what they had, a forked one is empty, and the layer says so."""
    layer, step, _, _ = sparse_step.demo_layer([130, 64], 128, 16, seed=17, temperature="logit", records="fp8", spare_blocks=1)
    layer.track_pages(max_rows=3)
    free = int((layer.page_set.refs == 0).sum())
    lens = step["seq_lens"]
    before = rows_of(layer, lens)
    rows, now = layer.fork(lens, torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda"), max_blocks_per_seq=40)
    assert rows.page_status() == 0 and now.tolist() == [64, 130, 64]      # one copy
    longer = torch.tensor([64 + 64 * free, 130, 65], dtype=torch.int32, device="cuda")
    rows.grow(now, longer)
    assert rows.page_status() != 0
    assert now.tolist() == [64, 130, 64]            # no row behind the first that finds too few gets any
    assert all(torch.equal(a[:len(b)], b) for a, b in zip(rows_of(rows, now), (before[1], before[0], before[1])))
