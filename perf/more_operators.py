"""Workloads of the 8-bit latent cache (append, read back, attention over selected
slots and over whole paged contexts) and of the pages that the caches share (fork,
copy, extend, free, compact).

Every case has a plain form in elementary torch operations and the framework's
own calls; `own` chooses.  Sizes follow the indexer's workloads (contexts of 2000
/ 4500 / 10000 / 22000 tokens, 131072 and 1048576 for long contexts, top-512 and
top-1024, 32 sequences a decode step) and generic head counts.

A record is scale * [c (512 e4m3) | p (64 bf16)], its scale a power of two in 32
bits.  A block of bs tokens holds bs records of 640 bytes and then bs scales,
rounded up to 128 bytes.
"""
import math

import torch

own = False

LATENT, PE, NOPE = 512, 64, 128
REC = LATENT + PE
ROW = LATENT + 2 * PE             # bytes of a record without its scale
ATT_SCALE = 1.0 / math.sqrt(NOPE + PE)
BASE = 160000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token of each of 32 sequences, and their last pages read back
        {"name": "append_decode_32", "op": "append", "n": 32, "bs": 64, "half": False, "max_pos": 131072,
         "factor": 40.0, "skip": False},
        # a prefill chunk, some tokens without a slot (prefix already cached); the next chunk's expanded attention reads
        # all of the prefix
        {"name": "append_prefill_8192", "op": "append", "n": 8192, "bs": 64, "half": False, "max_pos": 22000,
         "factor": 40.0, "skip": True},
        # one decode step over the indexer's top-512, all heads on one card
        {"name": "slots_decode_b32_top512_h128", "op": "slots", "T": 32, "H": 128, "topk": 512, "S": 10000, "bs": 64,
         "causal": False},
        # few rows, heads that fill no tile, rows with few or no selected keys
        {"name": "slots_decode_b7_top1000_h20", "op": "slots", "T": 7, "H": 20, "topk": 1000, "S": 1200, "bs": 32,
         "causal": True},
        # a prefill chunk over the indexer's top-1024
        {"name": "slots_prefill_t4096_top1024_h128", "op": "slots", "T": 4096, "H": 128, "topk": 1024, "S": 22000,
         "bs": 64, "causal": True},
        # one decode step over whole contexts, the heads of one card of eight
        {"name": "paged_decode_b32_s4500_10000_h16", "op": "paged", "lens": "4500,10000", "B": 32, "H": 16, "bs": 64},
        # short, odd and empty contexts, every head
        {"name": "paged_decode_b13_ragged_h128", "op": "paged", "lens": "1,2000,65,0,777,4500,31", "B": 13, "H": 128,
         "bs": 32},
        # a long-context decode step, ragged
        {"name": "paged_decode_b9_s131072_1048576_h16", "op": "paged",
         "lens": "131072,131072,131072,131072,131072,131072,131072,131072,1048576", "B": 9, "H": 16, "bs": 64},
        # 32 sequences of the decode batch, four sampled continuations of each: the last step's continuations end, new
        # ones are forked off in the pools of eight layers, and get room for the tokens they will draft
        {"name": "fork_b32_x4_s4500_10000_l8", "op": "fork", "lens": "4500,10000", "B": 32, "kids": 4, "grow": 40,
         "layers": 8, "bs": 64, "spare": 512, "none": 0.0},
        # long contexts, odd sizes, some continuations not taken up
        {"name": "fork_b9_x3_s131072_1048576_l1", "op": "fork",
         "lens": "131071,131072,130000,70001,1,131072,64,0,1048575", "B": 9, "kids": 3, "grow": 1000, "layers": 1,
         "bs": 64, "spare": 1024, "none": 0.2},
        # a small pool of blocks of 32, one layer in four of them fragmented by requests that ended
        {"name": "compact_777_pages_l4", "op": "compact", "pages": 777, "rows": 20, "most": 50, "live": 0.3, "layers": 4,
         "bs": 32},
        # a large pool half empty
        {"name": "compact_16384_pages_l1", "op": "compact", "pages": 16384, "rows": 96, "most": 300, "live": 0.5,
         "layers": 1, "bs": 64},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "slots", "slots", "slots", "paged", "paged", "paged", "fork", "fork", "compact"])
    if op == "append":
        return {"op": op, "n": _log_int(rng, 1, 8192), "bs": rng.choice([32, 64]), "half": rng.random() < 0.5,
                "max_pos": _log_int(rng, 2000, 1048576), "factor": rng.choice([1.0, 40.0]), "skip": rng.random() < 0.5}
    if op == "slots":
        topk = _log_int(rng, 64, 2048)
        H = rng.choice([1, 8, 16, 20, 32, 64, 128])
        T = min(_log_int(rng, 1, 4096), max(1, 4096 * 1024 * 128 // (topk * max(H, 64))))
        return {"op": op, "T": T, "H": H, "topk": topk, "S": _log_int(rng, max(100, topk // 2), 22000),
                "bs": rng.choice([32, 64]), "causal": rng.random() < 0.7}
    if op == "paged":
        B = _log_int(rng, 1, 64)
        top = min(131072, 1000000 // B)
        lens = [_log_int(rng, 1, top) for _ in range(min(B, 8))]
        return {"op": op, "lens": ",".join(str(x) for x in lens), "B": B, "H": rng.choice([1, 8, 16, 20, 32, 64, 128]),
                "bs": rng.choice([32, 64])}
    if op == "fork":
        B = _log_int(rng, 1, 64)
        top = min(131072, 600000 // B)
        lens = [rng.choice([0, 64, _log_int(rng, 1, top), _log_int(rng, 1, top)]) for _ in range(min(B, 8))]
        return {"op": op, "lens": ",".join(str(x) for x in lens), "B": B, "kids": rng.randint(1, 8),
                "grow": _log_int(rng, 1, 1000), "layers": rng.choice([1, 1, 2, 3]), "bs": rng.choice([32, 64]),
                "spare": _log_int(rng, 1, 1024), "none": rng.choice([0.0, 0.3])}
    n = _log_int(rng, 10, 12000)
    return {"op": op, "pages": n, "rows": rng.randint(1, 100), "most": rng.randint(1, 300), "live": rng.uniform(0.05, 0.95),
            "layers": rng.choice([1, 1, 2]) if n < 6000 else 1, "bs": rng.choice([32, 64])}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lens(case):
    some = _ints(case["lens"])
    return [some[i % len(some)] for i in range(case["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _block_bytes(bs):
    return (bs * (ROW + 4) + 127) // 128 * 128


def _views(pool, bs):
    """Codes, position values and scales of a pool [blocks, block bytes] of bytes, one row a slot's block."""
    nb = pool.shape[0]
    rows = pool[:, :bs * ROW].view(nb, bs, ROW)
    scales = pool[:, bs * ROW:bs * (ROW + 4)].view(torch.float32)
    return rows[:, :, :LATENT].view(torch.float8_e4m3fn), rows[:, :, LATENT:].view(torch.bfloat16), scales


def _encode(c, p):
    """c [n, 512], p [n, 64] in 32 bits -> codes, position values and scales: the least power of two that brings the
    latents to 448 or below, 1 for none."""
    top = c.abs().amax(1)
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875).int()).clamp(-32, 119)
    s = torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, 0))
    return (c / s[:, None]).to(torch.float8_e4m3fn), (p / s[:, None]).to(torch.bfloat16), s


def _filled(g, nb, bs):
    """A pool of records as layers make them: latents behind a norm with its own gain a channel, some tokens larger."""
    pool = torch.zeros(nb, _block_bytes(bs), dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.5 * torch.randn(LATENT, generator=g, device="cuda"))
    step = max(1, 262144 // bs)
    codes, pe, scales = _views(pool, bs)
    for b in range(0, nb, step):
        n = min(step, nb - b) * bs
        c = torch.randn(n, LATENT, generator=g, device="cuda") * gain
        c *= torch.exp(0.4 * torch.randn(n, 1, generator=g, device="cuda"))
        q, p, s = _encode(c.bfloat16().float(), torch.randn(n, PE, generator=g, device="cuda").bfloat16().float())
        codes[b:b + step].view(torch.uint8).copy_(q.view(torch.uint8).view(-1, bs, LATENT))
        pe[b:b + step].copy_(p.view(-1, bs, PE))
        scales[b:b + step].copy_(s.view(-1, bs))
    return pool


def _noise(g, nb, nbytes):
    """A pool whose contents do not matter: nb pages of whole words, small enough to be exact in any type."""
    return torch.randint(0, 1 << 20, (nb, nbytes // 4), generator=g, device="cuda", dtype=torch.int32)


def _selection(g, T, topk, S, causal, slot_of):
    """Distinct random visible positions a row, -1 behind them; causal rows end at the last T positions."""
    last = torch.arange(S - T, S, device="cuda") if causal else torch.full((T,), S - 1, device="cuda")
    score = torch.rand(T, S, generator=g, device="cuda")
    score.masked_fill_(torch.arange(S, device="cuda")[None, :] > last[:, None], -1.0)
    k = min(topk, S)
    v, i = score.topk(k, dim=1)
    s = torch.where(v < 0, -1, slot_of[i])
    return torch.cat([s, s.new_full((T, topk - k), -1)], 1).contiguous()


def _tables(g, nblk, pages):
    """A block table [rows, most] of rows of nblk pages taken from the page ids given, -1 behind them."""
    table = torch.full((len(nblk), max(max(nblk), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(nblk):
        table[b, :k] = pages[at:at + k]
        at += k
    return table


def _fork_sizes(case):
    """Pages of each trunk row, pages a continuation needs on its own, pages of the pool."""
    bs, lens = case["bs"], _lens(case)
    trunk = [(x + bs - 1) // bs for x in lens]
    more = max((x + case["grow"] + bs - 1) // bs - x // bs for x in lens)
    return trunk, more, sum(trunk) + len(lens) * case["kids"] * more + case["spare"]


def prepare(case, seed):
    g = _gen(seed)
    op, bs = case["op"], case["bs"]
    st = {"case": case, "op": op}
    if own:
        from sparse_attention_top_idx_gb300 import dsaidx, latent, pages
        st["lib"], st["pages"] = latent, pages
    if op == "append":
        n = case["n"]
        if own:
            st["plan"] = latent.rope_plan(PE, base=BASE, scaling="yarn" if case["factor"] > 1.0 else "none",
                                          factor=case["factor"], original_max_pos=4096)
        kv = _normal(g, n, REC)
        kv[:, :LATENT] *= torch.exp(0.4 * torch.randn(n, 1, generator=g, device="cuda")).bfloat16()
        st["latent"], st["pe"] = kv[:, :LATENT], kv[:, LATENT:]
        st["pos"] = torch.randint(0, case["max_pos"], (n,), generator=g, device="cuda")
        nb = (n + bs - 1) // bs + 2
        order = torch.randperm(nb * bs, generator=g, device="cuda")
        slots = order[:n].clone()
        if case["skip"]:
            slots[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
            order[torch.rand(nb * bs, generator=g, device="cuda") < 0.01] = -1
        st["slots"], st["order"] = slots, order
        st["pool"] = _filled(g, nb, bs)
        st["out"] = torch.empty(nb * bs, REC, dtype=torch.bfloat16, device="cuda")
        if own:
            st["cache"] = latent.QuantLatentCache(st["pool"], bs)
    elif op == "slots":
        T, H, S = case["T"], case["H"], case["S"]
        nb = (S + bs - 1) // bs
        at = torch.arange(S, device="cuda")
        slot_of = torch.randperm(nb, generator=g, device="cuda")[at // bs] * bs + at % bs
        st["pool"] = _filled(g, nb, bs)
        st["ql"], st["qp"] = _normal(g, H, T, LATENT).transpose(0, 1), _normal(g, T, H, PE)
        st["slots"] = _selection(g, T, case["topk"], S, case["causal"] and T <= S, slot_of)
        if T > 3 and case["causal"]:
            st["slots"][1] = -1
            st["slots"][2, 1:] = -1
        st["out"] = torch.empty(T, H, LATENT, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
        if own:
            st["cache"] = latent.QuantLatentCache(st["pool"], bs)
            st["ws"] = dsaidx.new_workspace(latent.workspace_bytes(T, H, case["topk"]))
    elif op == "paged":
        lens, H = _lens(case), case["H"]
        B = len(lens)
        nblk = [(x + bs - 1) // bs for x in lens]
        st["table"] = _tables(g, nblk, torch.randperm(sum(nblk), generator=g, device="cuda").to(torch.int32))
        st["pool"] = _filled(g, max(sum(nblk), 1), bs)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["max"] = max(lens)
        st["ql"], st["qp"] = _normal(g, H, B, LATENT).transpose(0, 1), _normal(g, B, H, PE)
        st["out"] = torch.empty(B, H, LATENT, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(B, H, dtype=torch.float32, device="cuda")
        if own:
            st["cache"] = latent.QuantLatentCache(st["pool"], bs)
            st["ws"] = dsaidx.new_workspace(latent.workspace_bytes(B, H, st["max"]))
    elif op == "fork":
        trunk, more, nb = _fork_sizes(case)
        lens = _lens(case)
        n = len(lens) * case["kids"]
        ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        st["table"] = _tables(g, trunk, ids)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["refs"] = torch.zeros(nb, dtype=torch.int32, device="cuda")
        st["refs"][ids[:sum(trunk)].long()] = 1
        # some of the spare pages belong to others
        others = ids[sum(trunk):sum(trunk) + case["spare"] // 2].long()
        st["refs"][others] = torch.randint(1, 4, (len(others),), generator=g, device="cuda", dtype=torch.int32)
        kids = torch.arange(n, device="cuda") // case["kids"]
        kids[torch.rand(n, generator=g, device="cuda") < case["none"]] = -1
        st["parents"] = kids.to(torch.int32)
        st["longer"] = torch.where(kids >= 0, st["lens"][kids.clamp_min(0)] + case["grow"], 0).to(torch.int32)
        st["table2"] = torch.full((n, max(trunk) + more), -1, dtype=torch.int32, device="cuda")
        st["lens2"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        st["pairs"] = torch.empty(n, 2, dtype=torch.int32, device="cuda")
        st["pools"] = [_noise(g, nb, b) for _ in range(case["layers"]) for b in (132 * bs, _block_bytes(bs))]
        if own:
            st["set"] = pages.PageSet(st["refs"], bs, st["pools"])
            st["ws"] = dsaidx.new_workspace(pages.workspace_bytes(nb, n))
    else:
        nb = case["pages"]
        st["refs"] = (torch.rand(nb, generator=g, device="cuda") < case["live"]).int()
        live = st["refs"].nonzero().squeeze(1)
        st["refs"][live] += torch.randint(0, 3, (len(live),), generator=g, device="cuda", dtype=torch.int32)
        at = torch.randint(0, max(len(live), 1), (case["rows"], case["most"]), generator=g, device="cuda")
        cut = torch.randint(0, case["most"] + 1, (case["rows"], 1), generator=g, device="cuda")
        st["table"] = torch.full((case["rows"], case["most"]), -1, dtype=torch.int32, device="cuda")
        if len(live):
            st["table"] = torch.where(torch.arange(case["most"], device="cuda") < cut, live[at], -1).to(torch.int32)
        st["refs2"], st["table2"] = torch.empty_like(st["refs"]), torch.empty_like(st["table"])
        st["map"] = torch.empty(nb, dtype=torch.int32, device="cuda")
        st["pairs"] = torch.empty(max(nb // 2, 1), 2, dtype=torch.int32, device="cuda")
        st["count"] = torch.empty(1, dtype=torch.int32, device="cuda")
        st["pools"] = [_noise(g, nb, b) for _ in range(case["layers"]) for b in (132 * bs, _block_bytes(bs))]
        if own:
            st["set"] = pages.PageSet(st["refs"], bs, st["pools"])
            st["ws"] = dsaidx.new_workspace(pages.workspace_bytes(nb, case["rows"]))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(positions, factor):
    """Angles of positions [T] in 64 bits, [T, 32], and the amplitude: yarn ramp over 4096 trained positions where
    factor > 1."""
    i = torch.arange(PE // 2, dtype=torch.float64, device=positions.device)
    f = torch.exp(i * (-2.0 * math.log(BASE) / PE))
    amp = 1.0
    if factor > 1.0:
        low = PE * math.log(4096 / (32.0 * 2 * math.pi)) / (2 * math.log(BASE))
        high = PE * math.log(4096 / (1.0 * 2 * math.pi)) / (2 * math.log(BASE))
        low, high = max(math.floor(low), 0), min(math.ceil(high), PE - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        amp = 0.1 * math.log(factor) + 1.0
    return positions.double()[:, None] * f[None, :], amp


def _turn(x, ang, amp, half):
    """x [..., 64] in 32 bits turned by ang [..., 32]."""
    c, s = (ang.cos() * amp).float(), (ang.sin() * amp).float()
    if half:
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _records(pool, bs, slots):
    """Records at slots [...] in 32 bits; zeros at negative ones."""
    codes, pe, scales = _views(pool, bs)
    at = slots.clamp_min(0)
    b, o = at // bs, at % bs
    s = torch.where(slots >= 0, scales[b, o], 0.0)[..., None]
    out = torch.empty(*slots.shape, REC, dtype=torch.float32, device=slots.device)
    torch.mul(codes.view(torch.uint8)[b, o].view(torch.float8_e4m3fn).float(), s, out=out[..., :LATENT])
    torch.mul(pe[b, o].float(), s, out=out[..., LATENT:])
    return out


def _soft(s):
    """exp(s - max), its sum, and lse over the last dimension; a row of -inf alone has zeros and lse -inf."""
    m = s.amax(-1, keepdim=True)
    p = (s - m.clamp_min(-3.0e38)).exp_()
    l = p.sum(-1, keepdim=True)
    return p, l, (m.clamp_min(-3.0e38) + l.log()).squeeze(-1)


def _absorbed(ql, qp, rec, valid):
    q = torch.cat([ql.float(), qp.float()], -1)
    s = (q @ rec.transpose(1, 2)) * ATT_SCALE
    s.masked_fill_(~valid[:, None, :], -math.inf)
    p, l, lse = _soft(s)
    return ((p @ rec[:, :, :LATENT]) / torch.where(l > 0, l, 1.0)).to(torch.bfloat16), lse


def _plain_fork(st):
    bs, refs, lens = st["case"]["bs"], st["refs"], st["lens"]
    t2 = st["table2"]
    # the continuations of the step before end
    held = t2[t2 >= 0].long()
    refs.index_add_(0, held, torch.full_like(held, -1).to(torch.int32))
    # new ones: full pages shared, the partly filled one new
    p = st["parents"].long()
    L = torch.where(p >= 0, lens[p.clamp_min(0)], 0)
    full, part = (L // bs).long(), L % bs > 0
    spare = (refs == 0).nonzero().squeeze(1)
    new = torch.where(part, spare[(part.long().cumsum(0) - 1).clamp_min(0)], -1)
    col = torch.arange(t2.shape[1], device="cuda")
    src = torch.nn.functional.pad(st["table"], (0, t2.shape[1] - st["table"].shape[1]), value=-1)[p.clamp_min(0)]
    keep = col[None, :] < full[:, None]
    t2.copy_(torch.where(keep, src, -1))
    shared = t2[keep].long()
    refs.index_add_(0, shared, torch.ones_like(shared).to(torch.int32))
    old = torch.where(part, src.gather(1, full[:, None]).squeeze(1).long(), -1)
    t2.scatter_(1, full[:, None], new[:, None].to(torch.int32))
    refs[new[part]] = 1
    st["pairs"].copy_(torch.stack([old, new], 1))
    for pool in st["pools"]:
        pool[new[part]] = pool[old[part]]
    # room for the tokens to come
    longer = st["longer"]
    grown = (col[None, :] >= ((L + bs - 1) // bs)[:, None]) & (col[None, :] < ((longer + bs - 1) // bs)[:, None])
    more = (refs == 0).nonzero().squeeze(1)[:int(grown.sum())]
    t2[grown] = more.to(torch.int32)
    refs[more] = 1
    st["lens2"].copy_(longer)
    return t2, st["lens2"], st["pairs"], refs, *st["pools"]


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    live = refs > 0
    ids = torch.arange(len(refs), device="cuda")
    n = live.sum()
    src, dst = (live & (ids >= n)).nonzero().squeeze(1), (~live & (ids < n)).nonzero().squeeze(1)
    new = torch.where(live, ids, -1)
    new[src] = dst
    st["map"].copy_(new)
    st["refs2"].zero_()
    st["refs2"][new[live]] = refs[live]
    st["table2"].copy_(torch.where(table >= 0, new[table.clamp_min(0).long()], -1))
    st["pairs"].fill_(-1)
    st["pairs"][:len(src)] = torch.stack([src, dst], 1).to(torch.int32)
    st["count"].fill_(len(src))
    for pool in st["pools"]:
        pool[dst] = pool[src]
    return st["table2"], st["refs2"], st["map"], st["pairs"], st["count"], *st["pools"]


def _plain(st):
    case, op, bs = st["case"], st["op"], st["case"]["bs"]
    if op == "append":
        ang, amp = _angles(st["pos"], case["factor"])
        pe = _turn(st["pe"].float(), ang, amp, case["half"]).to(torch.bfloat16).float()
        q, p, s = _encode(st["latent"].float(), pe)
        codes, pes, scales = _views(st["pool"], bs)
        keep = st["slots"] >= 0
        at = st["slots"][keep]
        codes.view(torch.uint8)[at // bs, at % bs] = q.view(torch.uint8)[keep]
        pes[at // bs, at % bs] = p[keep]
        scales[at // bs, at % bs] = s[keep]
        st["out"].copy_(_records(st["pool"], bs, st["order"]))
        return st["out"]
    if op == "slots":
        return _absorbed(st["ql"], st["qp"], _records(st["pool"], bs, st["slots"]), st["slots"] >= 0)
    if op == "paged":
        pos = torch.arange(st["max"], device="cuda")
        valid = pos[None, :] < st["lens"][:, None]
        slots = st["table"].clamp_min(0)[:, pos // bs].long() * bs + pos % bs
        return _absorbed(st["ql"], st["qp"], _records(st["pool"], bs, torch.where(valid, slots, -1)), valid)
    return _plain_fork(st) if op == "fork" else _plain_compact(st)


def run(state):
    if not own:
        return _plain(state)
    lib, pages, case, op = state["lib"], state["pages"], state["case"], state["op"]
    if op == "append":
        lib.latent_append(state["cache"], state["latent"], state["pe"], state["pos"], state["slots"], state["plan"],
                          layout=lib.HALF if case["half"] else lib.INTERLEAVED)
        lib.latent_read(state["cache"], state["order"], state["out"])
        return state["out"]
    if op == "slots":
        lib.latent_attend_slots(state["cache"], state["ql"], state["qp"], state["slots"], ATT_SCALE, state["out"],
                                state["ws"], lse=state["lse"])
        return state["out"], state["lse"]
    if op == "paged":
        lib.latent_attend_paged(state["cache"], state["ql"], state["qp"], state["table"], state["lens"], state["max"],
                                ATT_SCALE, state["out"], state["ws"], lse=state["lse"])
        return state["out"], state["lse"]
    if op == "fork":
        pages.free(state["set"], state["table2"], state["lens2"])
        pages.fork(state["set"], state["table"], state["lens"], state["parents"], state["table2"], state["lens2"],
                   state["pairs"], state["ws"])
        pages.copy(state["set"], state["pairs"])
        pages.extend(state["set"], state["table2"], state["lens2"], state["longer"], state["ws"])
        return state["table2"], state["lens2"], state["pairs"], state["refs"], *state["pools"]
    pages.compact(state["set"], state["table"], state["refs2"], state["table2"], state["map"], state["pairs"],
                  state["count"], state["ws"])
    pages.copy(state["set"], state["pairs"], count=state["count"])
    return state["table2"], state["refs2"], state["map"], state["pairs"], state["count"], *state["pools"]


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def _picked(case):
    """Valid (row, key) pairs of a slots case."""
    T, S, k = case["T"], case["S"], case["topk"]
    if not (case["causal"] and T <= S):
        n = [min(k, S)] * T
    else:
        n = [min(k, S - T + t + 1) for t in range(T)]
    if T > 3 and case["causal"]:
        n[1], n[2] = 0, min(n[2], 1)
    return sum(n)


def work(case):
    op, bs = case["op"], case["bs"]
    rec = ROW + 4
    if op == "append":
        n, m = case["n"], ((case["n"] + bs - 1) // bs + 2) * bs
        return {"bytes": n * (2 * REC + rec + 16) + m * (rec + 2 * REC + 8), "flops": n * (3 * PE + LATENT) + m * REC}
    if op == "slots":
        T, H, pairs = case["T"], case["H"], _picked(case)
        return {"bytes": T * H * (2 * REC + 2 * LATENT + 4) + 8 * T * case["topk"] + rec * min(pairs, case["S"]),
                "flops": 2 * (REC + LATENT) * H * pairs}
    if op == "paged":
        H, lens = case["H"], _lens(case)
        return {"bytes": len(lens) * H * (2 * REC + 2 * LATENT + 4) + rec * sum(lens),
                "flops": 2 * (REC + LATENT) * H * sum(lens)}
    page = case["layers"] * (132 * bs + _block_bytes(bs))
    if op == "fork":
        trunk, more, nb = _fork_sizes(case)
        lens, kids = _lens(case), case["kids"] * (1.0 - case["none"])
        cells = sum(trunk) + int(sum(trunk) * kids) + int(len(lens) * kids * more)
        copied = int(kids * sum(1 for x in lens if x % bs))
        # tables read and written, the counts read once and the pages' own changed
        return {"bytes": 2 * copied * page + 4 * (cells + 2 * nb), "flops": cells + nb}
    nb, cells = case["pages"], case["rows"] * case["most"]
    moved = int(nb * case["live"] * (1.0 - case["live"]))
    return {"bytes": 2 * moved * page + 4 * (2 * cells + 3 * nb), "flops": cells + nb}


def _turned64(x, pos, factor, half):
    """The rotation as a product of complex numbers."""
    n = PE // 2
    f = [BASE ** (-2.0 * i / PE) for i in range(n)]
    amp = 1.0
    if factor > 1.0:
        turn = lambda r: PE * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        a, b = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), PE - 1)
        r = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(n)]
        f = [(1.0 - t) * w + t * w / factor for w, t in zip(f, r)]
        amp += 0.1 * math.log(factor)
    ang = pos.double().unsqueeze(1) * torch.tensor(f, dtype=torch.float64, device=pos.device)
    z = torch.polar(torch.full_like(ang, amp), ang)
    x = x.double()
    x = x.reshape(-1, 2, n).movedim(-2, -1) if half else x.reshape(-1, n, 2)
    y = torch.complex(x[..., 0].contiguous(), x[..., 1].contiguous()) * z
    y = torch.stack([y.real, y.imag], -2 if half else -1)
    return y.reshape(-1, PE)


def _e4m3():
    """Values of the 256 codes from their bits: bias 7, three fraction bits, no infinities."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _stored64(pool, bs, slots):
    """Records at slots [n], none negative, from the pool's bytes, in 64 bits."""
    raw = pool.view(-1)
    first = (slots // bs) * pool.shape[1]
    rows = raw[(first + slots % bs * ROW)[:, None] + torch.arange(ROW, device="cuda")]
    scale = raw[(first + bs * ROW + slots % bs * 4)[:, None] + torch.arange(4, device="cuda")].contiguous().view(torch.float32)
    c = _e4m3()[rows[:, :LATENT].long()]
    p = rows[:, LATENT:].contiguous().view(torch.bfloat16).double()
    return torch.cat([c, p], 1) * scale.double()


def _append64(case, st):
    """Records as appended: each latent goes to the nearest multiple of its binade's step under the token's scale."""
    want = torch.zeros(st["pool"].shape[0] * case["bs"], REC, dtype=torch.float64, device="cuda")
    every = torch.arange(len(want), device="cuda")
    want[:] = _stored64(st["pool"], case["bs"], every)
    c = st["latent"].double()
    top = c.abs().amax(1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)), 0.0)
    e = e.clamp(-32, 119) * (top > 0)
    x = c / 2.0 ** e
    step = 2.0 ** (torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    c = torch.round(x / step) * step * 2.0 ** e
    at = (st["slots"] >= 0).nonzero().squeeze(1)
    want[st["slots"][at]] = torch.cat([c, _turned64(st["pe"], st["pos"], case["factor"], case["half"])], 1)[at]
    return torch.where((st["order"] >= 0)[:, None], want[st["order"].clamp_min(0)], 0.0)


def _fork_by_hand(case, st):
    """Page by page on the host."""
    bs = case["bs"]
    table, lens, parents, longer = (st[k].tolist() for k in ("table", "lens", "parents", "longer"))
    refs, width = st["refs"].tolist(), st["table2"].shape[1]
    pools = [p.clone() for p in st["pools"]]
    free = iter([i for i, r in enumerate(refs) if r == 0])
    rows, pairs = [], []
    for p in parents:
        n = lens[p] if p >= 0 else 0
        row = table[p][:n // bs] if p >= 0 else []
        for x in row:
            refs[x] += 1
        pairs.append((-1, -1))
        if n % bs:
            pairs[-1] = (table[p][n // bs], next(free))
            row = row + [pairs[-1][1]]
            refs[row[-1]] = 1
        rows.append(row)
    for row, n in zip(rows, longer):
        while len(row) * bs < n:
            row.append(next(free))
            refs[row[-1]] = 1
    for pool in pools:
        for a, b in pairs:
            if a >= 0:
                pool[b] = pool[a]
    t2 = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32, device="cuda")
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return t2, st["longer"].clone(), whole(pairs), whole(refs), *pools


def _compact_by_hand(case, st):
    refs, table = st["refs"].tolist(), st["table"].tolist()
    n = sum(1 for r in refs if r)
    holes = iter([i for i in range(n) if not refs[i]])
    new = [(i if i < n else next(holes)) if r else -1 for i, r in enumerate(refs)]
    moved = [(i, k) for i, k in enumerate(new) if k >= 0 and k != i]
    after = [0] * len(refs)
    for i, k in enumerate(new):
        if k >= 0:
            after[k] = refs[i]
    pools = [p.clone() for p in st["pools"]]
    for pool in pools:
        for a, b in moved:
            pool[b] = pool[a]
    rest = len(st["pairs"]) - len(moved)
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return (whole([[new[x] if x >= 0 else -1 for x in row] for row in table]), whole(after), whole(new),
            whole(moved + [(-1, -1)] * rest), whole([len(moved)]), *pools)


def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    op, bs = case["op"], case["bs"]
    if op == "append":
        return _append64(case, st)
    if op == "fork":
        return _fork_by_hand(case, st)
    if op == "compact":
        return _compact_by_hand(case, st)
    outs, lses = [], []
    for t in range(st["ql"].shape[0]):
        if op == "slots":
            at = st["slots"][t][st["slots"][t] >= 0]
        else:
            i = torch.arange(int(st["lens"][t]), device="cuda")
            at = st["table"][t].long()[i // bs] * bs + i % bs
        q = torch.cat([st["ql"][t], st["qp"][t]], 1).double()
        if len(at) == 0:
            outs.append(q.new_zeros(q.shape[0], LATENT))
            lses.append(q.new_full((q.shape[0],), -math.inf))
            continue
        # in pieces of the context, each with its own statistics
        o, l = [], []
        for some in at.split(131072):
            rec = _stored64(st["pool"], bs, some)
            s = torch.einsum("hd,nd->hn", q, rec) * ATT_SCALE
            l.append(torch.logsumexp(s, 1))
            o.append(torch.softmax(s, 1) @ rec[:, :LATENT])
        lse = torch.logsumexp(torch.stack(l), 0)
        outs.append(sum(a * torch.exp(b - lse)[:, None] for a, b in zip(o, l)))
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)
