"""Workloads of the latent-attention operators: rotary positions, the append to
the paged latent cache, attention over selected slots and over whole paged
contexts (absorbed form), and causal prompts (expanded form).

Every case has a plain form in elementary torch operations and the
framework's own calls; `own` chooses.  Sizes follow the indexer's workloads
(contexts of 2000 / 4500 / 10000 / 22000 tokens, 131072 and 1048576 for long
contexts, top-512 and top-1024, 32 sequences a decode step) and generic head
counts.
"""
import math

import torch

own = False

LATENT, PE, NOPE, VDIM = 512, 64, 128, 128
REC = LATENT + PE
ATT_SCALE = 1.0 / math.sqrt(NOPE + PE)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the rotary part of one decode step's queries, cut out of the projection's output
        {"name": "rope_decode_32x128", "op": "rope", "T": 32, "H": 128, "D": 64, "rot": 64, "pad": 128, "offset": 0,
         "half": False, "dtype": "bfloat16", "max_pos": 1048576, "factor": 40.0, "transpose": False},
        # a prefill chunk's index queries, first half of each head rotated in halves, the rest copied
        {"name": "rope_prefill_8192x64_half", "op": "rope", "T": 8192, "H": 64, "D": 128, "rot": 64, "pad": 0,
         "offset": 0, "half": True, "dtype": "bfloat16", "max_pos": 22000, "factor": 1.0, "transpose": False},
        # the gradient of such a rotation in 32 bits, odd counts
        {"name": "rope_grad_1001x9_f32", "op": "rope", "T": 1001, "H": 9, "D": 96, "rot": 48, "pad": 0, "offset": 40,
         "half": False, "dtype": "float32", "max_pos": 131072, "factor": 4.0, "transpose": True},
        # one new token of each of 32 sequences
        {"name": "append_decode_32", "op": "append", "n": 32, "bs": 64, "half": False, "max_pos": 131072,
         "factor": 40.0, "skip": False},
        # a prefill chunk, some tokens without a slot (prefix already cached)
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
        # a long-context decode step, ragged
        {"name": "paged_decode_b9_s131072_1048576_h16", "op": "paged",
         "lens": "131072,131072,131072,131072,131072,131072,131072,131072,1048576", "B": 9, "H": 16, "bs": 64},
        # prompts of many lengths packed together, some empty or of one token
        {"name": "expanded_ragged_h8", "op": "expanded", "q": "1,500,77,2000,0,129,1023", "past": "0,0,300,0,0,64,1",
         "H": 8},
        # a chunk of 8192 tokens behind 13808 cached ones, the heads of one card of eight
        {"name": "expanded_t8192_s22000_h16", "op": "expanded", "q": "8192", "past": "13808", "H": 16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "slots", "slots", "paged", "paged", "expanded", "expanded"])
    if op == "rope":
        rot = 2 * rng.randint(8, 64)
        D = rot + 2 * rng.randint(0, 32)
        H = rng.choice([1, 3, 8, 16, 64, 128])
        T = min(_log_int(rng, 1, 8192), 67108864 // (H * D))
        return {"op": op, "T": T, "H": H, "D": D, "rot": rot, "pad": rng.choice([0, 0, 64, 128]),
                "offset": rng.choice([0, D - rot]), "half": rng.random() < 0.5,
                "dtype": rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                "max_pos": _log_int(rng, 2000, 1048576), "factor": rng.choice([1.0, 4.0, 40.0]),
                "transpose": rng.random() < 0.25}
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
    n = rng.randint(1, 6)
    q = [_log_int(rng, 1, 4096 // n) for _ in range(n)]
    past = [rng.choice([0, 0, _log_int(rng, 1, 4096 // n)]) for _ in range(n)]
    return {"op": op, "q": ",".join(map(str, q)), "past": ",".join(map(str, past)), "H": rng.choice([1, 4, 8, 16, 24])}


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


def _perm_slots(g, n_tokens, bs):
    """Slots of logical positions 0..n-1 in randomly permuted blocks; the block ids; the number of blocks."""
    nb = max(1, (n_tokens + bs - 1) // bs)
    blocks = torch.randperm(nb, generator=g, device="cuda")
    pos = torch.arange(n_tokens, device="cuda")
    return blocks[pos // bs] * bs + pos % bs, blocks, nb


def _selection(g, T, topk, S, causal, slot_of):
    """Distinct random visible positions a row, -1 behind them; causal rows end at the last T positions."""
    last = torch.arange(S - T, S, device="cuda") if causal else torch.full((T,), S - 1, device="cuda")
    score = torch.rand(T, S, generator=g, device="cuda")
    score.masked_fill_(torch.arange(S, device="cuda")[None, :] > last[:, None], -1.0)
    k = min(topk, S)
    v, i = score.topk(k, dim=1)
    s = torch.where(v < 0, -1, slot_of[i])
    return torch.cat([s, s.new_full((T, topk - k), -1)], 1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if own:
        from sparse_attention_top_idx_gb300 import dsaidx, latent
        st["lib"] = latent
    if op in ("rope", "append"):
        dim = case["rot"] if op == "rope" else PE
        st["dim"], st["factor"] = dim, case["factor"]
        if own:
            st["plan"] = latent.rope_plan(dim, base=160000.0, scaling="yarn" if case["factor"] > 1.0 else "none",
                                          factor=case["factor"], original_max_pos=4096)
    if op == "rope":
        dt = getattr(torch, case["dtype"])
        x = _normal(g, case["T"], case["H"], case["pad"] + case["D"], dtype=dt)
        st["x"] = x[:, :, case["pad"]:]
        st["pos"] = torch.randint(0, case["max_pos"], (case["T"],), generator=g, device="cuda")
        st["out"] = torch.empty(case["T"], case["H"], case["D"], dtype=dt, device="cuda")
    elif op == "append":
        n, bs = case["n"], case["bs"]
        kv = _normal(g, n, REC)
        st["latent"], st["pe"] = kv[:, :LATENT], kv[:, LATENT:]
        st["pos"] = torch.randint(0, case["max_pos"], (n,), generator=g, device="cuda")
        nb = (n + bs - 1) // bs + 2
        slots = torch.randperm(nb * bs, generator=g, device="cuda")[:n]
        if case["skip"]:
            slots[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
        st["slots"] = slots.contiguous()
        st["pool"] = _normal(g, nb, bs, REC)
        if own:
            st["cache"] = latent.LatentCache(st["pool"])
    elif op == "slots":
        T, H, S = case["T"], case["H"], case["S"]
        slot_of, _, nb = _perm_slots(g, S, case["bs"])
        pool = _normal(g, nb, case["bs"], REC)
        st["pool"] = pool
        st["ql"], st["qp"] = _normal(g, H, T, LATENT).transpose(0, 1), _normal(g, T, H, PE)
        causal = case["causal"] and T <= S
        st["slots"] = _selection(g, T, case["topk"], S, causal, slot_of)
        if T > 3 and case["causal"]:
            st["slots"][1] = -1
            st["slots"][2, 1:] = -1
        st["out"] = torch.empty(T, H, LATENT, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
        if own:
            st["cache"] = latent.LatentCache(pool)
            st["ws"] = dsaidx.new_workspace(latent.workspace_bytes(T, H, case["topk"]))
    elif op == "paged":
        lens, bs, H = _lens(case), case["bs"], case["H"]
        B, mx = len(lens), max(lens)
        nblk = [(x + bs - 1) // bs for x in lens]
        perm = torch.randperm(sum(nblk), generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(nblk)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(nblk):
            table[b, :k] = perm[at:at + k]
            at += k
        st["pool"] = _normal(g, sum(nblk), bs, REC)
        st["table"] = table
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["max"] = mx
        st["ql"], st["qp"] = _normal(g, H, B, LATENT).transpose(0, 1), _normal(g, B, H, PE)
        st["out"] = torch.empty(B, H, LATENT, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(B, H, dtype=torch.float32, device="cuda")
        if own:
            st["cache"] = latent.LatentCache(st["pool"])
            st["ws"] = dsaidx.new_workspace(latent.workspace_bytes(B, H, mx))
    else:
        nq, past, H = _ints(case["q"]), _ints(case["past"]), case["H"]
        nk = [a + b for a, b in zip(nq, past)]
        T, S = sum(nq), sum(nk)
        st["q"] = _normal(g, T, H, NOPE + PE)
        kv = _normal(g, S, H, NOPE + VDIM)
        st["k"], st["v"] = kv[:, :, :NOPE], kv[:, :, NOPE:]
        st["pe"] = _normal(g, S, PE)
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["cuq"] = torch.cat([zero, torch.tensor(nq, device="cuda").cumsum(0).to(torch.int32)])
        st["cuk"] = torch.cat([zero, torch.tensor(nk, device="cuda").cumsum(0).to(torch.int32)])
        st["out"] = torch.empty(T, H, VDIM, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(positions, dim, factor):
    """Angles of positions [T] in 64 bits, [T, dim / 2], and the amplitude: base 160000, yarn ramp over 4096 trained
    positions where factor > 1."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=positions.device)
    f = torch.exp(i * (-2.0 * math.log(160000.0) / dim))
    amp = 1.0
    if factor > 1.0:
        low = dim * math.log(4096 / (32.0 * 2 * math.pi)) / (2 * math.log(160000.0))
        high = dim * math.log(4096 / (1.0 * 2 * math.pi)) / (2 * math.log(160000.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), dim - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        amp = 0.1 * math.log(factor) + 1.0
    return positions.double()[:, None] * f[None, :], amp


def _turn(x, ang, amp, half, sign=1.0):
    """x [..., dim] in 32 bits turned by ang [..., dim / 2]."""
    c, s = (ang.cos() * amp).float(), (ang.sin() * (amp * sign)).float()
    if half:
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


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


def _plain(st):
    case, op = st["case"], st["op"]
    if op == "rope":
        x, o, r = st["x"].float(), case["offset"], case["rot"]
        ang, amp = _angles(st["pos"], st["dim"], st["factor"])
        y = _turn(x[..., o:o + r], ang[:, None, :], amp, case["half"], -1.0 if case["transpose"] else 1.0)
        st["out"].copy_(torch.cat([x[..., :o], y, x[..., o + r:]], -1))
        return st["out"]
    if op == "append":
        ang, amp = _angles(st["pos"], st["dim"], st["factor"])
        pe = _turn(st["pe"].float(), ang, amp, case["half"]).to(torch.bfloat16)
        keep = st["slots"] >= 0
        st["pool"].view(-1, REC)[st["slots"][keep]] = torch.cat([st["latent"], pe], -1)[keep]
        return st["pool"]
    if op == "slots":
        valid = st["slots"] >= 0
        rec = st["pool"].view(-1, REC)[st["slots"].clamp_min(0)].float()
        return _absorbed(st["ql"], st["qp"], rec, valid)
    if op == "paged":
        pos = torch.arange(st["max"], device="cuda")
        bs = case["bs"]
        valid = pos[None, :] < st["lens"][:, None]
        slots = st["table"].clamp_min(0)[:, pos // bs].long() * bs + pos % bs
        rec = st["pool"].view(-1, REC)[slots].float()
        return _absorbed(st["ql"], st["qp"], rec, valid)
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    T, S = q.shape[0], k.shape[0]
    ti, si = torch.arange(T, device="cuda"), torch.arange(S, device="cuda")
    cuq, cuk = st["cuq"].long(), st["cuk"].long()
    tb = torch.searchsorted(cuq[1:], ti, right=True)
    sb = torch.searchsorted(cuk[1:], si, right=True)
    back = cuk[1:][tb] - (cuq[1:][tb] - ti)
    valid = (tb[:, None] == sb[None, :]) & (si[None, :] <= back[:, None])
    s = q[:, :, :NOPE].transpose(0, 1) @ k.permute(1, 2, 0) + q[:, :, NOPE:].transpose(0, 1) @ st["pe"].float().T
    s = (s * ATT_SCALE).masked_fill_(~valid[None], -math.inf)
    p, l, lse = _soft(s)
    o = (p @ v.transpose(0, 1)) / torch.where(l > 0, l, 1.0)
    return o.transpose(0, 1).to(torch.bfloat16), lse.T


def run(state):
    if not own:
        return _plain(state)
    lib, case, op = state["lib"], state["case"], state["op"]
    if op == "rope":
        lib.rope(state["x"], state["pos"], state["plan"], layout=lib.HALF if case["half"] else lib.INTERLEAVED,
                 offset=case["offset"], out=state["out"], transpose=case["transpose"])
        return state["out"]
    if op == "append":
        lib.latent_append(state["cache"], state["latent"], state["pe"], state["pos"], state["slots"], state["plan"],
                          layout=lib.HALF if case["half"] else lib.INTERLEAVED)
        return state["pool"]
    if op == "slots":
        lib.latent_attend_slots(state["cache"], state["ql"], state["qp"], state["slots"], ATT_SCALE, state["out"],
                                state["ws"], lse=state["lse"])
    elif op == "paged":
        lib.latent_attend_paged(state["cache"], state["ql"], state["qp"], state["table"], state["lens"], state["max"],
                                ATT_SCALE, state["out"], state["ws"], lse=state["lse"])
    else:
        lib.latent_attend_expanded(state["q"], state["k"], state["pe"], state["v"], state["cuq"], state["cuk"],
                                   ATT_SCALE, state["out"], lse=state["lse"])
    return state["out"], state["lse"]


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def _visible(case):
    """Causal (query, key) pairs of an expanded case."""
    return sum(n * p + n * (n + 1) // 2 for n, p in zip(_ints(case["q"]), _ints(case["past"])))


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
    op = case["op"]
    if op == "rope":
        e = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * case["T"] * case["H"] * case["D"] * e + 8 * case["T"],
                "flops": 3 * case["T"] * case["H"] * case["rot"]}
    if op == "append":
        return {"bytes": case["n"] * (2 * 2 * REC + 16), "flops": 3 * case["n"] * PE}
    if op == "slots":
        T, H, pairs = case["T"], case["H"], _picked(case)
        return {"bytes": T * H * (2 * REC + 2 * LATENT + 4) + 8 * T * case["topk"] + 2 * REC * min(pairs, case["S"]),
                "flops": 2 * (REC + LATENT) * H * pairs}
    if op == "paged":
        H, lens = case["H"], _lens(case)
        return {"bytes": len(lens) * H * (2 * REC + 2 * LATENT + 4) + 2 * REC * sum(lens),
                "flops": 2 * (REC + LATENT) * H * sum(lens)}
    H, nq = case["H"], _ints(case["q"])
    S = sum(nq) + sum(_ints(case["past"]))
    return {"bytes": sum(nq) * H * (2 * (NOPE + PE) + 2 * VDIM + 4) + S * (H * 2 * (NOPE + VDIM) + 2 * PE),
            "flops": 2 * (NOPE + PE + VDIM) * H * _visible(case)}


def _turned64(x, pos, dim, factor, half, back):
    """The rotation as a product of complex numbers."""
    n = dim // 2
    f = [160000.0 ** (-2.0 * i / dim) for i in range(n)]
    amp = 1.0
    if factor > 1.0:
        turn = lambda r: dim * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(160000.0))  # noqa: E731
        a, b = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), dim - 1)
        r = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(n)]
        f = [(1.0 - t) * w + t * w / factor for w, t in zip(f, r)]
        amp += 0.1 * math.log(factor)
    ang = pos.double().unsqueeze(1) * torch.tensor(f, dtype=torch.float64, device=pos.device)
    z = torch.polar(torch.full_like(ang, amp), -ang if back else ang)
    x = x.double()
    shape = x.shape[:-1]
    x = x.reshape(*shape, 2, n).movedim(-2, -1) if half else x.reshape(*shape, n, 2)
    y = torch.complex(x[..., 0].contiguous(), x[..., 1].contiguous()) * z.reshape(z.shape[0], *([1] * (len(shape) - 1)), n)
    y = torch.stack([y.real, y.imag], -2 if half else -1)
    return y.reshape(*shape, dim)


def _attend64(q, k, v):
    """One row's attention: q [H, d], k [n, d], v [n, e] in 64 bits -> [H, e], [H]."""
    if k.shape[0] == 0:
        return q.new_zeros(q.shape[0], v.shape[1]), q.new_full((q.shape[0],), -math.inf)
    s = torch.einsum("hd,nd->hn", q, k) * ATT_SCALE
    return torch.softmax(s, 1) @ v, torch.logsumexp(s, 1)


def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        o, r = case["offset"], case["rot"]
        y = st["x"].double().clone()
        y[..., o:o + r] = _turned64(st["x"][..., o:o + r], st["pos"], r, case["factor"], case["half"], case["transpose"])
        return y
    if op == "append":
        pool = st["pool"].double()
        pe = _turned64(st["pe"], st["pos"], PE, case["factor"], case["half"], False)
        flat = pool.view(-1, REC)
        ok = (st["slots"] >= 0).nonzero().squeeze(1)
        flat[st["slots"][ok]] = torch.cat([st["latent"].double(), pe], 1)[ok]
        return pool
    outs, lses = [], []
    if op in ("slots", "paged"):
        flat = st["pool"].view(-1, REC)
        for t in range(st["ql"].shape[0]):
            if op == "slots":
                at = st["slots"][t][st["slots"][t] >= 0]
            else:
                i = torch.arange(int(st["lens"][t]), device="cuda")
                at = st["table"][t].long()[i // case["bs"]] * case["bs"] + i % case["bs"]
            rec = flat[at].double()
            o, l = _attend64(torch.cat([st["ql"][t], st["qp"][t]], 1).double(), rec, rec[:, :LATENT])
            outs.append(o)
            lses.append(l)
        return torch.stack(outs), torch.stack(lses)
    T, H = st["q"].shape[:2]
    out = torch.zeros(T, H, VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n, p in zip(_ints(case["q"]), _ints(case["past"])):
        S = n + p
        see = torch.ones(n, S, dtype=torch.bool, device="cuda").tril(p)
        for h in range(H if n else 0):
            k = torch.cat([st["k"][k0:k0 + S, h], st["pe"][k0:k0 + S]], 1).double()
            s = (st["q"][q0:q0 + n, h].double() @ k.T * ATT_SCALE).masked_fill(~see, -math.inf)
            out[q0:q0 + n, h] = torch.softmax(s, 1) @ st["v"][k0:k0 + S, h].double()
            lse[q0:q0 + n, h] = torch.logsumexp(s, 1)
        q0, k0 = q0 + n, k0 + S
    return out, lse
