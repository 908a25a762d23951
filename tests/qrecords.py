"""Records of the 8-bit latent cache from their definition, for the tests: an
encoder and a decoder in 64 bits over the pool's bytes, and the attention's
tolerances."""
import math

import torch

from sparse_attention_top_idx_gb300 import latent

REC, LAT, PE = latent.RECORD, latent.LATENT_DIM, latent.PE_DIM
ROW = LAT + 2 * PE
SCALE = 1.0 / math.sqrt(192)


def block_bytes(bs):
    return (bs * (ROW + 4) + 127) // 128 * 128


def e4m3_values():
    """The 256 codes: bias 7, three fraction bits, S.1111.111 is NaN, no infinities."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 127 == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def nearest_codes(x):
    """Codes nearest to x (64 bits, |x| <= 448), ties to the even one, by trying them all."""
    values = e4m3_values()[:127].to(x.device)
    at = torch.bucketize(x.abs(), values)                       # values[at - 1] < |x| <= values[at]
    lo, hi = (at - 1).clamp_min(0), at.clamp_max(126)
    a, b = x.abs() - values[lo], values[hi] - x.abs()
    code = torch.where((b < a) | ((b == a) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * torch.signbit(x)).to(torch.uint8)


def encode(c, p):
    """Codes, position values and scales of latents c [n, 512] and position parts p [n, 64] (bf16)."""
    finite = torch.where(c.isfinite(), c, 0).double()
    top = finite.abs().amax(1)
    e = [0 if t == 0 else min(max(math.frexp(t)[1] - 9 + (math.frexp(t)[0] > 0.875), -32), 120) for t in top.tolist()]
    s = torch.tensor([2.0 ** x for x in e], dtype=torch.float64, device=c.device)
    codes = nearest_codes(finite / s[:, None])
    codes = torch.where(c.isfinite(), codes, 127)
    return codes, (p.double() / s[:, None]).to(torch.bfloat16), s.float()


def put(pool, bs, slots, codes, p, s):
    """Writes records into the pool's bytes."""
    flat = pool.view(-1)
    first = slots // bs * pool.shape[1]
    at = first + slots % bs * ROW
    rows = torch.cat([codes, p.contiguous().view(torch.uint8)], 1)
    flat[(at[:, None] + torch.arange(ROW, device=at.device)).view(-1)] = rows.view(-1)
    at = first + bs * ROW + slots % bs * 4
    flat[(at[:, None] + torch.arange(4, device=at.device)).view(-1)] = s.contiguous().view(torch.uint8)


def take(pool, bs, slots):
    """(codes, position values, scales) at slots, as they are held."""
    flat = pool.view(-1)
    first = slots // bs * pool.shape[1]
    rows = flat[(first + slots % bs * ROW)[:, None] + torch.arange(ROW, device=slots.device)]
    s = flat[(first + bs * ROW + slots % bs * 4)[:, None] + torch.arange(4, device=slots.device)]
    return rows[:, :LAT], rows[:, LAT:].contiguous().view(torch.bfloat16), s.contiguous().view(torch.float32).view(-1)


def records(pool, bs, slots):
    """Records at slots in 64 bits, and their scales."""
    codes, p, s = take(pool, bs, slots)
    x = torch.cat([e4m3_values().to(codes.device)[codes.long()], p.double()], 1)
    return x * s.double()[:, None], s.double()


def filled(g, nb, bs, spread=0.4, dtype=torch.bfloat16):
    """A cache of nb blocks with a record in every slot; scales spread over exp(spread N(0, 1))."""
    pool = torch.zeros(nb, block_bytes(bs), dtype=torch.uint8, device="cuda")
    for a in range(0, nb * bs, 65536):
        n = min(65536, nb * bs - a)
        c = torch.randn(n, LAT, generator=g, device="cuda") * torch.exp(spread * torch.randn(n, 1, generator=g, device="cuda"))
        p = torch.randn(n, PE, generator=g, device="cuda").to(dtype)
        put(pool, bs, torch.arange(a, a + n, device="cuda"), *encode(c.to(dtype), p))
    return latent.QuantLatentCache(pool, bs)


def attend64(q, rec, s, scale):
    """q [H, 576], rec [n, 576] and its scales [n] in 64 bits: out, lse and their tolerances.

    * A score sums 2 * 576 products in fp32 (the query is held as two numbers), each exact: terms * 2^-23 of the sum of
      magnitudes; a query element is off by 2^-22 of its head's largest, or by 2^-74: the power of two that brings the
      largest to [128, 256) is 2^60 at most, and of the lower e4m3, held times 16, half of the least step 2^-9 is
      2^-14 2^-60.  Together delta; a weight changes by exp(delta).
    * Weights times scales are rounded to fp16 and then, up or down, to the third of three e5m2: 2^-11 + 2^-8 of sum
      p |c| at most.  The smallest e5m2 is 2^-16, and the largest product of a head over the n keys worked on together is
      held at 2^(15 - G) or more, G <= 20, n <= 4^(23 - G): smaller products w are off by up to a step
      q = 2^-(31 - G) of it.  Which way is set by the key's place, independent of its values: independent errors of zero
      mean and variance min(q / 4, w) q.  A sum of them with variance V, none above M, passes 9 sqrt(V) + 20 M with a
      probability below 1e-13 (Bernstein).  The step is 2^-11 for 64 keys and halves at most where their number
      quadruples; so for any pieces V is at most 4 times what pieces of 64 keys have.
    * The result is rounded to bf16: 2^-8.
    """
    H = q.shape[0]
    if rec.shape[0] == 0:
        z = q.new_zeros(H, LAT)
        return z, q.new_full((H,), -math.inf), z, q.new_zeros(H)
    y = q @ rec.T * scale
    big = q[:, :LAT].abs().amax(1)
    delta = ((q.abs() @ rec.abs().T) * (2 * REC * 2.0 ** -23) + (big * 2.0 ** -22).clamp_min(2.0 ** -74)[:, None] * rec[:, :LAT].abs().sum(1)).amax(1) * abs(scale)
    lse = torch.logsumexp(y, 1)
    p = torch.exp(y - lse[:, None])
    v = rec[:, :LAT]
    o = p @ v
    codes = v / torch.where(s > 0, s, 1.0)[:, None]
    var, most = torch.zeros_like(o), torch.zeros_like(o)
    for a in range(0, len(s), 64):
        w = (p * s)[:, a:a + 64]
        c, step = codes[a:a + 64], 2.0 ** -11 * w.amax(1, keepdim=True)
        var += 4 * torch.minimum(step / 4, w) * step @ c.square()
        most = torch.maximum(most, step * c.abs().amax(0))
    floor = 9 * var.sqrt() + 20 * most
    tol = (2.0 ** -8 + 2.0 ** -11 + 2 * (2 * delta).expm1())[:, None] * (p @ v.abs()) + floor + 2.0 ** -8 * o.abs() + 1e-30
    return o, lse, tol, delta + lse.abs() * 2.0 ** -22 + 2.0 ** -19


def want_slots(cache, ql, qp, slots, scale=SCALE):
    n = cache.num_blocks * cache.block_size
    res = []
    for t in range(ql.shape[0]):
        at = slots[t][(slots[t] >= 0) & (slots[t] < n)]
        res.append(attend64(torch.cat([ql[t], qp[t]], 1).double(), *records(cache.pool, cache.block_size, at), scale))
    return res


def want_paged(cache, ql, qp, slots, scale=SCALE):
    return [attend64(torch.cat([ql[b], qp[b]], 1).double(), *records(cache.pool, cache.block_size, s), scale)
            for b, s in enumerate(slots)]
