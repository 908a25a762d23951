"""The indexer, the cache and the attention together: a decode step and a
prompt through the public calls, against plain formulas in 64 bits."""
import pytest
import torch

from sparse_attention_top_idx_gb300 import latent, sparse_step
from tests.test_gpu_latent import attend64, check_attend, check_expanded, turned

pytestmark = pytest.mark.gpu


def plan_freqs():
    """Steps of the layer's plan as radians a position."""
    steps, amp = latent.rope_steps(64, 160000.0, "yarn", 40.0, 4096)
    f = torch.tensor([(s & (2 ** 64 - 1)) / 2.0 ** 64 * 6.283185307179586 for s in steps.tolist()], dtype=torch.float64)
    return f, amp


def test_decode_step_selects_then_attends():
    lens, topk, heads = [300, 2000, 64, 5000], 256, 20
    layer, step, kv, positions = sparse_step.demo_layer(lens, topk, heads, seed=5)
    out, lse, idx, slots = layer.decode(**step)
    f, amp = plan_freqs()
    # what the cache holds and what the queries became are bf16 roundings of
    # the definition (checked with the rope and append tests); the attention is
    # compared on them
    kp = turned(kv[:, None, 512:], positions, 64, 0, False, amp=amp, freqs=f)[0].bfloat16()
    qp = turned(step["q_pe"], step["positions"], 64, 0, False, amp=amp, freqs=f)[0].bfloat16()
    start, want = 0, []
    for b, n in enumerate(lens):
        sel = idx[b][idx[b] >= 0].long()
        assert sel.numel() == min(topk, n)
        bs = layer.records.block_size
        assert torch.equal(slots[b][:sel.numel()], layer.block_table[b].long()[sel // bs] * bs + sel % bs)
        rec = layer.records.pool.view(-1, 576)[slots[b][:sel.numel()]]
        assert torch.equal(rec[:, :512], kv[start + sel, :512])
        ulp = (rec[:, 512:].double() - kp[start + sel, 0].double()).abs()
        assert bool((ulp <= kp[start + sel, 0].double().abs() * 2.0 ** -7 + 1e-6).all())
        q = torch.cat([step["q_latent"][b], latent.rope(step["q_pe"][b:b + 1], step["positions"][b:b + 1], layer.plan,
                                                        out=torch.empty(1, heads, 64, dtype=torch.bfloat16, device="cuda"))[0]], 1)
        assert bool(((q[:, 512:].double() - qp[b].double()).abs() <= qp[b].double().abs() * 2.0 ** -7 + 1e-6).all())
        want.append(attend64(q.double(), rec.double(), rec[:, :512].double(), sparse_step.SCALE))
        start += n
    check_attend(out, lse, want)


def test_prompt_expanded():
    lens, heads = [100, 1, 333], 3
    layer, _, kv, positions = sparse_step.demo_layer(lens, 512, 4, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    n = sum(lens)
    q = torch.randn(n, heads, 192, generator=g, device="cuda").bfloat16()
    up = (torch.randn(2, heads, 512, 128, generator=g, device="cuda") / 512 ** 0.5).bfloat16()
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    out = sparse_step.prompt(layer, q, up[0], up[1], kv[:, :512], kv[:, 512:], positions, cu)
    k, v = (torch.einsum("tc,hcd->thd", kv[:, :512], u) for u in up)
    kp = latent.rope(kv[:, None, 512:], positions, layer.plan, out=torch.empty(n, 1, 64, dtype=torch.bfloat16, device="cuda"))[:, 0]
    o, lse = torch.empty_like(out), torch.empty(n, heads, device="cuda")
    latent.latent_attend_expanded(q, k, kp, v, cu, cu, sparse_step.SCALE, o, lse=lse)   # q was turned in place
    assert torch.equal(o, out)
    check_expanded(out, lse, q, k, kp, v, lens, lens)


def test_selected_slots_and_whole_context_agree_when_everything_is_selected():
    lens = [200, 31]
    layer, step, _, _ = sparse_step.demo_layer(lens, 256, 16, seed=8)
    out, lse, _, _ = layer.decode(**step)
    tq = latent.rope(step["q_pe"], step["positions"], layer.plan, out=torch.empty(2, 16, 64, dtype=torch.bfloat16, device="cuda"))
    dense, dense_lse = layer.decode_dense(step["q_latent"], tq, step["seq_lens"], 200)
    # the same sums in another order: weights and results rounded to bf16 on both sides
    assert bool(((out.double() - dense.double()).abs() <= 2.0 ** -6 * dense.double().abs() + 2.0 ** -7).all())
    assert bool(((lse - dense_lse).abs() <= 2.0 ** -17).all())
