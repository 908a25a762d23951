"""What the calls of a sparse layer do to their arguments, and the temperature of its softmax."""
import math

import pytest
import torch

from sparse_attention_top_idx_gb300 import latent, sparse_step
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
