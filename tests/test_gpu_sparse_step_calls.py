"""What the calls of a sparse layer do to their arguments."""
import pytest
import torch

from sparse_attention_top_idx_gb300 import sparse_step

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
