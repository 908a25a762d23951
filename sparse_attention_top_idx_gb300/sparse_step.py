"""One sparse-attention decode step and one prompt, from the indexer to the
attention, through the public calls:

    python -m sparse_attention_top_idx_gb300.sparse_step

The index keys and the latent records of a token share its slot: both pools
have the same blocks, so the slots the score call returns name the records
the attention reads.  Inputs are seeded and synthetic.
"""
from __future__ import annotations

import dataclasses
import math

import torch

from . import dsaidx, latent
from . import workloads as wl
from .host import bf16_tensor

SCALE = 1.0 / math.sqrt(latent.NOPE_DIM + latent.PE_DIM)


@dataclasses.dataclass
class SparseLayer:
    """The caches of one layer and what a serving process keeps beside them."""
    index: dsaidx.IndexCache
    records: latent.LatentCache
    plan: latent.RopePlan
    block_table: torch.Tensor
    topk: int
    scale: float = SCALE

    @staticmethod
    def allocate(num_blocks: int, block_size: int, block_table: torch.Tensor, topk: int, key_dtype: int = dsaidx.FP8,
                 temperature: str = "logit"):
        """YaRN's temperature multiplies the whole logit by amplitude^2.  Where all of a head is turned, turning it to
        the length amplitude does that; here 64 of a key's 576 elements are turned, so the turned elements keep their
        length and the softmax scale carries it.  temperature="turn" is for a model whose turned elements alone are
        lengthened (their part of the logit then counts amplitude^2 times as much against the latent's)."""
        if temperature not in ("logit", "turn"):
            raise ValueError('temperature must be "logit" or "turn"')
        yarn = dict(base=160000.0, scaling="yarn", factor=40.0, original_max_pos=4096)
        amplitude = latent.rope_steps(latent.PE_DIM, **yarn)[1]
        whole = temperature == "logit"
        return SparseLayer(dsaidx.IndexCache.allocate(num_blocks, block_size, key_dtype),
                           latent.LatentCache.allocate(num_blocks, block_size),
                           latent.rope_plan(latent.PE_DIM, amplitude=1.0 if whole else amplitude, **yarn),
                           block_table, topk, SCALE * amplitude ** 2 if whole else SCALE)

    def append(self, index_keys, c, k_pe, positions, slots):
        """Store the index keys [n, 128] and the records (c [n, 512], k_pe [n, 64] not yet turned) of n tokens."""
        dsaidx.store_keys(self.index, index_keys, slots)
        latent.latent_append(self.records, c, k_pe, positions, slots, self.plan)

    def decode(self, index_q, index_w, q_latent, q_pe, seq_lens, positions, max_seq_len: int):
        """One query a sequence: select its top-k keys, turn q_pe [batch, heads, 64], attend over the selected
        records.  Returns (out [batch, heads, 512], lse, selected positions, their slots)."""
        B, H = q_latent.shape[:2]
        k, dev = self.topk, q_latent.device
        idx = torch.empty(B, k, dtype=torch.int32, device=dev)
        slots = torch.empty(B, k, dtype=torch.int64, device=dev)
        ws = dsaidx.new_workspace(dsaidx.workspace_bytes_decode(self.index, B, max_seq_len, index_q.shape[1], k))
        dsaidx.score_topk_decode(self.index, index_q, index_w, self.block_table, seq_lens, max_seq_len, k, idx, ws,
                                 out_slot=slots)
        turned = latent.rope(q_pe, positions, self.plan, out=torch.empty_like(q_pe, memory_format=torch.contiguous_format))
        out = torch.empty(B, H, latent.LATENT_DIM, dtype=torch.bfloat16, device=dev)
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
        aws = dsaidx.new_workspace(latent.workspace_bytes(B, H, k))
        latent.latent_attend_slots(self.records, q_latent, turned, slots, self.scale, out, aws, lse=lse)
        return out, lse, idx, slots

    def decode_dense(self, q_latent, turned_q_pe, seq_lens, max_seq_len: int):
        """The same attention over every record of each sequence."""
        B, H = q_latent.shape[:2]
        out = torch.empty(B, H, latent.LATENT_DIM, dtype=torch.bfloat16, device=q_latent.device)
        lse = torch.empty(B, H, dtype=torch.float32, device=q_latent.device)
        ws = dsaidx.new_workspace(latent.workspace_bytes(B, H, max_seq_len))
        latent.latent_attend_paged(self.records, q_latent, turned_q_pe, self.block_table, seq_lens, max_seq_len, self.scale,
                                   out, ws, lse=lse)
        return out, lse


def prompt(layer: SparseLayer, q, k_up, v_up, c, k_pe, positions, cu_seqlens, in_place: bool = True):
    """Prompts no longer than the top-k select every key: expanded attention, without the indexer.  q [tokens,
    heads, 192] with its last 64 elements not yet turned, c [tokens, 512], k_up and v_up [heads, 512, 128].

    q is the projection's output, which nothing else reads, so those 64 elements are turned where they are: the
    caller's q has changed afterwards and must not be passed again.  in_place=False turns a copy and leaves q as
    it was."""
    if not in_place:
        q = q.clone()
    latent.rope(q[:, :, latent.NOPE_DIM:], positions, layer.plan)
    kp = latent.rope(k_pe[:, None], positions, layer.plan, out=torch.empty_like(k_pe)[:, None])[:, 0]
    k_nope = torch.einsum("tc,hcd->thd", c, k_up)
    v = torch.einsum("tc,hcd->thd", c, v_up)
    out = torch.empty(*v.shape, dtype=torch.bfloat16, device=q.device)
    latent.latent_attend_expanded(q, k_nope, kp, v, cu_seqlens, cu_seqlens, layer.scale, out)
    return out


def demo_layer(seq_lens, topk: int, heads: int, seed: int = 0, block_size: int = 64,
               temperature: str = "turn"):
    """A layer filled with seq_lens tokens a sequence and the inputs of one decode step.  The records are synthetic;
    temperature is SparseLayer.allocate's."""
    W = wl.make_workload("step", seq_lens, [1] * len(seq_lens), topk=topk, bs=block_size, seed=seed)
    dev = "cuda"
    layer = SparseLayer.allocate(W.num_blocks, block_size, torch.from_numpy(W.block_table).to(dev), topk,
                                 temperature=temperature)
    g = torch.Generator(device=dev).manual_seed(seed)
    n = sum(seq_lens)
    kv = torch.randn(n, latent.RECORD, generator=g, device=dev).bfloat16()
    positions = torch.cat([torch.arange(s, device=dev) for s in seq_lens])
    layer.append(bf16_tensor(W.all_keys()), kv[:, :latent.LATENT_DIM], kv[:, latent.LATENT_DIM:], positions,
                 torch.from_numpy(W.all_slots()).to(dev))
    B = len(seq_lens)
    q = torch.randn(B, heads, latent.RECORD, generator=g, device=dev).bfloat16()
    step = dict(index_q=bf16_tensor(W.q), index_w=torch.from_numpy(W.w).to(dev), q_latent=q[:, :, :latent.LATENT_DIM],
                q_pe=q[:, :, latent.LATENT_DIM:], seq_lens=torch.tensor(seq_lens, dtype=torch.int32, device=dev),
                positions=torch.tensor(seq_lens, device=dev) - 1, max_seq_len=max(seq_lens))
    return layer, step, kv, positions


def main():
    layer, step, _, _ = demo_layer([4500, 10000] * 4, topk=512, heads=128, temperature="logit")
    out, lse, idx, _ = layer.decode(**step)
    turned = latent.rope(step["q_pe"], step["positions"], layer.plan, out=torch.empty_like(step["q_pe"]))
    dense, dense_lse = layer.decode_dense(step["q_latent"], turned, step["seq_lens"], step["max_seq_len"])
    torch.cuda.synchronize()
    share = torch.exp(lse - dense_lse).mean()
    print("8 sequences of 4500 / 10000 keys, top-512, 128 heads: selected keys hold %.1f%% of the softmax weight, "
          "|sparse - dense| / |dense| = %.3f" % (100 * float(share), float((out - dense).norm() / dense.norm())))


if __name__ == "__main__":
    main()
