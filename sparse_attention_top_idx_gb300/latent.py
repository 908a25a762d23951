"""ctypes binding of libdsaidx's latent attention (include/dsaidx_latent.h):
rotary positions, the append to a paged latent cache, and attention over the
indexer's selected slots, over whole paged contexts (absorbed form) and over
prompts (expanded form).

Argument marshalling only, as in dsaidx: tensors are checked for device, dtype
and shape and passed as raw pointers and strides with the current CUDA stream;
there is no fallback.  Workspaces come from dsaidx.new_workspace.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

from . import dsaidx
from .dsaidx import _check, _need, _ptr, _stream

HEADER = os.path.join(os.path.dirname(dsaidx.HEADER), "dsaidx_latent.h")

LATENT_DIM = 512
PE_DIM = 64
RECORD = LATENT_DIM + PE_DIM
NOPE_DIM = 128
V_DIM = 128

INTERLEAVED = 0   # pairs (2 i, 2 i + 1)
HALF = 1          # pairs (i, i + rot_dim / 2); IDX_ROPE_HALF
_TRANSPOSE = 2    # IDX_ROPE_TRANSPOSE

_SCALING = {"none": 0, "linear": 1, "yarn": 2}
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class _Pool(ctypes.Structure):
    _fields_ = [("data_dev", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int)]


_bound = None


def load():
    """The library with the argument types of the calls of this module."""
    global _bound
    L = dsaidx.load()
    if _bound is L:
        return L
    P, I, I64, SZ, D, F, U = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_double,
                              ctypes.c_float, ctypes.c_uint)
    POOL = ctypes.POINTER(_Pool)
    L.idx_rope_steps.argtypes = [I, D, I, D, D, D, D, P, ctypes.POINTER(F)]
    L.idx_rope.argtypes = [P, I64, I64, P, I64, I64, I, I64, I, I, P, P, I, I, F, U, P]
    L.idx_latent_append.argtypes = [POOL, P, I64, P, I64, P, P, I64, P, F, U, P, P]
    L.idx_latent_workspace_bytes.argtypes = [I64, I, I64]
    L.idx_latent_workspace_bytes.restype = SZ
    L.idx_latent_attend_slots.argtypes = [POOL, P, I64, I64, P, I64, I64, P, I64, I64, I, I, F, P, P, P, SZ, P]
    L.idx_latent_attend_paged.argtypes = [POOL, P, I64, I64, P, I64, I64, P, I, P, I, I, I, F, P, P, P, SZ, P]
    L.idx_latent_attend_expanded.argtypes = [P, I64, I64, P, I64, I64, P, I64, P, I64, I64, P, P, I, I64, I64, I, F,
                                             P, P, P, P]
    for f in (L.idx_rope_steps, L.idx_rope, L.idx_latent_append, L.idx_latent_attend_slots,
              L.idx_latent_attend_paged, L.idx_latent_attend_expanded):
        f.restype = I
    _bound = L
    return L


def header_functions():
    """Names of the functions include/dsaidx_latent.h declares."""
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(idx_[a-z_]+)\s*\(", src)))


def _strided(t: torch.Tensor, dtype, name: str, shape):
    """A CUDA tensor of that type and shape whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.numel() and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


class RopePlan:
    """Rotary steps in device memory (a uint64 fraction of a turn a pair, held as int64) and the amplitude."""

    def __init__(self, steps: torch.Tensor, amplitude: float):
        self.steps = steps
        self.amplitude = amplitude
        self.rot_dim = 2 * steps.numel()


def rope_steps(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_max_pos: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """idx_rope_steps on the host: (steps as a CPU int64 tensor of uint64 bits, amplitude)."""
    if scaling not in _SCALING:
        raise ValueError("scaling must be one of %s" % sorted(_SCALING))
    steps = torch.zeros(max(rot_dim // 2, 1), dtype=torch.int64)
    amp = ctypes.c_float(0.0)
    _check(load().idx_rope_steps(rot_dim, base, _SCALING[scaling], factor, original_max_pos, beta_fast, beta_slow,
                                 _ptr(steps), ctypes.byref(amp)), "idx_rope_steps")
    return steps, float(amp.value)


def rope_plan(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
              original_max_pos: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
              amplitude: Optional[float] = None, device="cuda") -> RopePlan:
    """The steps of idx_rope_steps on the device; scaling "none", "linear" or
    "yarn"; amplitude overrides the scaling's own."""
    steps, amp = rope_steps(rot_dim, base, scaling, factor, original_max_pos, beta_fast, beta_slow)
    return RopePlan(steps.to(device), amp if amplitude is None else float(amplitude))


def rope(x: torch.Tensor, positions: torch.Tensor, plan: RopePlan, layout: int = INTERLEAVED, offset: int = 0,
         out: Optional[torch.Tensor] = None, transpose: bool = False, stream=None) -> torch.Tensor:
    """idx_rope: turn elements [offset, offset + plan.rot_dim) of every head of
    x [tokens, heads, head_dim] (bf16, fp16 or fp32, any strides) by its token's
    position [tokens] int64; into out (which gets the other elements too) or
    in place.  transpose=True applies the transposed map: the gradient of the
    turn with respect to x, given the gradient of its result."""
    if x.dim() != 3 or x.dtype not in _DTYPE:
        raise TypeError("x must be [tokens, heads, head_dim] of bfloat16, float16 or float32")
    if layout not in (INTERLEAVED, HALF):
        raise ValueError("layout must be INTERLEAVED or HALF")
    T, H, D = x.shape
    out = x if out is None else out
    _strided(x, x.dtype, "x", (T, H, D))
    _strided(out, x.dtype, "out", (T, H, D))
    _need(positions, torch.int64, "positions", (T,))
    _need(plan.steps, torch.int64, "plan.steps")
    _check(load().idx_rope(_ptr(x), x.stride(0), x.stride(1), _ptr(out), out.stride(0), out.stride(1),
                           _DTYPE[x.dtype], T, H, D, _ptr(positions), _ptr(plan.steps), plan.rot_dim, offset,
                           plan.amplitude, layout | (_TRANSPOSE if transpose else 0), _stream(stream)), "idx_rope")
    return out


class LatentCache:
    """A caller-owned pool of latent records: a bf16 CUDA tensor
    [num_blocks, block_size, 576], each record [latent 512 | turned key 64]."""

    def __init__(self, pool: torch.Tensor):
        _need(pool, torch.bfloat16, "pool")
        if pool.dim() != 3 or pool.shape[2] != RECORD:
            raise ValueError("pool must be [num_blocks, block_size, %d]" % RECORD)
        self.pool = pool
        self.num_blocks, self.block_size = int(pool.shape[0]), int(pool.shape[1])
        self._desc = _Pool(pool.data_ptr(), self.num_blocks, self.block_size)

    @staticmethod
    def allocate(num_blocks: int, block_size: int, device="cuda"):
        return LatentCache(torch.zeros(num_blocks, block_size, RECORD, dtype=torch.bfloat16, device=device))

    @property
    def desc(self):
        return ctypes.byref(self._desc)


def latent_append(cache: LatentCache, latent: torch.Tensor, k_pe: torch.Tensor, positions: Optional[torch.Tensor],
                  slot_mapping: torch.Tensor, plan: Optional[RopePlan], layout: int = INTERLEAVED,
                  status: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_append: write n tokens' records (latent [n, 512], k_pe
    [n, 64], rows may be strided) to their slots, k_pe turned by positions
    [n] int64 on the way (copied where plan is None)."""
    n = latent.shape[0]
    _strided(latent, torch.bfloat16, "latent", (n, LATENT_DIM))
    _strided(k_pe, torch.bfloat16, "k_pe", (n, PE_DIM))
    _need(slot_mapping, torch.int64, "slot_mapping", (n,))
    if layout not in (INTERLEAVED, HALF):
        raise ValueError("layout must be INTERLEAVED or HALF")
    if plan is not None:
        if plan.rot_dim != PE_DIM:
            raise ValueError("plan must turn %d elements" % PE_DIM)
        _need(positions, torch.int64, "positions", (n,))
        _need(plan.steps, torch.int64, "plan.steps")
    if status is not None:
        _need(status, torch.int32, "status")
    _check(load().idx_latent_append(cache.desc, _ptr(latent), latent.stride(0), _ptr(k_pe), k_pe.stride(0),
                                    _ptr(positions if plan is not None else None), _ptr(slot_mapping), n,
                                    _ptr(plan.steps if plan is not None else None),
                                    plan.amplitude if plan is not None else 1.0, layout, _ptr(status),
                                    _stream(stream)), "idx_latent_append")


def workspace_bytes(rows: int, heads: int, max_keys: int) -> int:
    """idx_latent_workspace_bytes: workspace of one absorbed attention call."""
    return int(load().idx_latent_workspace_bytes(rows, heads, max_keys))


def _absorbed_tensors(q_latent, q_pe, out, lse, workspace):
    if q_latent.dim() != 3:
        raise ValueError("q_latent must be [rows, heads, %d]" % LATENT_DIM)
    T, H = q_latent.shape[0], q_latent.shape[1]
    _strided(q_latent, torch.bfloat16, "q_latent", (T, H, LATENT_DIM))
    _strided(q_pe, torch.bfloat16, "q_pe", (T, H, PE_DIM))
    _need(out, torch.bfloat16, "out", (T, H, LATENT_DIM))
    if lse is not None:
        _need(lse, torch.float32, "lse", (T, H))
    _need(workspace, torch.uint8, "workspace")
    return T, H


def latent_attend_slots(cache: LatentCache, q_latent: torch.Tensor, q_pe: torch.Tensor, slots: torch.Tensor,
                        scale: float, out: torch.Tensor, workspace: torch.Tensor,
                        lse: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_attend_slots: each row's queries (q_latent [rows, heads, 512],
    q_pe [rows, heads, 64]) attend over the records at its slots [rows, topk]
    int64 (the out_slot of the score calls; negative entries are skipped).
    out [rows, heads, 512] bf16, lse [rows, heads] fp32."""
    T, H = _absorbed_tensors(q_latent, q_pe, out, lse, workspace)
    if slots.dim() != 2:
        raise ValueError("slots must be [rows, topk]")
    _strided(slots, torch.int64, "slots", (T, slots.shape[1]))
    _check(load().idx_latent_attend_slots(cache.desc, _ptr(q_latent), q_latent.stride(0), q_latent.stride(1),
                                          _ptr(q_pe), q_pe.stride(0), q_pe.stride(1), _ptr(slots), slots.stride(0), T,
                                          H, slots.shape[1], scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                          workspace.numel(), _stream(stream)), "idx_latent_attend_slots")


def latent_attend_paged(cache: LatentCache, q_latent: torch.Tensor, q_pe: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, max_seq_len: int, scale: float, out: torch.Tensor,
                        workspace: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_attend_paged: one query a sequence over all its records
    (block_table [batch, max_blocks_per_seq], seq_lens [batch] int32)."""
    T, H = _absorbed_tensors(q_latent, q_pe, out, lse, workspace)
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens", (T,))
    if block_table.dim() != 2 or block_table.shape[0] != T:
        raise ValueError("block_table must be [batch, max_blocks_per_seq]")
    _check(load().idx_latent_attend_paged(cache.desc, _ptr(q_latent), q_latent.stride(0), q_latent.stride(1),
                                          _ptr(q_pe), q_pe.stride(0), q_pe.stride(1), _ptr(block_table),
                                          block_table.shape[1], _ptr(seq_lens), T, max_seq_len, H, scale, _ptr(out),
                                          _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)),
           "idx_latent_attend_paged")


def latent_attend_expanded(q: torch.Tensor, k_nope: torch.Tensor, k_pe: torch.Tensor, v: torch.Tensor,
                           cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, scale: float, out: torch.Tensor,
                           lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_attend_expanded: causal attention of packed prompts, q
    [total_q, heads, 192], k_nope and v [total_k, heads, 128], k_pe
    [total_k, 64] shared by the heads; a sequence's queries are its last
    positions.  out [total_q, heads, 128] bf16, lse [total_q, heads] fp32."""
    if q.dim() != 3 or k_nope.dim() != 3:
        raise ValueError("q and k_nope must be [tokens, heads, dim]")
    T, H, S = q.shape[0], q.shape[1], k_nope.shape[0]
    _strided(q, torch.bfloat16, "q", (T, H, NOPE_DIM + PE_DIM))
    _strided(k_nope, torch.bfloat16, "k_nope", (S, H, NOPE_DIM))
    _strided(k_pe, torch.bfloat16, "k_pe", (S, PE_DIM))
    _strided(v, torch.bfloat16, "v", (S, H, V_DIM))
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    B = cu_seqlens_q.numel() - 1
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", (B + 1,))
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k", (B + 1,))
    _need(out, torch.bfloat16, "out", (T, H, V_DIM))
    if lse is not None:
        _need(lse, torch.float32, "lse", (T, H))
    if status is not None:
        _need(status, torch.int32, "status")
    _check(load().idx_latent_attend_expanded(_ptr(q), q.stride(0), q.stride(1), _ptr(k_nope), k_nope.stride(0),
                                             k_nope.stride(1), _ptr(k_pe), k_pe.stride(0), _ptr(v), v.stride(0),
                                             v.stride(1), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, T, S, H, scale,
                                             _ptr(out), _ptr(lse), _ptr(status), _stream(stream)),
           "idx_latent_attend_expanded")
