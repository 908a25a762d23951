"""ctypes binding of libdsaidx's latent attention (include/dsaidx_latent.h and,
for records in 8 bits, include/dsaidx_qlatent.h): rotary positions, the append
to a paged latent cache, and attention over the indexer's selected slots, over
whole paged contexts (absorbed form) and over prompts (expanded form).  The
calls on a cache take a LatentCache (bf16) or a QuantLatentCache (8 bits).

Argument marshalling only, as in dsaidx: tensors are checked for device (one
for all of a call's tensors, the current one), dtype and shape and passed as
raw pointers and strides with the current CUDA stream; there is no fallback.  Workspaces come from dsaidx.new_workspace.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

from . import dsaidx
from .dsaidx import IdxError

HEADER = os.path.join(os.path.dirname(dsaidx.HEADER), "dsaidx_latent.h")
QUANT_HEADER = os.path.join(os.path.dirname(dsaidx.HEADER), "dsaidx_qlatent.h")

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
    L.idx_qlatent_block_bytes.argtypes = [I]
    L.idx_qlatent_block_bytes.restype = SZ
    L.idx_qlatent_append.argtypes = L.idx_latent_append.argtypes
    L.idx_qlatent_read.argtypes = [POOL, P, I64, P, I64, P, P]
    L.idx_qlatent_attend_slots.argtypes = L.idx_latent_attend_slots.argtypes
    L.idx_qlatent_attend_paged.argtypes = L.idx_latent_attend_paged.argtypes
    for f in (L.idx_rope_steps, L.idx_rope, L.idx_latent_append, L.idx_latent_attend_slots,
              L.idx_latent_attend_paged, L.idx_latent_attend_expanded, L.idx_qlatent_append, L.idx_qlatent_read,
              L.idx_qlatent_attend_slots, L.idx_qlatent_attend_paged):
        f.restype = I
    _bound = L
    return L


def header_functions(header: str = HEADER):
    """Names of the functions include/dsaidx_latent.h (or another header) declares."""
    src = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(idx_[a-z_]+)\s*\(", src)))


# The calls below take a few microseconds on the GPU, so the checks are written
# for speed: one pass over what has to hold, the message only where it fails.
# Every tensor of a call has to be on the device of its first one (dev), which
# has to be the current one: the kernels are launched there.
_Tensor = torch.Tensor      # a name less to look up in each check


def _refuse(t, dtype, name: str, shape, dense: bool, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the call's other tensors on cuda:%d" % (name, t.get_device(), dev))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous%s" % (name, "" if dense else " in its last dimension"))


def _dev(t, name: str) -> int:
    """Index of the device of a call's first tensor."""
    dev = t.get_device() if isinstance(t, _Tensor) else -1
    if dev < 0:
        raise TypeError("%s must be a CUDA tensor" % name)
    return dev


def _dense(t: torch.Tensor, dtype, name: str, dev: int, shape=None) -> int:
    """Address of a contiguous tensor of that type (and shape) on that device."""
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        _refuse(t, dtype, name, shape, True, dev)
    return t.data_ptr()


def _strided(t: torch.Tensor, dtype, name: str, dev: int, shape):
    """Address and strides of a tensor of that type and shape on that device whose last dimension is contiguous."""
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape):
        _refuse(t, dtype, name, shape, False, dev)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel():
        _refuse(t, dtype, name, shape, False, dev)
    return t.data_ptr(), st


def _maybe(t, dtype, name: str, dev: int, shape=None):
    """_dense of an optional tensor: None where there is none."""
    return None if t is None else _dense(t, dtype, name, dev, shape)


def _elsewhere(name: str, held: int, dev: int):
    raise ValueError("the %s is on cuda:%d, the call's tensors on cuda:%d" % (name, held, dev))


def _check(code: int, what: str):
    if code:
        raise IdxError(code, what)


def _stream(stream, dev: int) -> int:
    """The stream's handle; the current one's without building a Stream object (2.9 us a call)."""
    if torch._C._cuda_getDevice() != dev or (stream is not None and stream.device_index != dev):
        raise ValueError("the tensors are on cuda:%d, which is not the current device%s"
                         % (dev, "" if stream is None else " and the stream's"))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream


class RopePlan:
    """Rotary steps in device memory (a uint64 fraction of a turn a pair, held as int64) and the amplitude."""

    def __init__(self, steps: torch.Tensor, amplitude: float):
        self.steps = steps
        self.amplitude = amplitude
        self.rot_dim = 2 * steps.numel()
        self.device = steps.get_device()
        self._address = _dense(steps, torch.int64, "plan.steps", self.device) if steps.is_cuda else None

    def on_device(self, dev: int) -> int:
        """Address of the steps; they have to be in that device's memory."""
        if self._address is None:
            raise TypeError("plan.steps must be a CUDA tensor")
        if self.device != dev:
            _elsewhere("plan", self.device, dev)
        return self._address


def rope_steps(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_max_pos: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """idx_rope_steps on the host: (steps as a CPU int64 tensor of uint64 bits, amplitude)."""
    if scaling not in _SCALING:
        raise ValueError("scaling must be one of %s" % sorted(_SCALING))
    steps = torch.zeros(max(rot_dim // 2, 1), dtype=torch.int64)
    amp = ctypes.c_float(0.0)
    _check(load().idx_rope_steps(rot_dim, base, _SCALING[scaling], factor, original_max_pos, beta_fast, beta_slow,
                                 steps.data_ptr(), ctypes.byref(amp)), "idx_rope_steps")
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
    in place.  What is written may not share elements between heads or tokens
    (an expanded tensor in place, an expanded out).  transpose=True applies the transposed map: the gradient of the
    turn with respect to x, given the gradient of its result."""
    dtype, shape = x.dtype, x.shape
    code = _DTYPE.get(dtype)
    if code is None or len(shape) != 3:
        raise TypeError("x must be [tokens, heads, head_dim] of bfloat16, float16 or float32")
    if layout != INTERLEAVED and layout != HALF:
        raise ValueError("layout must be INTERLEAVED or HALF")
    T, H, D = shape
    dev = _dev(x, "x")
    xp, xs = _strided(x, dtype, "x", dev, shape)
    if out is None:
        out, yp, ys = x, xp, xs
    else:
        yp, ys = _strided(out, dtype, "out", dev, shape)
    err = (_bound or load()).idx_rope(xp, xs[0], xs[1], yp, ys[0], ys[1], code, T, H, D,
                                      _dense(positions, torch.int64, "positions", dev, (T,)), plan.on_device(dev),
                                      plan.rot_dim, offset, plan.amplitude, layout | _TRANSPOSE if transpose else layout,
                                      _stream(stream, dev))
    if err:
        raise IdxError(err, "idx_rope")
    return out


class LatentCache:
    """A caller-owned pool of latent records: a bf16 CUDA tensor
    [num_blocks, block_size, 576], each record [latent 512 | turned key 64]."""
    calls = ("idx_latent_append", "idx_latent_attend_slots", "idx_latent_attend_paged")

    def __init__(self, pool: torch.Tensor):
        self.device = _dev(pool, "pool")
        _dense(pool, torch.bfloat16, "pool", self.device)
        if pool.dim() != 3 or pool.shape[2] != RECORD:
            raise ValueError("pool must be [num_blocks, block_size, %d]" % RECORD)
        self.pool = pool
        self.num_blocks, self.block_size = int(pool.shape[0]), int(pool.shape[1])
        self._desc = _Pool(pool.data_ptr(), self.num_blocks, self.block_size)
        self.desc = ctypes.byref(self._desc)   # what the calls take

    @staticmethod
    def allocate(num_blocks: int, block_size: int, device="cuda"):
        return LatentCache(torch.zeros(num_blocks, block_size, RECORD, dtype=torch.bfloat16, device=device))


def quant_block_bytes(block_size: int) -> int:
    """idx_qlatent_block_bytes: bytes of a block of records in 8 bits (0: no such size)."""
    return int(load().idx_qlatent_block_bytes(block_size))


class QuantLatentCache:
    """A caller-owned pool of latent records in 8 bits: a uint8 CUDA tensor
    [num_blocks, quant_block_bytes(block_size)], each record scale * [512 codes
    (e4m3) | turned key 64 (bf16)].  For latent_append, latent_read,
    latent_attend_slots and latent_attend_paged."""
    calls = ("idx_qlatent_append", "idx_qlatent_attend_slots", "idx_qlatent_attend_paged")

    def __init__(self, pool: torch.Tensor, block_size: int):
        self.device = _dev(pool, "pool")
        _dense(pool, torch.uint8, "pool", self.device)
        nb = quant_block_bytes(block_size)
        if nb == 0 or pool.dim() != 2 or pool.shape[1] != nb:
            raise ValueError("pool must be [num_blocks, %d] for blocks of %d tokens" % (nb, block_size))
        self.pool = pool
        self.num_blocks, self.block_size = int(pool.shape[0]), block_size
        self._desc = _Pool(pool.data_ptr(), self.num_blocks, block_size)
        self.desc = ctypes.byref(self._desc)   # what the calls take

    @staticmethod
    def allocate(num_blocks: int, block_size: int, device="cuda"):
        return QuantLatentCache(torch.zeros(num_blocks, quant_block_bytes(block_size), dtype=torch.uint8, device=device),
                                block_size)


def latent_append(cache, latent: torch.Tensor, k_pe: torch.Tensor, positions: Optional[torch.Tensor],
                  slot_mapping: torch.Tensor, plan: Optional[RopePlan], layout: int = INTERLEAVED,
                  status: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_append, idx_qlatent_append: write n tokens' records (latent
    [n, 512], k_pe [n, 64], rows may be strided) to their slots, k_pe turned by
    positions [n] int64 on the way (copied where plan is None), in the cache's format."""
    n, dev = latent.shape[0], _dev(latent, "latent")
    if cache.device != dev:
        _elsewhere("cache", cache.device, dev)
    lp, ls = _strided(latent, torch.bfloat16, "latent", dev, (n, LATENT_DIM))
    kp, ks = _strided(k_pe, torch.bfloat16, "k_pe", dev, (n, PE_DIM))
    if layout != INTERLEAVED and layout != HALF:
        raise ValueError("layout must be INTERLEAVED or HALF")
    pos = steps = None
    amplitude = 1.0
    if plan is not None:
        if plan.rot_dim != PE_DIM:
            raise ValueError("plan must turn %d elements" % PE_DIM)
        pos, steps = _dense(positions, torch.int64, "positions", dev, (n,)), plan.on_device(dev)
        amplitude = plan.amplitude
    name = cache.calls[0]
    err = getattr(_bound or load(), name)(cache.desc, lp, ls[0], kp, ks[0], pos,
                                          _dense(slot_mapping, torch.int64, "slot_mapping", dev, (n,)), n, steps,
                                          amplitude, layout, _maybe(status, torch.int32, "status", dev),
                                          _stream(stream, dev))
    if err:
        raise IdxError(err, name)


def latent_read(cache: QuantLatentCache, slots: torch.Tensor, out: torch.Tensor,
                status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """idx_qlatent_read: the records at slots [n] int64 into out [n, 576] bf16
    (rows may be strided), [latent 512 | turned key 64]; zeros where a slot is negative."""
    if not isinstance(cache, QuantLatentCache):
        raise TypeError("cache must be a QuantLatentCache")
    n, dev = slots.shape[0], _dev(slots, "slots")
    if cache.device != dev:
        _elsewhere("cache", cache.device, dev)
    op, os_ = _strided(out, torch.bfloat16, "out", dev, (n, RECORD))
    err = (_bound or load()).idx_qlatent_read(cache.desc, _dense(slots, torch.int64, "slots", dev, (n,)), n, op,
                                              os_[0] if n > 1 else RECORD, _maybe(status, torch.int32, "status", dev),
                                              _stream(stream, dev))
    if err:
        raise IdxError(err, "idx_qlatent_read")
    return out


def workspace_bytes(rows: int, heads: int, max_keys: int) -> int:
    """idx_latent_workspace_bytes: workspace of one absorbed attention call over either kind of cache."""
    return int(load().idx_latent_workspace_bytes(rows, heads, max_keys))


def _absorbed(cache, q_latent, q_pe, out, lse, workspace):
    """Checks what the two absorbed calls share: device, rows, heads and their common arguments."""
    dev = _dev(q_latent, "q_latent")
    if cache.device != dev:
        _elsewhere("cache", cache.device, dev)
    if q_latent.dim() != 3:
        raise ValueError("q_latent must be [rows, heads, %d]" % LATENT_DIM)
    T, H, _ = q_latent.shape
    lp, ls = _strided(q_latent, torch.bfloat16, "q_latent", dev, (T, H, LATENT_DIM))
    kp, ks = _strided(q_pe, torch.bfloat16, "q_pe", dev, (T, H, PE_DIM))
    return (dev, T, H, (lp, ls[0], ls[1], kp, ks[0], ks[1]),
            (_dense(out, torch.bfloat16, "out", dev, (T, H, LATENT_DIM)), _maybe(lse, torch.float32, "lse", dev, (T, H)),
             _dense(workspace, torch.uint8, "workspace", dev), workspace.numel()))


def latent_attend_slots(cache, q_latent: torch.Tensor, q_pe: torch.Tensor, slots: torch.Tensor,
                        scale: float, out: torch.Tensor, workspace: torch.Tensor,
                        lse: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_attend_slots, idx_qlatent_attend_slots: each row's queries (q_latent [rows, heads, 512],
    q_pe [rows, heads, 64]) attend over the records at its slots [rows, topk]
    int64 (the out_slot of the score calls; negative entries are skipped).
    out [rows, heads, 512] bf16, lse [rows, heads] fp32."""
    dev, T, H, query, result = _absorbed(cache, q_latent, q_pe, out, lse, workspace)
    if slots.dim() != 2:
        raise ValueError("slots must be [rows, topk]")
    topk = slots.shape[1]
    sp, ss = _strided(slots, torch.int64, "slots", dev, (T, topk))
    name = cache.calls[1]
    _check(getattr(load(), name)(cache.desc, *query, sp, ss[0], T, H, topk, scale, *result, _stream(stream, dev)), name)


def latent_attend_paged(cache, q_latent: torch.Tensor, q_pe: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, max_seq_len: int, scale: float, out: torch.Tensor,
                        workspace: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    """idx_latent_attend_paged, idx_qlatent_attend_paged: one query a sequence over all its records
    (block_table [batch, max_blocks_per_seq], seq_lens [batch] int32)."""
    dev, T, H, query, result = _absorbed(cache, q_latent, q_pe, out, lse, workspace)
    if block_table.dim() != 2 or block_table.shape[0] != T:
        raise ValueError("block_table must be [batch, max_blocks_per_seq]")
    name = cache.calls[2]
    _check(getattr(load(), name)(cache.desc, *query, _dense(block_table, torch.int32, "block_table", dev),
                                 block_table.shape[1], _dense(seq_lens, torch.int32, "seq_lens", dev, (T,)), T,
                                 max_seq_len, H, scale, *result, _stream(stream, dev)), name)


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
    dev, bf16, B = _dev(q, "q"), torch.bfloat16, cu_seqlens_q.numel() - 1
    qp, qs = _strided(q, bf16, "q", dev, (T, H, NOPE_DIM + PE_DIM))
    np_, ns = _strided(k_nope, bf16, "k_nope", dev, (S, H, NOPE_DIM))
    pp, ps = _strided(k_pe, bf16, "k_pe", dev, (S, PE_DIM))
    vp, vs = _strided(v, bf16, "v", dev, (S, H, V_DIM))
    _check(load().idx_latent_attend_expanded(qp, qs[0], qs[1], np_, ns[0], ns[1], pp, ps[0], vp, vs[0], vs[1],
                                             _dense(cu_seqlens_q, torch.int32, "cu_seqlens_q", dev, (B + 1,)),
                                             _dense(cu_seqlens_k, torch.int32, "cu_seqlens_k", dev, (B + 1,)), B, T, S, H,
                                             scale, _dense(out, bf16, "out", dev, (T, H, V_DIM)),
                                             _maybe(lse, torch.float32, "lse", dev, (T, H)),
                                             _maybe(status, torch.int32, "status", dev), _stream(stream, dev)),
           "idx_latent_attend_expanded")
