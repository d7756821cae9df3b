"""context_long_sequence_zigzag_gb300 — Python binding of libcpattn.

Context-parallel exact causal attention on one GB300: a (packed) sequence is
cut into C context-parallel shards (contiguous, zigzag or striped); the C virtual ranks
share one GPU and the KV ring is the order in which the kernels visit the
HBM-resident KV shards.  The C ABI (``include/cp_attn.h``) is the product;
this module only marshals torch tensors into its pointers and sizes.  Every
step runs in the library's CUDA kernels; there is no fallback: importing this
module fails if ``libcpattn.so`` has not been built, and every call raises on
a non-OK status.

Functions carry the C names: ``cp_shard_permute``, ``cp_attn_block_fwd``,
``cp_lse_merge``, ``cp_attn_fwd``, ``cp_attn_bwd``, ``cp_workspace_size``,
``cp_shard_offsets``, ``cp_rank_block_counts``, ``cp_rank_fwd_key_tiles``, ``cp_device_status``,
``cp_check_bounded_wait``, ``cp_status_string``, ``cp_validate``, ``cp_ulysses_a2a``,
``cp_ulysses_attn_fwd``, ``cp_ulysses_attn_bwd``, ``cp_ring_attn_fwd``, ``cp_lin_attn_fwd``,
``cp_attn_key_weights``, and for decoding over a 4-bit key/value cache (``Kv4Cache``) ``cp_kv4_append``,
``cp_kv4_read``, ``cp_kv4_attn``, ``cp_kv4_evict``, ``cp_kv4_block_bytes``, ``cp_kv4_validate``,
``cp_kv4_workspace_size``.  Over a cache in the model's own type (``KvCache``): ``cp_kv_append``, ``cp_kv_attn``,
``cp_kv_validate``, ``cp_kv_workspace_size``; rotary positions (``Rope``): ``cp_rope``, ``cp_rope_turns``; pages that
sequences share (``PagePool``): ``cp_pages_reserve``, ``cp_pages_fork``, ``cp_pages_compact``, ``cp_pages_copy``,
``cp_pages_validate``, ``cp_pages_workspace_size``.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcpattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python context_long_sequence_zigzag_gb300/build.py` (no CPU fallback exists)")

_lib = ctypes.CDLL(LIB_PATH)

CP_OK, CP_ERR_INVALID_ARG, CP_ERR_UNSUPPORTED, CP_ERR_CUDA, CP_ERR_DEVICE_TIMEOUT, CP_ERR_WORKSPACE = range(6)
CP_LAYOUT_CONTIGUOUS, CP_LAYOUT_ZIGZAG, CP_LAYOUT_STRIPED = 0, 1, 2
CP_DT_F32, CP_DT_BF16 = 0, 1
CP_GQA_BLOCKED, CP_GQA_INTERLEAVED = 0, 1
CP_OP_FWD, CP_OP_BWD, CP_OP_BLOCK_FWD, CP_OP_PERMUTE, CP_OP_BWD_DKDV, CP_OP_BWD_DQ = 0, 1, 2, 3, 4, 5
CP_OP_ULYSSES_A2A, CP_OP_ULYSSES_FWD, CP_OP_ULYSSES_BWD, CP_OP_LIN_FWD, CP_OP_RING_FWD = 6, 7, 8, 9, 10
CP_OP_KEY_WEIGHTS = 11
CP_KV4_PAGE, CP_KV4_GROUP, CP_KV4_MAX_QUERIES = 64, 64, 16
CP_ROPE_HALVES, CP_ROPE_ADJACENT = 0, 1
CP_ROPE_MAX_AXES, CP_ROPE_MAX_DIMS, CP_PAGES_MAX_BUFFERS = 4, 512, 128

EXPORTED = [
    "cp_status_string", "cp_validate", "cp_workspace_size", "cp_shard_offsets",
    "cp_rank_block_counts", "cp_rank_fwd_key_tiles", "cp_shard_permute", "cp_attn_block_fwd", "cp_lse_merge",
    "cp_attn_fwd", "cp_attn_bwd", "cp_device_status", "cp_check_bounded_wait",
    "cp_attn_fwd_noalloc", "cp_attn_bwd_prep", "cp_attn_bwd_dkdv", "cp_attn_bwd_dq",
    "cp_ulysses_a2a", "cp_ulysses_attn_fwd", "cp_ulysses_attn_bwd", "cp_lin_attn_fwd", "cp_ring_attn_fwd",
    "cp_set_debug_checks", "cp_attn_key_weights",
    "cp_kv4_block_bytes", "cp_kv4_validate", "cp_kv4_workspace_size", "cp_kv4_append", "cp_kv4_read", "cp_kv4_attn",
    "cp_kv4_evict",
    "cp_rope_turns", "cp_rope", "cp_kv_validate", "cp_kv_workspace_size", "cp_kv_append", "cp_kv_attn",
    "cp_pages_validate", "cp_pages_workspace_size", "cp_pages_reserve", "cp_pages_fork", "cp_pages_compact",
    "cp_pages_copy",
]


class cp_desc_t(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("hq", ctypes.c_int32),
        ("hkv", ctypes.c_int32),
        ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
        ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("cp_size", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("gqa", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class cp_kv4_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("hq", ctypes.c_int32),
        ("hkv", ctypes.c_int32),
        ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("gqa", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("pages", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
    ]


class cp_rope_t(ctypes.Structure):
    _fields_ = [
        ("first", ctypes.c_int32),
        ("dims", ctypes.c_int32),
        ("pairing", ctypes.c_int32),
        ("axes", ctypes.c_int32),
        ("factor", ctypes.c_float),
        ("turns", ctypes.c_void_p),
        ("axis", ctypes.c_void_p),
    ]


class cp_kv_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("hq", ctypes.c_int32),
        ("hkv", ctypes.c_int32),
        ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("gqa", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("k_pages", ctypes.c_void_p),
        ("v_pages", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
    ]


class cp_pages_t(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("refs", ctypes.c_void_p),
        ("num_buffers", ctypes.c_int32),
        ("base", ctypes.POINTER(ctypes.c_void_p)),
        ("bytes", ctypes.POINTER(ctypes.c_int64)),
    ]


_P = ctypes.c_void_p
_DP = ctypes.POINTER(cp_desc_t)
_KP = ctypes.POINTER(cp_kv4_t)
_RP, _CP, _GP = ctypes.POINTER(cp_rope_t), ctypes.POINTER(cp_kv_t), ctypes.POINTER(cp_pages_t)
_I = ctypes.c_int32
_sigs = {
    "cp_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cp_validate": (ctypes.c_int, [_DP]),
    "cp_workspace_size": (ctypes.c_int, [_DP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "cp_shard_offsets": (ctypes.c_int, [_DP, ctypes.POINTER(ctypes.c_int64)]),
    "cp_rank_block_counts": (ctypes.c_int, [_DP, ctypes.POINTER(ctypes.c_int64)]),
    "cp_rank_fwd_key_tiles": (ctypes.c_int, [_DP, ctypes.POINTER(ctypes.c_int64)]),
    "cp_shard_permute": (ctypes.c_int, [_DP, _P, _P, ctypes.c_int64, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "cp_attn_block_fwd": (ctypes.c_int, [_DP, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                         ctypes.c_size_t, _P]),
    "cp_lse_merge": (ctypes.c_int, [_DP, ctypes.c_int64, _P, _P, _P, _P, _P]),
    "cp_attn_fwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_attn_bwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_device_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "cp_check_bounded_wait": (ctypes.c_int, [ctypes.c_int64, ctypes.POINTER(ctypes.c_int32), _P]),
    "cp_attn_fwd_noalloc": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P]),
    "cp_attn_bwd_prep": (ctypes.c_int, [_DP, _P, _P, _P, _P]),
    "cp_attn_bwd_dkdv": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_attn_bwd_dq": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_ulysses_a2a": (ctypes.c_int, [_DP, _P, _P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P,
                                      ctypes.c_size_t, _P]),
    "cp_ulysses_attn_fwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_lin_attn_fwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_ulysses_attn_bwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_ring_attn_fwd": (ctypes.c_int, [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "cp_set_debug_checks": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "cp_attn_key_weights": (ctypes.c_int, [_DP, ctypes.c_int64, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_kv4_block_bytes": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "cp_kv4_validate": (ctypes.c_int, [_KP]),
    "cp_kv4_workspace_size": (ctypes.c_int, [_KP, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "cp_kv4_append": (ctypes.c_int, [_KP, _P, _P, _P, ctypes.c_int64, _P, _P, _P, ctypes.c_int64, _P]),
    "cp_kv4_read": (ctypes.c_int, [_KP, _P, _P, ctypes.c_int64, _P, _P, _P]),
    "cp_kv4_attn": (ctypes.c_int, [_KP, ctypes.c_int32, _P, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, _P,
                                   ctypes.c_size_t, _P]),
    "cp_kv4_evict": (ctypes.c_int, [_KP, _P, ctypes.c_int32, ctypes.c_int32, _KP, _P, _P, _P]),
    "cp_rope_turns": (ctypes.c_int, [_P, _I, _P]),
    "cp_rope": (ctypes.c_int, [_RP, ctypes.c_int64, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P]),
    "cp_kv_validate": (ctypes.c_int, [_CP]),
    "cp_kv_workspace_size": (ctypes.c_int, [_CP, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "cp_kv_append": (ctypes.c_int, [_CP, _P, _P, ctypes.c_int64, _P, _P, _P, ctypes.c_int64, _RP, _P, _I, _P]),
    "cp_kv_attn": (ctypes.c_int, [_CP, _I, _P, _P, _P, _I, _P, _P, ctypes.c_size_t, _P]),
    "cp_pages_validate": (ctypes.c_int, [_GP]),
    "cp_pages_workspace_size": (ctypes.c_int, [_GP, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "cp_pages_reserve": (ctypes.c_int, [_GP, _I, _I, _P, _P, _P, _P, _P]),
    "cp_pages_fork": (ctypes.c_int, [_GP, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_pages_compact": (ctypes.c_int, [_GP, _I, _I, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "cp_pages_copy": (ctypes.c_int, [_GP, _GP, _I, _P, _P, _P]),
}
for _name, (_res, _args) in _sigs.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class CpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {cp_status_string(status)}")


def cp_status_string(status: int) -> str:
    return _lib.cp_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != CP_OK:
        raise CpError(status, where)


class Problem:
    """Holds a cp_desc_t and the host cu_seqlens it points at.

    cu_seqlens : global-order int32 prefix sums (list / tensor), or None for
                 one sequence of ``total_tokens``.
    """

    def __init__(self, total_tokens: int, hq: int, hkv: int, d_qk: int, d_v: int, cp_size: int,
                 layout: str = "zigzag", cu_seqlens=None, causal: bool = True,
                 scale: Optional[float] = None, gqa: str = "blocked", dtype=torch.bfloat16):
        if cu_seqlens is None:
            cu = [0, int(total_tokens)]
        else:
            cu = [int(x) for x in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
        self.cu = cu
        self._cu_arr = (ctypes.c_int32 * len(cu))(*cu)
        self.torch_dtype = dtype
        self.desc = cp_desc_t(
            total_tokens=int(total_tokens), num_seqs=len(cu) - 1, hq=hq, hkv=hkv,
            cu_seqlens=ctypes.cast(self._cu_arr, ctypes.POINTER(ctypes.c_int32)),
            d_qk=d_qk, d_v=d_v, cp_size=cp_size,
            layout={"contiguous": CP_LAYOUT_CONTIGUOUS, "zigzag": CP_LAYOUT_ZIGZAG,
                    "striped": CP_LAYOUT_STRIPED}[layout],
            causal=int(bool(causal)),
            scale=float(scale if scale is not None else 1.0 / math.sqrt(d_qk)),
            gqa={"blocked": CP_GQA_BLOCKED, "interleaved": CP_GQA_INTERLEAVED}[gqa],
            dtype={torch.float32: CP_DT_F32, torch.bfloat16: CP_DT_BF16}[dtype])
        self._key_weights_bytes = None

    @classmethod
    def from_workload(cls, w, cu_seqlens=None) -> "Problem":
        from_cu = cu_seqlens if cu_seqlens is not None else _cu_of(w.lengths())
        return cls(w.total_tokens, w.hq, w.hkv, w.d_qk, w.d_v, w.cp_size, w.layout, from_cu,
                   w.causal, w.scale, "blocked",
                   torch.float32 if w.dtype == "f32" else torch.bfloat16)

    @property
    def ptr(self):
        return ctypes.byref(self.desc)

    @property
    def T(self) -> int:
        return int(self.desc.total_tokens)


def _cu_of(lengths):
    cu = [0]
    for L in lengths:
        cu.append(cu[-1] + int(L))
    return cu


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.is_cuda and not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def cp_validate(prob: Problem) -> int:
    return _lib.cp_validate(prob.ptr)


def cp_workspace_size(prob: Problem, op: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.cp_workspace_size(prob.ptr, int(op), ctypes.byref(n)), "cp_workspace_size")
    return int(n.value)


def cp_shard_offsets(prob: Problem) -> list:
    arr = (ctypes.c_int64 * (prob.desc.cp_size + 1))()
    _check(_lib.cp_shard_offsets(prob.ptr, arr), "cp_shard_offsets")
    return list(arr)


def cp_rank_block_counts(prob: Problem) -> list:
    arr = (ctypes.c_int64 * prob.desc.cp_size)()
    _check(_lib.cp_rank_block_counts(prob.ptr, arr), "cp_rank_block_counts")
    return list(arr)


def cp_rank_fwd_key_tiles(prob: Problem) -> list:
    arr = (ctypes.c_int64 * prob.desc.cp_size)()
    _check(_lib.cp_rank_fwd_key_tiles(prob.ptr, arr), "cp_rank_fwd_key_tiles")
    return list(arr)


def workspace(prob: Problem, op: int, device=None) -> torch.Tensor:
    """A device buffer of cp_workspace_size bytes (256-byte aligned)."""
    n = max(cp_workspace_size(prob, op), 1)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def cp_shard_permute(prob: Problem, x: torch.Tensor, inverse: bool = False, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows (first dim, T) of x from global to sharded order (inverse: back)."""
    if out is None:
        out = torch.empty_like(x)
    row_bytes = x[0].numel() * x.element_size() if x.shape[0] else x.element_size() * 16
    if ws is None:
        ws = workspace(prob, CP_OP_PERMUTE, x.device)
    _check(_lib.cp_shard_permute(prob.ptr, _ptr(x), _ptr(out), row_bytes, int(bool(inverse)), _ptr(ws),
                                 ws.numel(), _stream(stream)), "cp_shard_permute")
    return out


def cp_attn_block_fwd(prob: Problem, q_rank: int, kv_rank: int, q, k, v, o_part=None, lse_part=None,
                      ws=None, stream=None):
    off = cp_shard_offsets(prob)
    Tr = off[q_rank + 1] - off[q_rank]
    d = prob.desc
    if o_part is None:
        o_part = torch.empty(Tr, d.hq, d.d_v, dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty(d.hq, Tr, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(prob, CP_OP_BLOCK_FWD, q.device)
    _check(_lib.cp_attn_block_fwd(prob.ptr, q_rank, kv_rank, _ptr(q), _ptr(k), _ptr(v), _ptr(o_part),
                                  _ptr(lse_part), _ptr(ws), ws.numel(), _stream(stream)), "cp_attn_block_fwd")
    return o_part, lse_part


def cp_lse_merge(prob: Problem, o_acc, lse_acc, o_part, lse_part, stream=None):
    rows = o_acc.shape[0]
    _check(_lib.cp_lse_merge(prob.ptr, rows, _ptr(o_acc), _ptr(lse_acc), _ptr(o_part), _ptr(lse_part),
                             _stream(stream)), "cp_lse_merge")
    return o_acc, lse_acc


def cp_attn_fwd(prob: Problem, q, k, v, o=None, lse=None, ws=None, stream=None):
    d = prob.desc
    if o is None:
        o = torch.empty(d.total_tokens, d.hq, d.d_v, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(d.hq, d.total_tokens, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(prob, CP_OP_FWD, q.device)
    _check(_lib.cp_attn_fwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                            _stream(stream)), "cp_attn_fwd")
    return o, lse


def cp_attn_bwd(prob: Problem, q, k, v, o, lse, dout, dq=None, dk=None, dv=None, ws=None, stream=None):
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    if ws is None:
        ws = workspace(prob, CP_OP_BWD, q.device)
    _check(_lib.cp_attn_bwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                            _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)), "cp_attn_bwd")
    return dq, dk, dv


def cp_ring_attn_fwd(prob: Problem, q, k, v, o=None, lse=None, ws=None, stream=None, comm_stream=None,
                     overlap: bool = True):
    """Ring forward with explicit KV transport: C steps, each rank's block
    against the shard it holds, while the shards move one rank on through
    device-to-device copies on ``comm_stream`` (a new high-priority stream
    when None and ``overlap``, so that the copies are not queued behind the
    attention kernel's waiting CTAs; ``overlap=False`` serialises the copies
    on ``stream``)."""
    d = prob.desc
    if o is None:
        o = torch.empty(d.total_tokens, d.hq, d.d_v, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(d.hq, d.total_tokens, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(prob, CP_OP_RING_FWD, q.device)
    if overlap and comm_stream is None:
        comm_stream = torch.cuda.Stream(device=q.device, priority=-1)
    xs = _stream(comm_stream) if overlap else None
    _check(_lib.cp_ring_attn_fwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                 _stream(stream), xs), "cp_ring_attn_fwd")
    return o, lse


def cp_ulysses_a2a(prob: Problem, x: torch.Tensor, inverse: bool = False, out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Ulysses all-to-all re-layout.  Forward: x [T, H, ...] in sharded order
    -> [C, T, H/C, ...] (rank r: heads r*H/C.., global token order).
    Inverse: [C, T, H/C, ...] -> [T, H, ...] sharded."""
    C = prob.desc.cp_size
    if inverse:
        heads = x.shape[2] * C
        shape = (x.shape[1], heads) + tuple(x.shape[3:])
    else:
        heads = x.shape[1]
        shape = (C, x.shape[0], heads // C) + tuple(x.shape[2:])
    head_bytes = (x[0, 0].numel() if not inverse else x[0, 0, 0].numel()) * x.element_size()
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    if ws is None:
        ws = workspace(prob, CP_OP_ULYSSES_A2A, x.device)
    _check(_lib.cp_ulysses_a2a(prob.ptr, _ptr(x), _ptr(out), heads, head_bytes, int(bool(inverse)), _ptr(ws),
                               ws.numel(), _stream(stream)), "cp_ulysses_a2a")
    return out


def cp_ulysses_attn_fwd(prob: Problem, q, k, v, o=None, lse=None, ws=None, stream=None):
    """cp_attn_fwd computed the Ulysses way (all-to-all, per-rank full-sequence
    attention, all-to-all back); same inputs and outputs."""
    d = prob.desc
    if o is None:
        o = torch.empty(d.total_tokens, d.hq, d.d_v, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(d.hq, d.total_tokens, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(prob, CP_OP_ULYSSES_FWD, q.device)
    _check(_lib.cp_ulysses_attn_fwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                    _stream(stream)), "cp_ulysses_attn_fwd")
    return o, lse


def cp_ulysses_attn_bwd(prob: Problem, q, k, v, o, lse, dout, dq=None, dk=None, dv=None, ws=None, stream=None):
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    if ws is None:
        ws = workspace(prob, CP_OP_ULYSSES_BWD, q.device)
    _check(_lib.cp_ulysses_attn_bwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                                    _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)), "cp_ulysses_attn_bwd")
    return dq, dk, dv


def cp_lin_attn_fwd(prob: Problem, q, k, v, g, o=None, ws=None, stream=None):
    """Decayed linear attention with AllGather CP (contiguous pieces).
    g: float32 [hq] on the device, log of the per-head decay."""
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if ws is None:
        ws = workspace(prob, CP_OP_LIN_FWD, q.device)
    _check(_lib.cp_lin_attn_fwd(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o), _ptr(ws), ws.numel(),
                                _stream(stream)), "cp_lin_attn_fwd")
    return o


def cp_attn_bwd_prep(prob: Problem, o, dout, dpsum=None, stream=None):
    """D = rowsum(dout * o) per (head, row): float32 [hq, T]."""
    d = prob.desc
    if dpsum is None:
        dpsum = torch.empty(d.hq, d.total_tokens, dtype=torch.float32, device=o.device)
    _check(_lib.cp_attn_bwd_prep(prob.ptr, _ptr(o), _ptr(dout), _ptr(dpsum), _stream(stream)), "cp_attn_bwd_prep")
    return dpsum


def cp_attn_bwd_dkdv(prob: Problem, q, k, v, lse, dpsum, dout, dk=None, dv=None, ws=None, stream=None):
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    if ws is None:
        ws = workspace(prob, CP_OP_BWD_DKDV, q.device)
    _check(_lib.cp_attn_bwd_dkdv(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(dpsum), _ptr(dout), _ptr(dk),
                                 _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)), "cp_attn_bwd_dkdv")
    return dk, dv


def cp_attn_bwd_dq(prob: Problem, q, k, v, lse, dpsum, dout, dq=None, ws=None, stream=None):
    if dq is None:
        dq = torch.empty_like(q)
    if ws is None:
        ws = workspace(prob, CP_OP_BWD_DQ, q.device)
    _check(_lib.cp_attn_bwd_dq(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(dpsum), _ptr(dout), _ptr(dq),
                               _ptr(ws), ws.numel(), _stream(stream)), "cp_attn_bwd_dq")
    return dq


def cp_attn_fwd_noalloc(prob: Problem, q, k, v, o, lse, stream=None):
    """Forward without a workspace: the tile plan lives in the library's fixed
    device scratch (CP_NOALLOC_SCRATCH_BYTES).  o and lse are caller-owned;
    nothing is allocated here or in the library."""
    _check(_lib.cp_attn_fwd_noalloc(prob.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream)),
           "cp_attn_fwd_noalloc")
    return o, lse


NOALLOC_SCRATCH_BYTES = 4 << 20


try:  # (torch.cuda.current_stream builds an object on every call)
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # a private name, and one that builds without CUDA lack

    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


_current_device = torch.cuda.current_device


def _order_after(on, dev: torch.device) -> None:
    """Stream `on` waits for the current one: what the allocator handed out
    there may still be in use by work queued there before.  (Not across a
    capture, which would drag the other stream into it.)"""
    with torch.cuda.device(dev):
        if torch.cuda.is_current_stream_capturing():
            return
        current = torch.cuda.current_stream()
        with torch.cuda.stream(on):
            if torch.cuda.is_current_stream_capturing():
                return
        on.wait_stream(current)


def _launch(dev: torch.device, stream, temps, name: str, *args) -> None:
    """Calls a library function with the stream appended, on device dev.
    ``temps`` (buffers allocated here) are kept until that stream is done."""
    index = dev.index
    handle = _raw_stream(index)
    if stream is not None:
        other = _stream(stream)
        if other != handle:
            if isinstance(stream, torch.cuda.Stream):
                on = stream
            else:  # (handle 0, the default stream, would make ExternalStream a stream of the pool)
                on = torch.cuda.ExternalStream(other, device=dev) if other else torch.cuda.default_stream(dev)
            if temps:
                _order_after(on, dev)
            for x in temps:
                x.record_stream(on)
            handle = other
    if _current_device() == index:
        status = _kv4_calls[name](*args, handle)
    else:
        with torch.cuda.device(dev):
            status = _kv4_calls[name](*args, handle)
    if status != CP_OK:
        raise CpError(status, name)


_kv4_calls = {n: getattr(_lib, n) for n in ("cp_attn_key_weights", "cp_kv4_append", "cp_kv4_read", "cp_kv4_attn",
                                            "cp_kv4_evict", "cp_rope", "cp_kv_append", "cp_kv_attn",
                                            "cp_pages_reserve", "cp_pages_fork", "cp_pages_compact",
                                            "cp_pages_copy")}


def _need(t, name: str, dtype, shape, device=None) -> int:
    """Data pointer of a contiguous CUDA tensor of this type and shape (None
    in the shape: any size); ValueError otherwise."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: a tensor on {device or 'a CUDA device'} is needed")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} is needed, got {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _need_workspace(ws, device) -> int:
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous tensor on {device} is needed")
    return ws.data_ptr()


def cp_attn_key_weights(prob: Problem, q, k, lse, last: Optional[int] = None, w=None, ws=None, stream=None):
    """Accumulated attention weight of every key, float32 [hkv, T] in sharded
    order: the attention probabilities summed over the query heads of the
    key's head and over the queries, or over the last ``last`` of every
    sequence.  lse: the forward's; +inf leaves a query out.  bfloat16 heads of 128 and 192 run on the
    tensor cores, others slowly on the CUDA cores.  Not for capture into a graph (as the other
    calls with tile plans)."""
    d = prob.desc
    if not isinstance(q, torch.Tensor) or not q.is_cuda:  # (the others have to be where q is)
        raise ValueError("q: a tensor on a CUDA device is needed")
    T, hkv, dev, dtype = d.total_tokens, d.hkv, q.device, prob.torch_dtype
    if last is not None and last < 1:
        raise ValueError("last: a positive number of queries, or None for all")
    pq = _need(q, "q", dtype, (T, d.hq, d.d_qk), dev)
    pk = _need(k, "k", dtype, (T, hkv, d.d_qk), dev)
    pl = _need(lse, "lse", torch.float32, (d.hq, T), dev)
    temps = []
    if w is None:
        w = torch.empty((hkv, T), dtype=torch.float32, device=dev)
        temps.append(w)
        pw = w.data_ptr()
    else:
        pw = _need(w, "w", torch.float32, (hkv, T), dev)
    if ws is None:
        if prob._key_weights_bytes is None:
            prob._key_weights_bytes = cp_workspace_size(prob, CP_OP_KEY_WEIGHTS)
        ws = torch.empty(max(prob._key_weights_bytes, 1), dtype=torch.uint8, device=dev)
        temps.append(ws)
    _launch(dev, stream, temps, "cp_attn_key_weights", prob.ptr, last or 0, pq, pk, pl, pw, _need_workspace(ws, dev),
            ws.numel() * ws.element_size())
    return w


def cp_kv4_block_bytes(d_qk: int, d_v: int) -> int:
    """Bytes of one page (64 tokens) of one key/value head."""
    n = ctypes.c_size_t(0)
    _check(_lib.cp_kv4_block_bytes(d_qk, d_v, ctypes.byref(n)), "cp_kv4_block_bytes")
    return int(n.value)


class Kv4Cache:
    """A paged key/value cache in 4 bits, or the part of it that a call deals
    with: the pool and the page table of the sequences in the batch.

    pages      : uint8 [num_pages, hkv, cp_kv4_block_bytes(d_qk, d_v)]
    page_table : int32 [num_seqs, max_pages], a page of 64 tokens an entry
    weights    : float32 [num_pages, hkv, 64], the tokens' accumulated attention weights, or None
    dtype      : of keys, values, queries and outputs (float32 or bfloat16)

    Holds the tensors; lengths stay with the caller.
    """

    def __init__(self, pages: torch.Tensor, page_table: torch.Tensor, hq: int, hkv: int, d_qk: int, d_v: int,
                 weights: Optional[torch.Tensor] = None, scale: Optional[float] = None, gqa: str = "blocked",
                 dtype=torch.bfloat16):
        block = cp_kv4_block_bytes(d_qk, d_v)
        p = _need(pages, "pages", torch.uint8, (None, hkv, block))
        t = _need(page_table, "page_table", torch.int32, (None, None), pages.device)
        w = None
        if weights is not None:
            w = _need(weights, "weights", torch.float32, (pages.shape[0], hkv, CP_KV4_PAGE), pages.device)
        self.pages, self.page_table, self.weights = pages, page_table, weights
        self.torch_dtype, self.device = dtype, pages.device
        self.num_seqs, self.hq, self.hkv, self.d_qk, self.d_v = page_table.shape[0], hq, hkv, d_qk, d_v
        self.desc = cp_kv4_t(
            num_seqs=page_table.shape[0], hq=hq, hkv=hkv, d_qk=d_qk, d_v=d_v,
            gqa={"blocked": CP_GQA_BLOCKED, "interleaved": CP_GQA_INTERLEAVED}[gqa],
            dtype={torch.float32: CP_DT_F32, torch.bfloat16: CP_DT_BF16}[dtype],
            scale=float(scale if scale is not None else 1.0 / math.sqrt(d_qk)),
            num_pages=pages.shape[0], max_pages=page_table.shape[1], pages=p, weights=w, page_table=t)
        self.ptr = ctypes.byref(self.desc)
        self._ws_bytes = {}
        _check(_lib.cp_kv4_validate(self.ptr), "cp_kv4_validate")


def cp_kv4_validate(cache: Kv4Cache) -> int:
    return _lib.cp_kv4_validate(cache.ptr)


def cp_kv4_workspace_size(cache: Kv4Cache, n_q: int = 1, accumulate: bool = False) -> int:
    n = ctypes.c_size_t(0)
    with torch.cuda.device(cache.device):  # (whose SMs it goes by)
        _check(_lib.cp_kv4_workspace_size(cache.ptr, n_q, int(bool(accumulate)), ctypes.byref(n)), "cp_kv4_workspace_size")
    return int(n.value)


def cp_kv4_append(cache: Kv4Cache, k, v, cu, start, w=None, rows=None, stream=None) -> None:
    """Quantises tokens into the cache: token t, cu[b] <= t < cu[b + 1], becomes
    slot start[b] + t - cu[b] of sequence b, from row rows[t] (or t) of k
    [n, hkv, d_qk], v [n, hkv, d_v] and w [hkv, n] (their first weights; None: 0).
    cu int32 [B + 1], start int32 [B], rows int32 [tokens], on the device."""
    dev, hkv, dtype, B = cache.device, cache.hkv, cache.torch_dtype, cache.num_seqs
    n = k.shape[0]
    pk = _need(k, "k", dtype, (n, hkv, cache.d_qk), dev)
    pv = _need(v, "v", dtype, (n, hkv, cache.d_v), dev)
    pw = None if w is None else _need(w, "w", torch.float32, (hkv, n), dev)
    tokens = n if rows is None else rows.shape[0]
    pr = None if rows is None else _need(rows, "rows", torch.int32, (tokens,), dev)
    _launch(dev, stream, (), "cp_kv4_append", cache.ptr, pk, pv, pw, n, pr, _need(cu, "cu", torch.int32, (B + 1,), dev),
            _need(start, "start", torch.int32, (B,), dev), tokens)


def cp_kv4_read(cache: Kv4Cache, cu, start, tokens: int, k=None, v=None, stream=None):
    """Slots start[b], start[b] + 1, ... of every sequence b as rows cu[b] .. cu[b + 1] - 1 of
    k [tokens, hkv, d_qk] and v [tokens, hkv, d_v].  Other rows (from cu[B] on, or of slots outside the cache) are not
    written: pass k and v where those should hold something."""
    dev, dtype, B = cache.device, cache.torch_dtype, cache.num_seqs
    temps = []
    shape = (tokens, cache.hkv, cache.d_qk)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
        temps.append(k)
        pk = k.data_ptr()
    else:
        pk = _need(k, "k", dtype, shape, dev)
    shape = (tokens, cache.hkv, cache.d_v)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=dev)
        temps.append(v)
        pv = v.data_ptr()
    else:
        pv = _need(v, "v", dtype, shape, dev)
    _launch(dev, stream, temps, "cp_kv4_read", cache.ptr, _need(cu, "cu", torch.int32, (B + 1,), dev),
            _need(start, "start", torch.int32, (B,), dev), tokens, pk, pv)
    return k, v


def cp_kv4_attn(cache: Kv4Cache, q, lengths, accumulate: bool = False, part: bool = False, o=None, lse=None, ws=None,
                stream=None):
    """Attention of q [B, n_q, hq, d_qk], the newest n_q tokens of every sequence, over the cache
    (lengths int32 [B]: tokens held, the new ones among them).  Returns o [B, n_q, hq, d_v] and
    lse [hq, B * n_q].  accumulate: the attention probabilities are added to cache.weights.
    part: o in float32, for cp_lse_merge (in a bfloat16 cache with the probabilities rounded to bfloat16 on the way all the
    same; a Kv4Cache of dtype float32 over the same pages takes float32 queries and keeps float32)."""
    dev, dtype, B, hq = cache.device, cache.torch_dtype, cache.num_seqs, cache.hq
    n_q = q.shape[1]
    pq = _need(q, "q", dtype, (B, n_q, hq, cache.d_qk), dev)
    o_dtype = torch.float32 if part else dtype
    accumulate = bool(accumulate)
    temps = []
    shape = (B, n_q, hq, cache.d_v)
    if o is None:
        o = torch.empty(shape, dtype=o_dtype, device=dev)
        temps.append(o)
        po = o.data_ptr()
    else:
        po = _need(o, "o", o_dtype, shape, dev)
    shape = (hq, B * n_q)
    if lse is None:
        lse = torch.empty(shape, dtype=torch.float32, device=dev)
        temps.append(lse)
        pl = lse.data_ptr()
    else:
        pl = _need(lse, "lse", torch.float32, shape, dev)
    if ws is None:
        size = cache._ws_bytes.get((n_q, accumulate))
        if size is None:
            size = cache._ws_bytes[n_q, accumulate] = max(cp_kv4_workspace_size(cache, n_q, accumulate), 1)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        temps.append(ws)
        pw = ws.data_ptr()
    else:
        pw, size = _need_workspace(ws, dev), ws.numel() * ws.element_size()
    _launch(dev, stream, temps, "cp_kv4_attn", cache.ptr, n_q, pq, _need(lengths, "lengths", torch.int32, (B,), dev), po,
            1 if part else 0, pl, 1 if accumulate else 0, pw, size)
    return o, lse


def cp_kv4_evict(cache: Kv4Cache, lengths, budget: int, recent: int, to: Kv4Cache, new_lengths=None, kept=None,
                 stream=None):
    """Keeps, for every sequence and head, the last ``recent`` slots and the budget - recent others of
    largest weight, copied in slot order into the pages of ``to`` (no page may be read and written).
    Returns new_lengths int32 [B] and kept int32 [B, hkv, budget], the slots kept (-1 behind the last)."""
    dev, B = cache.device, cache.num_seqs
    temps = []
    if new_lengths is None:
        new_lengths = torch.empty(B, dtype=torch.int32, device=dev)
        temps.append(new_lengths)
    shape = (B, cache.hkv, max(budget, 0))
    if kept is None:
        kept = torch.empty(shape, dtype=torch.int32, device=dev)
        temps.append(kept)
    if to.device != dev:
        raise ValueError(f"to: a cache on {dev} is needed")
    _launch(dev, stream, temps, "cp_kv4_evict", cache.ptr, _need(lengths, "lengths", torch.int32, (B,), dev), budget,
            recent, to.ptr, _need(new_lengths, "new_lengths", torch.int32, (B,), dev),
            _need(kept, "kept", torch.int32, shape, dev))
    return new_lengths, kept


_DTYPES = {torch.float32: CP_DT_F32, torch.bfloat16: CP_DT_BF16}


def cp_rope_turns(inv_freq) -> list:
    """Frequencies (radians a position) as 64-bit fractions of a turn a position."""
    f = [float(x) for x in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
    got = (ctypes.c_uint64 * len(f))()
    _check(_lib.cp_rope_turns((ctypes.c_double * len(f))(*f), len(f), got), "cp_rope_turns")
    return list(got)


class Rope:
    """Rotary positions: which channels of a head turn, in which pairs and how fast.

    inv_freq : frequency of every pair (radians a position; taken in 64 bits), list or tensor
    axis     : the position axis that every pair follows (time, height, width, ...), or None: 0
    first    : first of the 2 * len(inv_freq) turned channels
    pairing  : "halves": channel i with i + len(inv_freq); "adjacent": 2i with 2i + 1
    factor   : on every turned channel
    """

    def __init__(self, inv_freq, axis=None, first: int = 0, pairing: str = "halves", factor: float = 1.0,
                 device="cuda"):
        turns = cp_rope_turns(inv_freq)
        axes = 1
        if axis is not None:
            axis = [int(x) for x in (axis.tolist() if hasattr(axis, "tolist") else axis)]
            if len(axis) != len(turns) or any(x < 0 or x >= CP_ROPE_MAX_AXES for x in axis):
                raise ValueError(f"axis: one of 0 .. {CP_ROPE_MAX_AXES - 1} for every frequency is needed")
            axes = max(axis, default=0) + 1
        if not turns or len(turns) * 2 > CP_ROPE_MAX_DIMS:
            raise ValueError(f"inv_freq: 1 to {CP_ROPE_MAX_DIMS // 2} frequencies are needed")
        if first < 0 or not math.isfinite(factor):
            raise ValueError("first: a channel, and factor: a finite number is needed")
        self.axes, self.first, self.dims = axes, first, 2 * len(turns)
        self.turns = torch.tensor([x - (x >> 63 << 64) for x in turns], dtype=torch.int64).to(device)
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.int32).to(device)
        self.device = self.turns.device
        if not self.turns.is_cuda:
            raise ValueError("device: a CUDA device is needed")
        self.desc = cp_rope_t(
            first=first, dims=self.dims, pairing={"halves": CP_ROPE_HALVES, "adjacent": CP_ROPE_ADJACENT}[pairing],
            axes=axes, factor=float(factor), turns=self.turns.data_ptr(),
            axis=None if axis is None else self.axis.data_ptr())
        self.ptr = ctypes.byref(self.desc)


def _sizes(t) -> tuple:
    """Shape of a tensor; () of anything else (which _need then refuses)."""
    return t.shape if isinstance(t, torch.Tensor) else ()


def _positions(rope: Rope, positions, rows: int, dev):
    """Pointer and row length of positions [rows, axes or more] (or [rows] on one axis)."""
    if rope.device != dev:
        raise ValueError(f"rope: a Rope on {dev} is needed")
    shape = _sizes(positions)
    if len(shape) == 1:
        wide = 1
        p = _need(positions, "positions", torch.int32, (rows,), dev)
    else:
        wide = shape[1] if len(shape) == 2 else rope.axes
        p = _need(positions, "positions", torch.int32, (rows, wide), dev)
    if wide < rope.axes:
        raise ValueError(f"positions: {rope.axes} columns are needed, got {wide}")
    return p, wide


def cp_rope(rope: Rope, positions, q, k=None, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """q [T, hq, d] and k [T, hkv, d] turned by their rows' positions (int32 [T, axes], or more columns, or [T]);
    inverse: turned back (the gradients of a call's inputs from those of its outputs).  q_out, k_out: q and k
    themselves for a call in place.  Returns q_out, or (q_out, k_out) with k."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:  # (the others have to be where q is)
        raise ValueError("q: a tensor on a CUDA device is needed")
    dev, dtype, shape = q.device, q.dtype, q.shape
    code = _DTYPES.get(dtype)
    if len(shape) != 3 or code is None:
        raise ValueError("q: float32 or bfloat16 [T, heads, d] is needed")
    T, hq, d = shape
    temps = []
    pq = _need(q, "q", dtype, shape, dev)
    if q_out is None:
        q_out = torch.empty_like(q)
        temps.append(q_out)
        po = q_out.data_ptr()
    else:
        po = _need(q_out, "q_out", dtype, shape, dev)
    hkv, pk, pko = 0, None, None
    if k is not None:
        kshape = _sizes(k)
        hkv = kshape[1] if len(kshape) == 3 else 0
        pk = _need(k, "k", dtype, (T, hkv, d), dev)
        if k_out is None:
            k_out = torch.empty_like(k)
            temps.append(k_out)
            pko = k_out.data_ptr()
        else:
            pko = _need(k_out, "k_out", dtype, kshape, dev)
    pp, wide = _positions(rope, positions, T, dev)
    _launch(dev, stream, temps, "cp_rope", rope.ptr, T, pp, wide, d, code, hq, pq, po, hkv, pk, pko,
            1 if inverse else 0)
    return q_out if k is None else (q_out, k_out)


class KvCache:
    """A paged key/value cache in float32 or bfloat16, or the part of it that a call deals with: the pools and the
    page table of the sequences in the batch.

    k_pages    : [num_pages, hkv, page_size, d_qk]
    v_pages    : [num_pages, hkv, page_size, d_v]
    page_table : int32 [num_seqs, max_pages], a page of page_size tokens an entry

    Holds the tensors; lengths stay with the caller.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, hq: int,
                 scale: Optional[float] = None, gqa: str = "blocked"):
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4 or k_pages.dtype not in _DTYPES:
            raise ValueError("k_pages: float32 or bfloat16 [num_pages, hkv, page_size, d_qk] is needed")
        dtype, (num_pages, hkv, page_size, d_qk) = k_pages.dtype, k_pages.shape
        pk = _need(k_pages, "k_pages", dtype, (None,) * 4, None if not k_pages.is_cuda else k_pages.device)
        pv = _need(v_pages, "v_pages", dtype, (num_pages, hkv, page_size, None), k_pages.device)
        t = _need(page_table, "page_table", torch.int32, (None, None), k_pages.device)
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.torch_dtype, self.device, self.page_size = dtype, k_pages.device, page_size
        self.num_seqs, self.hq, self.hkv, self.d_qk, self.d_v = page_table.shape[0], hq, hkv, d_qk, v_pages.shape[3]
        self.desc = cp_kv_t(
            num_seqs=page_table.shape[0], hq=hq, hkv=hkv, d_qk=d_qk, d_v=self.d_v,
            gqa={"blocked": CP_GQA_BLOCKED, "interleaved": CP_GQA_INTERLEAVED}[gqa], dtype=_DTYPES[dtype],
            scale=float(scale if scale is not None else 1.0 / math.sqrt(d_qk)), page_size=page_size,
            num_pages=num_pages, max_pages=page_table.shape[1], k_pages=pk, v_pages=pv, page_table=t)
        self.ptr = ctypes.byref(self.desc)
        self._ws_bytes = {}
        _check(_lib.cp_kv_validate(self.ptr), "cp_kv_validate")


def cp_kv_validate(cache: KvCache) -> int:
    return _lib.cp_kv_validate(cache.ptr)


def cp_kv_workspace_size(cache: KvCache, n_q: int = 1) -> int:
    n = ctypes.c_size_t(0)
    with torch.cuda.device(cache.device):  # (whose SMs it goes by)
        _check(_lib.cp_kv_workspace_size(cache.ptr, n_q, ctypes.byref(n)), "cp_kv_workspace_size")
    return int(n.value)


def cp_kv_append(cache: KvCache, k, v, cu, start, rows=None, rope: Optional[Rope] = None, positions=None,
                 stream=None) -> None:
    """Writes tokens into the cache: token t, cu[b] <= t < cu[b + 1], becomes slot start[b] + t - cu[b] of
    sequence b, from row rows[t] (or t) of k [n, hkv, d_qk] and v [n, hkv, d_v].  rope: keys are turned on the way
    by positions (int32 [n, axes] or [n], in k's rows; None: by their slots).
    cu int32 [B + 1], start int32 [B], rows int32 [tokens], on the device."""
    dev, hkv, dtype, B = cache.device, cache.hkv, cache.torch_dtype, cache.num_seqs
    n = (_sizes(k) or (0,))[0]
    pk = _need(k, "k", dtype, (n, hkv, cache.d_qk), dev)
    pv = _need(v, "v", dtype, (n, hkv, cache.d_v), dev)
    tokens, pr = n, None
    if rows is not None:
        tokens = (_sizes(rows) or (0,))[0]
        pr = _need(rows, "rows", torch.int32, (tokens,), dev)
    ptr, pp, wide = None, None, 0
    if rope is not None:
        ptr = rope.ptr
        if positions is not None:
            pp, wide = _positions(rope, positions, n, dev)
        elif rope.device != dev:
            raise ValueError(f"rope: a Rope on {dev} is needed")
    elif positions is not None:
        raise ValueError("positions: they need a rope")
    _launch(dev, stream, (), "cp_kv_append", cache.ptr, pk, pv, n, pr, _need(cu, "cu", torch.int32, (B + 1,), dev),
            _need(start, "start", torch.int32, (B,), dev), tokens, ptr, pp, wide)


def cp_kv_attn(cache: KvCache, q, lengths, part: bool = False, o=None, lse=None, ws=None, stream=None):
    """Attention of q [B, n_q, hq, d_qk], the newest n_q tokens of every sequence, over the cache
    (lengths int32 [B]: tokens held, the new ones among them).  Returns o [B, n_q, hq, d_v] and
    lse [hq, B * n_q].  part: o in float32, for cp_lse_merge."""
    dev, dtype, B, hq = cache.device, cache.torch_dtype, cache.num_seqs, cache.hq
    shape = _sizes(q)
    n_q = shape[1] if len(shape) == 4 else 1
    pq = _need(q, "q", dtype, (B, n_q, hq, cache.d_qk), dev)
    o_dtype = torch.float32 if part else dtype
    temps = []
    shape = (B, n_q, hq, cache.d_v)
    if o is None:
        o = torch.empty(shape, dtype=o_dtype, device=dev)
        temps.append(o)
        po = o.data_ptr()
    else:
        po = _need(o, "o", o_dtype, shape, dev)
    shape = (hq, B * n_q)
    if lse is None:
        lse = torch.empty(shape, dtype=torch.float32, device=dev)
        temps.append(lse)
        pl = lse.data_ptr()
    else:
        pl = _need(lse, "lse", torch.float32, shape, dev)
    if ws is None:
        size = cache._ws_bytes.get(n_q)
        if size is None:
            size = cache._ws_bytes[n_q] = cp_kv_workspace_size(cache, n_q)
        pw = None
        if size:
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
            temps.append(ws)
            pw = ws.data_ptr()
    else:
        pw, size = _need_workspace(ws, dev), ws.numel() * ws.element_size()
    _launch(dev, stream, temps, "cp_kv_attn", cache.ptr, n_q, pq, _need(lengths, "lengths", torch.int32, (B,), dev), po,
            1 if part else 0, pl, pw, size)
    return o, lse


class PagePool:
    """Pages that several sequences may hold, of either cache.

    refs      : int32 [num_pages], the table entries that hold a page (0: it is free)
    buffers   : tensors [num_pages, ...] that a page consists of (K and V pages of one or all layers, a 4-bit
                cache's pages and weights)
    page_size : tokens of a page

    Holds the tensors; tables and lengths stay with the caller.
    """

    def __init__(self, refs: torch.Tensor, buffers: Sequence[torch.Tensor], page_size: int = CP_KV4_PAGE):
        r = _need(refs, "refs", torch.int32, (None,), refs.device if isinstance(refs, torch.Tensor) and refs.is_cuda else None)
        self.refs, self.buffers, self.device, self.num_pages = refs, list(buffers), refs.device, refs.shape[0]
        self.page_size = page_size
        base, size = [], []
        for x in self.buffers:
            base.append(_need(x, "buffers", x.dtype if isinstance(x, torch.Tensor) else None,
                              (self.num_pages,) + (None,) * (x.dim() - 1 if isinstance(x, torch.Tensor) else 0), refs.device))
            size.append(x[0].numel() * x.element_size() if self.num_pages else 16)
        n = len(base)
        self._base, self._bytes = (ctypes.c_void_p * n)(*base), (ctypes.c_int64 * n)(*size)
        self.desc = cp_pages_t(num_pages=self.num_pages, page_size=page_size, refs=r, num_buffers=n,
                               base=ctypes.cast(self._base, ctypes.POINTER(ctypes.c_void_p)),
                               bytes=ctypes.cast(self._bytes, ctypes.POINTER(ctypes.c_int64)))
        self.ptr = ctypes.byref(self.desc)
        self._ws_bytes = {}
        _check(_lib.cp_pages_validate(self.ptr), "cp_pages_validate")

    def _workspace(self, num_seqs: int, ws, temps):
        if ws is not None:
            return _need_workspace(ws, self.device), ws.numel() * ws.element_size()
        size = self._ws_bytes.get(num_seqs)
        if size is None:
            size = self._ws_bytes[num_seqs] = cp_pages_workspace_size(self, num_seqs)
        ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        temps.append(ws)
        return ws.data_ptr(), size

    def _out(self, t, name, shape, temps):
        if t is None:
            t = torch.empty(shape, dtype=torch.int32, device=self.device)
            temps.append(t)
            return t, t.data_ptr()
        return t, _need(t, name, torch.int32, shape, self.device)


def cp_pages_validate(pool: PagePool) -> int:
    return _lib.cp_pages_validate(pool.ptr)


def cp_pages_workspace_size(pool: PagePool, num_seqs: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.cp_pages_workspace_size(pool.ptr, num_seqs, ctypes.byref(n)), "cp_pages_workspace_size")
    return int(n.value)


def _rows_of(table, dev):
    shape = _sizes(table)
    B, columns = shape if len(shape) == 2 else (0, 0)
    return B, columns, _need(table, "table", torch.int32, (B, columns), dev)


def cp_pages_reserve(pool: PagePool, table, lengths, extra, counts=None, stream=None):
    """Gives every sequence b of lengths[b] tokens the pages that extra[b] more need, or takes those back that it needs
    no more (extra below 0), in table [B, max_pages] (in place).  Returns counts int32 [2]: pages in use, and entries
    that got none (they are -1)."""
    dev, temps = pool.device, []
    B, columns, pt = _rows_of(table, dev)
    counts, pc = pool._out(counts, "counts", (2,), temps)
    _launch(dev, stream, temps, "cp_pages_reserve", pool.ptr, B, columns, pt,
            _need(lengths, "lengths", torch.int32, (B,), dev), _need(extra, "extra", torch.int32, (B,), dev), pc)
    return counts


def cp_pages_fork(pool: PagePool, table, lengths, parents, new_table=None, new_lengths=None, counts=None, ws=None,
                  stream=None):
    """New sequence b goes on from old sequence parents[b] (below 0: it is empty); the old ones let go of their
    pages.  Whole pages are shared, a partly filled one is copied for all but the first that takes it.  Returns
    new_table [len(parents), columns] (-1 behind the last page), new_lengths and counts int32 [2]: pages in use,
    and entries that got none."""
    dev, temps = pool.device, []
    B, columns, pt = _rows_of(table, dev)
    n = (_sizes(parents) or (0,))[0]
    pp = _need(parents, "parents", torch.int32, (n,), dev)
    shape = _sizes(new_table)
    new_table, pn = pool._out(new_table, "new_table", (n, shape[1] if len(shape) == 2 else columns), temps)
    new_lengths, pl = pool._out(new_lengths, "new_lengths", (n,), temps)
    counts, pc = pool._out(counts, "counts", (2,), temps)
    pw, size = pool._workspace(max(B, n), ws, temps)
    _launch(dev, stream, temps, "cp_pages_fork", pool.ptr, B, columns, pt,
            _need(lengths, "lengths", torch.int32, (B,), dev), n, new_table.shape[1], pp, pn, pl, pc, pw, size)
    return new_table, new_lengths, counts


def cp_pages_compact(pool: PagePool, table, lengths, new_table=None, moved=None, counts=None, ws=None, stream=None):
    """Moves the pages in use to the front of the pool.  Returns new_table, the table of the sequences after it (table
    itself may be given), moved int32 [num_pages], every page's new place (-1: it was free), and counts int32 [2]:
    pages in use, and 0."""
    dev, temps = pool.device, []
    B, columns, pt = _rows_of(table, dev)
    new_table, pn = pool._out(new_table, "new_table", (B, columns), temps)
    moved, pm = pool._out(moved, "moved", (pool.num_pages,), temps)
    counts, pc = pool._out(counts, "counts", (2,), temps)
    pw, size = pool._workspace(B, ws, temps)
    _launch(dev, stream, temps, "cp_pages_compact", pool.ptr, B, columns, pt,
            _need(lengths, "lengths", torch.int32, (B,), dev), pn, pm, pc, pw, size)
    return new_table, moved, counts


def cp_pages_copy(pool: PagePool, src, dst, to: Optional[PagePool] = None, stream=None) -> None:
    """Copies page src[i] to page dst[i] of pool ``to`` (None: the same; pairs with a negative page are skipped).  No
    page may be written twice, or read and written, in one call.  refs are not looked at."""
    dev = pool.device
    if to is not None and to.device != dev:
        raise ValueError(f"to: a pool on {dev} is needed")
    n = (_sizes(src) or (0,))[0]
    ps = _need(src, "src", torch.int32, (n,), dev)
    _launch(dev, stream, (), "cp_pages_copy", pool.ptr, (to or pool).ptr, n, ps,
            _need(dst, "dst", torch.int32, (n,), dev))


def cp_set_debug_checks(on: bool) -> bool:
    """Turns the plan checks on or off for later calls; returns the former setting."""
    prev = ctypes.c_int32(0)
    _check(_lib.cp_set_debug_checks(int(bool(on)), ctypes.byref(prev)), "cp_set_debug_checks")
    return bool(prev.value)


def cp_device_status(stream=None) -> int:
    code = ctypes.c_int32(0)
    st = _lib.cp_device_status(_stream(stream), ctypes.byref(code))
    if st not in (CP_OK, CP_ERR_DEVICE_TIMEOUT):
        _check(st, "cp_device_status")
    return int(code.value)


def cp_check_bounded_wait(timeout_ns: int = 20_000_000, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(_lib.cp_check_bounded_wait(int(timeout_ns), ctypes.byref(code), _stream(stream)),
           "cp_check_bounded_wait")
    return int(code.value)


__all__ = ["Problem", "Kv4Cache", "KvCache", "PagePool", "Rope", "CpError", "workspace", "LIB_PATH", "EXPORTED"] + EXPORTED
