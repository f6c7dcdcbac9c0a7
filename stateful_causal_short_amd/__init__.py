"""MI355X (gfx950) stateful causal short convolution, and the operators that
take its outputs: the gated delta rule (prefill, update, speculative update),
head norms with rotation and cache write (bf16 or quantised), the quantised
cache's read, paged decode attention, and attention over shared prefixes.

Thin Python binding of ``libstatefulconv.so`` (C ABI in
``include/statefulconv.h``). Every function here only marshals arguments —
device pointers, sizes, strides, the current HIP stream — and calls the
library; every step of the computation runs in the library's HIP kernels.
PyTorch provides device memory and streams. There is no CPU fallback: if the
library is missing, import-time loading fails loudly.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libstatefulconv.so")

SC_OK = 0
SC_ABI_VERSION = 3   # the struct layouts and signatures below
STATUS = {0: "SC_OK", -1: "SC_ERR_NULL_ARG", -2: "SC_ERR_INVALID_ARG",
          -3: "SC_ERR_DTYPE", -4: "SC_ERR_STATE_CAPACITY",
          -5: "SC_ERR_UNSUPPORTED", -6: "SC_ERR_HIP"}
SC_DTYPE_F32, SC_DTYPE_BF16 = 0, 1
SC_ACT_NONE, SC_ACT_SILU = 0, 1
SC_STATE_DS, SC_STATE_SD = 0, 1

EXPORTS = ("sc_conv_prefill_varlen", "sc_conv_update", "sc_conv_update_spec",
           "sc_conv_update_spec_varlen", "sc_validate_metadata", "sc_state_gather",
           "sc_state_scatter", "sc_cca_qk_conv", "sc_gdn_workspace_bytes",
           "sc_gdn_prefill_varlen", "sc_gdn_update", "sc_gdn_update_spec",
           "sc_qk_norm_rope", "sc_paged_attn_workspace_bytes", "sc_paged_attn_decode",
           "sc_qk_norm_rope_fp8", "sc_paged_cache_read_fp8", "sc_paged_attn_fp8_workspace_bytes",
           "sc_paged_attn_decode_fp8", "sc_paged_attn_prefix_workspace_bytes",
           "sc_paged_attn_prefix", "sc_paged_attn_prefix_fp8", "sc_status_string", "sc_abi_version")


class ScError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib().sc_status_string(status).decode()
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")


class sc_conv_desc(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32), ("width", ctypes.c_int32),
                ("dilation", ctypes.c_int32), ("state_len", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("x_row_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
                ("state_indices_stride", ctypes.c_int64), ("state_layout", ctypes.c_int32)]


class sc_ckpt_desc(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_int32), ("cu_ckpt", ctypes.c_void_p),
                ("ckpt_slots", ctypes.c_void_p)]


class sc_conv_fuse(ctypes.Structure):
    _fields_ = [("token_indices", ctypes.c_void_p), ("num_physical_rows", ctypes.c_int64),
                ("accumulate", ctypes.c_int32), ("outer_residual", ctypes.c_void_p),
                ("outer_row_stride", ctypes.c_int64)]


class sc_cca_desc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("t0", ctypes.c_int32),
                ("t1", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
                ("v_cur_row_stride", ctypes.c_int64), ("v_del_row_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("decode_slot_stride", ctypes.c_int64),
                ("prefill_slot_stride", ctypes.c_int64)]


class sc_gdn_desc(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
                ("qk_l2norm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
                ("v_row_stride", ctypes.c_int64), ("a_row_stride", ctypes.c_int64),
                ("b_row_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
                ("state_indices_stride", ctypes.c_int64)]


class sc_paged_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class sc_qk_norm_desc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("table_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
                ("v_row_stride", ctypes.c_int64), ("q_out_row_stride", ctypes.c_int64),
                ("k_out_row_stride", ctypes.c_int64), ("table_row_stride", ctypes.c_int64),
                ("max_position", ctypes.c_int64)]


class sc_paged_attn_desc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q_row_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("block_table_row_stride", ctypes.c_int64)]


class sc_paged_cache_fp8(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("scale_block_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64)]


class sc_cache_read_desc(ctypes.Structure):
    _fields_ = [("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("k_row_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64),
                ("block_table_row_stride", ctypes.c_int64)]


_lib = None


def lib():
    """Load libstatefulconv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        # torch first: it carries its own HIP runtime, and the library must
        # bind to that one (loaded first, the library would pull in the
        # system runtime and the process would hold two, whose device
        # pointers and streams the other does not know)
        _torch()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(sc_conv_desc)
        L.sc_conv_prefill_varlen.restype = I32
        F = ctypes.POINTER(sc_conv_fuse)
        L.sc_conv_prefill_varlen.argtypes = [D, P, P, P, P, P, I32, P, P, P, I32, I64,
                                             ctypes.POINTER(sc_ckpt_desc), F, P]
        L.sc_conv_update.restype = I32
        L.sc_conv_update.argtypes = [D, P, P, P, P, P, I32, P, P, I32, I32, F, P]
        L.sc_conv_update_spec.restype = I32
        L.sc_conv_update_spec.argtypes = [D, P, P, P, P, P, I32, P, P, I32, I32, F, P]
        L.sc_conv_update_spec_varlen.restype = I32
        L.sc_conv_update_spec_varlen.argtypes = [D, P, P, P, P, P, I32, P, P, P, I32, I64, I32,
                                                 F, P]
        L.sc_validate_metadata.restype = I32
        L.sc_validate_metadata.argtypes = [P, P, I64, I32, I64, I32, P]
        L.sc_state_gather.restype = I32
        L.sc_state_gather.argtypes = [P, I32, I64, P, I64, I32, P, P]
        L.sc_state_scatter.restype = I32
        L.sc_state_scatter.argtypes = [P, I64, P, I64, I32, P, I32, P]
        L.sc_cca_qk_conv.restype = I32
        L.sc_cca_qk_conv.argtypes = [ctypes.POINTER(sc_cca_desc), P, P, P, P, P, P, P,
                                     P, P, P, P, P, I32, I32, P, I32, P, P, P, I64, P]
        G = P     # a descriptor's address, or its bytes
        L.sc_gdn_workspace_bytes.restype = I32
        L.sc_gdn_workspace_bytes.argtypes = [G, I32, I64, ctypes.POINTER(I64)]
        L.sc_gdn_prefill_varlen.restype = I32
        L.sc_gdn_prefill_varlen.argtypes = [G, P, P, P, P, P, P, P, P, P, I32, P, P, P, I32,
                                            I64, P, I64, P]
        L.sc_gdn_update.restype = I32
        L.sc_gdn_update.argtypes = [G, P, P, P, P, P, P, P, P, P, I32, P, P, I32, I32, P]
        L.sc_gdn_update_spec.restype = I32
        L.sc_gdn_update_spec.argtypes = [G, P, P, P, P, P, P, P, P, P, I32, P, P, I32, I32, P]
        PC = PA = P
        L.sc_qk_norm_rope.restype = I32
        L.sc_qk_norm_rope.argtypes = [P, P, P, P, P, P, P, P, P, P,
                                      P, PC, PC, I64, P]
        L.sc_paged_attn_workspace_bytes.restype = I32
        L.sc_paged_attn_workspace_bytes.argtypes = [PA, I32, I32, I32, ctypes.POINTER(I64)]
        L.sc_paged_attn_decode.restype = I32
        L.sc_paged_attn_decode.argtypes = [PA, P, P, PC, PC, P, I32, P, I32, I32, I32, P, I64, P]
        L.sc_qk_norm_rope_fp8.restype = I32
        L.sc_qk_norm_rope_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, P, PC, PC, I64, P]
        L.sc_paged_cache_read_fp8.restype = I32
        L.sc_paged_cache_read_fp8.argtypes = [P, PC, PC, P, P, P, I32, P, P, I32, I64, P]
        L.sc_paged_attn_fp8_workspace_bytes.restype = I32
        L.sc_paged_attn_fp8_workspace_bytes.argtypes = [PA, I32, I32, I32, ctypes.POINTER(I64)]
        L.sc_paged_attn_decode_fp8.restype = I32
        L.sc_paged_attn_decode_fp8.argtypes = [PA, P, P, PC, PC, P, I32, P, I32, I32, I32, P, I64,
                                               P]
        L.sc_paged_attn_prefix_workspace_bytes.restype = I32
        L.sc_paged_attn_prefix_workspace_bytes.argtypes = [PA, I32, I32, I32, I32, I32,
                                                           ctypes.POINTER(I64)]
        for name in ("sc_paged_attn_prefix", "sc_paged_attn_prefix_fp8"):
            fn = getattr(L, name)
            fn.restype = I32
            fn.argtypes = [PA, P, P, PC, PC, P, I32, P, P, P, I32, I32, I32, I32, I32, P, I64, P]
        L.sc_status_string.restype = ctypes.c_char_p
        L.sc_status_string.argtypes = [I32]
        L.sc_abi_version.restype = I32
        L.sc_abi_version.argtypes = []
        if L.sc_abi_version() != SC_ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI version {L.sc_abi_version()}, the binding "
                               f"expects {SC_ABI_VERSION}: rebuild the library")
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
_torch_mod = None
_dtype_codes = None


def _torch():
    global _torch_mod
    if _torch_mod is None:
        import torch
        _torch_mod = torch
    return _torch_mod


def _ptr(t) -> Optional[int]:
    """Device address of a tensor (None passes through). Every tensor argument
    is read or written by a kernel, so a host tensor is rejected here rather
    than handed to the GPU as an address."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"expected a tensor on the GPU, got one on {t.device}")
    return t.data_ptr()


def _stream(stream, like=None) -> Optional[int]:
    """Raw HIP stream: the given one, else torch's current stream on the device
    of tensor `like` (or the current device)."""
    torch = _torch()
    if like is not None and not like.is_cuda:
        raise ValueError(f"expected a tensor on the GPU, got one on {like.device}")
    cur = torch.cuda.current_device()
    if like is not None and like.get_device() != cur:
        # the library launches on the current device
        raise ValueError(f"tensors are on cuda:{like.get_device()} but the current device is "
                         f"cuda:{cur}; call under torch.cuda.device({like.get_device()})")
    if stream is not None:
        if getattr(stream, "device_index", cur) != cur:
            raise ValueError(f"the stream is on cuda:{stream.device_index} but the current device "
                             f"is cuda:{cur}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(cur)


def _dtype_code(t) -> int:
    global _dtype_codes
    if _dtype_codes is None:
        torch = _torch()
        _dtype_codes = {torch.bfloat16: SC_DTYPE_BF16, torch.float32: SC_DTYPE_F32}
    return _dtype_codes.get(t.dtype, -1)


def _rows(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    if t.numel() == 0:
        return t.shape[1]        # no rows to address (zero-work calls are no-ops)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected a 2-D tensor with unit channel stride")
    # with at most one row the row stride is never used
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _index_stride(t, name) -> int:
    """Row stride of int32 slot indices: 1-D, or 2-D whose column 0 holds the slot."""
    torch = _torch()
    if t.dtype != torch.int32:
        raise ValueError(f"{name}: expected int32")
    if t.dim() not in (1, 2):
        raise ValueError(f"{name}: expected a 1-D or 2-D tensor")
    # with at most one row the stride is never used (empty tensors may report 0)
    return t.stride(0) if t.shape[0] > 1 else 1


def _index(t, name) -> Tuple[int, int]:
    return _ptr(t), _index_stride(t, name)


def _flags(t, name):
    torch = _torch()
    if t is None:
        return None
    if t.dtype not in (torch.bool, torch.uint8) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous bool/uint8 tensor")
    return _ptr(t)


def _check(fn: str, status: int):
    if status != SC_OK:
        raise ScError(fn, status)


def _fuse(x, out, token_indices, accumulate, outer_residual):
    """The optional residual-fusion / row-map descriptor (None = plain call)."""
    if token_indices is None and not accumulate and outer_residual is None:
        return None
    torch = _torch()
    if token_indices is not None and (token_indices.dtype != torch.int32 or
                                      not token_indices.is_contiguous()):
        raise ValueError("token_indices: expected a contiguous int32 tensor")
    if outer_residual is not None and (outer_residual.shape[0] != out.shape[0] or
                                       outer_residual.dtype != x.dtype):
        raise ValueError("outer_residual: expected as many rows as out, in x's dtype")
    if token_indices is not None and out.shape[0] != x.shape[0]:
        raise ValueError("with token_indices, x and out are the full batch tensors")
    return ctypes.byref(sc_conv_fuse(
        token_indices=_ptr(token_indices), num_physical_rows=x.shape[0],
        accumulate=1 if accumulate else 0, outer_residual=_ptr(outer_residual),
        outer_row_stride=0 if outer_residual is None else _rows(outer_residual, "outer_residual")))


def _covers(batch, **tensors):
    """Per-request arrays (slots, flags, counts) must hold at least `batch`
    entries: the kernels read entry r for every request r."""
    for name, t in tensors.items():
        if t is not None and t.shape[0] < batch:
            raise ValueError(f"{name}: {t.shape[0]} entries for {batch} requests")


def _conv_desc(x, out, weight, state_pool, dilation, activation, state_indices,
               state_layout="ds", bias=None):
    C = x.shape[1]
    K = weight.shape[-1]
    act = {"silu": SC_ACT_SILU, "none": SC_ACT_NONE, None: SC_ACT_NONE}[activation]
    # one dtype for every float tensor: the library reads them all as x's
    for name, t in (("out", out), ("weight", weight), ("bias", bias),
                    ("state_pool", state_pool)):
        if t is not None and t.dtype != x.dtype:
            raise ValueError(f"{name}: dtype {t.dtype} differs from x's {x.dtype}")
    if out.dim() != 2 or out.shape[1] != C or out.shape[0] < x.shape[0]:
        raise ValueError("out: expected at least as many (rows, C) as x")
    if weight.numel() != C * K or not weight.is_contiguous():
        raise ValueError("weight: expected a contiguous (C, K) or (C, 1, K) tensor")
    if bias is not None and (bias.numel() != C or not bias.is_contiguous()):
        raise ValueError("bias: expected a contiguous tensor of C entries")
    sd = {"ds": False, "sd": True}[state_layout]
    if not state_pool.is_contiguous() or state_pool.dim() != 3 or \
            state_pool.shape[2 if sd else 1] != C:
        raise ValueError("state_pool: expected a contiguous (num_slots, C, S) tensor, or "
                         "(num_slots, S, C) with state_layout='sd'")
    sst = _index_stride(state_indices, "state_indices")
    return sc_conv_desc(channels=C, width=K, dilation=dilation,
                        state_len=state_pool.shape[1 if sd else 2], dtype=_dtype_code(x),
                        activation=act, x_row_stride=_rows(x, "x"),
                        out_row_stride=_rows(out, "out"), state_indices_stride=sst,
                        state_layout=SC_STATE_SD if sd else SC_STATE_DS)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def sc_conv_prefill_varlen(x, out, weight, bias, state_pool, query_start_loc,
                           state_indices, has_initial_state, *, dilation: int = 1,
                           activation: Optional[str] = "silu", ckpt=None, token_indices=None,
                           accumulate: bool = False, outer_residual=None,
                           state_layout: str = "ds", stream=None):
    """Varlen prefill conv; updates ``state_pool`` in place.

    x, out: (num_tokens, C); weight (C, K); bias (C) or None; state_pool
    (num_slots, C, S), S >= (K-1)*dilation (window in the first (K-1)*dilation
    entries of each row); query_start_loc int32 (B+1);
    state_indices int32 (B) or (B, n) using column 0; has_initial_state
    bool/uint8 (B); ckpt = None or (grid, cu_ckpt int32 (B+1), ckpt_slots int32).
    token_indices (int32, one per logical row) maps the call's rows to rows of
    x / out / outer_residual; accumulate adds the result to out's contents;
    outer_residual is added too.
    """
    desc = _conv_desc(x, out, weight, state_pool, dilation, activation, state_indices,
                      state_layout, bias)
    _covers(query_start_loc.shape[0] - 1, state_indices=state_indices,
            has_initial_state=has_initial_state)
    cd = None
    if ckpt is not None:
        grid, cu, slots = ckpt
        if grid:
            _covers(query_start_loc.shape[0], cu_ckpt=cu)
        cd = ctypes.byref(sc_ckpt_desc(grid=grid, cu_ckpt=_ptr(cu), ckpt_slots=_ptr(slots)))
    st = lib().sc_conv_prefill_varlen(
        ctypes.byref(desc), _ptr(x), _ptr(out), _ptr(weight), _ptr(bias),
        _ptr(state_pool), state_pool.shape[0], _ptr(query_start_loc),
        _index(state_indices, "state_indices")[0],
        _flags(has_initial_state, "has_initial_state"),
        query_start_loc.shape[0] - 1,
        x.shape[0] if token_indices is None else token_indices.shape[0], cd,
        _fuse(x, out, token_indices, accumulate, outer_residual), _stream(stream, x))
    _check("sc_conv_prefill_varlen", st)


def sc_conv_update(x, out, weight, bias, state_pool, state_indices,
                   has_initial_state=None, *, q: int = 1, dilation: int = 1,
                   activation: Optional[str] = "silu", token_indices=None,
                   accumulate: bool = False, outer_residual=None, state_layout: str = "ds",
                   stream=None):
    """Decode / multi-token update: x (B*q, C) rows, request r owns rows
    [r*q, (r+1)*q) (logical rows, mapped by token_indices when given);
    updates ``state_pool`` in place."""
    rows = x.shape[0] if token_indices is None else token_indices.shape[0]
    if rows % max(q, 1):
        raise ValueError("rows must be a multiple of q")
    desc = _conv_desc(x, out, weight, state_pool, dilation, activation, state_indices,
                      state_layout, bias)
    B = rows // q if q else 0
    _covers(B, state_indices=state_indices, has_initial_state=has_initial_state)
    st = lib().sc_conv_update(
        ctypes.byref(desc), _ptr(x), _ptr(out), _ptr(weight), _ptr(bias),
        _ptr(state_pool), state_pool.shape[0], _index(state_indices, "state_indices")[0],
        _flags(has_initial_state, "has_initial_state"), B, q,
        _fuse(x, out, token_indices, accumulate, outer_residual), _stream(stream, x))
    _check("sc_conv_update", st)


def sc_conv_update_spec(x, out, weight, bias, state_pool, state_indices, num_accepted_tokens,
                        *, q: int, dilation: int = 1, activation: Optional[str] = "silu",
                        token_indices=None, accumulate: bool = False, outer_residual=None,
                        state_layout: str = "ds", stream=None):
    """Speculative update on a rolling buffer: x (B*q, C) rows, request r owns
    rows [r*q, (r+1)*q); state_pool (num_slots, C, S) with S >= (K-1)*dilation;
    num_accepted_tokens int32 (B). Updates ``state_pool`` in place."""
    rows = x.shape[0] if token_indices is None else token_indices.shape[0]
    if q < 1 or rows % q:
        raise ValueError("rows must be a positive multiple of q")
    torch = _torch()
    if num_accepted_tokens.dtype != torch.int32 or not num_accepted_tokens.is_contiguous():
        raise ValueError("num_accepted_tokens: expected a contiguous int32 tensor")
    desc = _conv_desc(x, out, weight, state_pool, dilation, activation, state_indices,
                      state_layout, bias)
    _covers(rows // q, state_indices=state_indices, num_accepted_tokens=num_accepted_tokens)
    st = lib().sc_conv_update_spec(
        ctypes.byref(desc), _ptr(x), _ptr(out), _ptr(weight), _ptr(bias),
        _ptr(state_pool), state_pool.shape[0], _index(state_indices, "state_indices")[0],
        _ptr(num_accepted_tokens), rows // q, q,
        _fuse(x, out, token_indices, accumulate, outer_residual), _stream(stream, x))
    _check("sc_conv_update_spec", st)


def sc_conv_update_spec_varlen(x, out, weight, bias, state_pool, state_indices,
                               num_accepted_tokens, query_start_loc, *, max_query_len: int,
                               dilation: int = 1, activation: Optional[str] = "silu",
                               token_indices=None, accumulate: bool = False,
                               outer_residual=None, state_layout: str = "ds", stream=None):
    """Speculative update with a draft count per request: request r owns rows
    [query_start_loc[r], query_start_loc[r+1]) of x (int32, batch+1 entries);
    max_query_len bounds every count (<= S). Updates ``state_pool`` in place."""
    torch = _torch()
    for name, t in (("num_accepted_tokens", num_accepted_tokens),
                    ("query_start_loc", query_start_loc)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous int32 tensor")
    batch = query_start_loc.shape[0] - 1
    if batch < 0:
        raise ValueError("query_start_loc: expected batch + 1 entries")
    rows = x.shape[0] if token_indices is None else token_indices.shape[0]
    desc = _conv_desc(x, out, weight, state_pool, dilation, activation, state_indices,
                      state_layout, bias)
    _covers(batch, state_indices=state_indices, num_accepted_tokens=num_accepted_tokens)
    st = lib().sc_conv_update_spec_varlen(
        ctypes.byref(desc), _ptr(x), _ptr(out), _ptr(weight), _ptr(bias),
        _ptr(state_pool), state_pool.shape[0], _index(state_indices, "state_indices")[0],
        _ptr(num_accepted_tokens), _ptr(query_start_loc), batch, rows, max_query_len,
        _fuse(x, out, token_indices, accumulate, outer_residual), _stream(stream, x))
    _check("sc_conv_update_spec_varlen", st)


def sc_validate_metadata(query_start_loc=None, state_indices=None, *, num_tokens: int = 0,
                         num_slots: int = 0, batch: Optional[int] = None, stream=None) -> bool:
    """Host check of the device-side preconditions (syncs the stream): True if
    query_start_loc runs non-decreasing from 0 to num_tokens and the
    non-negative state indices are distinct and below num_slots."""
    torch = _torch()
    if batch is None:
        batch = (query_start_loc.shape[0] - 1) if query_start_loc is not None else \
            (state_indices.shape[0] if state_indices is not None else 0)
    if query_start_loc is not None and (query_start_loc.dtype != torch.int32 or
                                        not query_start_loc.is_contiguous()):
        raise ValueError("query_start_loc: expected a contiguous int32 tensor")
    p, s = _index(state_indices, "state_indices") if state_indices is not None else (None, 1)
    like = query_start_loc if query_start_loc is not None else state_indices
    st = lib().sc_validate_metadata(_ptr(query_start_loc), p, s, batch, num_tokens, num_slots,
                                    None if like is None else _stream(stream, like))
    if st == -2:
        return False
    _check("sc_validate_metadata", st)
    return True


def _copy_rows(state_pool, idx, dense) -> int:
    """Bytes per slot row; the pool and the dense buffer must agree on it, be
    contiguous, and the dense buffer must hold a row per index."""
    for name, t in (("state_pool", state_pool), ("dense", dense)):
        if not t.is_contiguous() or t.dim() < 1:
            raise ValueError(f"{name}: expected a contiguous tensor of rows")
    row_of = lambda t: (t.numel() // t.shape[0] if t.shape[0] else
                        math.prod(t.shape[1:])) * t.element_size()
    if row_of(state_pool) != row_of(dense):
        raise ValueError(f"state_pool rows hold {row_of(state_pool)} bytes, dense rows "
                         f"{row_of(dense)}")
    _covers(idx.shape[0], dense=dense)
    return max(row_of(dense), 1)


def sc_state_gather(state_pool, idx, dense, *, stream=None):
    """dense[i] = state_pool[idx[i]] (zeros for an index outside the pool)."""
    row = _copy_rows(state_pool, idx, dense)
    p, s = _index(idx, "idx")
    st = lib().sc_state_gather(_ptr(state_pool), state_pool.shape[0], row, p, s,
                               idx.shape[0], _ptr(dense), _stream(stream, dense))
    _check("sc_state_gather", st)


def sc_state_scatter(dense, idx, state_pool, *, stream=None):
    """state_pool[idx[i]] = dense[i] (indices outside the pool skipped)."""
    row = _copy_rows(state_pool, idx, dense)
    p, s = _index(idx, "idx")
    st = lib().sc_state_scatter(_ptr(dense), row, p, s, idx.shape[0], _ptr(state_pool),
                                state_pool.shape[0], _stream(stream, dense))
    _check("sc_state_scatter", st)


def _cca_shapes(q, k, v_cur, v_del, out, w_dw, b_dw, w_gr, b_gr, delayed_init, conv_state,
                delayed_state, nq, nkv, hd, t0, t1):
    """The CCA kernels address every tensor from the head counts and the token
    count (q's rows): each tensor must hold what they reach."""
    if nq < 1 or nkv < 1 or hd < 2 or nq % nkv or hd % 2 or t0 < 1 or t1 < 1:
        raise ValueError("expected num_q_heads a multiple of num_kv_heads, an even "
                         "head_dim and kernel widths >= 1")
    C, vd, W, n = (nq + nkv) * hd, nkv * hd // 2, (nq + 2 * nkv) * hd, t0 + t1 - 2
    T = q.shape[0] if q.dim() == 2 else -1
    for name, t, cols in (("q", q, nq * hd), ("k", k, nkv * hd), ("v_cur", v_cur, vd),
                          ("v_del", v_del, vd), ("out", out, W)):
        if t.dim() != 2 or t.shape[1] != cols or t.shape[0] != T:
            raise ValueError(f"{name}: expected ({T}, {cols}), got {tuple(t.shape)}")
    for name, t, numel in (("w_dw", w_dw, C * t0), ("b_dw", b_dw, C),
                           ("w_gr", w_gr, C * hd * t1), ("b_gr", b_gr, C),
                           ("delayed_init", delayed_init, vd)):
        if t is not None and t.numel() != numel:
            raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    slots = conv_state.shape[0] if conv_state.dim() else 0
    if conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (C, n):
        raise ValueError(f"conv_state: expected (num_slots, {C}, {n}), got "
                         f"{tuple(conv_state.shape)}")
    if delayed_state.dim() != 2 or tuple(delayed_state.shape) != (slots, vd):
        raise ValueError(f"delayed_state: expected ({slots}, {vd}), got "
                         f"{tuple(delayed_state.shape)}")


def sc_cca_qk_conv(q, k, v_cur, v_del, out, w_dw, b_dw, w_gr, b_gr, delayed_init,
                   conv_state, delayed_state, decode_slots, prefill_qsl, prefill_slots,
                   prefill_has_initial_state, *, num_q_heads: int, num_kv_heads: int,
                   head_dim: int, t0: int, t1: int, stream=None):
    """CCA q/k conv with per-request state; updates both state pools in place.

    Rows: len(decode_slots) one-token decodes, then prefills (prefill_qsl
    rebased to 0). Pass decode_slots / prefill tensors as None when absent."""
    _cca_shapes(q, k, v_cur, v_del, out, w_dw, b_dw, w_gr, b_gr, delayed_init, conv_state,
                delayed_state, num_q_heads, num_kv_heads, head_dim, t0, t1)
    nd = 0 if decode_slots is None else decode_slots.shape[0]
    npf = 0 if prefill_qsl is None else prefill_qsl.shape[0] - 1
    dp, ds = _index(decode_slots, "decode_slots") if nd else (None, 1)
    pp, ps = _index(prefill_slots, "prefill_slots") if npf else (None, 1)
    desc = sc_cca_desc(num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                       head_dim=head_dim, t0=t0, t1=t1, dtype=_dtype_code(q),
                       q_row_stride=_rows(q, "q"), k_row_stride=_rows(k, "k"),
                       v_cur_row_stride=_rows(v_cur, "v_cur"),
                       v_del_row_stride=_rows(v_del, "v_del"),
                       out_row_stride=_rows(out, "out"), decode_slot_stride=ds,
                       prefill_slot_stride=ps)
    for name, t in (("w_dw", w_dw), ("b_dw", b_dw), ("w_gr", w_gr), ("b_gr", b_gr),
                    ("conv_state", conv_state), ("delayed_state", delayed_state)):
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
    # one dtype for every float tensor: the library reads them all as q's
    for name, t in (("k", k), ("v_cur", v_cur), ("v_del", v_del), ("out", out),
                    ("w_dw", w_dw), ("b_dw", b_dw), ("w_gr", w_gr), ("b_gr", b_gr),
                    ("delayed_init", delayed_init), ("conv_state", conv_state),
                    ("delayed_state", delayed_state)):
        if t is not None and t.dtype != q.dtype:
            raise ValueError(f"{name}: dtype {t.dtype} differs from q's {q.dtype}")
    if npf:
        _covers(npf, prefill_slots=prefill_slots,
                prefill_has_initial_state=prefill_has_initial_state)
    st = lib().sc_cca_qk_conv(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v_cur), _ptr(v_del), _ptr(out),
        _ptr(w_dw), _ptr(b_dw), _ptr(w_gr), _ptr(b_gr), _ptr(delayed_init),
        _ptr(conv_state), _ptr(delayed_state), conv_state.shape[0], nd, dp, npf,
        _ptr(prefill_qsl), pp, _flags(prefill_has_initial_state, "prefill_has_initial_state"),
        q.shape[0], _stream(stream, q))
    _check("sc_cca_qk_conv", st)


# The calls below marshal a dozen small things each, and a decode step is as
# long as its marshalling: descriptors are packed as bytes, in the layout of the
# structures above, and each tensor's shape and strides are read once.
def _packer(structure) -> struct.Struct:
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    # native alignment, the end included ("0q")
    return struct.Struct("@" + "".join(codes[t] for _, t in structure._fields_) + "0q")


_GDN_DESC = _packer(sc_gdn_desc)
_QK_NORM_DESC = _packer(sc_qk_norm_desc)
_ATTN_DESC = _packer(sc_paged_attn_desc)
_CACHE_DESC = _packer(sc_paged_cache)
_CACHE_FP8_DESC = _packer(sc_paged_cache_fp8)
_CACHE_READ_DESC = _packer(sc_cache_read_desc)


def _addresses(device, *tensors):
    """Device addresses; every tensor must be on the call's device (None passes
    through)."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.get_device() != device:
            raise ValueError(f"expected a tensor on the GPU cuda:{device}, got one on {t.device}")
        else:
            out.append(t.data_ptr())
    return out


def _device(t) -> int:
    """Index of the GPU that tensor t is on."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"expected a tensor on the GPU, got one on {t.device}")
    return d


def _row_stride(t, name, width, rows, dtype) -> int:
    """Row stride of a 2-D tensor of at least `rows` rows of `width` values."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or shape[0] < rows or t.dtype != dtype:
        raise ValueError(f"{name}: expected ({rows}, {width}) of {dtype}, got {tuple(shape)} of "
                         f"{t.dtype}")
    if shape[0] == 0:
        return width             # no rows to address
    stride = t.stride()
    if stride[1] != 1 and width > 1:
        raise ValueError(f"{name}: expected a unit stride within a row")
    # with one row the row stride is never used
    return stride[0] if shape[0] > 1 else width


def _vector(t, name, n, dtype):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of {n} entries of {dtype}")


def _gdn_desc(query, key, value, a, b, A_log, dt_bias, out, state_pool, index_stride, scale,
              qk_l2norm):
    """Packed descriptor of a gated delta rule call; the heads follow from the
    pool's shape (num_slots, HV, DV, DK) and the width of query."""
    torch = _torch()
    shape = state_pool.shape
    if len(shape) != 4 or state_pool.dtype != torch.float32 or not state_pool.is_contiguous():
        raise ValueError("state_pool: expected a contiguous float32 (num_slots, HV, DV, DK) "
                         "tensor")
    _, hv, dv, dk = shape
    if query.dim() != 2:
        raise ValueError("query: expected a 2-D tensor")
    rows, kw = query.shape
    if dk < 1 or kw % dk or kw == 0:
        raise ValueError(f"query: expected rows of HK * {dk} values")
    dtype, gate = query.dtype, a.dtype
    _vector(A_log, "A_log", hv, torch.float32)
    _vector(dt_bias, "dt_bias", hv, torch.float32)
    return _GDN_DESC.pack(
        kw // dk, hv, dk, dv, _dtype_code(query), _dtype_code(a), 1 if qk_l2norm else 0,
        dk ** -0.5 if scale is None else scale, _row_stride(query, "query", kw, rows, dtype),
        _row_stride(key, "key", kw, rows, dtype),
        _row_stride(value, "value", hv * dv, rows, dtype), _row_stride(a, "a", hv, rows, gate),
        _row_stride(b, "b", hv, rows, gate), _row_stride(out, "out", hv * dv, rows, dtype),
        index_stride)


def _workspace(workspace, need, like, stream):
    """The given workspace, or a new one of `need` bytes from torch's allocator,
    in the memory of the stream that the call runs on: a block that another
    stream has freed may still be in use there, and one freed here is not
    handed out before the call has run."""
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=like.device)
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=like.device)
    if not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return workspace


def _fits(bits, **sizes):
    """Sizes that no tensor bounds: the call's C integers would cut them."""
    for name, n in sizes.items():
        if not -(1 << bits - 1) <= n < 1 << bits - 1:
            raise ValueError(f"{name}: {n} does not fit {bits} bits")


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def sc_gdn_workspace_bytes(num_tokens: int, batch: int, *, num_k_heads: int, num_v_heads: int,
                           head_k_dim: int, head_v_dim: int) -> int:
    """Bytes of workspace that sc_gdn_prefill_varlen needs for a batch of
    `batch` requests with `num_tokens` tokens in all."""
    _fits(32, batch=batch)
    _fits(64, num_tokens=num_tokens)
    kw, vw = num_k_heads * head_k_dim, num_v_heads * head_v_dim
    return _gdn_need(_GDN_DESC.pack(num_k_heads, num_v_heads, head_k_dim, head_v_dim,
                                    SC_DTYPE_BF16, SC_DTYPE_BF16, 1, 1.0, kw, kw, vw, num_v_heads,
                                    num_v_heads, vw, 1), batch, num_tokens)


def _gdn_need(desc, batch, num_tokens) -> int:
    n = ctypes.c_int64(0)
    st = lib().sc_gdn_workspace_bytes(desc, batch, num_tokens, ctypes.byref(n))
    if st != SC_OK:
        raise ScError("sc_gdn_workspace_bytes", st)
    return n.value


def sc_gdn_prefill_varlen(query, key, value, a, b, A_log, dt_bias, out, state_pool,
                          query_start_loc, state_indices, has_initial_state, *,
                          scale: Optional[float] = None, qk_l2norm: bool = True,
                          workspace=None, stream=None):
    """Gated delta rule over a varlen batch; updates ``state_pool`` in place.

    query, key: (T, HK * DK) bf16; value, out: (T, HV * DV) bf16 (column blocks
    of the conv's output rows will do); a, b: (T, HV) bf16 or fp32; A_log,
    dt_bias: (HV) fp32; state_pool: (num_slots, HV, DV, DK) fp32;
    query_start_loc int32 (B+1); state_indices int32 (B) or column 0 of (B, n);
    has_initial_state bool/uint8 (B). scale defaults to DK ** -0.5.
    workspace: None, or a tensor of sc_gdn_workspace_bytes bytes to reuse
    (one for each call that may run at the same time).
    """
    torch = _torch()
    if query_start_loc.dtype != torch.int32 or not query_start_loc.is_contiguous() or \
            query_start_loc.dim() != 1 or query_start_loc.shape[0] < 1:
        raise ValueError("query_start_loc: expected a contiguous int32 tensor of batch + 1 "
                         "entries")
    desc = _gdn_desc(query, key, value, a, b, A_log, dt_bias, out, state_pool,
                     _index_stride(state_indices, "state_indices"), scale, qk_l2norm)
    batch, T = query_start_loc.shape[0] - 1, query.shape[0]
    _covers(batch, state_indices=state_indices, has_initial_state=has_initial_state)
    _flags(has_initial_state, "has_initial_state")
    dev = _device(query)
    raw = _stream(stream, query)
    if workspace is None:
        workspace = _workspace(None, _gdn_need(desc, batch, T), query, stream)
    else:
        _workspace(workspace, 0, query, stream)
    ptr = _addresses(dev, query, key, value, a, b, A_log, dt_bias, out, state_pool,
                     query_start_loc, state_indices, has_initial_state, workspace)
    st = lib().sc_gdn_prefill_varlen(desc, *ptr[:9], state_pool.shape[0], *ptr[9:12], batch, T,
                                     ptr[12], _nbytes(workspace), raw)
    if st != SC_OK:
        raise ScError("sc_gdn_prefill_varlen", st)


def sc_gdn_update(query, key, value, a, b, A_log, dt_bias, out, state_pool, state_indices,
                  has_initial_state=None, *, q: int = 1, scale: Optional[float] = None,
                  qk_l2norm: bool = True, stream=None):
    """Gated delta rule for `q` tokens of each request (rows [r*q, (r+1)*q));
    updates ``state_pool`` in place. Tensors as for sc_gdn_prefill_varlen."""
    if q < 1 or query.shape[0] % q:
        raise ValueError("rows must be a multiple of q >= 1")
    desc = _gdn_desc(query, key, value, a, b, A_log, dt_bias, out, state_pool,
                     _index_stride(state_indices, "state_indices"), scale, qk_l2norm)
    batch = query.shape[0] // q
    _covers(batch, state_indices=state_indices, has_initial_state=has_initial_state)
    _flags(has_initial_state, "has_initial_state")
    dev = _device(query)
    ptr = _addresses(dev, query, key, value, a, b, A_log, dt_bias, out, state_pool, state_indices,
                     has_initial_state)
    st = lib().sc_gdn_update(desc, *ptr[:9], state_pool.shape[0], *ptr[9:], batch, q,
                             _stream(stream, query))
    if st != SC_OK:
        raise ScError("sc_gdn_update", st)


def sc_gdn_update_spec(query, key, value, a, b, A_log, dt_bias, out, state_pool, state_indices,
                       num_accepted_tokens, *, q: int, scale: Optional[float] = None,
                       qk_l2norm: bool = True, stream=None):
    """Speculative gated delta rule: request r has q drafts (rows [r*q, (r+1)*q))
    and q state slots, state_indices int32 (B, q). It starts from the slot of its
    last accepted draft (entry num_accepted_tokens[r] - 1; int32 (B)) and leaves
    the state after draft t in slot t's row."""
    torch = _torch()
    if q < 1 or query.shape[0] % q:
        raise ValueError("rows must be a multiple of q >= 1")
    if state_indices.dim() != 2 or state_indices.shape[1] < q or \
            (state_indices.shape[1] > 1 and state_indices.numel() and
             state_indices.stride(1) != 1):
        raise ValueError("state_indices: expected (B, q) with adjacent entries")
    if num_accepted_tokens.dtype != torch.int32 or not num_accepted_tokens.is_contiguous():
        raise ValueError("num_accepted_tokens: expected a contiguous int32 tensor")
    stride = _index_stride(state_indices, "state_indices")
    if state_indices.shape[0] <= 1:
        stride = state_indices.shape[1]      # never used; the library wants a row's length
    desc = _gdn_desc(query, key, value, a, b, A_log, dt_bias, out, state_pool, stride, scale,
                     qk_l2norm)
    batch = query.shape[0] // q
    _covers(batch, state_indices=state_indices, num_accepted_tokens=num_accepted_tokens)
    dev = _device(query)
    ptr = _addresses(dev, query, key, value, a, b, A_log, dt_bias, out, state_pool, state_indices,
                     num_accepted_tokens)
    st = lib().sc_gdn_update_spec(desc, *ptr[:9], state_pool.shape[0], *ptr[9:], batch, q,
                                  _stream(stream, query))
    if st != SC_OK:
        raise ScError("sc_gdn_update_spec", st)


def _given(t, name):
    if t is None:
        raise ValueError(f"{name}: expected a tensor")
    return t


def _paged(cache, name, blocks, block_size, nkv, hd, dtype):
    """Packed descriptor of a (num_blocks, block_size, nkv, hd) cache tensor."""
    if cache.shape != (blocks, block_size, nkv, hd) or cache.dtype != dtype:
        raise ValueError(f"{name}: expected ({blocks}, {block_size}, {nkv}, {hd}) of {dtype}")
    st = cache.stride()
    if st[3] != 1:
        raise ValueError(f"{name}: expected a unit stride in head_dim")
    # the stride of a dimension of one entry is never used
    return _CACHE_DESC.pack(cache.data_ptr(), st[0] if blocks > 1 else 0,
                            st[1] if block_size > 1 else 0, st[2] if nkv > 1 else 0)


def _paged_fp8(cache, scale, name, blocks, block_size, nkv, hd):
    """Packed descriptor of a quantised cache: codes as for _paged, and the scales'
    bytes (num_blocks, nkv, block_size)."""
    torch = _torch()
    if cache.shape != (blocks, block_size, nkv, hd) or cache.dtype != torch.float8_e4m3fn:
        raise ValueError(f"{name}_cache: expected ({blocks}, {block_size}, {nkv}, {hd}) of "
                         f"{torch.float8_e4m3fn}")
    if scale.shape != (blocks, nkv, block_size) or \
            scale.dtype not in (torch.float8_e8m0fnu, torch.uint8):
        raise ValueError(f"{name}_scale: expected ({blocks}, {nkv}, {block_size}) of "
                         f"{torch.float8_e8m0fnu} or {torch.uint8}")
    st, sc = cache.stride(), scale.stride()
    if st[3] != 1:
        raise ValueError(f"{name}_cache: expected a unit stride in head_dim")
    if sc[2] != 1 and block_size > 1:
        raise ValueError(f"{name}_scale: expected a unit stride over a block's tokens")
    # the stride of a dimension of one entry is never used
    return _CACHE_FP8_DESC.pack(
        cache.data_ptr(), st[0] if blocks > 1 else 0, st[1] if block_size > 1 else 0,
        st[2] if nkv > 1 else 0, scale.data_ptr(), sc[0] if blocks > 1 else 0,
        sc[1] if nkv > 1 else 0)


def _norm_call(name, query, key, value, q_out, k_out, q_weight, k_weight, cos_sin, positions,
               slots, k_cache, k_scale, v_cache, v_scale, head_dim, eps, interleaved, stream):
    """Marshals a norm, rotation and cache write, into either cache."""
    torch = _torch()
    if query.ndim != 2 or key.ndim != 2:
        raise ValueError("query, key: expected 2-D tensors")
    T, qw = query.shape
    kw = key.shape[1]
    if head_dim < 1 or qw % head_dim or kw % head_dim:
        raise ValueError(f"query, key: expected rows of heads of {head_dim} values")
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache, v_cache: expected both or neither")
    dtype, nkv = query.dtype, kw // head_dim
    if q_weight is not None:
        _vector(q_weight, "q_weight", head_dim, dtype)
    if k_weight is not None:
        _vector(k_weight, "k_weight", head_dim, dtype)
    kc = vc = None
    v_rs, blocks, block_size = 0, 0, 1
    if k_cache is None:
        value = slots = None
    else:
        pool = k_cache.shape
        if len(pool) != 4:
            raise ValueError("k_cache: expected (num_blocks, block_size, nkv, head_dim)")
        if value is None or slots is None:
            raise ValueError("value, slots: expected with the caches")
        blocks, block_size = pool[0], pool[1]
        if k_scale is None:
            kc = _paged(k_cache, "k_cache", blocks, block_size, nkv, head_dim, dtype)
            vc = _paged(v_cache, "v_cache", blocks, block_size, nkv, head_dim, dtype)
        else:
            kc = _paged_fp8(k_cache, k_scale, "k", blocks, block_size, nkv, head_dim)
            vc = _paged_fp8(v_cache, v_scale, "v", blocks, block_size, nkv, head_dim)
        v_rs = _row_stride(value, "value", kw, T, dtype)
        if slots.dtype != torch.int64 or slots.ndim != 1 or slots.shape[0] < T or \
                not slots.is_contiguous():
            raise ValueError(f"slots: expected a contiguous int64 tensor of {T} entries")
    rot, t_rs, top, t_code = 0, 0, 0, SC_DTYPE_F32
    if cos_sin is None:
        positions = None
    else:
        top, rot = cos_sin.shape
        t_rs, t_code = _row_stride(cos_sin, "cos_sin", rot, top, cos_sin.dtype), _dtype_code(cos_sin)
        if positions is None or positions.dtype != torch.int64 or positions.ndim != 1 or \
                positions.shape[0] < T or not positions.is_contiguous():
            raise ValueError(f"positions: expected a contiguous int64 tensor of {T} entries")
    desc = _QK_NORM_DESC.pack(
        qw // head_dim, nkv, head_dim, rot, 1 if interleaved else 0, _dtype_code(query), t_code,
        eps, block_size, blocks, _row_stride(query, "query", qw, T, dtype),
        _row_stride(key, "key", kw, T, dtype), v_rs, _row_stride(q_out, "q_out", qw, T, dtype),
        0 if k_out is None else _row_stride(k_out, "k_out", kw, T, dtype), t_rs, top)
    dev = _device(query)
    ptr = _addresses(dev, query, key, value, q_out, k_out, q_weight, k_weight, cos_sin, positions,
                     slots, k_cache, v_cache)
    if k_scale is not None:
        _addresses(dev, k_scale, v_scale)
    st = getattr(lib(), name)(desc, *ptr[:10], kc, vc, T, _stream(stream, query))
    if st != SC_OK:
        raise ScError(name, st)


def sc_qk_norm_rope(query, key, value, q_out, k_out, q_weight, k_weight, cos_sin, positions,
                    slots, k_cache, v_cache, *, head_dim: int, eps: float = 1e-6,
                    interleaved: bool = False, stream=None):
    """Norms of the query and key heads, position rotation, and the write of keys
    and values into a paged cache.

    query (T, nq * head_dim), key, value (T, nkv * head_dim) bf16 rows (column
    blocks of sc_cca_qk_conv's output rows will do); q_out like query; k_out
    like key or None; q_out = query or k_out = key work in place. q_weight,
    k_weight: (head_dim) bf16 or None. cos_sin: (positions, rotary_dim) fp32 or
    bf16, cos then sin, or None (no rotation). positions, slots: int64 (T); slot
    -1 is not written. k_cache, v_cache: (num_blocks, block_size, nkv,
    head_dim), or None for both (value and slots are then not read).
    """
    _norm_call("sc_qk_norm_rope", query, key, value, q_out, k_out, q_weight, k_weight, cos_sin,
               positions, slots, k_cache, None, v_cache, None, head_dim, eps, interleaved, stream)


def sc_qk_norm_rope_fp8(query, key, value, q_out, k_out, q_weight, k_weight, cos_sin, positions,
                        slots, k_cache, k_scale, v_cache, v_scale, *, head_dim: int,
                        eps: float = 1e-6, interleaved: bool = False, stream=None):
    """sc_qk_norm_rope into a quantised cache: k_cache, v_cache (num_blocks,
    block_size, nkv, head_dim) float8_e4m3fn, k_scale, v_scale (num_blocks, nkv,
    block_size) float8_e8m0fnu or its bytes as uint8, a power of two for each
    token's head. The other arguments are those of sc_qk_norm_rope.
    """
    _norm_call("sc_qk_norm_rope_fp8", query, key, value, q_out, k_out, q_weight, k_weight, cos_sin,
               positions, slots, _given(k_cache, "k_cache"), _given(k_scale, "k_scale"),
               _given(v_cache, "v_cache"), _given(v_scale, "v_scale"), head_dim, eps, interleaved,
               stream)


def _block_table(table, batch) -> Tuple[int, int]:
    """Row stride and row length of a block table of at least `batch` rows."""
    shape = table.shape
    if len(shape) != 2 or shape[0] < batch or table.dtype != _torch().int32:
        raise ValueError(f"block_table: expected int32 ({batch}, max_blocks)")
    rs, cs = table.stride()
    if shape[1] > 1 and cs != 1 and shape[0]:
        raise ValueError("block_table: expected adjacent entries in a row")
    return (rs if shape[0] > 1 else max(shape[1], 1)), shape[1]


def _counts(t, name, n):
    """A contiguous int32 tensor of at least n entries."""
    if t.dtype != _torch().int32 or t.dim() != 1 or t.shape[0] < n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor of {n} entries")


def sc_paged_cache_read_fp8(k_cache, k_scale, v_cache, v_scale, k_out, v_out, block_table,
                            start_loc, first_tokens=None, *, stream=None):
    """Reads tokens of requests back from a quantised cache, as bf16 rows.

    k_out, v_out (rows, nkv * head_dim) bf16: row start_loc[r] + i becomes token
    first_tokens[r] + i of request r; rows of no request are left as they were.
    start_loc int32 (B + 1); block_table int32 (B, max_blocks); first_tokens int32 (B),
    or None: from the first token on. Caches as for sc_qk_norm_rope_fp8.
    """
    torch = _torch()
    for t, name in ((k_cache, "k_cache"), (k_scale, "k_scale"), (v_cache, "v_cache"),
                    (v_scale, "v_scale"), (k_out, "k_out"), (v_out, "v_out"),
                    (block_table, "block_table"), (start_loc, "start_loc")):
        _given(t, name)
    if k_cache.dim() != 4:
        raise ValueError("k_cache: expected (num_blocks, block_size, nkv, head_dim)")
    blocks, block_size, nkv, hd = k_cache.shape
    if k_out.dim() != 2:
        raise ValueError("k_out: expected a 2-D tensor")
    if start_loc.dim() != 1 or start_loc.shape[0] < 1:
        raise ValueError("start_loc: expected a contiguous int32 tensor of batch + 1 entries")
    rows, batch = k_out.shape[0], start_loc.shape[0] - 1
    _counts(start_loc, "start_loc", batch + 1)
    t_rs, width = _block_table(block_table, batch)
    if first_tokens is not None:
        _counts(first_tokens, "first_tokens", batch)
    kc = _paged_fp8(k_cache, k_scale, "k", blocks, block_size, nkv, hd)
    vc = _paged_fp8(v_cache, v_scale, "v", blocks, block_size, nkv, hd)
    desc = _CACHE_READ_DESC.pack(
        nkv, hd, block_size, blocks, _row_stride(k_out, "k_out", nkv * hd, rows, torch.bfloat16),
        _row_stride(v_out, "v_out", nkv * hd, rows, torch.bfloat16), t_rs)
    ptr = _addresses(_device(k_cache), k_out, v_out, block_table, start_loc, first_tokens, k_scale,
                     v_cache, v_scale)
    st = lib().sc_paged_cache_read_fp8(desc, kc, vc, ptr[0], ptr[1], ptr[2], width, ptr[3], ptr[4],
                                       batch, rows, _stream(stream, k_cache))
    if st != SC_OK:
        raise ScError("sc_paged_cache_read_fp8", st)


def _workspace_need(name, desc, *sizes) -> int:
    n = ctypes.c_int64(0)
    st = getattr(lib(), name)(desc, *sizes, ctypes.byref(n))
    if st != SC_OK:
        raise ScError(name, st)
    return n.value


def _heads_desc(num_q_heads, num_kv_heads, head_dim):
    """Descriptor of these heads, for the sizes of a workspace."""
    w = num_q_heads * head_dim
    return _ATTN_DESC.pack(num_q_heads, num_kv_heads, head_dim, SC_DTYPE_BF16, 16, 1, 1.0, w, w, 1)


def sc_paged_attn_workspace_bytes(batch: int, *, q: int = 1, max_seq_len: int, num_q_heads: int,
                                  num_kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that sc_paged_attn_decode needs for these sizes on the
    current device (0 where the cache's length is not split)."""
    _fits(32, batch=batch, q=q, max_seq_len=max_seq_len)
    return _workspace_need("sc_paged_attn_workspace_bytes",
                           _heads_desc(num_q_heads, num_kv_heads, head_dim), batch, q, max_seq_len)


def sc_paged_attn_fp8_workspace_bytes(batch: int, *, q: int = 1, max_seq_len: int,
                                      num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """The same for sc_paged_attn_decode_fp8."""
    _fits(32, batch=batch, q=q, max_seq_len=max_seq_len)
    return _workspace_need("sc_paged_attn_fp8_workspace_bytes",
                           _heads_desc(num_q_heads, num_kv_heads, head_dim), batch, q, max_seq_len)


def sc_paged_attn_prefix_workspace_bytes(batch: int, *, q: int = 1, max_seq_len: int,
                                         num_groups: int, max_prefix_len: int, num_q_heads: int,
                                         num_kv_heads: int, head_dim: int) -> int:
    """The same for sc_paged_attn_prefix and sc_paged_attn_prefix_fp8."""
    _fits(32, batch=batch, q=q, max_seq_len=max_seq_len, num_groups=num_groups,
          max_prefix_len=max_prefix_len)
    return _workspace_need("sc_paged_attn_prefix_workspace_bytes",
                           _heads_desc(num_q_heads, num_kv_heads, head_dim), batch, q, max_seq_len,
                           num_groups, max_prefix_len)


def _attn_call(name, need, query, out, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens,
               max_seq_len, q, scale, workspace, stream, groups=None):
    """Marshals an attention call over either cache; `groups`: (group_start_loc,
    prefix_lens, their number, max_prefix_len) of one with shared prefixes. The checks
    stand here one after another: a decode step is as long as its marshalling."""
    torch = _torch()
    pool, shape = k_cache.shape, query.shape
    if len(pool) != 4:
        raise ValueError("k_cache: expected (num_blocks, block_size, nkv, head_dim)")
    if len(shape) != 2:
        raise ValueError("query: expected a 2-D tensor")
    (blocks, block_size, nkv, hd), (rows, qw) = pool, shape
    if hd < 1 or qw % hd or qw == 0:
        raise ValueError(f"query: expected rows of heads of {hd} values")
    if q < 1 or rows % q:
        raise ValueError("rows must be a multiple of q >= 1")
    if not 0 <= max_seq_len < 1 << 31:
        raise ValueError("max_seq_len: expected 0 .. 2^31 - 1")
    batch, dtype = rows // q, query.dtype
    table = block_table.shape
    if len(table) != 2 or table[0] < batch or block_table.dtype != torch.int32:
        raise ValueError(f"block_table: expected int32 ({batch}, max_blocks)")
    t_rs, t_cs = block_table.stride()
    if table[1] > 1 and t_cs != 1 and table[0]:
        raise ValueError("block_table: expected adjacent entries in a row")
    if seq_lens.dtype != torch.int32 or seq_lens.ndim != 1 or seq_lens.shape[0] < batch or \
            not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens: expected a contiguous int32 tensor of {batch} entries")
    desc = _ATTN_DESC.pack(
        qw // hd, nkv, hd, _dtype_code(query), block_size, blocks,
        hd ** -0.5 if scale is None else scale, _row_stride(query, "query", qw, rows, dtype),
        _row_stride(out, "out", qw, rows, dtype), t_rs if table[0] > 1 else max(table[1], 1))
    if k_scale is None:
        kc = _paged(k_cache, "k_cache", blocks, block_size, nkv, hd, dtype)
        vc = _paged(v_cache, "v_cache", blocks, block_size, nkv, hd, dtype)
    else:
        kc = _paged_fp8(k_cache, k_scale, "k", blocks, block_size, nkv, hd)
        vc = _paged_fp8(v_cache, v_scale, "v", blocks, block_size, nkv, hd)
    dev = _device(query)
    raw = _stream(stream, query)
    library = lib()
    if workspace is None:
        sizes = (batch, q, max_seq_len) if groups is None else (batch, q, max_seq_len, *groups[2:])
        n = ctypes.c_int64(0)
        st = getattr(library, need)(desc, *sizes, ctypes.byref(n))
        if st != SC_OK:
            raise ScError(need, st)
        if n.value:
            workspace = _workspace(None, n.value, query, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ptr = _addresses(dev, query, out, block_table, seq_lens, workspace, k_cache, v_cache)
    if k_scale is not None:
        _addresses(dev, k_scale, v_scale)
    if groups is None:
        st = getattr(library, name)(desc, ptr[0], ptr[1], kc, vc, ptr[2], table[1], ptr[3], batch,
                                    q, max_seq_len, ptr[4], nbytes, raw)
    else:
        starts, lens, n_groups, longest = groups
        st = getattr(library, name)(desc, ptr[0], ptr[1], kc, vc, ptr[2], table[1], ptr[3],
                                    *_addresses(dev, starts, lens), n_groups, batch, q,
                                    max_seq_len, longest, ptr[4], nbytes, raw)
    if st != SC_OK:
        raise ScError(name, st)


def sc_paged_attn_decode(query, out, k_cache, v_cache, block_table, seq_lens, *,
                         max_seq_len: int, q: int = 1, scale: Optional[float] = None,
                         workspace=None, stream=None):
    """Attention of each request's `q` newest tokens over its paged cache.

    query, out: (B * q, nq * hd) bf16, request r owning rows [r*q, (r+1)*q);
    k_cache, v_cache: (num_blocks, block_size, nkv, hd), block_size a multiple
    of 16; block_table int32 (B, max_blocks); seq_lens int32 (B), the tokens in
    the cache with the new ones last; max_seq_len bounds them. scale defaults
    to hd ** -0.5. workspace: None, or a tensor of
    sc_paged_attn_workspace_bytes bytes to reuse (one for each call that may
    run at the same time).
    """
    _attn_call("sc_paged_attn_decode", "sc_paged_attn_workspace_bytes", query, out, k_cache, None,
               v_cache, None, block_table, seq_lens, max_seq_len, q, scale, workspace, stream)


def sc_paged_attn_decode_fp8(query, out, k_cache, k_scale, v_cache, v_scale, block_table,
                             seq_lens, *, max_seq_len: int, q: int = 1,
                             scale: Optional[float] = None, workspace=None, stream=None):
    """sc_paged_attn_decode over quantised caches (as for sc_qk_norm_rope_fp8); its
    workspace has sc_paged_attn_fp8_workspace_bytes bytes."""
    _attn_call("sc_paged_attn_decode_fp8", "sc_paged_attn_fp8_workspace_bytes", query, out,
               _given(k_cache, "k_cache"), _given(k_scale, "k_scale"), _given(v_cache, "v_cache"),
               _given(v_scale, "v_scale"), block_table, seq_lens, max_seq_len, q, scale, workspace,
               stream)


def _prefix_call(name, query, out, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens,
                 group_start_loc, prefix_lens, max_seq_len, max_prefix_len, q, scale, workspace,
                 stream):
    for t, given in ((k_cache, "k_cache"), (v_cache, "v_cache"),
                     (group_start_loc, "group_start_loc"), (prefix_lens, "prefix_lens")):
        _given(t, given)
    if prefix_lens.dim() != 1:
        raise ValueError("prefix_lens: expected a 1-D tensor")
    groups = prefix_lens.shape[0]
    _counts(prefix_lens, "prefix_lens", groups)
    _counts(group_start_loc, "group_start_loc", groups + 1)
    if not 0 <= max_prefix_len < 1 << 31:
        raise ValueError("max_prefix_len: expected 0 .. 2^31 - 1")
    _attn_call(name, "sc_paged_attn_prefix_workspace_bytes", query, out, k_cache, k_scale, v_cache,
               v_scale, block_table, seq_lens, max_seq_len, q, scale, workspace, stream,
               (group_start_loc, prefix_lens, groups, max_prefix_len))


def sc_paged_attn_prefix(query, out, k_cache, v_cache, block_table, seq_lens, group_start_loc,
                         prefix_lens, *, max_seq_len: int, max_prefix_len: int, q: int = 1,
                         scale: Optional[float] = None, workspace=None, stream=None):
    """sc_paged_attn_decode for requests that share the beginning of their caches,
    which is read once for each group of them.

    group_start_loc int32 (G + 1): group g is requests [group_start_loc[g],
    group_start_loc[g+1]); prefix_lens int32 (G): their first tokens that are the
    same, at most max_prefix_len. block_table rows hold whole caches, the prefix
    first; requests too short to see the whole prefix, and those of no group, are
    taken by themselves (long ones beside large groups end sooner in a call of
    sc_paged_attn_decode). workspace: None, or a tensor of
    sc_paged_attn_prefix_workspace_bytes bytes. The other arguments are those of
    sc_paged_attn_decode.
    """
    _prefix_call("sc_paged_attn_prefix", query, out, k_cache, None, v_cache, None, block_table,
                 seq_lens, group_start_loc, prefix_lens, max_seq_len, max_prefix_len, q, scale,
                 workspace, stream)


def sc_paged_attn_prefix_fp8(query, out, k_cache, k_scale, v_cache, v_scale, block_table,
                             seq_lens, group_start_loc, prefix_lens, *, max_seq_len: int,
                             max_prefix_len: int, q: int = 1, scale: Optional[float] = None,
                             workspace=None, stream=None):
    """sc_paged_attn_prefix over quantised caches (as for sc_qk_norm_rope_fp8)."""
    _prefix_call("sc_paged_attn_prefix_fp8", query, out, k_cache, _given(k_scale, "k_scale"),
                 v_cache, _given(v_scale, "v_scale"), block_table, seq_lens, group_start_loc,
                 prefix_lens, max_seq_len, max_prefix_len, q, scale, workspace, stream)


__all__ = ["lib", "ScError", "LIB_PATH", "EXPORTS", "sc_conv_desc", "sc_ckpt_desc",
           "sc_cca_desc", "sc_conv_fuse", "sc_gdn_desc", "sc_qk_norm_desc", "sc_paged_cache",
           "sc_paged_attn_desc", "sc_conv_prefill_varlen", "sc_conv_update",
           "sc_conv_update_spec", "sc_conv_update_spec_varlen", "sc_validate_metadata",
           "sc_state_gather", "sc_state_scatter", "sc_cca_qk_conv", "sc_gdn_workspace_bytes",
           "sc_gdn_prefill_varlen", "sc_gdn_update", "sc_gdn_update_spec", "sc_qk_norm_rope",
           "sc_paged_attn_workspace_bytes", "sc_paged_attn_decode", "sc_paged_cache_fp8",
           "sc_cache_read_desc", "sc_qk_norm_rope_fp8", "sc_paged_cache_read_fp8",
           "sc_paged_attn_fp8_workspace_bytes", "sc_paged_attn_decode_fp8",
           "sc_paged_attn_prefix_workspace_bytes", "sc_paged_attn_prefix",
           "sc_paged_attn_prefix_fp8"]
