"""ctypes binding of librra_gb300.so: the C entry points under the same names.

Argument marshalling only: shapes are read from the torch tensors, pointers and the
current CUDA stream are passed through, and a non-zero status raises RraError. Every
step of the decode path runs in the library's CUDA kernels; there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import _build

RRA_F32, RRA_BF16 = 0, 1
RRA_ERR_POSITION, RRA_ERR_BLOCK_ID, RRA_ERR_SEQ_LEN, RRA_ERR_TIMEOUT, RRA_ERR_WORKSPACE = 1, 2, 4, 8, 16
RRA_ERR_TOKEN, RRA_ERR_PROBS = 32, 64

_lib: Optional[ctypes.CDLL] = None

_c_int, _c_i64, _c_u64, _c_size, _c_f32, _c_f64, _vp = (ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                                         ctypes.c_size_t, ctypes.c_float, ctypes.c_double,
                                                         ctypes.c_void_p)
_SIGNATURES = {
    "rra_rope_append": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                 _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _c_int, _vp, _vp]),
    "rra_decode_attn_contig": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f32,
                                        _c_int, _vp, _c_size, _c_int, _vp, _vp]),
    "rra_decode_attn_paged": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _vp, _c_int, _c_int,
                                       _c_int, _c_int, _c_f32, _c_int, _vp, _c_size, _c_int, _vp, _vp]),
    "rra_kv_bytes": (_c_u64, [_c_int, _c_int, _c_int, _c_i64, _c_int, _c_int]),
    "rra_decode_num_splits": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int]),
    "rra_decode_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "rra_status_str": (ctypes.c_char_p, [_c_int]),
    "rra_last_cuda_error": (ctypes.c_char_p, []),
    "rra_use_device": (_c_int, [_c_int]),
    "rra_test_hold_append": (_c_int, [_c_int]),
    "rra_rope_phi": (_c_int, [_c_int, _c_f64, _vp]),
    "rra_rope_cos_sin_host": (_c_int, [_c_int, _vp, _vp]),
    "rra_rope_cos_sin": (_c_int, [_vp, _c_int, _c_int, _c_f64, _vp, _vp]),
    "rra_decode_step_contig": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int,
                                        _c_int, _c_f64, _c_int, _c_f32, _c_int, _vp, _c_size, _c_int, _vp, _vp]),
    "rra_decode_step_paged": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_int,
                                       _c_int, _c_int, _c_int, _c_f64, _c_int, _c_f32, _c_int, _vp, _c_size, _c_int,
                                       _vp, _vp]),
    "rra_rope_append_q8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int,
                                    _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _vp,
                                    _vp]),
    "rra_decode_attn_q8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _vp, _c_int, _c_int,
                                    _c_int, _vp, _c_int, _c_int, _c_int, _c_int, _c_f32, _c_int, _vp, _c_size, _vp,
                                    _vp]),
    "rra_decode_step_q8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int,
                                    _c_int, _c_int, _c_int, _vp, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int,
                                    _c_f32, _c_int, _vp, _c_size, _vp, _vp]),
    "rra_decode_q8_num_splits": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int]),
    "rra_rope_append_q4": None, "rra_decode_attn_q4": None, "rra_decode_step_q4": None,
    "rra_decode_q4_num_splits": None,
    "rra_rope_append_verify": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                        _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _c_int, _vp, _vp]),
    "rra_verify_attn": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _c_int,
                                 _c_int, _c_int, _c_int, _c_f32, _c_int, _vp, _c_size, _vp, _vp]),
    "rra_verify_step": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _c_f32, _c_int, _vp, _c_size,
                                 _vp, _vp]),
    "rra_verify_num_splits": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int]),
    "rra_verify_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "rra_prefill_attn": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _c_int,
                                  _c_int, _c_int, _c_int, _c_f32, _vp, _vp]),
    "rra_prefill_step": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp,
                                  _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _c_f32, _vp, _vp]),
    "rra_shared_prefix_attn": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _vp, _c_int, _c_int, _vp, _c_int,
                                        _c_int, _c_int, _c_int, _c_int, _c_f32, _c_int, _c_int, _vp, _c_size, _vp,
                                        _vp]),
    "rra_shared_prefix_step": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int,
                                        _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _c_f32, _c_int,
                                        _c_int, _vp, _c_size, _vp, _vp]),
    "rra_shared_prefix_append": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int,
                                          _c_int, _c_int, _c_int, _c_int, _c_int, _c_f64, _c_int, _vp, _vp]),
    "rra_accept_draft": (_c_int, [_vp, _c_i64, _c_i64, _vp, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "rra_shared_prefix_plan": (_c_int, [_c_int] * 10 + [_vp, _vp, _vp]),
}


class RraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        detail = lib().rra_status_str(status).decode()
        if status == -5:
            detail += ": " + lib().rra_last_cuda_error().decode()
        super().__init__(f"{fn} returned {status} ({detail})")
        self.status = status


def lib_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """Load the library (it must have been built; see __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB_PATH):
            raise RuntimeError(f"{_build.LIB_PATH} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        handle = ctypes.CDLL(_build.LIB_PATH)
        for name in [n for n, sig in _SIGNATURES.items() if sig is None]:   # INT4 twins of the INT8 calls
            _SIGNATURES[name] = _SIGNATURES[name.replace("_q4", "_q8")]
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RRA_BF16
    if t.dtype == torch.float32:
        return RRA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the decode kernels must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


_device_of_thread = threading.local()


def use_device_of(t: torch.Tensor) -> None:
    """Selects tensor ``t``'s device in the library for this thread."""
    dev = t.get_device()
    if getattr(_device_of_thread, "dev", None) != dev:
        _check("rra_use_device", lib().rra_use_device(dev))
        _device_of_thread.dev = dev


def _stream(stream, t: torch.Tensor) -> Optional[int]:
    """The stream handle for a call on tensor ``t``'s device (selecting that device in the
    library when the call runs on the default stream, which carries no device)."""
    use_device_of(t)
    if stream is None:  # the handle alone: torch.cuda.current_stream builds a Stream object, 2 us of a call
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(name: str, status: int) -> None:
    if status != 0:
        raise RraError(name, status)


# --------------------------------------------------------------------------- host-only helpers
def rra_kv_bytes(n_layers: int, n_kv_heads: int, head_dim: int, seq_len: int, batch: int, dtype_bytes: int) -> int:
    return int(lib().rra_kv_bytes(n_layers, n_kv_heads, head_dim, seq_len, batch, dtype_bytes))


def rra_decode_num_splits(B: int, Hq: int, Hkv: int, D: int, max_tokens: int, block_size: int,
                          num_splits: int, dtype: int) -> int:
    r = lib().rra_decode_num_splits(B, Hq, Hkv, D, max_tokens, block_size, num_splits, dtype)
    _check("rra_decode_num_splits", min(r, 0))
    return r


def rra_decode_workspace_bytes(B: int, Hq: int, D: int, splits: int) -> int:
    return int(lib().rra_decode_workspace_bytes(B, Hq, D, splits))


def rra_test_hold_append(hold: bool) -> None:
    """Test hook of the bounded-wait timeout path: while held, fused bf16 steps never release
    their append barrier, so their waits run out (~1 s) and set RRA_ERR_TIMEOUT."""
    _check("rra_test_hold_append", lib().rra_test_hold_append(1 if hold else 0))


def rra_rope_phi(head_dim: int, rope_base: float = 10000.0) -> list:
    """theta_i / 2pi (i < head_dim/2) as 96-bit fractions: [[w0, w1, w2], ...], w0 least significant."""
    buf = (ctypes.c_uint32 * (3 * (head_dim // 2) if head_dim > 0 else 1))()
    _check("rra_rope_phi", lib().rra_rope_phi(head_dim, rope_base, ctypes.cast(buf, _vp)))
    return [[int(buf[3 * i + w]) for w in range(3)] for i in range(head_dim // 2)]


def rra_rope_cos_sin_host(position: int, phi) -> tuple:
    """(cos hi, cos lo, sin hi, sin lo) of 2pi * (position * phi mod 1), by the kernels' float32 steps."""
    ph = (ctypes.c_uint32 * 3)(*[int(w) & 0xffffffff for w in phi])
    out = (ctypes.c_float * 4)()
    _check("rra_rope_cos_sin_host",
           lib().rra_rope_cos_sin_host(int(position), ctypes.cast(ph, _vp), ctypes.cast(out, _vp)))
    return tuple(float(x) for x in out)


def rra_status_str(status: int) -> str:
    return lib().rra_status_str(status).decode()


# --------------------------------------------------------------------------- device entry points
def rra_rope_cos_sin(positions: torch.Tensor, head_dim: int, rope_base: float = 10000.0, out=None,
                     stream=None) -> torch.Tensor:
    """cos hi, cos lo, sin hi, sin lo of positions[p] * theta_i on the device: float32 [n, 4, head_dim/2]."""
    if positions.dtype != torch.int32 or not positions.is_cuda or not positions.is_contiguous():
        raise ValueError("positions: a contiguous int32 CUDA tensor")
    n = positions.numel()
    if out is None:
        out = torch.empty(n, 4, head_dim // 2, dtype=torch.float32, device=positions.device)
    _check("rra_rope_cos_sin", lib().rra_rope_cos_sin(positions.data_ptr(), n, head_dim, rope_base, out.data_ptr(),
                                                      _stream(stream, positions)))
    return out


def rra_rope_append(q, k_new, v_new, positions, q_out, k_cache, v_cache, block_table=None,
                    rope_base: float = 10000.0, rope_style: int = 0, err_flag=None, stream=None) -> None:
    """RoPE on q / k_new at ``positions`` and append of rotated k and raw v into the cache.

    Contiguous cache: k_cache/v_cache [B, Hkv, max_len, D]. Paged: pools
    [num_blocks, block_size, Hkv, D] plus ``block_table`` [B, max_blocks_per_seq] int32.
    """
    B, Hq, D = q.shape
    Hkv = k_new.shape[1]
    if block_table is not None:
        num_blocks, block_size = k_cache.shape[0], k_cache.shape[1]
        mbps, max_len = block_table.shape[1], 0
    else:
        num_blocks = block_size = mbps = 0
        max_len = k_cache.shape[2]
    st = lib().rra_rope_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_cache),
                               _ptr(v_cache), _ptr(block_table), mbps, block_size, num_blocks, max_len, B, Hq, Hkv,
                               D, float(rope_base), int(rope_style), _dtype_code(q), _ptr(err_flag), _stream(stream, q))
    _check("rra_rope_append", st)


def rra_decode_attn_contig(q_rot, k_cache, v_cache, seq_lens, out, scale: float = 0.0, num_splits: int = 0,
                           workspace=None, err_flag=None, stream=None) -> None:
    """out = GQA softmax attention of q_rot over the first seq_lens[b] slots of a contiguous cache."""
    B, Hq, D = q_rot.shape
    Hkv, max_len = k_cache.shape[1], k_cache.shape[2]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_decode_attn_contig(_ptr(q_rot), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), _ptr(out), B, Hq,
                                      Hkv, D, max_len, float(scale), int(num_splits), _ptr(workspace), ws_bytes,
                                      _dtype_code(q_rot), _ptr(err_flag), _stream(stream, q_rot))
    _check("rra_decode_attn_contig", st)


def rra_decode_attn_paged(q_rot, k_pool, v_pool, block_table, seq_lens, out, scale: float = 0.0,
                          num_splits: int = 0, workspace=None, err_flag=None, stream=None) -> None:
    """out = GQA softmax attention of q_rot over each sequence's blocks of a paged pool."""
    B, Hq, D = q_rot.shape
    num_blocks, block_size, Hkv = k_pool.shape[0], k_pool.shape[1], k_pool.shape[2]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_decode_attn_paged(_ptr(q_rot), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                     block_table.shape[1], _ptr(seq_lens), block_size, num_blocks, _ptr(out), B, Hq,
                                     Hkv, D, float(scale), int(num_splits), _ptr(workspace), ws_bytes,
                                     _dtype_code(q_rot), _ptr(err_flag), _stream(stream, q_rot))
    _check("rra_decode_attn_paged", st)


def rra_decode_step_contig(q, k_new, v_new, positions, q_out, k_cache, v_cache, out, rope_base: float = 10000.0,
                           rope_style: int = 0, scale: float = 0.0, num_splits: int = 0, workspace=None,
                           err_flag=None, stream=None) -> None:
    """The whole decode step on a contiguous cache: RoPE, append at positions, attention over positions+1."""
    B, Hq, D = q.shape
    Hkv, max_len = k_cache.shape[1], k_cache.shape[2]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_decode_step_contig(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_cache),
                                      _ptr(v_cache), max_len, _ptr(out), B, Hq, Hkv, D, float(rope_base),
                                      int(rope_style), float(scale), int(num_splits), _ptr(workspace), ws_bytes,
                                      _dtype_code(q), _ptr(err_flag), _stream(stream, q))
    _check("rra_decode_step_contig", st)


def rra_decode_step_paged(q, k_new, v_new, positions, q_out, k_pool, v_pool, block_table, out,
                          rope_base: float = 10000.0, rope_style: int = 0, scale: float = 0.0, num_splits: int = 0,
                          workspace=None, err_flag=None, stream=None) -> None:
    """The whole decode step on a paged pool: RoPE, append at positions, attention over positions+1."""
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv = k_pool.shape[0], k_pool.shape[1], k_pool.shape[2]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_decode_step_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_pool),
                                     _ptr(v_pool), _ptr(block_table), block_table.shape[1], block_size, num_blocks,
                                     _ptr(out), B, Hq, Hkv, D, float(rope_base), int(rope_style), float(scale),
                                     int(num_splits), _ptr(workspace), ws_bytes, _dtype_code(q), _ptr(err_flag),
                                     _stream(stream, q))
    _check("rra_decode_step_paged", st)


# --------------------------------------------------------------------------- INT8 KV cache
def _q8_layout(codes, block_table, D: int, bits: int):
    """(block_table columns, block_size, num_blocks, max_len) of an INT8 / INT4 code cache, whose
    rows must hold D * bits / 8 bytes (one code per byte, or two)."""
    if codes.shape[-1] * codes.element_size() != D * bits // 8:
        raise ValueError(f"a {bits}-bit code cache of head dim {D} has rows of {D * bits // 8} bytes, "
                         f"got {codes.shape[-1] * codes.element_size()}")
    if block_table is not None:
        return block_table.shape[1], codes.shape[1], codes.shape[0], 0
    return 0, 0, 0, codes.shape[2]


def _qfn(name: str, bits: int):
    """The INT8 (bits 8) or INT4 (bits 4) entry point of a quantised-cache call."""
    if bits not in (8, 4):
        raise ValueError("code width must be 8 or 4 bits")
    full = name if bits == 8 else name.replace("_q8", "_q4")
    return full, getattr(lib(), full)


def rra_decode_q8_num_splits(B: int, Hq: int, Hkv: int, D: int, max_tokens: int, block_size: int, num_splits: int,
                             window: int, bits: int = 8) -> int:
    name, fn = _qfn("rra_decode_q8_num_splits", bits)
    r = fn(B, Hq, Hkv, D, max_tokens, block_size, num_splits, window)
    _check(name, min(r, 0))
    return r


def rra_rope_append_q8(q, k_new, v_new, positions, q_out, k_codes, v_codes, k_scale, v_scale, k_win=None, v_win=None,
                       block_table=None, rope_base: float = 10000.0, rope_style: int = 0, err_flag=None,
                       stream=None, bits: int = 8) -> None:
    """RoPE on bf16 q / k_new, then quantised append into the INT8 (or INT4) caches and the bf16 rings."""
    B, Hq, D = q.shape
    Hkv = k_new.shape[1]
    window = k_win.shape[2] if k_win is not None else 0
    mbps, bs, nblk, max_len = _q8_layout(k_codes, block_table, D, bits)
    name, fn = _qfn("rra_rope_append_q8", bits)
    st = fn(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_codes),
                                  _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), _ptr(k_win), _ptr(v_win), window,
                                  _ptr(block_table), mbps, bs, nblk, max_len, B, Hq, Hkv, D, float(rope_base),
                                  int(rope_style), _ptr(err_flag), _stream(stream, q))
    _check(name, st)


def rra_decode_attn_q8(q_rot, k_codes, v_codes, k_scale, v_scale, seq_lens, out, k_win=None, v_win=None,
                       block_table=None, scale: float = 0.0, num_splits: int = 0, workspace=None, err_flag=None,
                       stream=None, bits: int = 8) -> None:
    """Attention of q_rot over the INT8 cache (tokens older than the window) and the bf16 rings."""
    B, Hq, D = q_rot.shape
    Hkv = k_codes.shape[2] if block_table is not None else k_codes.shape[1]
    window = k_win.shape[2] if k_win is not None else 0
    mbps, bs, nblk, max_len = _q8_layout(k_codes, block_table, D, bits)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    name, fn = _qfn("rra_decode_attn_q8", bits)
    st = fn(_ptr(q_rot), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                                  _ptr(k_win), _ptr(v_win), window, _ptr(block_table), mbps, _ptr(seq_lens), bs, nblk,
                                  max_len, _ptr(out), B, Hq, Hkv, D, float(scale), int(num_splits), _ptr(workspace),
                                  ws_bytes, _ptr(err_flag), _stream(stream, q_rot))
    _check(name, st)


def rra_decode_step_q8(q, k_new, v_new, positions, q_out, k_codes, v_codes, k_scale, v_scale, out, k_win=None,
                       v_win=None, block_table=None, rope_base: float = 10000.0, rope_style: int = 0,
                       scale: float = 0.0, num_splits: int = 0, workspace=None, err_flag=None, stream=None,
                       bits: int = 8) -> None:
    """The whole step on an INT8 cache in one kernel: RoPE, quantised append, attention over positions + 1."""
    B, Hq, D = q.shape
    Hkv = k_new.shape[1]
    window = k_win.shape[2] if k_win is not None else 0
    mbps, bs, nblk, max_len = _q8_layout(k_codes, block_table, D, bits)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    name, fn = _qfn("rra_decode_step_q8", bits)
    st = fn(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_codes),
                                  _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), _ptr(k_win), _ptr(v_win), window,
                                  _ptr(block_table), mbps, bs, nblk, max_len, _ptr(out), B, Hq, Hkv, D,
                                  float(rope_base), int(rope_style), float(scale), int(num_splits), _ptr(workspace),
                                  ws_bytes, _ptr(err_flag), _stream(stream, q))
    _check(name, st)


# --------------------------------------------------------------------------- speculative verify
def _cache_layout(k_cache, block_table):
    """(block_table columns, block_size, num_blocks, max_len, Hkv) of a bf16 / fp32 cache."""
    if block_table is not None:
        return block_table.shape[1], k_cache.shape[1], k_cache.shape[0], 0, k_cache.shape[2]
    return 0, 0, 0, k_cache.shape[2], k_cache.shape[1]


def rra_verify_num_splits(B: int, gamma: int, Hq: int, Hkv: int, D: int, max_tokens: int, block_size: int,
                          num_splits: int) -> int:
    r = lib().rra_verify_num_splits(B, gamma, Hq, Hkv, D, max_tokens, block_size, num_splits)
    _check("rra_verify_num_splits", min(r, 0))
    return r


def rra_verify_workspace_bytes(B: int, gamma: int, Hq: int, Hkv: int, D: int, splits: int) -> int:
    return int(lib().rra_verify_workspace_bytes(B, gamma, Hq, Hkv, D, splits))


def rra_rope_append_verify(q, k_new, v_new, positions, q_out, k_cache, v_cache, block_table=None,
                           rope_base: float = 10000.0, rope_style: int = 0, err_flag=None, stream=None) -> None:
    """RoPE on q / k_new [B, gamma, H, D] (token j at positions[b] + j) and append of the gamma tokens."""
    B, gamma, Hq, D = q.shape
    mbps, bs, nblk, max_len, Hkv = _cache_layout(k_cache, block_table)
    st = lib().rra_rope_append_verify(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(block_table), mbps, bs, nblk, max_len, B, gamma, Hq, Hkv, D,
                                      float(rope_base), int(rope_style), _dtype_code(q), _ptr(err_flag),
                                      _stream(stream, q))
    _check("rra_rope_append_verify", st)


def rra_verify_attn(q_rot, k_cache, v_cache, positions, out, block_table=None, scale: float = 0.0, num_splits: int = 0,
                    workspace=None, err_flag=None, stream=None) -> None:
    """out[b, j] = attention of q_rot[b, j] over tokens [0, positions[b] + j] (bf16 caches)."""
    B, gamma, Hq, D = q_rot.shape
    mbps, bs, nblk, max_len, Hkv = _cache_layout(k_cache, block_table)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_verify_attn(_ptr(q_rot), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps, _ptr(positions), bs,
                               nblk, max_len, _ptr(out), B, gamma, Hq, Hkv, D, float(scale), int(num_splits),
                               _ptr(workspace), ws_bytes, _ptr(err_flag), _stream(stream, q_rot))
    _check("rra_verify_attn", st)


def rra_verify_step(q, k_new, v_new, positions, q_out, k_cache, v_cache, out, block_table=None,
                    rope_base: float = 10000.0, rope_style: int = 0, scale: float = 0.0, num_splits: int = 0,
                    workspace=None, err_flag=None, stream=None) -> None:
    """The whole speculative-verify step: RoPE + append of the gamma tokens, then their causal attention."""
    B, gamma, Hq, D = q.shape
    mbps, bs, nblk, max_len, Hkv = _cache_layout(k_cache, block_table)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().rra_verify_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_cache),
                               _ptr(v_cache), _ptr(block_table), mbps, bs, nblk, max_len, _ptr(out), B, gamma, Hq, Hkv,
                               D, float(rope_base), int(rope_style), float(scale), int(num_splits), _ptr(workspace),
                               ws_bytes, _ptr(err_flag), _stream(stream, q))
    _check("rra_verify_step", st)


# --------------------------------------------------------------------------- shared prefix
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _shared_layout(q, k_pool, v_pool, prefix_blocks, prefix_len: int, block_table, lens, out):
    """(B, gamma, Hq, D, num_blocks, block_size, Hkv, block-table columns) of a shared-prefix call; queries
    [B, Hq, D] are one new token per sequence. The C calls take no element types, so they are checked
    here, with the shapes."""
    shape, pool, table = q.shape, k_pool.shape, block_table.shape
    if len(shape) == 4:
        B, gamma, Hq, D = shape
    elif len(shape) == 3:
        (B, Hq, D), gamma = shape, 1
    else:
        raise ValueError("q: [B, gamma, Hq, D] or [B, Hq, D]")
    if not (q.dtype == k_pool.dtype == v_pool.dtype == out.dtype == _BF16):
        raise TypeError("shared-prefix attention takes bf16 queries, caches and outputs")
    if not block_table.dtype == lens.dtype == _I32:
        raise TypeError("block_table, seq_lens and positions are int32")
    if len(pool) != 4 or v_pool.shape != pool or pool[3] != D or out.shape != shape:
        raise ValueError("k_pool and v_pool: [num_blocks, block_size, Hkv, D]; out: the shape of q")
    if len(table) != 2 or table[0] != B or lens.numel() != B:
        raise ValueError("block_table: [B, max_blocks_per_seq]; one length or position per sequence")
    if prefix_len > 0 and (prefix_blocks is None or prefix_blocks.dtype != _I32 or
                           prefix_blocks.numel() * pool[1] < prefix_len):
        raise ValueError("prefix_blocks: int32, a block for every block_size tokens of the prefix")
    return B, gamma, Hq, D, pool[0], pool[1], pool[2], table[1]


def rra_shared_prefix_plan(B: int, gamma: int, Hq: int, Hkv: int, D: int, prefix_len: int, max_blocks_per_seq: int,
                           block_size: int, num_splits: int = 0, prefix_splits: int = 0) -> tuple:
    """(splits of the sequences' own tokens, prefix chunks, workspace bytes) of the shared-prefix calls."""
    own, chunks, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    _check("rra_shared_prefix_plan",
           lib().rra_shared_prefix_plan(B, gamma, Hq, Hkv, D, prefix_len, max_blocks_per_seq, block_size, num_splits,
                                        prefix_splits, ctypes.byref(own), ctypes.byref(chunks), ctypes.byref(ws)))
    return own.value, chunks.value, ws.value


def rra_shared_prefix_attn(q_rot, k_pool, v_pool, prefix_blocks, prefix_len: int, block_table, seq_lens, out,
                           scale: float = 0.0, num_splits: int = 0, prefix_splits: int = 0, workspace=None,
                           err_flag=None, stream=None) -> None:
    """out[b, j] = attention of q_rot[b, j] over the first seq_lens[b] - gamma + 1 + j tokens, of which the
    first prefix_len are in prefix_blocks for every sequence (read once for the batch)."""
    B, gamma, Hq, D, num_blocks, block_size, Hkv, cols = _shared_layout(q_rot, k_pool, v_pool, prefix_blocks,
                                                                        prefix_len, block_table, seq_lens, out)
    st = lib().rra_shared_prefix_attn(_ptr(q_rot), _ptr(k_pool), _ptr(v_pool), _ptr(prefix_blocks), prefix_len,
                                      _ptr(block_table), cols, _ptr(seq_lens), block_size, num_blocks, _ptr(out), B,
                                      gamma, Hq, Hkv, D, scale, num_splits, prefix_splits, _ptr(workspace),
                                      workspace.nbytes if workspace is not None else 0, _ptr(err_flag),
                                      _stream(stream, q_rot))
    if st != 0:
        raise RraError("rra_shared_prefix_attn", st)


def _new_tokens(q, k_new, v_new, q_out, Hkv: int) -> None:
    """Checks the new tokens' types and shapes beside queries that _shared_layout has looked at."""
    if not k_new.dtype == v_new.dtype == q_out.dtype == _BF16:
        raise TypeError("shared-prefix attention takes bf16 new tokens")
    if k_new.numel() * q.shape[-2] != q.numel() * Hkv or v_new.shape != k_new.shape or q_out.shape != q.shape:
        raise ValueError("k_new and v_new: [B, gamma, Hkv, D]; q_out: the shape of q")


def rra_shared_prefix_append(q, k_new, v_new, positions, q_out, k_pool, v_pool, prefix_len: int, block_table,
                             rope_base: float = 10000.0, rope_style: int = 0, err_flag=None, stream=None) -> None:
    """RoPE on q and k_new (token j at positions[b] + j) and append of the gamma new tokens, but for those at
    positions below prefix_len (a multiple of the block size), which are refused."""
    B, gamma, Hq, D, num_blocks, block_size, Hkv, cols = _shared_layout(q, k_pool, v_pool, None, 0, block_table,
                                                                        positions, q_out)
    _new_tokens(q, k_new, v_new, q_out, Hkv)
    st = lib().rra_shared_prefix_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_pool),
                                        _ptr(v_pool), prefix_len, _ptr(block_table), cols, block_size, num_blocks, B,
                                        gamma, Hq, Hkv, D, rope_base, rope_style, _ptr(err_flag), _stream(stream, q))
    if st != 0:
        raise RraError("rra_shared_prefix_append", st)


def rra_shared_prefix_step(q, k_new, v_new, positions, q_out, k_pool, v_pool, prefix_blocks, prefix_len: int,
                           block_table, out, rope_base: float = 10000.0, rope_style: int = 0, scale: float = 0.0,
                           num_splits: int = 0, prefix_splits: int = 0, workspace=None, err_flag=None,
                           stream=None) -> None:
    """RoPE + append of the gamma new tokens at positions[b] (at least prefix_len), then their attention."""
    B, gamma, Hq, D, num_blocks, block_size, Hkv, cols = _shared_layout(q, k_pool, v_pool, prefix_blocks, prefix_len,
                                                                        block_table, positions, out)
    _new_tokens(q, k_new, v_new, q_out, Hkv)
    st = lib().rra_shared_prefix_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_pool),
                                      _ptr(v_pool), _ptr(prefix_blocks), prefix_len, _ptr(block_table), cols,
                                      block_size, num_blocks, _ptr(out), B, gamma, Hq, Hkv, D, rope_base, rope_style,
                                      scale, num_splits, prefix_splits, _ptr(workspace),
                                      workspace.nbytes if workspace is not None else 0, _ptr(err_flag),
                                      _stream(stream, q))
    if st != 0:
        raise RraError("rra_shared_prefix_step", st)


# --------------------------------------------------------------------------- draft acceptance
def _i32(t, shape, what: str) -> int:
    """The pointer of a contiguous int32 tensor of this shape."""
    if t.dtype != _I32 or t.shape != shape:
        raise ValueError(f"{what}: an int32 tensor of shape {tuple(shape)}")
    return _ptr(t)


def rra_accept_draft(target_probs, draft_tokens, u_accept, u_sample, draft_probs=None, draft_lens=None,
                     positions=None, tokens_out=None, n_accepted=None, positions_out=None, err_flag=None,
                     stream=None) -> tuple:
    """(tokens [B, gamma + 1], kept [B]), and with ``positions`` the next positions [B]: the drafted tokens the
    target keeps, the one drawn after them, then -1.

    target_probs [B, gamma + 1, V] and draft_probs [B, gamma, V] (or None: a drafter without
    probabilities) are bf16 or fp32 with a unit last stride; u_accept [B, gamma] and u_sample [B] are
    uniform random numbers in [0, 1). Outputs are made where they are not given; positions_out may be
    positions.
    """
    ids = draft_tokens.shape
    B, gamma = ids
    V, dt = target_probs.shape[-1], target_probs.dtype
    code = RRA_F32 if dt == _F32 else _dtype_code(target_probs)
    if target_probs.shape != (B, gamma + 1, V):
        raise ValueError("target_probs: [B, gamma + 1, V]")
    pb, pt, p1 = target_probs.stride()
    if not target_probs.is_cuda or (p1 != 1 and V > 1):
        raise ValueError("target_probs: a CUDA tensor with a unit last stride")
    q_ptr, qb, qt = None, 0, 0
    if draft_probs is not None:
        if draft_probs.shape != (B, gamma, V) or draft_probs.dtype != dt:
            raise ValueError("draft_probs: [B, gamma, V], of target_probs' type")
        qb, qt, q1 = draft_probs.stride()
        if not draft_probs.is_cuda or (q1 != 1 and V > 1):
            raise ValueError("draft_probs: a CUDA tensor with a unit last stride")
        q_ptr = draft_probs.data_ptr()
    if not u_accept.dtype == u_sample.dtype == _F32:
        raise TypeError("u_accept and u_sample are float32")
    if u_accept.shape != ids or u_sample.shape != (B,):
        raise ValueError("u_accept: [B, gamma]; u_sample: [B]")
    row, device = (B,), target_probs.device
    if tokens_out is None:  # (made here, so not checked below: the call takes longer on the host than on the GPU)
        tokens_out = torch.empty((B, gamma + 1), dtype=_I32, device=device)
        tokens_ptr = tokens_out.data_ptr()
    else:
        tokens_ptr = _i32(tokens_out, (B, gamma + 1), "tokens_out")
    if n_accepted is None:
        n_accepted = torch.empty(row, dtype=_I32, device=device)
        kept_ptr = n_accepted.data_ptr()
    else:
        kept_ptr = _i32(n_accepted, row, "n_accepted")
    next_ptr = None
    if positions_out is not None:
        next_ptr = _i32(positions_out, row, "positions_out")
    elif positions is not None:
        positions_out = torch.empty(row, dtype=_I32, device=device)
        next_ptr = positions_out.data_ptr()
    st = lib().rra_accept_draft(
        target_probs.data_ptr(), pb, pt, q_ptr, qb, qt, _i32(draft_tokens, ids, "draft_tokens"),
        _i32(draft_lens, row, "draft_lens") if draft_lens is not None else None, _ptr(u_accept), _ptr(u_sample),
        _i32(positions, row, "positions") if positions is not None else None, tokens_ptr, kept_ptr, next_ptr, B, gamma,
        V, code, _ptr(err_flag), _stream(stream, target_probs))
    if st != 0:
        raise RraError("rra_accept_draft", st)
    return (tokens_out, n_accepted) if positions_out is None else (tokens_out, n_accepted, positions_out)


# --------------------------------------------------------------------------- prefill
def rra_prefill_attn(q_rot, k_cache, v_cache, positions, out, block_table=None, scale: float = 0.0, err_flag=None,
                     stream=None) -> None:
    """out[b, t] = causal attention of prompt token t (q_rot [B, T, Hq, D]) over tokens [0, positions[b] + t]."""
    B, T, Hq, D = q_rot.shape
    mbps, bs, nblk, max_len, Hkv = _cache_layout(k_cache, block_table)
    st = lib().rra_prefill_attn(_ptr(q_rot), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps, _ptr(positions), bs,
                                nblk, max_len, _ptr(out), B, T, Hq, Hkv, D, float(scale), _ptr(err_flag),
                                _stream(stream, q_rot))
    _check("rra_prefill_attn", st)


def rra_prefill_step(q, k_new, v_new, positions, q_out, k_cache, v_cache, out, block_table=None,
                     rope_base: float = 10000.0, rope_style: int = 0, scale: float = 0.0, err_flag=None,
                     stream=None) -> None:
    """RoPE + append of the T prompt tokens, then their causal attention."""
    B, T, Hq, D = q.shape
    mbps, bs, nblk, max_len, Hkv = _cache_layout(k_cache, block_table)
    st = lib().rra_prefill_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q_out), _ptr(k_cache),
                                _ptr(v_cache), _ptr(block_table), mbps, bs, nblk, max_len, _ptr(out), B, T, Hq, Hkv, D,
                                float(rope_base), int(rope_style), float(scale), _ptr(err_flag), _stream(stream, q))
    _check("rra_prefill_step", st)
