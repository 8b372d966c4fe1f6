"""ctypes binding of libkvarn.so (include/kvarn.h): argument marshalling only.

Every function takes torch CUDA tensors, checks dtypes and shapes, passes raw
pointers and the current CUDA stream to the C ABI, and raises KVarNError on a
non-zero status. There is no fallback: if the library is missing the first
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvarn.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kvarn.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE = 0, -1, -2, -3, -4
DEVERR_BLOCK_ID, DEVERR_POSITION, DEVERR_NONFINITE, DEVERR_WAIT_TIMEOUT = 0x1, 0x2, 0x4, 0x8
BF16, FP32 = 0, 1
KIND_K, KIND_V = 0, 1
FLAG_NO_ROTATION, FLAG_NO_TOKEN_PASS, FLAG_NO_CHANNEL_PASS = 0x1, 0x2, 0x4
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
FLAG_TEST_WAIT_TIMEOUT = 0x100   # test only: the decode kernel's first copy waits give up at once


class KVarNError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({status_string(status)})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("varn_iters", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("sign_bits", ctypes.c_uint32 * 4), ("flags", ctypes.c_uint32)]


class Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("turns", ctypes.c_uint64 * 64)]


def make_config(n_q_heads: int, n_kv_heads: int, block_size: int, varn_iters: int,
                sign_bits: Sequence[int], sm_scale: float = 0.0, head_dim: int = 128,
                group_size: int = 32, bits: int = 2, flags: int = 0) -> Config:
    c = Config()
    c.flags = flags
    c.head_dim, c.block_size, c.group_size, c.bits = head_dim, block_size, group_size, bits
    c.varn_iters, c.n_q_heads, c.n_kv_heads, c.sm_scale = varn_iters, n_q_heads, n_kv_heads, sm_scale
    for i in range(4):
        c.sign_bits[i] = int(sign_bits[i]) & 0xFFFFFFFF
    return c


_lib = None
_vp = ctypes.c_void_p
_i32, _i64, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_cfgp = ctypes.POINTER(Config)

_SIGS = {
    "kvarn_version": (ctypes.c_char_p, []),
    "kvarn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kvarn_head_block_bytes": (_sz, [_cfgp]),
    "kvarn_block_bytes": (_sz, [_cfgp]),
    "kvarn_staging_bytes": (_sz, [_cfgp, _i32]),
    "kvarn_workspace_bytes": (_sz, [_cfgp, _i32, _i32]),
    "kvarn_prefill_workspace_bytes": (_sz, [_cfgp, _i32, _i32, _i32]),
    "kvarn_quantize_block": (ctypes.c_int, [_cfgp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "kvarn_append": (ctypes.c_int, [_cfgp, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "kvarn_rope_init": (ctypes.c_int, [ctypes.POINTER(Rope), _i32, _i32, ctypes.POINTER(ctypes.c_double),
                                       ctypes.c_float, ctypes.c_float]),
    "kvarn_append_rope": (ctypes.c_int, [_cfgp, ctypes.POINTER(Rope), _vp, _i64, _vp, _vp, _i32, _vp, _vp, _vp, _i64,
                                         _i32, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp]),
    "kvarn_append_rope_bf16": (ctypes.c_int, [_cfgp, ctypes.POINTER(Rope), _vp, _i64, _vp, _i32, _vp, _vp, _vp, _i64,
                                              _i32, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp]),
    "kvarn_decode_attn": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _vp,
                                         _sz, _vp]),
    "kvarn_prefill_attn": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _i32, _i32, _vp,
                                          _vp, _sz, _vp]),
    "kvarn_dequantize": (ctypes.c_int, [_cfgp, _i32, _vp, _vp, _i64, _i32, _vp, _vp]),
    "kvarn_decode_attn_bf16": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _i32, _vp, _i32, _vp, _vp,
                                              _sz, _vp]),
    "kvarn_decode_attn_noalloc": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _i32, _vp,
                                                 _vp, _vp]),
    "kvarn_prefix_workspace_bytes": (_sz, [_cfgp, _i32, _i32]),
    "kvarn_prefix_attn": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp,
                                         _i32, _vp, _sz, _vp]),
    "kvarn_prefix_attn_bf16": (ctypes.c_int, [_cfgp, _vp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp,
                                              _i32, _vp, _sz, _vp]),
    "kvarn_error_decomposition": (ctypes.c_int, [_cfgp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "kvarn_read_error": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]),
    "kvarn_clear_error": (ctypes.c_int, [_vp, _vp]),
}


def lib():
    """Load libkvarn.so (built by bit_kv_cache_08_gb300.build.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with bit_kv_cache_08_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_symbols() -> list:
    """Names of the functions include/kvarn.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"\b(kvarn_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().kvarn_status_string(status).decode()


def version() -> str:
    return lib().kvarn_version().decode()


def _check(status: int, what: str):
    if status != OK:
        raise KVarNError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream():
    """The current stream of the current device (a Stream object takes 3 us of a 4 us launch to make)."""
    if _raw_stream is None or _raw_device is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _need_cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ sizes

def head_block_bytes(cfg: Config) -> int:
    return int(lib().kvarn_head_block_bytes(ctypes.byref(cfg)))


def block_bytes(cfg: Config) -> int:
    return int(lib().kvarn_block_bytes(ctypes.byref(cfg)))


def staging_bytes(cfg: Config, max_seqs: int) -> int:
    return int(lib().kvarn_staging_bytes(ctypes.byref(cfg), max_seqs))


def workspace_bytes(cfg: Config, batch: int, max_blocks_per_seq: int) -> int:
    return int(lib().kvarn_workspace_bytes(ctypes.byref(cfg), batch, max_blocks_per_seq))


# ------------------------------------------------------------------ buffers

def prefill_workspace_bytes(cfg: Config, batch: int, chunk: int, max_blocks_per_seq: int) -> int:
    return int(lib().kvarn_prefill_workspace_bytes(ctypes.byref(cfg), batch, chunk, max_blocks_per_seq))


def alloc_prefill_workspace(cfg: Config, batch: int, chunk: int, max_blocks_per_seq: int,
                            device="cuda") -> torch.Tensor:
    n = prefill_workspace_bytes(cfg, batch, chunk, max_blocks_per_seq)
    if n == 0:
        raise ValueError("kvarn_prefill_workspace_bytes: invalid config or sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def prefix_workspace_bytes(cfg: Config, batch: int, prefix_blocks: int) -> int:
    return int(lib().kvarn_prefix_workspace_bytes(ctypes.byref(cfg), batch, prefix_blocks))


def alloc_prefix_workspace(cfg: Config, batch: int, prefix_blocks: int, device="cuda") -> torch.Tensor:
    n = prefix_workspace_bytes(cfg, batch, prefix_blocks)
    if n == 0:
        raise KVarNError(ERR_CUDA, "kvarn_prefix_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_workspace(cfg: Config, batch: int, max_blocks_per_seq: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(cfg, batch, max_blocks_per_seq)
    if n == 0:
        raise KVarNError(ERR_CUDA, "kvarn_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_pool(cfg: Config, n_blocks: int, device="cuda") -> torch.Tensor:
    return torch.zeros(n_blocks, block_bytes(cfg), dtype=torch.uint8, device=device)


def alloc_staging(cfg: Config, max_seqs: int, device="cuda") -> torch.Tensor:
    return torch.zeros(max_seqs, cfg.n_kv_heads, 2, cfg.block_size, 128, dtype=torch.bfloat16,
                       device=device)


# ------------------------------------------------------------------ entry points

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _blocks_in(src: torch.Tensor, cfg: Config, n_head_blocks: Optional[int], block_stride: Optional[int],
               token_stride: int):
    """(n, block stride) for a source of head-blocks read from src's first
    element at the given strides (elements); n defaults to every whole block a
    contiguous src holds. Raises if block n-1 would read past src's storage."""
    B = cfg.block_size
    explicit = block_stride is not None or token_stride != 128
    if not explicit and not src.is_contiguous():
        raise ValueError("src must be contiguous unless its strides are given")
    bstride = B * 128 if block_stride is None else block_stride
    if n_head_blocks is None:
        if explicit:
            raise ValueError("n_head_blocks is required with explicit strides")
        n = src.numel() // (B * 128)
    else:
        n = n_head_blocks
    room = src.untyped_storage().nbytes() // src.element_size() - src.storage_offset()
    if n > 0 and (n - 1) * bstride + (B - 1) * token_stride + 128 > room:
        raise ValueError("src holds fewer elements than n_head_blocks blocks at these strides")
    return n, bstride


def quantize_block(cfg: Config, kind: int, src: torch.Tensor, dst_base: torch.Tensor,
                   workspace: torch.Tensor, dst_offsets: Optional[torch.Tensor] = None,
                   n_head_blocks: Optional[int] = None, block_stride: Optional[int] = None,
                   token_stride: int = 128):
    """src: contiguous bf16|fp32 values, head-block i at element i * block_stride
    (default B * 128) with token rows token_stride apart; n_head_blocks defaults
    to the whole blocks src holds. dst_base: uint8 buffer."""
    _need_cuda(dst_base, "dst_base", torch.uint8)
    if not src.is_cuda:
        raise ValueError("src must be a CUDA tensor")
    n, bstride = _blocks_in(src, cfg, n_head_blocks, block_stride, token_stride)
    if dst_offsets is not None:
        _need_cuda(dst_offsets, "dst_offsets", torch.int64)
    _check(lib().kvarn_quantize_block(ctypes.byref(cfg), kind, _ptr(src), _dtype_code(src), n, bstride,
                                      token_stride, _ptr(dst_base), _ptr(dst_offsets), _ptr(workspace),
                                      _stream()), "kvarn_quantize_block")


def append(cfg: Config, pool: torch.Tensor, staging: torch.Tensor, block_table: torch.Tensor,
           pos: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, workspace: torch.Tensor):
    _need_cuda(pool, "pool", torch.uint8)
    _need_cuda(staging, "staging", torch.bfloat16)
    _need_cuda(block_table, "block_table", torch.int32)
    _need_cuda(pos, "pos", torch.int32)
    _need_cuda(k_new, "k_new", torch.bfloat16)
    _need_cuda(v_new, "v_new", torch.bfloat16)
    batch = pos.shape[0]
    _check(lib().kvarn_append(ctypes.byref(cfg), _ptr(pool), pool.shape[0], _ptr(staging), _ptr(block_table),
                              block_table.shape[1], _ptr(pos), _ptr(k_new), _ptr(v_new), batch,
                              _ptr(workspace), _stream()), "kvarn_append")


def make_rope(inv_freq: Sequence[float], layout: int = ROPE_HALF, scale: float = 1.0, eps: float = 1e-6) -> Rope:
    """Rotary positions over the first 2 * len(inv_freq) channels of a head
    (radians per position, float64; rope_frequencies gives the usual ones),
    and the epsilon of the head norms."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.ndim != 1 or f.size > 64:
        raise ValueError("inv_freq must be a vector of at most 64 rates")
    r = Rope()
    _check(lib().kvarn_rope_init(ctypes.byref(r), 2 * f.size, layout, f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                 scale, eps), "kvarn_rope_init")
    return r


def rope_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_ctx: int = 0, low: float = 1.0, high: float = 32.0):
    """(inv_freq [rotary_dim / 2] float64, scale of cos and sin) for rates
    theta^(-2i / rotary_dim), stretched for contexts `factor` times as long:

    "none"    as they are
    "linear"  every rate divided by factor (positions interpolated)
    "ntk"     theta raised so that the slowest rate is divided by factor and the fastest is kept
    "bands"   per pair, by its turns within original_ctx: divided by factor below `low` turns, kept above
              `high`, a blend linear in the number of turns between
    "yarn"    the same with cos and sin times 0.1 ln(factor) + 1 (Peng et al. 2023, "YaRN")

    "yarn" blends by a pair's turns, as the paper writes it. A model trained with a blend linear in the pair's index
    (between the pairs of `high` and of `low` turns) has other rates in between: give make_rope that model's own.
    """
    if rotary_dim < 2 or rotary_dim % 2 or not theta > 0 or not factor >= 1.0:
        raise ValueError("rotary_dim must be even and positive, theta positive, factor at least 1")
    i = np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("ntk scaling needs two pairs")
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    f = theta ** -i
    if scaling in ("none", "ntk"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling not in ("yarn", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if original_ctx < 1 or not 0 < low < high:
        raise ValueError("yarn and bands need original_ctx and 0 < low < high")
    keep = np.clip((original_ctx * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    return f * (keep + (1 - keep) / factor), 1.0 if scaling == "bands" else 0.1 * float(np.log(factor)) + 1.0


@functools.lru_cache(maxsize=64)
def _block_bytes_of(n_kv: int, block_size: int, bits: int) -> int:
    """block_bytes, which depends on these alone (a call into the library each time: 1 us)."""
    return block_bytes(make_config(n_kv, n_kv, block_size, 1, [0, 0, 0, 0], bits=bits))


def _need_packed(cfg, pool, staging, batch: int, of: str):
    """The packed pool and the staging buffer of `batch` sequences (their device is checked with the others')."""
    n_kv, B = cfg.n_kv_heads, cfg.block_size
    try:
        _, row = pool.shape
        good = (pool.dtype is _u8 and staging.dtype is _bf16 and pool.is_contiguous() and staging.is_contiguous()
                and staging.numel() >= batch * n_kv * 256 * B and row == _block_bytes_of(n_kv, B, cfg.bits))
    except (AttributeError, TypeError, ValueError, KVarNError):
        good = False
    if not good:
        _need_cuda(pool, "pool", _u8)
        _need_cuda(staging, "staging", _bf16)
        if pool.dim() != 2 or pool.shape[1] != block_bytes(cfg):
            raise ValueError("pool must be [n_blocks][block_bytes]")
        raise ValueError(f"staging holds fewer sequences than {of}")


def _need_pages(cfg, kv_pool):
    if (not isinstance(kv_pool, torch.Tensor) or kv_pool.dtype is not _bf16 or not kv_pool.is_contiguous()
            or kv_pool.shape[1:] != (cfg.n_kv_heads, 2, cfg.block_size, 128)):
        _need_cuda(kv_pool, "kv_pool", _bf16)
        raise ValueError("kv_pool must be [n_blocks][n_kv][2][B][128]")


def _stream_of(dev: int) -> int:
    """The current stream of the current device `dev`, which the caller's tensors are on."""
    return _stream() if _raw_stream is None else _raw_stream(dev)


def _current_device() -> int:
    return torch.cuda.current_device() if _raw_device is None else _raw_device()


def _need_device(*tensors):
    """The library launches on the current device: every buffer must be on it."""
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _need_vec(t, name: str, dtype, n: int):
    _need_cuda(t, name, dtype)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")


_bf16, _i32t, _u8, _f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32


def _need_rows(t: torch.Tensor, name: str, shape: tuple):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not _bf16:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name}: the heads of a token must be contiguous")


def _refuse_append(cfg, pool, staging, block_table, pos, q, k, v, q_out, workspace, cu_tokens, rope_pos, q_weight,
                   k_weight):
    """Why _append_rope's arguments do not pass: always raises."""
    _need_cuda(block_table, "block_table", _i32t)
    _need_cuda(pos, "pos", _i32t)
    _need_cuda(workspace, "workspace", _u8)
    for t, name in ((k, "k"), (v, "v")) + (((q, "q"),) if q is not None else ()):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be [n_tokens][heads][128]")
    batch, n = pos.numel(), k.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] < batch:
        raise ValueError("block_table must be [batch][max_blocks]")
    if cu_tokens is not None:
        _need_vec(cu_tokens, "cu_tokens", _i32t, batch + 1)
    elif n != batch:
        raise ValueError("without cu_tokens there is one token per sequence")
    if rope_pos is not None:
        _need_vec(rope_pos, "rope_pos", _i32t, batch)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need_vec(w, name, _bf16, 128)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q_out is not None:
        _need_cuda(q_out, "q_out")
        _dtype_code(q_out)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
    if workspace.numel() < 256:
        raise ValueError("workspace must hold 256 bytes")
    _need_device(pool, staging, block_table, pos, cu_tokens, rope_pos, q, k, v, q_weight, k_weight, q_out, workspace)
    if q is not None and (q.dtype is not _bf16 or q.shape != (n, cfg.n_q_heads, 128) or not _heads_together(q)):
        _need_rows(q, "q", (n, cfg.n_q_heads, 128))
    if k.dtype is not _bf16 or k.shape != (n, cfg.n_kv_heads, 128) or not _heads_together(k):
        _need_rows(k, "k", (n, cfg.n_kv_heads, 128))
    _need_rows(v, "v", (n, cfg.n_kv_heads, 128))


def _heads_together(t) -> bool:
    _, s1, s2 = t.stride()
    return s2 == 1 and (s1 == 128 or t.shape[1] == 1)


def _append_rope(cfg, rope, pool, staging, block_table, pos, q, k, v, q_out, workspace, cu_tokens, rope_pos, q_weight,
                 k_weight):
    # A decode step's call takes as long as its checks, so each attribute is read
    # once (a CPU tensor's get_device() is -1) and the words for what does not
    # pass are found apart.
    dev, i32, bf16 = _current_device(), _i32t, _bf16
    args = (cfg, pool, staging, block_table, pos, q, k, v, q_out, workspace, cu_tokens, rope_pos, q_weight, k_weight)
    cu_ptr = rope_ptr = qw_ptr = kw_ptr = q_ptr = out_ptr = None
    qs, out_code = 0, BF16
    try:
        batch, (n, kh, kd), n_kv = pos.numel(), k.shape, cfg.n_kv_heads
        rows, max_blocks = block_table.shape
        ks, k1, k2 = k.stride()
        vs, v1, v2 = v.stride()
        good = (dev == pool.get_device() == block_table.get_device() == pos.get_device() == k.get_device()
                == v.get_device() == workspace.get_device()
                and block_table.dtype is i32 and pos.dtype is i32 and k.dtype is bf16 and v.dtype is bf16
                and workspace.dtype is _u8 and kh == n_kv and kd == 128 and v.shape == k.shape and rows >= batch
                and k2 == 1 and v2 == 1 and (k1 == v1 == 128 or n_kv == 1) and workspace.numel() >= 256
                and block_table.is_contiguous() and pos.is_contiguous() and workspace.is_contiguous()
                and (staging is None or staging.get_device() == dev))
        if cu_tokens is not None:
            good = (good and cu_tokens.dtype is i32 and cu_tokens.get_device() == dev and cu_tokens.numel() == batch + 1
                    and cu_tokens.is_contiguous())
            cu_ptr = cu_tokens.data_ptr()
        else:
            good = good and n == batch
        if rope_pos is not None:
            good = (good and rope_pos.dtype is i32 and rope_pos.get_device() == dev and rope_pos.numel() == batch
                    and rope_pos.is_contiguous())
            rope_ptr = rope_pos.data_ptr()
        if q_weight is not None:
            good = (good and q_weight.dtype is bf16 and q_weight.get_device() == dev and q_weight.numel() == 128
                    and q_weight.is_contiguous())
            qw_ptr = q_weight.data_ptr()
        if k_weight is not None:
            good = (good and k_weight.dtype is bf16 and k_weight.get_device() == dev and k_weight.numel() == 128
                    and k_weight.is_contiguous())
            kw_ptr = k_weight.data_ptr()
        if q is not None and q_out is not None:
            shape, n_q, out_type = q.shape, cfg.n_q_heads, q_out.dtype
            qs, q1, q2 = q.stride()
            good = (good and q.get_device() == dev == q_out.get_device() and q.dtype is bf16
                    and (out_type is bf16 or out_type is _f32) and shape == (n, n_q, 128) and q_out.shape == shape
                    and q2 == 1 and (q1 == 128 or n_q == 1) and q_out.is_contiguous())
            if out_type is _f32:
                out_code = FP32
            if n == 1:
                qs = n_q * 128
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        else:
            good = good and q is None and q_out is None
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_append(*args)
    if n == 1:   # (a single row's stride is not looked at)
        ks = vs = n_kv * 128
    tail = (block_table.data_ptr(), max_blocks, pos.data_ptr(), rope_ptr, cu_ptr, n, batch, q_ptr, k.data_ptr(),
            v.data_ptr(), qs, ks, vs, qw_ptr, kw_ptr, out_ptr, out_code, workspace.data_ptr(), _stream_of(dev))
    if staging is None:
        r = lib().kvarn_append_rope_bf16(ctypes.byref(cfg), ctypes.byref(rope), pool.data_ptr(), pool.shape[0], *tail)
        if r:
            _check(r, "kvarn_append_rope_bf16")
    else:
        r = lib().kvarn_append_rope(ctypes.byref(cfg), ctypes.byref(rope), pool.data_ptr(), pool.shape[0],
                                    staging.data_ptr(), *tail)
        if r:
            _check(r, "kvarn_append_rope")


def append_rope(cfg: Config, rope: Rope, pool: torch.Tensor, staging: torch.Tensor, block_table: torch.Tensor,
                pos: torch.Tensor, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                q_out: Optional[torch.Tensor], workspace: torch.Tensor, *, cu_tokens: Optional[torch.Tensor] = None,
                rope_pos: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                k_weight: Optional[torch.Tensor] = None):
    """One step's keys and values into the packed cache, normed and rotated on
    the way, and its queries into q_out. q [tokens][n_q][128], k and v
    [tokens][n_kv][128]: bf16, token rows at any stride that is a multiple of
    8 (columns of one projection's output). cu_tokens int32 [batch + 1]: ragged
    runs of tokens; None: one token per sequence. rope_pos int32 [batch]: the
    position of each sequence's first new token (default: pos)."""
    _need_packed(cfg, pool, staging, pos.numel(), "pos")
    _append_rope(cfg, rope, pool, staging, block_table, pos, q, k, v, q_out, workspace, cu_tokens, rope_pos, q_weight,
                 k_weight)


def append_rope_bf16(cfg: Config, rope: Rope, kv_pool: torch.Tensor, block_table: torch.Tensor, pos: torch.Tensor,
                     q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, q_out: Optional[torch.Tensor],
                     workspace: torch.Tensor, *, cu_tokens: Optional[torch.Tensor] = None,
                     rope_pos: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None):
    """append_rope into the bf16 pages [n_blocks][n_kv][2][B][128] of decode_attn_bf16."""
    _need_pages(cfg, kv_pool)
    _append_rope(cfg, rope, kv_pool, None, block_table, pos, q, k, v, q_out, workspace, cu_tokens, rope_pos, q_weight,
                 k_weight)


def decode_attn(cfg: Config, q: torch.Tensor, pool: torch.Tensor, staging: torch.Tensor,
                block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                workspace: torch.Tensor):
    _need_cuda(q, "q")
    _need_cuda(pool, "pool", torch.uint8)
    _need_cuda(staging, "staging", torch.bfloat16)
    _need_cuda(block_table, "block_table", torch.int32)
    _need_cuda(seq_lens, "seq_lens", torch.int32)
    _need_cuda(out, "out", torch.float32)
    _need_cuda(workspace, "workspace", torch.uint8)
    _check(lib().kvarn_decode_attn(ctypes.byref(cfg), _ptr(q), _dtype_code(q), _ptr(pool), pool.shape[0],
                                   _ptr(staging), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                                   q.shape[0], _ptr(out), _ptr(workspace), workspace.numel(), _stream()),
           "kvarn_decode_attn")


def prefill_attn(cfg: Config, q: torch.Tensor, pool: torch.Tensor, staging: torch.Tensor,
                 block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor):
    """q: [batch][chunk][n_q][128] (bf16|fp32) queries of each sequence's last
    chunk tokens; out: fp32 [batch][chunk][n_q][128]."""
    _need_cuda(q, "q")
    _need_cuda(pool, "pool", torch.uint8)
    _need_cuda(staging, "staging", torch.bfloat16)
    _need_cuda(block_table, "block_table", torch.int32)
    _need_cuda(seq_lens, "seq_lens", torch.int32)
    _need_cuda(out, "out", torch.float32)
    _need_cuda(workspace, "workspace", torch.uint8)
    if q.dim() != 4 or out.shape != q.shape:
        raise ValueError("q and out must be [batch][chunk][n_q][128]")
    _check(lib().kvarn_prefill_attn(ctypes.byref(cfg), _ptr(q), _dtype_code(q), _ptr(pool), pool.shape[0],
                                    _ptr(staging), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                                    q.shape[0], q.shape[1], _ptr(out), _ptr(workspace), workspace.numel(),
                                    _stream()),
           "kvarn_prefill_attn")


def decode_attn_bf16(cfg: Config, q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                     seq_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor):
    """kv_pool: bf16 [n_blocks][n_kv][2][B][128]."""
    _need_cuda(q, "q")
    _need_cuda(kv_pool, "kv_pool", torch.bfloat16)
    _need_cuda(block_table, "block_table", torch.int32)
    _need_cuda(seq_lens, "seq_lens", torch.int32)
    _need_cuda(out, "out", torch.float32)
    _need_cuda(workspace, "workspace", torch.uint8)
    _check(lib().kvarn_decode_attn_bf16(ctypes.byref(cfg), _ptr(q), _dtype_code(q), _ptr(kv_pool),
                                        kv_pool.shape[0], _ptr(block_table), block_table.shape[1],
                                        _ptr(seq_lens), q.shape[0], _ptr(out), _ptr(workspace),
                                        workspace.numel(), _stream()), "kvarn_decode_attn_bf16")


def _refuse_prefix(cfg, q, pool, staging, prefix_table, prefix_lens, block_table, seq_lens, out, workspace):
    """Why _prefix_args does not pass its arguments: always raises."""
    _need_cuda(q, "q")
    _need_cuda(out, "out")
    _dtype_code(q), _dtype_code(out)
    _need_cuda(prefix_table, "prefix_table", _i32t)
    _need_cuda(prefix_lens, "prefix_lens", _i32t)
    _need_cuda(block_table, "block_table", _i32t)
    _need_cuda(seq_lens, "seq_lens", _i32t)
    _need_cuda(workspace, "workspace", _u8)
    _need_device(pool, staging, q, out, prefix_table, prefix_lens, block_table, seq_lens, workspace)
    if q.dim() != 3 or q.shape[1:] != (cfg.n_q_heads, 128) or out.shape != q.shape:
        raise ValueError("q and out must be [batch][n_q][128]")
    raise ValueError("prefix_lens, seq_lens and block_table must have a row for each sequence of q")


def _prefix_args(cfg, q, pool, staging, prefix_table, prefix_lens, block_table, seq_lens, out, workspace):
    # (as in _append_rope: each attribute read once)
    dev, i32 = _current_device(), _i32t
    try:
        shape, q_type, out_type = q.shape, q.dtype, out.dtype
        batch, n_q, d = shape
        rows, max_blocks = block_table.shape
        n_prefix, n_workspace = prefix_table.numel(), workspace.numel()
        good = (dev == pool.get_device() == q.get_device() == out.get_device() == prefix_table.get_device()
                == prefix_lens.get_device() == block_table.get_device() == seq_lens.get_device()
                == workspace.get_device() and (staging is None or staging.get_device() == dev)
                and prefix_table.dtype is i32 and prefix_lens.dtype is i32 and block_table.dtype is i32
                and seq_lens.dtype is i32 and workspace.dtype is _u8 and (q_type is _bf16 or q_type is _f32)
                and (out_type is _bf16 or out_type is _f32) and n_q == cfg.n_q_heads and d == 128 and out.shape == shape
                and prefix_lens.numel() == batch == seq_lens.numel() and rows == batch and q.is_contiguous()
                and out.is_contiguous() and prefix_table.is_contiguous() and prefix_lens.is_contiguous()
                and block_table.is_contiguous() and seq_lens.is_contiguous() and workspace.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_prefix(cfg, q, pool, staging, prefix_table, prefix_lens, block_table, seq_lens, out, workspace)
    return (FP32 if q_type is _f32 else BF16,
            (prefix_table.data_ptr(), n_prefix, prefix_lens.data_ptr(), block_table.data_ptr(), max_blocks,
             seq_lens.data_ptr(), batch, out.data_ptr(), FP32 if out_type is _f32 else BF16, workspace.data_ptr(),
             n_workspace, _stream_of(dev)))


def prefix_attn(cfg: Config, q: torch.Tensor, pool: torch.Tensor, staging: torch.Tensor, prefix_table: torch.Tensor,
                prefix_lens: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                workspace: torch.Tensor):
    """decode_attn for a batch that shares a prefix: sequence b sees the first
    prefix_lens[b] tokens of the blocks prefix_table [prefix_blocks], then its
    own seq_lens[b] tokens. q (bf16|fp32) and out (bf16|fp32): [batch][n_q][128]."""
    _need_packed(cfg, pool, staging, seq_lens.numel(), "q")
    code, rest = _prefix_args(cfg, q, pool, staging, prefix_table, prefix_lens, block_table, seq_lens, out, workspace)
    r = lib().kvarn_prefix_attn(ctypes.byref(cfg), q.data_ptr(), code, pool.data_ptr(), pool.shape[0],
                                staging.data_ptr(), *rest)
    if r:
        _check(r, "kvarn_prefix_attn")


def prefix_attn_bf16(cfg: Config, q: torch.Tensor, kv_pool: torch.Tensor, prefix_table: torch.Tensor,
                     prefix_lens: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                     workspace: torch.Tensor):
    """prefix_attn over the bf16 pages [n_blocks][n_kv][2][B][128] of decode_attn_bf16."""
    _need_pages(cfg, kv_pool)
    code, rest = _prefix_args(cfg, q, kv_pool, None, prefix_table, prefix_lens, block_table, seq_lens, out, workspace)
    r = lib().kvarn_prefix_attn_bf16(ctypes.byref(cfg), q.data_ptr(), code, kv_pool.data_ptr(), kv_pool.shape[0], *rest)
    if r:
        _check(r, "kvarn_prefix_attn_bf16")


def decode_attn_noalloc(cfg: Config, q: torch.Tensor, pool: torch.Tensor, staging: torch.Tensor,
                        block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                        error_word: Optional[torch.Tensor] = None):
    """kvarn_decode_attn with the library's built-in scratch (no workspace):
    for callers that cannot allocate device memory."""
    _need_cuda(q, "q")
    _need_cuda(pool, "pool", torch.uint8)
    _need_cuda(staging, "staging", torch.bfloat16)
    _need_cuda(block_table, "block_table", torch.int32)
    _need_cuda(seq_lens, "seq_lens", torch.int32)
    _need_cuda(out, "out", torch.float32)
    if error_word is not None:
        _need_cuda(error_word, "error_word", torch.int32)
    _check(lib().kvarn_decode_attn_noalloc(ctypes.byref(cfg), _ptr(q), _dtype_code(q), _ptr(pool),
                                           pool.shape[0], _ptr(staging), _ptr(block_table),
                                           block_table.shape[1], _ptr(seq_lens), q.shape[0], _ptr(out),
                                           _ptr(error_word), _stream()), "kvarn_decode_attn_noalloc")


def dequantize(cfg: Config, kind: int, src_base: torch.Tensor, out: torch.Tensor, rotated: bool,
               src_offsets: Optional[torch.Tensor] = None, n_head_blocks: Optional[int] = None):
    _need_cuda(src_base, "src_base", torch.uint8)
    _need_cuda(out, "out", torch.float32)
    n = out.shape[0] if n_head_blocks is None else n_head_blocks
    if src_offsets is not None:
        _need_cuda(src_offsets, "src_offsets", torch.int64)
    _check(lib().kvarn_dequantize(ctypes.byref(cfg), kind, _ptr(src_base), _ptr(src_offsets), n,
                                  1 if rotated else 0, _ptr(out), _stream()), "kvarn_dequantize")


def error_decomposition(cfg: Config, kind: int, src: torch.Tensor, packed_base: torch.Tensor, out: torch.Tensor,
                        packed_offsets: Optional[torch.Tensor] = None, n_head_blocks: Optional[int] = None,
                        block_stride: Optional[int] = None, token_stride: int = 128):
    """src: the n head-blocks' values before quantisation, block i at element
    i * block_stride (default B * 128), token rows token_stride apart; out:
    fp32 [n][B][4] = (|x|, |x^|, |E_M|, |E_D|) per token. n defaults to
    out.shape[0]."""
    _need_cuda(packed_base, "packed_base", torch.uint8)
    _need_cuda(out, "out", torch.float32)
    if not src.is_cuda:
        raise ValueError("src must be a CUDA tensor")
    n, bstride = _blocks_in(src, cfg, out.shape[0] if n_head_blocks is None else n_head_blocks, block_stride,
                            token_stride)
    if out.numel() < n * cfg.block_size * 4:
        raise ValueError("out holds fewer than n_head_blocks x B x 4 values")
    if packed_offsets is not None:
        _need_cuda(packed_offsets, "packed_offsets", torch.int64)
    _check(lib().kvarn_error_decomposition(ctypes.byref(cfg), kind, _ptr(src), _dtype_code(src), n, bstride,
                                           token_stride, _ptr(packed_base), _ptr(packed_offsets), _ptr(out),
                                           _stream()), "kvarn_error_decomposition")


def read_error(workspace: torch.Tensor) -> int:
    code = ctypes.c_uint32(0)
    _check(lib().kvarn_read_error(_ptr(workspace), ctypes.byref(code), _stream()), "kvarn_read_error")
    return code.value


def clear_error(workspace: torch.Tensor):
    _check(lib().kvarn_clear_error(_ptr(workspace), _stream()), "kvarn_clear_error")
