"""Thin ctypes binding of libpkv.so (declared in include/pkv.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors; the stream defaults to torch's
current stream.  If the library has not been built, the first call raises --
there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpkv.so")

PKV_F32, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2
ALGOS = {"auto": 0, "simt": 1, "mma": 2, "tc": 3}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace", 4: "cuda error",
          5: "device bounds", 6: "out of blocks", 7: "inconsistent"}
ERRBIT_BLOCK_ID, ERRBIT_SLOT, ERRBIT_SEQ_LEN, ERRBIT_TIMEOUT = 1, 2, 4, 8
ERRBIT_POSITION, ERRBIT_STEP, ERRBIT_GROUP, ERRBIT_OFFSETS = 16, 32, 64, 128

# Every symbol include/pkv.h declares.
EXPORTS = ("kv_pool_create", "kv_pool_destroy", "kv_pool_tensor_bytes", "kv_bytes_per_token",
           "kv_append", "paged_decode_plan", "paged_decode_algo", "paged_decode_attention",
           "paged_multi_query_plan", "paged_multi_query_algo", "paged_multi_query_attention",
           "paged_decode_append_attention",
           "paged_prefix_decode_plan", "paged_prefix_decode_algo", "paged_prefix_decode_attention",
           "kv_append_norm_rope", "kv_tables_grow", "kv_tables_release",
           "kv_quant_pool_create", "kv_quant_pool_destroy", "kv_quant_pool_bytes", "kv_quant_append", "kv_read",
           "kv_quant_read", "paged_quant_decode_plan", "paged_quant_decode_attention", "prompt_attention_plan",
           "prompt_attention",
           "paged_decode_attention_static_ws", "pkv_set_first_wait_limit_for_testing", "pkv_status_string",
           "pkv_last_cuda_error",
           "kv_block_manager_create", "kv_block_manager_destroy", "kv_bm_num_free", "kv_bm_add_sequence",
           "kv_bm_free_sequence", "kv_bm_grow", "kv_bm_decode_slots", "kv_bm_match_prefix", "kv_bm_seq_len",
           "kv_bm_block_tables", "kv_bm_free_list", "kv_bm_block_ref", "kv_bm_check")
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024
ALGO_NAMES = {1: "simt", 2: "mma", 3: "tc"}


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = "%s failed: %s" % (what, STATUS.get(status, str(status)))
        if status == 4 and _lib is not None:
            msg += " (%s)" % _lib.pkv_last_cuda_error().decode()
        super().__init__(msg)


class PoolDesc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kv_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("k_base", ctypes.c_void_p), ("v_base", ctypes.c_void_p),
                ("error_word", ctypes.c_void_p)]


class NormRopeDesc(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 3),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


class QuantPoolDesc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_params", ctypes.c_void_p),
                ("v_params", ctypes.c_void_p), ("error_word", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpkv.so (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libpkv.so is not built (run __graft_entry__.build() or "
                           "python -m paged_kv_cache_194_gb300.build); no fallback exists")
    L = ctypes.CDLL(LIB_PATH)
    c, P = ctypes, ctypes.c_void_p
    L.kv_pool_create.restype = c.c_int
    L.kv_pool_create.argtypes = [c.POINTER(PoolDesc), c.POINTER(P)]
    L.kv_pool_destroy.restype = None
    L.kv_pool_destroy.argtypes = [P]
    L.kv_pool_tensor_bytes.restype = c.c_size_t
    L.kv_pool_tensor_bytes.argtypes = [c.POINTER(PoolDesc)]
    L.kv_bytes_per_token.restype = c.c_int64
    L.kv_bytes_per_token.argtypes = [c.c_int32, c.c_int32, c.c_int32, c.c_int]
    L.kv_append.restype = c.c_int
    L.kv_append.argtypes = [P, c.c_int32, P, P, c.c_int, P, c.c_int32, P]
    L.paged_decode_plan.restype = c.c_int
    L.paged_decode_plan.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
                                    c.POINTER(c.c_int32), c.POINTER(c.c_int32), c.POINTER(c.c_size_t)]
    L.paged_decode_attention.restype = c.c_int
    L.paged_decode_attention.argtypes = [P, c.c_int, P, c.c_int32, P, c.c_int32, P, c.c_int32,
                                         c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int, P,
                                         c.c_size_t, P, P]
    L.paged_multi_query_plan.restype = c.c_int
    L.paged_multi_query_plan.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int32,
                                         c.POINTER(c.c_int32), c.POINTER(c.c_int32), c.POINTER(c.c_size_t)]
    L.paged_multi_query_attention.restype = c.c_int
    L.paged_multi_query_attention.argtypes = [P, c.c_int, P, c.c_int32, P, c.c_int32, P, c.c_int32, c.c_int32,
                                              c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int, P,
                                              c.c_size_t, P, P]
    L.paged_multi_query_algo.restype = c.c_int32
    L.paged_multi_query_algo.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.c_int]
    L.paged_decode_append_attention.restype = c.c_int
    L.paged_decode_append_attention.argtypes = [P, c.c_int, P, P, c.c_int, P, c.c_int32, P, c.c_int32, P,
                                                c.c_int32, c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int,
                                                P, c.c_size_t, P, P]
    L.paged_decode_attention_static_ws.restype = c.c_int
    L.paged_decode_attention_static_ws.argtypes = [P, c.c_int, P, c.c_int32, P, c.c_int32, P, c.c_int32,
                                                   c.c_int32, c.c_int32, c.c_float, c.c_int32, c.c_int, P, P]
    L.paged_decode_algo.restype = c.c_int32
    L.paged_decode_algo.argtypes = [P, c.c_int32, c.c_int]
    L.paged_prefix_decode_plan.restype = c.c_int
    L.paged_prefix_decode_plan.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.POINTER(c.c_size_t)]
    L.paged_prefix_decode_algo.restype = c.c_int32
    L.paged_prefix_decode_algo.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int]
    L.paged_prefix_decode_attention.restype = c.c_int
    L.paged_prefix_decode_attention.argtypes = [P, c.c_int, P, c.c_int32, P, c.c_int32, P, c.c_int32, c.c_int32,
                                                c.c_int32, P, P, c.c_int32, c.c_float, c.c_int, P, c.c_size_t, P, P]
    L.kv_append_norm_rope.restype = c.c_int
    L.kv_append_norm_rope.argtypes = [P, c.c_int32, P, P, P, c.c_int, c.c_int64, c.c_int64, c.c_int64, P, P,
                                      c.c_int32, c.c_int32, c.POINTER(NormRopeDesc), P, P]
    L.kv_tables_grow.restype = c.c_int
    L.kv_tables_grow.argtypes = [P, P, c.c_int32, P, P, c.c_int32, P, c.c_int32, P, c.c_int32, P, P, P, P, P, P, P, P]
    L.kv_tables_release.restype = c.c_int
    L.kv_tables_release.argtypes = [P, P, c.c_int32, P, P, P, c.c_int32, P, c.c_int32, P, P, P, P]
    L.kv_quant_pool_create.restype = c.c_int
    L.kv_quant_pool_create.argtypes = [c.POINTER(QuantPoolDesc), c.POINTER(P)]
    L.kv_quant_pool_destroy.restype = None
    L.kv_quant_pool_destroy.argtypes = [P]
    L.kv_quant_pool_bytes.restype = c.c_int
    L.kv_quant_pool_bytes.argtypes = [c.POINTER(QuantPoolDesc), c.POINTER(c.c_size_t), c.POINTER(c.c_size_t)]
    L.kv_quant_append.restype = c.c_int
    L.kv_quant_append.argtypes = [P, c.c_int32, P, P, c.c_int, c.c_int64, c.c_int64, P, c.c_int32, P]
    for read in (L.kv_read, L.kv_quant_read):
        read.restype = c.c_int
        read.argtypes = [P, c.c_int32, P, c.c_int32, P, c.c_int32, c.c_int32, P, P, P]
    L.paged_quant_decode_plan.restype = c.c_int
    L.paged_quant_decode_plan.argtypes = [P, c.c_int32, c.c_int32, c.c_int32, c.POINTER(c.c_size_t)]
    L.paged_quant_decode_attention.restype = c.c_int
    L.paged_quant_decode_attention.argtypes = [P, c.c_int, P, c.c_int32, P, c.c_int32, P, c.c_int32, c.c_int32,
                                               c.c_int32, c.c_float, P, c.c_size_t, P, P]
    L.prompt_attention_plan.restype = c.c_int
    L.prompt_attention_plan.argtypes = [c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_int,
                                        c.POINTER(c.c_size_t)]
    L.prompt_attention.restype = c.c_int
    L.prompt_attention.argtypes = [P, P, P, c.c_int, c.c_int64, c.c_int64, c.c_int64, P, P, c.c_int32, c.c_int32,
                                   c.c_int32, c.c_int32, c.c_int32, c.c_int32, c.c_float, P, c.c_size_t, P, P, P]
    L.pkv_set_first_wait_limit_for_testing.restype = None
    L.pkv_set_first_wait_limit_for_testing.argtypes = [c.c_int32, c.c_int32]
    L.pkv_status_string.restype = c.c_char_p
    L.pkv_status_string.argtypes = [c.c_int]
    L.pkv_last_cuda_error.restype = c.c_char_p
    L.pkv_last_cuda_error.argtypes = []
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != 0:
        raise PkvError(rc, what)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return PKV_F32
    if t == torch.bfloat16:
        return PKV_BF16
    if t in (torch.float8_e4m3fn, torch.uint8):
        return PKV_FP8_E4M3
    raise ValueError("unsupported dtype %s" % t)


_POOL_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
_POOL_CODE = {"f32": PKV_F32, "bf16": PKV_BF16, "fp8": PKV_FP8_E4M3}


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> ctypes.c_void_p:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def kv_bytes_per_token(num_layers: int, num_kv_heads: int, head_dim: int, kv_dtype: str) -> int:
    return int(lib().kv_bytes_per_token(num_layers, num_kv_heads, head_dim, _POOL_CODE[kv_dtype]))


class KVPool:
    """K and V pools [layers][blocks][kv_heads][block_size][head_dim] plus the
    library's handle.  FP8 pools hold raw E4M3 bytes (torch.uint8)."""

    def __init__(self, num_layers: int, num_blocks: int, block_size: int, num_kv_heads: int,
                 head_dim: int, kv_dtype: str, k_scale: float = 1.0, v_scale: float = 1.0,
                 device: str = "cuda", fill: Optional[int] = None):
        self.num_layers, self.num_blocks, self.block_size = num_layers, num_blocks, block_size
        self.num_kv_heads, self.head_dim, self.kv_dtype = num_kv_heads, head_dim, kv_dtype
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        shape = (num_layers, num_blocks, num_kv_heads, block_size, head_dim)
        dt = _POOL_TORCH[kv_dtype]
        self.k = torch.empty(shape, dtype=dt, device=device)
        self.v = torch.empty(shape, dtype=dt, device=device)
        if fill is not None:
            self.k.view(torch.uint8).fill_(fill)
            self.v.view(torch.uint8).fill_(fill)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)
        self._desc = PoolDesc(num_layers, num_blocks, block_size, num_kv_heads, head_dim,
                              _POOL_CODE[kv_dtype], self.k_scale, self.v_scale, self.k.data_ptr(),
                              self.v.data_ptr(), self.error_word.data_ptr())
        h = ctypes.c_void_p()
        _check(lib().kv_pool_create(ctypes.byref(self._desc), ctypes.byref(h)), "kv_pool_create")
        self.handle = h
        # for the native calls
        self.address = h.value
        self.device = self.k.device
        self.device_index = self.k.device.index if self.k.is_cuda else -1

    @property
    def tensor_bytes(self) -> int:
        return int(lib().kv_pool_tensor_bytes(ctypes.byref(self._desc)))

    def errors(self) -> int:
        """Read (synchronously) the error bits the kernels have set."""
        return int(self.error_word.item())

    def clear_errors(self):
        self.error_word.zero_()

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().kv_pool_destroy(self.handle)
            self.handle = self.address = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def kv_append(pool: KVPool, layer: int, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
              stream=None) -> None:
    """Write k, v [T, Hkv, D] (f32 or bf16) into the pool at slot_mapping [T] (int64)."""
    T = slot_mapping.shape[0]
    if k.shape != (T, pool.num_kv_heads, pool.head_dim) or v.shape != k.shape:
        raise ValueError("k/v must be [T, num_kv_heads, head_dim]")
    if k.dtype != v.dtype:
        raise ValueError("k and v must share a dtype")
    rc = lib().kv_append(pool.handle, layer, _dev(k, "k"), _dev(v, "v"), _dtype_code(k.dtype),
                         _dev(slot_mapping, "slot_mapping", torch.int64), T, _stream_ptr(stream))
    _check(rc, "kv_append")


def decode_plan(pool: KVPool, num_seqs: int, num_q_heads: int, max_seq_len: int,
                split_tokens: int = 0) -> Tuple[int, int, int]:
    """(split_tokens used, number of splits, workspace bytes)."""
    S, NS, ws = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t()
    _check(lib().paged_decode_plan(pool.handle, num_seqs, num_q_heads, max_seq_len, split_tokens,
                                   ctypes.byref(S), ctypes.byref(NS), ctypes.byref(ws)),
           "paged_decode_plan")
    return S.value, NS.value, ws.value


def decode_algo(pool: KVPool, num_q_heads: int, algo: str = "auto") -> str:
    """Name of the kernel design a call with this request would run."""
    r = lib().paged_decode_algo(pool.handle, num_q_heads // pool.num_kv_heads, ALGOS[algo])
    if r < 0:
        raise PkvError(2, "paged_decode_algo")
    return ALGO_NAMES[r]


def workspace_for(pool: KVPool, num_seqs: int, num_q_heads: int, max_seq_len: int,
                  split_tokens: int = 0) -> Optional[torch.Tensor]:
    _, _, ws = decode_plan(pool, num_seqs, num_q_heads, max_seq_len, split_tokens)
    if ws == 0:
        return None
    # the leading per-sequence counters must start at zero
    return torch.zeros(ws, dtype=torch.uint8, device=pool.k.device)


def paged_decode_attention(q: torch.Tensor, pool: KVPool, layer: int, block_tables: torch.Tensor,
                           seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           split_tokens: int = 0, algo: str = "auto", stream=None) -> torch.Tensor:
    """out[b, hq] = softmax(scale * q[b, hq] . K^T) V over the first seq_lens[b]
    tokens of sequence b, gathered through block_tables [B, max_blocks] (int32)."""
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = workspace_for(pool, B, Hq, max_seq_len, split_tokens)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().paged_decode_attention(
        _dev(q, "q"), _dtype_code(q.dtype), pool.handle, layer, _dev(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _dev(seq_lens, "seq_lens", torch.int32), B, Hq, max_seq_len, float(scale),
        split_tokens, ALGOS[algo], ws_ptr, ws_bytes, _dev(out, "out", q.dtype), _stream_ptr(stream))
    _check(rc, "paged_decode_attention")
    return out


def paged_decode_append_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, pool: KVPool,
                                  layer: int, block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                  scale: float, out: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None, split_tokens: int = 0,
                                  algo: str = "auto", stream=None) -> torch.Tensor:
    """One launch: write k_new / v_new [B, Hkv, D] (bf16 or f32) at position
    seq_lens[b] - 1 of each sequence, then paged_decode_attention over
    seq_lens[b] tokens (tensor-core design only)."""
    B, Hq, D = q.shape
    if tuple(k_new.shape) != (B, pool.num_kv_heads, D) or k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new / v_new must both be [num_seqs, num_kv_heads, head_dim] of one dtype")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = workspace_for(pool, B, Hq, max_seq_len, split_tokens)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().paged_decode_append_attention(
        _dev(q, "q"), _dtype_code(q.dtype), _dev(k_new, "k_new"), _dev(v_new, "v_new"), _dtype_code(k_new.dtype),
        pool.handle, layer, _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(seq_lens, "seq_lens", torch.int32), B, Hq, max_seq_len, float(scale), split_tokens, ALGOS[algo],
        ws_ptr, ws_bytes, _dev(out, "out", q.dtype), _stream_ptr(stream))
    _check(rc, "paged_decode_append_attention")
    return out


def paged_decode_attention_static_ws(q: torch.Tensor, pool: KVPool, layer: int, block_tables: torch.Tensor,
                                     seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                                     out: Optional[torch.Tensor] = None, split_tokens: int = 0,
                                     algo: str = "auto", stream=None) -> torch.Tensor:
    """paged_decode_attention whose split partials live in the library's own
    fixed device array (no workspace argument; the call allocates nothing on
    the device beyond `out` when `out` is not given).  Calls that overlap on
    the GPU share that array and race."""
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    rc = lib().paged_decode_attention_static_ws(
        _dev(q, "q"), _dtype_code(q.dtype), pool.handle, layer, _dev(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _dev(seq_lens, "seq_lens", torch.int32), B, Hq, max_seq_len, float(scale),
        split_tokens, ALGOS[algo], _dev(out, "out", q.dtype), _stream_ptr(stream))
    _check(rc, "paged_decode_attention_static_ws")
    return out


def set_first_wait_limit_for_testing(polls: int, cta: int = -1) -> None:
    """Make the first stage wait of the tensor-core designs (decode, shared prefixes, prompts) give up after
    `polls` polls in CTA `cta` (every CTA when negative) for later calls from
    this thread; polls < 0 restores the normal bound (test hook)."""
    lib().pkv_set_first_wait_limit_for_testing(int(polls), int(cta))


def multi_query_plan(pool: KVPool, num_seqs: int, num_queries: int, num_q_heads: int, max_seq_len: int,
                     split_tokens: int = 0) -> Tuple[int, int, int]:
    S, NS, ws = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t()
    _check(lib().paged_multi_query_plan(pool.handle, num_seqs, num_queries, num_q_heads, max_seq_len, split_tokens,
                                        ctypes.byref(S), ctypes.byref(NS), ctypes.byref(ws)),
           "paged_multi_query_plan")
    return S.value, NS.value, ws.value


def multi_query_algo(pool: KVPool, num_queries: int, num_q_heads: int, split_tokens: int = 0,
                     algo: str = "auto") -> str:
    """Name of the kernel design a multi-query call with this request would run."""
    r = lib().paged_multi_query_algo(pool.handle, num_queries, num_q_heads, split_tokens, ALGOS[algo])
    if r < 0:
        raise PkvError(2, "no kernel design serves this request")
    return ALGO_NAMES[r]


def paged_multi_query_attention(q: torch.Tensor, pool: KVPool, layer: int, block_tables: torch.Tensor,
                                seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                split_tokens: int = 0, algo: str = "auto", stream=None) -> torch.Tensor:
    """q [B, C, Hq, D]: the last C tokens of each sequence, each attending
    causally (query c at position seq_lens[b] - C + c).  Returns [B, C, Hq, D]."""
    B, C, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        _, _, ws = multi_query_plan(pool, B, C, Hq, max_seq_len, split_tokens)
        workspace = torch.zeros(ws, dtype=torch.uint8, device=q.device) if ws else None
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().paged_multi_query_attention(
        _dev(q, "q"), _dtype_code(q.dtype), pool.handle, layer, _dev(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _dev(seq_lens, "seq_lens", torch.int32), B, C, Hq, max_seq_len, float(scale),
        split_tokens, ALGOS[algo], ws_ptr, ws_bytes, _dev(out, "out", q.dtype), _stream_ptr(stream))
    _check(rc, "paged_multi_query_attention")
    return out


# ------------------------------------------------------------- one decode step
# The calls below check that every tensor lies on the pool's device and launch
# there, whatever device is current; what they allocate belongs to the stream
# they run on.  Their argument checks are native (csrc_python/step_calls.cpp).

_step_module = None


def _step():
    """Load _pkvstep.so (raises if it is missing)."""
    global _step_module
    if _step_module is None:
        lib()
        path = os.path.join(HERE, "_pkvstep.so")
        if not os.path.exists(path):
            raise RuntimeError("_pkvstep.so is not built (run __graft_entry__.build() or "
                               "python -m paged_kv_cache_194_gb300.build); no fallback exists")
        spec = importlib.util.spec_from_file_location(__package__ + "._pkvstep", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _step_module = module
    return _step_module


# The current device, and (device index) -> handle of its current stream, without
# the objects and checks of the public calls, which take longer than some of the
# kernels below.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _here(pool, stream) -> bool:
    """Whether a call needs no other device or stream than the current ones."""
    return stream is None and (pool.device_index < 0 or pool.device_index == _current_device())


def _on(pool, stream):
    """Context in which the pool's device is current, and `stream` when given
    (so that allocations belong to it)."""
    return _on_device(pool.device, stream, "the pool")


def _on_device(device: torch.device, stream, whose: str):
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream must be on %s, %s's device, not %s" % (device, whose, stream.device))
        return torch.cuda.stream(stream)
    return torch.cuda.device(device)


def _stream_handle(pool) -> int:
    return _raw_stream(pool.device_index) if pool.device_index >= 0 else 0


def prefix_decode_workspace(pool: KVPool, num_seqs: int, num_groups: int, num_q_heads: int,
                            max_seq_len: int) -> Optional[torch.Tensor]:
    """A zeroed workspace for paged_prefix_decode_attention calls of this size."""
    if not _here(pool, None):
        with _on(pool, None):
            return prefix_decode_workspace(pool, num_seqs, num_groups, num_q_heads, max_seq_len)
    ws = ctypes.c_size_t()
    _check(lib().paged_prefix_decode_plan(pool.handle, num_seqs, num_groups, num_q_heads, max_seq_len,
                                          ctypes.byref(ws)), "paged_prefix_decode_plan")
    return torch.zeros(ws.value, dtype=torch.uint8, device=pool.k.device) if ws.value else None


def prefix_decode_algo(pool: KVPool, num_seqs: int, num_groups: int, num_q_heads: int, max_seq_len: int,
                       algo: str = "auto") -> str:
    """Kernel design of such a call: "tc" shares the prefixes."""
    r = lib().paged_prefix_decode_algo(pool.handle, num_seqs, num_groups, num_q_heads, max_seq_len, ALGOS[algo])
    if r < 0:
        raise PkvError(2, "no kernel design serves this request")
    return ALGO_NAMES[r]


def paged_prefix_decode_attention(q: torch.Tensor, pool: KVPool, layer: int, block_tables: torch.Tensor,
                                  seq_lens: torch.Tensor, max_seq_len: int, group_offsets: torch.Tensor,
                                  prefix_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None, algo: str = "auto",
                                  stream=None) -> torch.Tensor:
    """paged_decode_attention for a batch whose sequences group_offsets[g] ..
    group_offsets[g + 1] - 1 share their first prefix_lens[g] tokens (int32
    tensors [groups + 1] and [groups]): each prefix is read once per group."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return paged_prefix_decode_attention(q, pool, layer, block_tables, seq_lens, max_seq_len, group_offsets,
                                                 prefix_lens, scale, out, workspace, algo)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None and q.dim() == 3:
        workspace = prefix_decode_workspace(pool, q.shape[0], prefix_lens.numel(), q.shape[1], max_seq_len)
    rc = _step().prefix_attention(pool.address, pool.device_index, pool.head_dim, layer, q, block_tables, seq_lens,
                                  max_seq_len, group_offsets, prefix_lens, scale, ALGOS[algo], workspace, out,
                                  _stream_handle(pool))
    if rc:
        raise PkvError(rc, "paged_prefix_decode_attention")
    return out


class RopeTable:
    """Cosines and sines of rotary positions: cos_sin [max_pos, rotary_dim]
    float32, cosines of the rotary_dim / 2 pairs, then sines.  sections: the
    pairs that follow each position axis, in order (default: all, one axis).
    interleaved: pairs are (2 j, 2 j + 1) instead of (j, j + rotary_dim / 2)."""

    def __init__(self, cos_sin: torch.Tensor, sections: Optional[Sequence[int]] = None, interleaved: bool = False):
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous float32 [max_pos, rotary_dim] tensor")
        self.cos_sin = cos_sin
        self.sections = tuple(int(s) for s in (sections if sections is not None else (cos_sin.shape[1] // 2,)))
        self.interleaved = bool(interleaved)
        if not 1 <= len(self.sections) <= 3 or min(self.sections) < 0 or 2 * sum(self.sections) != cos_sin.shape[1]:
            raise ValueError("sections must be 1 to 3 counts of pairs that sum to rotary_dim / 2")
        # as the native call takes them: number of axes, 20 bits per section
        self._axes = len(self.sections)
        self._packed = sum(n << (20 * i) for i, n in enumerate(self.sections))

    @classmethod
    def create(cls, max_pos: int, rotary_dim: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None,
               interleaved: bool = False, device="cuda") -> "RopeTable":
        """The usual table: pair j of position p turns by p * base^(-2 j /
        rotary_dim), the angle taken in 64 bits (a 32-bit one is off by 0.004
        at position 65536)."""
        j = torch.arange(rotary_dim // 2, dtype=torch.float64)
        a = torch.arange(max_pos, dtype=torch.float64)[:, None] * float(base) ** (-2.0 * j / rotary_dim)
        return cls(torch.cat([a.cos(), a.sin()], 1).to(torch.float32).to(device), sections, interleaved)


def kv_append_norm_rope(pool: KVPool, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        positions: torch.Tensor, slot_mapping: torch.Tensor, rope: RopeTable,
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """RMS norm of every query and key head (with weights [head_dim]; none: no
    norm), rotary positions for both, and kv_append of K and V, in one launch.
    q [T, Hq, D], k and v [T, Hkv, D] may be slices of one projection's rows;
    positions int32 [axes, T] (or [T] for one axis).  Returns the queries [T,
    Hq, D] in the dtype attention takes; `out` may be a contiguous q itself."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return kv_append_norm_rope(pool, layer, q, k, v, positions, slot_mapping, rope, q_weight, k_weight, eps, out)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if pool.kv_dtype == "f32" else torch.bfloat16, device=q.device)
    rc = _step().norm_rope(pool.address, pool.device_index, pool.num_kv_heads, pool.head_dim, pool.kv_dtype == "f32",
                           layer, q, k, v, positions, slot_mapping, rope.cos_sin, rope._axes, rope._packed,
                           rope.interleaved, q_weight, k_weight, eps, out, _stream_handle(pool))
    if rc:
        raise PkvError(rc, "kv_append_norm_rope")
    return out


class StepTables(NamedTuple):
    """What kv_tables_grow writes (beside the block tables)."""
    slot_mapping: torch.Tensor    # int64 [max_tokens]
    positions: torch.Tensor       # int32 [max_tokens]
    token_seqs: torch.Tensor      # int32 [max_tokens]
    token_offsets: torch.Tensor   # int32 [num_seqs + 1]
    granted: torch.Tensor         # int32 [num_seqs]
    seq_lens: torch.Tensor        # int32 [num_seqs]
    free_state: torch.Tensor      # int32 [2]

    @classmethod
    def empty(cls, num_seqs: int, max_tokens: int, device="cuda") -> "StepTables":
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=device)
        return cls(torch.empty(max_tokens, dtype=torch.int64, device=device), i32(max_tokens), i32(max_tokens),
                   i32(num_seqs + 1), i32(num_seqs), i32(num_seqs), i32(2))


def kv_tables_grow(pool: KVPool, block_tables: torch.Tensor, seq_lens: torch.Tensor, new_tokens: torch.Tensor,
                   free_ring: torch.Tensor, free_state: torch.Tensor, max_tokens: int,
                   out: Optional[StepTables] = None, stream=None) -> StepTables:
    """Reserve the next new_tokens[b] positions of every request on the device:
    blocks from the free ring into block_tables (in place), the slot, position
    and request of every token row, the new lengths and free state.  All int32
    tensors but the slots.  `out` may hold seq_lens and free_state themselves."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return kv_tables_grow(pool, block_tables, seq_lens, new_tokens, free_ring, free_state, max_tokens, out)
    if out is None:
        out = StepTables.empty(seq_lens.numel(), max_tokens, device=pool.k.device)
    rc = _step().tables_grow(pool.address, pool.device_index, block_tables, seq_lens, new_tokens, free_ring, free_state,
                             max_tokens, *out, _stream_handle(pool))
    if rc:
        raise PkvError(rc, "kv_tables_grow")
    return out


def kv_tables_release(pool: KVPool, block_tables: torch.Tensor, seq_lens: torch.Tensor, finished: torch.Tensor,
                      free_ring: torch.Tensor, free_state: torch.Tensor, keep_blocks: Optional[torch.Tensor] = None,
                      seq_lens_out: Optional[torch.Tensor] = None, free_state_out: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Return the blocks of every request with finished[b] != 0, but for the
    first keep_blocks[b] of its row, to the free ring (in place).  Returns the
    new lengths and free state; the outputs may be the inputs themselves."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return kv_tables_release(pool, block_tables, seq_lens, finished, free_ring, free_state, keep_blocks,
                                     seq_lens_out, free_state_out)
    seq_lens_out = torch.empty_like(seq_lens) if seq_lens_out is None else seq_lens_out
    free_state_out = torch.empty_like(free_state) if free_state_out is None else free_state_out
    rc = _step().tables_release(pool.address, pool.device_index, block_tables, seq_lens, finished, keep_blocks, free_ring,
                                free_state, seq_lens_out, free_state_out, _stream_handle(pool))
    if rc:
        raise PkvError(rc, "kv_tables_release")
    return seq_lens_out, free_state_out


# ------------------------------------------------- a quantised cache, whole prompts
class QuantKVPool:
    """A paged KV cache of 4- or 8-bit codes: k_codes and v_codes [layers, blocks,
    kv_heads, block_size, head_dim * bits / 8] (torch.uint8; 4 bits: element 2 j
    in the low half of byte j) and k_params and v_params [layers, blocks,
    kv_heads, block_size, 2] (bfloat16: scale and offset of each row).  A code c
    stands for offset + scale * c."""

    def __init__(self, num_layers: int, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int, bits: int,
                 device: str = "cuda", fill: Optional[int] = None):
        self.num_layers, self.num_blocks, self.block_size = num_layers, num_blocks, block_size
        self.num_kv_heads, self.head_dim, self.bits = num_kv_heads, head_dim, bits
        self.kv_dtype = "q%d" % bits
        self.handle = self.address = None
        self._desc = QuantPoolDesc(num_layers, num_blocks, block_size, num_kv_heads, head_dim, bits)
        _check(lib().kv_quant_pool_bytes(ctypes.byref(self._desc), None, None), "kv_quant_pool_bytes")
        rows = (num_layers, num_blocks, num_kv_heads, block_size)
        self.k_codes, self.v_codes = (torch.empty(rows + (head_dim * bits // 8,), dtype=torch.uint8, device=device)
                                      for _ in range(2))
        self.k_params, self.v_params = (torch.empty(rows + (2,), dtype=torch.bfloat16, device=device) for _ in range(2))
        if fill is not None:
            for x in (self.k_codes, self.v_codes, self.k_params, self.v_params):
                x.view(torch.uint8).fill_(fill)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)
        for name in ("k_codes", "v_codes", "k_params", "v_params", "error_word"):
            setattr(self._desc, name, getattr(self, name).data_ptr())
        h = ctypes.c_void_p()
        _check(lib().kv_quant_pool_create(ctypes.byref(self._desc), ctypes.byref(h)), "kv_quant_pool_create")
        self.handle, self.address = h, h.value
        self.device = self.k_codes.device
        self.device_index = self.device.index if self.k_codes.is_cuda else -1

    def errors(self) -> int:
        """Read (synchronously) the error bits the kernels have set."""
        return int(self.error_word.item())

    def clear_errors(self):
        self.error_word.zero_()

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().kv_quant_pool_destroy(self.handle)
            self.handle = self.address = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def kv_quant_append(pool: QuantKVPool, layer: int, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                    stream=None) -> None:
    """Quantise k, v [T, Hkv, D] (float32 or bfloat16, possibly slices of one
    projection's rows) into the pool at slot_mapping [T] (int64; -1: skipped),
    each row with a scale and an offset of its own."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return kv_quant_append(pool, layer, k, v, slot_mapping)
    rc = _step().quant_append(pool.address, pool.device_index, pool.num_kv_heads, pool.head_dim, layer, k, v, slot_mapping,
                              _stream_handle(pool))
    if rc:
        raise PkvError(rc, "kv_quant_append")


def kv_read(pool, layer: int, block_tables: torch.Tensor, offsets: torch.Tensor, num_rows: int,
            k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of a batch read back from a KVPool or a QuantKVPool, packed: rows
    offsets[b] .. offsets[b + 1] - 1 (int32 [B + 1]) are the first tokens of
    sequence b, gathered through block_tables [B, max_blocks] (int32).  Returns
    k, v [num_rows, Hkv, D], float32 from a float32 pool, else bfloat16; rows of
    no sequence keep what k_out and v_out held."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return kv_read(pool, layer, block_tables, offsets, num_rows, k_out, v_out)
    shape, f32 = (num_rows, pool.num_kv_heads, pool.head_dim), pool.kv_dtype == "f32"
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.float32 if f32 else torch.bfloat16, device=pool.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.float32 if f32 else torch.bfloat16, device=pool.device)
    rc = _step().read_rows(pool.address, isinstance(pool, QuantKVPool), pool.device_index, pool.num_kv_heads, pool.head_dim,
                           f32, layer, block_tables, offsets, num_rows, k_out, v_out, _stream_handle(pool))
    if rc:
        raise PkvError(rc, "kv_read")
    return k_out, v_out


def _counters_zeroed(size: int, device) -> Optional[torch.Tensor]:
    if not size:
        return None
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    ws[:65536].zero_()
    return ws


def quant_decode_workspace(pool: QuantKVPool, num_seqs: int, num_q_heads: int, max_seq_len: int) -> Optional[torch.Tensor]:
    """A workspace (its counters zeroed) for paged_quant_decode_attention calls of this size; stream-ordered calls of it
    and of prompt_attention may share one that is large enough for each."""
    if not _here(pool, None):
        with _on(pool, None):
            return quant_decode_workspace(pool, num_seqs, num_q_heads, max_seq_len)
    ws = ctypes.c_size_t()
    _check(lib().paged_quant_decode_plan(pool.handle, num_seqs, num_q_heads, max_seq_len, ctypes.byref(ws)),
           "paged_quant_decode_plan")
    return _counters_zeroed(ws.value, pool.device)


def paged_quant_decode_attention(q: torch.Tensor, pool: QuantKVPool, layer: int, block_tables: torch.Tensor,
                                 seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """paged_decode_attention over a quantised cache: q [B, Hq, D] bfloat16."""
    if not _here(pool, stream):
        with _on(pool, stream):
            return paged_quant_decode_attention(q, pool, layer, block_tables, seq_lens, max_seq_len, scale, out, workspace)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None and q.dim() == 3:
        workspace = quant_decode_workspace(pool, q.shape[0], q.shape[1], max_seq_len)
    rc = _step().quant_attention(pool.address, pool.device_index, pool.head_dim, layer, q, block_tables, seq_lens,
                                 max_seq_len, scale, workspace, out, _stream_handle(pool))
    if rc:
        raise PkvError(rc, "paged_quant_decode_attention")
    return out


def prompt_attention_workspace(q: torch.Tensor, num_seqs: int, num_kv_heads: int) -> Optional[torch.Tensor]:
    """A workspace (its counters zeroed) for prompt_attention calls of this size; stream-ordered calls of it and of
    paged_quant_decode_attention may share one that is large enough for each."""
    index = q.device.index if q.is_cuda else -1
    if index >= 0 and index != _current_device():
        with torch.cuda.device(index):
            return prompt_attention_workspace(q, num_seqs, num_kv_heads)
    if q.dim() != 3 or q.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("q must be [rows, num_q_heads, head_dim], float32 or bfloat16")
    ws = ctypes.c_size_t()
    _check(lib().prompt_attention_plan(num_seqs, q.shape[0], q.shape[1], num_kv_heads, q.shape[2], _dtype_code(q.dtype),
                                       ctypes.byref(ws)), "prompt_attention_plan")
    return _counters_zeroed(ws.value, q.device)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor, k_offsets: torch.Tensor,
                     scale: float, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     error_word: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts: sequence b's queries are rows
    q_offsets[b] .. q_offsets[b + 1] - 1 of q [Tq, Hq, D], its keys and values
    rows k_offsets[b] .. k_offsets[b + 1] - 1 of k and v [Tk, Hkv, D] (bfloat16
    or float32, possibly slices of one projection's rows); its queries are the
    last of its positions.  Returns [Tq, Hq, D]; rows of no sequence keep what
    `out` held.  error_word: int32 [1], gets ERRBIT_OFFSETS where offsets do not
    ascend within the rows, ERRBIT_TIMEOUT where a wait expired (whose rows are NaN)."""
    index = q.device.index if q.is_cuda else -1
    if stream is not None or (index >= 0 and index != _current_device()):
        with _on_device(q.device, stream, "q"):
            return prompt_attention(q, k, v, q_offsets, k_offsets, scale, out, workspace, error_word)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None and q.dim() == 3 and k.dim() == 3:
        workspace = prompt_attention_workspace(q, max(0, q_offsets.numel() - 1), k.shape[1])
    rc = _step().prompt_attention(index, q, k, v, q_offsets, k_offsets, scale, workspace, out, error_word,
                                  _raw_stream(index) if index >= 0 else 0)
    if rc:
        raise PkvError(rc, "prompt_attention")
    return out
