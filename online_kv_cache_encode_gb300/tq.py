"""Python binding of the C ABI in ``include/tq.h`` (ctypes, argument marshalling only).

PyTorch supplies device memory and the current CUDA stream; every step of
encode and decode runs in the library's CUDA kernels.  The binding refuses to
work without ``libtq.so``: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA, TQ_ERR_WORKSPACE = range(5)
FLAG_OVERFLOW, FLAG_BAD_SLOT, FLAG_NONFINITE, FLAG_TIMEOUT, FLAG_INTERNAL = 1, 2, 4, 8, 16
TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
NOALLOC_WORKSPACE_BYTES = 4 << 20  # TQ_NOALLOC_WORKSPACE_BYTES

# every exported symbol of include/tq.h: (restype, argtypes)
_P, _I, _I64, _U64, _F, _SZ, _D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                   ctypes.c_float, ctypes.c_size_t, ctypes.c_double)
SIGNATURES = {
    "tq_codebook_init": (_I, [_I, _I, ctypes.POINTER(_P)]),
    "tq_codebook_get": (_I, [_P, _P, _P, _P]),
    "tq_codebook_free": (None, [_P]),
    "tq_page_bytes": (_I64, [_I, _I, _I, _I, _I]),
    "tq_cache_create": (_I, [_P, _I64, _I, _I, _I, _I, _I, _I, _U64, ctypes.POINTER(_P)]),
    "tq_cache_free": (None, [_P]),
    "tq_method_constants": (_I, [_I, _I, _U64, _P, _P]),
    "tq_cache_signs": (_I, [_P, _P]),
    "tq_cache_gaussian": (_I, [_P, _P]),
    "tq_encode_kv": (_I, [_P, _P, _P, _I, _I64, _P, _P, _P]),
    "tq_decode_workspace_bytes": (_SZ, [_P, _I, _I, _I]),
    "tq_decode_attention": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _F, _P, _P, _SZ, _P, _P]),
    "tq_decode_attention_noalloc": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _F, _P, _P, _P]),
    "tq_decode_attention_append": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _F, _P, _P, _SZ, _P, _P]),
    "tq_decode_attention_ring_append": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _F, _P, _P, _SZ, _P,
                                             _P]),
    "tq_cache_create_octopus": (_I, [_P, ctypes.c_int64, _I, _I, _I, _I, _I, ctypes.c_uint64, ctypes.POINTER(_P)]),
    "tq_octopus_page_bytes": (ctypes.c_int64, [_I, _I, _I, _I]),
    "tq_octopus_codebook": (_I, [_I, _I, _I, _P]),
    "tq_prefill_workspace_bytes": (_SZ, [_P, _I, _I, _I]),
    "tq_prefill_attention": (_I, [_P, _P, _I, _I, _I, _P, _I, _I, _F, _P, _P, _SZ, _P, _P]),
    "tq_fp8_cache_create": (_I, [_P, _P, _I64, _I, _I, _I, ctypes.POINTER(_P)]),
    "tq_fp8_cache_free": (None, [_P]),
    "tq_fp8_write": (_I, [_P, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P]),
    "tq_fp8_read": (_I, [_P, _P, _P, _I, _I64, _I, _P, _P, _P, _I, _P, _P]),
    "tq_fp8_decode_workspace_bytes": (_SZ, [_P, _I, _I]),
    "tq_fp8_decode_counters_offset": (_SZ, [_P]),
    "tq_fp8_decode_attention": (_I, [_P, _P, _I, _I64, _I64, _I, _I, _P, _I, _P, _F, _P, _P, _SZ, _P, _P]),
    "tq_fp8_prefill_workspace_bytes": (_SZ, [_P, _I64, _I, _I]),
    "tq_fp8_prefill_attention": (_I, [_P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _P, _P, _I, _F, _P, _P, _SZ, _P, _P]),
    "tq_rotary_frequencies": (_I, [_I, _D, _I, _D, _D, _D, _D, _P]),
    "tq_rotary_table": (_I, [_P, _I, _D, _I64, _P, _P]),
    "tq_rotary": (_I, [_P, _I, _I64, _I64, _I64, _I, _I, _P, _P, _I64, _I, _I, _I, _P, _I64, _I64, _P, _P]),
    "tq_fp8_append": (_I, [_P, _P, _P, _I, _I64, _I64, _I64, _I64, _P, _I64, _I64, _I, _P, _I64, _I64, _I64, _I, _P, _P, _P, _I,
                           _P, _P, _I64, _I, _I, _P, _P]),
    "tq_fp8_tree_workspace_bytes": (_SZ, [_P, _I64, _I, _I]),
    "tq_fp8_tree_attention": (_I, [_P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _P, _P, _I, _P, _I, _F, _P, _P, _SZ, _P, _P]),
    "tq_fp8_keep": (_I, [_P, _I64, _I, _P, _P, _P, _P, _I, _P, _P]),
    "tq_device_accessible": (_I, [_P, ctypes.POINTER(_I)]),
    "tq_test_stall_waits": (None, [_I64]),
    "tq_selftest_tcgen05": (_I, [_P, _P, _P, _P, _P]),
    "tq_status_string": (ctypes.c_char_p, [_I]),
    "tq_last_error": (ctypes.c_char_p, []),
}

_lock = threading.Lock()
_lib = None


class TQError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"tq status {status}: {detail}")
        self.status = status


def lib():
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:  # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def _check(st: int):
    if st != TQ_OK:
        raise TQError(st, lib().tq_last_error().decode())


_DTYPE_CODES = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}


def _dtype_code(t: torch.Tensor) -> int:
    return _DTYPE_CODES[t.dtype]


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    # a plain int: the c_void_p argtypes convert it
    return None if t is None else t.data_ptr()


def device_accessible(t: torch.Tensor) -> bool:
    """Whether the decode kernels can read / write tensor t in place: a CUDA
    tensor, or a pinned host tensor mapped into the device's address space
    (the kernel then reaches it over the host link, with no copy launch)."""
    if t.is_cuda:
        return True
    if not t.is_pinned():
        return False
    a = ctypes.c_int(0)
    _check(lib().tq_device_accessible(_ptr(t), ctypes.byref(a)))
    return a.value == 1


def set_test_stall(cycles: int) -> None:
    """Test hook of the device-side timeout path (tq_test_stall_waits): with
    cycles > 0 every later decode launch lets warp 0 of each odd split give up
    a bounded wait; 0 turns it off."""
    lib().tq_test_stall_waits(int(cycles))


def selftest_tcgen05(A: torch.Tensor, B: torch.Tensor, status: torch.Tensor | None = None) -> torch.Tensor:
    """tq_selftest_tcgen05: A [128, 256] and B [256, 16] fp16 (CUDA) -> out [6, 128, 16] fp32."""
    assert A.is_cuda and A.dtype == torch.float16 and A.shape == (128, 256) and A.is_contiguous()
    assert B.is_cuda and B.dtype == torch.float16 and B.shape == (256, 16) and B.is_contiguous()
    out = torch.full((6, 128, 16), float("nan"), dtype=torch.float32, device=A.device)
    _check(lib().tq_selftest_tcgen05(_ptr(A), _ptr(B), _ptr(out), _ptr(status), _stream()))
    return out


def ring_slots(block_row, positions, window: int, block_size: int = 16):
    """Slots of token positions in a sequence's ring of `window` slots (its
    block-table row block_row): position t lives in slot t % window."""
    r = positions % window
    return block_row[r // block_size] * block_size + r % block_size


def page_bytes(d: int, key_bits: int, value_bits: int, qjl_m: int = 0, block_size: int = 16) -> int:
    return int(lib().tq_page_bytes(d, key_bits, value_bits, qjl_m, block_size))


class Codebook:
    """Host Lloyd-Max codebook (centroids, boundaries, passes)."""

    def __init__(self, d: int, bits: int):
        h = ctypes.c_void_p()
        _check(lib().tq_codebook_init(d, bits, ctypes.byref(h)))
        try:
            n = 1 << bits
            self.centroids = np.empty(n, dtype=np.float64)
            self.boundaries = np.empty(n - 1, dtype=np.float64)
            passes = ctypes.c_int()
            _check(lib().tq_codebook_get(h, self.centroids.ctypes.data_as(_P),
                                         self.boundaries.ctypes.data_as(_P), ctypes.byref(passes)))
            self.passes = passes.value
        finally:
            lib().tq_codebook_free(h)


def method_constants(d: int, m: int, seed: int):
    """(signs[d] int8, S[m, d] float64) that a seed defines (host, no GPU)."""
    s = np.empty(d, dtype=np.int8)
    S = np.empty((m, d), dtype=np.float64)
    _check(lib().tq_method_constants(d, m, seed, s.ctypes.data_as(_P), S.ctypes.data_as(_P) if m else None))
    return s, S


def new_status(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


class Cache:
    """A compressed paged KV cache on the current CUDA device.

    pool: uint8 [num_blocks * num_kv_heads * page_bytes], allocated here unless given.
    """

    def __init__(self, num_blocks: int, num_kv_heads: int, key_bits: int = 4, value_bits: int = 4,
                 qjl_m: int = 0, seed: int = 0, block_size: int = 16, d: int = 128,
                 pool: torch.Tensor | None = None, device="cuda"):
        self.num_blocks, self.hkv, self.kb, self.vb = num_blocks, num_kv_heads, key_bits, value_bits
        self.m, self.seed, self.bs, self.d = qjl_m, seed, block_size, d
        self.page_bytes = page_bytes(d, key_bits, value_bits, qjl_m, block_size)
        if self.page_bytes < 0:
            raise TQError(TQ_ERR_INVALID_ARG, "invalid geometry")
        nbytes = self.page_bytes * num_kv_heads * num_blocks
        if pool is None:
            pool = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        assert pool.dtype == torch.uint8 and pool.numel() >= nbytes and pool.is_contiguous()
        self.pool = pool
        self._h = ctypes.c_void_p()
        _check(lib().tq_cache_create(_ptr(pool), num_blocks, block_size, num_kv_heads, d, key_bits,
                                     value_bits, qjl_m, seed, ctypes.byref(self._h)))
        self._ws = None

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.tq_cache_free(h)
            self._h = None

    # ---- derived constants (host copies) ----
    def signs(self) -> np.ndarray:
        s = np.empty(self.d, dtype=np.int8)
        _check(lib().tq_cache_signs(self._h, s.ctypes.data_as(_P)))
        return s

    def gaussian(self) -> np.ndarray:
        S = np.empty((self.m, self.d), dtype=np.float64)
        _check(lib().tq_cache_gaussian(self._h, S.ctypes.data_as(_P)))
        return S

    # ---- encode ----
    def encode(self, K: torch.Tensor, V: torch.Tensor, slot_mapping: torch.Tensor,
               status: torch.Tensor | None = None):
        """K, V: [T, num_kv_heads, d] (f32/bf16/f16, CUDA); slot_mapping: int64 [T]."""
        assert K.is_cuda and K.shape == V.shape and K.dtype == V.dtype
        assert K.dim() == 3 and K.shape[1] == self.hkv and K.shape[2] == self.d
        assert K.is_contiguous() and V.is_contiguous()
        assert slot_mapping.dtype == torch.int64 and slot_mapping.is_contiguous()
        assert slot_mapping.numel() == K.shape[0]
        _check(lib().tq_encode_kv(self._h, _ptr(K), _ptr(V), _dtype_code(K), K.shape[0],
                                  _ptr(slot_mapping), _ptr(status), _stream()))

    # ---- decode ----
    def workspace_bytes(self, batch: int, num_q_heads: int, max_blocks_per_seq: int) -> int:
        return int(lib().tq_decode_workspace_bytes(self._h, batch, num_q_heads, max_blocks_per_seq))

    def new_workspace(self, batch: int, num_q_heads: int, max_blocks_per_seq: int) -> torch.Tensor:
        n = self.workspace_bytes(batch, num_q_heads, max_blocks_per_seq)
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=self.pool.device)

    def decode(self, q: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
               sm_scale: float | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
        """q: [B, Hq, d]; block_table: int32 [B, max_blocks]; lens: int32 [B] -> out fp32 [B, Hq, d].
        q and out may be pinned host tensors (see device_accessible)."""
        assert device_accessible(q) and q.dim() == 3 and q.shape[2] == self.d and q.is_contiguous()
        B, hq, _ = q.shape
        assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B
        assert block_table.is_contiguous() and lens.dtype == torch.int32 and lens.numel() == B
        mb = block_table.shape[1]
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.d)
        if out is None:
            out = torch.empty((B, hq, self.d), dtype=torch.float32, device=self.pool.device)
        assert device_accessible(out)
        if workspace is None:
            key = (B, hq, mb)
            if self._ws is None or self._ws[0] != key:
                self._ws = (key, self.new_workspace(B, hq, mb))
            workspace = self._ws[1]
        _check(lib().tq_decode_attention(self._h, _ptr(q), _dtype_code(q), B, hq, _ptr(block_table), mb,
                                         _ptr(lens), float(sm_scale), _ptr(out), _ptr(workspace),
                                         workspace.numel(), _ptr(status), _stream()))
        return out

    def decode_append(self, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor, block_table: torch.Tensor,
                      lens: torch.Tensor, sm_scale: float | None = None, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      window: int | None = None) -> torch.Tensor:
        """One decode step: append the new token of every sequence (k_new, v_new:
        [B, num_kv_heads, d], position lens[b] - 1) and attend over lens[b] tokens.
        With `window`, each sequence's blocks form a ring of `window` slots: the
        token goes to slot (lens[b] - 1) % window and the query attends over the
        min(lens[b], window) tokens the ring holds."""
        assert device_accessible(k_new) and device_accessible(v_new)
        assert k_new.shape == v_new.shape and k_new.dtype == v_new.dtype
        assert k_new.dim() == 3 and k_new.shape[1] == self.hkv and k_new.shape[2] == self.d
        assert k_new.is_contiguous() and v_new.is_contiguous()
        assert device_accessible(q) and q.dim() == 3 and q.shape[2] == self.d and q.is_contiguous()
        B, hq, _ = q.shape
        assert k_new.shape[0] == B
        assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B
        assert block_table.is_contiguous() and lens.dtype == torch.int32 and lens.numel() == B
        mb = block_table.shape[1]
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.d)
        if out is None:
            out = torch.empty((B, hq, self.d), dtype=torch.float32, device=self.pool.device)
        assert device_accessible(out)
        if workspace is None:
            key = (B, hq, mb)
            if self._ws is None or self._ws[0] != key:
                self._ws = (key, self.new_workspace(B, hq, mb))
            workspace = self._ws[1]
        if window is None:
            _check(lib().tq_decode_attention_append(self._h, _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _ptr(q),
                                                    _dtype_code(q), B, hq, _ptr(block_table), mb, _ptr(lens),
                                                    float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                                    _ptr(status), _stream()))
        else:
            _check(lib().tq_decode_attention_ring_append(self._h, _ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                                         _ptr(q), _dtype_code(q), B, hq, _ptr(block_table), mb,
                                                         _ptr(lens), int(window), float(sm_scale), _ptr(out),
                                                         _ptr(workspace), workspace.numel(), _ptr(status),
                                                         _stream()))
        return out

    def prefill(self, q: torch.Tensor, block_row: torch.Tensor, first_position: int, sm_scale: float | None = None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                status: torch.Tensor | None = None) -> torch.Tensor:
        """Causal attention of the query positions first_position .. first_position + C - 1
        (q: [C, Hq, d]) of one sequence over its cached tokens (the chunk's own
        keys and values already encoded); block_row: int32 [max_blocks]."""
        assert q.is_cuda and q.dim() == 3 and q.shape[2] == self.d and q.is_contiguous()
        assert block_row.dtype == torch.int32 and block_row.dim() == 1 and block_row.is_contiguous()
        C, hq, _ = q.shape
        mb = block_row.shape[0]
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.d)
        if out is None:
            out = torch.empty((C, hq, self.d), dtype=torch.float32, device=q.device)
        if workspace is None:
            n = int(lib().tq_prefill_workspace_bytes(self._h, C, hq, mb))
            workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
        _check(lib().tq_prefill_attention(self._h, _ptr(q), _dtype_code(q), C, hq, _ptr(block_row), mb,
                                          int(first_position), float(sm_scale), _ptr(out), _ptr(workspace),
                                          workspace.numel(), _ptr(status), _stream()))
        return out

    def decode_noalloc(self, q: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                       sm_scale: float | None = None, out: torch.Tensor = None,
                       status: torch.Tensor | None = None) -> torch.Tensor:
        """decode() through tq_decode_attention_noalloc: the library's fixed
        workspace instead of a caller one (for callers that must not allocate).
        `out` must be given: this call allocates nothing, here or in the library."""
        assert out is not None and out.dtype == torch.float32 and out.is_contiguous()
        assert q.is_cuda and q.dim() == 3 and q.shape[2] == self.d and q.is_contiguous()
        B, hq, _ = q.shape
        assert out.shape == (B, hq, self.d)
        assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous()
        assert lens.dtype == torch.int32 and lens.numel() == B
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(self.d)
        _check(lib().tq_decode_attention_noalloc(self._h, _ptr(q), _dtype_code(q), B, hq, _ptr(block_table),
                                                 block_table.shape[1], _ptr(lens), float(sm_scale), _ptr(out),
                                                 _ptr(status), _stream()))
        return out


class OctopusCache(Cache):
    """A cache whose keys use the OCTOPUS triplet codec (bits 2..4 per
    coordinate on average: (bits + 1)-bit direction codes, (bits - 1)-bit norm
    codes per triplet); values keep min-max codes.  encode / decode as Cache."""

    def __init__(self, num_blocks: int, num_kv_heads: int, bits: int = 4, value_bits: int = 4, seed: int = 0,
                 block_size: int = 16, d: int = 128, pool: torch.Tensor | None = None, device="cuda"):
        self.num_blocks, self.hkv, self.kb, self.vb = num_blocks, num_kv_heads, bits, value_bits
        self.m, self.seed, self.bs, self.d = 0, seed, block_size, d
        self.page_bytes = int(lib().tq_octopus_page_bytes(d, bits, value_bits, block_size))
        if self.page_bytes < 0:
            raise TQError(TQ_ERR_INVALID_ARG, "invalid geometry")
        nbytes = self.page_bytes * num_kv_heads * num_blocks
        if pool is None:
            pool = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        assert pool.dtype == torch.uint8 and pool.numel() >= nbytes and pool.is_contiguous()
        self.pool = pool
        self._h = ctypes.c_void_p()
        _check(lib().tq_cache_create_octopus(_ptr(pool), num_blocks, block_size, num_kv_heads, d, bits, value_bits,
                                             seed, ctypes.byref(self._h)))
        self._ws = None


def octopus_codebook(d: int, bits: int, kind: int) -> np.ndarray:
    """The library's host-computed OCTOPUS levels (kind 0: xi / eta, kind 1: triplet norm)."""
    out = np.empty(1 << bits, dtype=np.float64)
    _check(lib().tq_octopus_codebook(d, bits, kind, out.ctypes.data_as(ctypes.c_void_p)))
    return out


_ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
_ROTARY_SCALINGS = {None: (0, 0), "linear": (1, 1), "base": (2, 1), "parts": (3, 4)}  # code, arguments


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: tuple | None = None) -> np.ndarray:
    """The dim / 2 frequencies (radians a position, float64) of rotated pairs.  scaling: None, ("linear", factor),
    ("base", factor) or ("parts", factor, original_positions, low_turns, high_turns), as tq_rotary_frequencies has them."""
    kind, *args = scaling or (None,)
    if kind not in _ROTARY_SCALINGS or len(args) != _ROTARY_SCALINGS[kind][1]:
        raise TQError(TQ_ERR_INVALID_ARG, f"bad rotary scaling {scaling!r}")
    factor, original, low, high = (*map(float, args), *(0.0,) * (4 - len(args)))
    out = np.empty(max(dim, 2) // 2, dtype=np.float64)
    _check(lib().tq_rotary_frequencies(dim, base, _ROTARY_SCALINGS[kind][0], factor, original, low, high,
                                       out.ctypes.data_as(ctypes.c_void_p)))
    return out


class Rotary:
    """Rotary positions 0 .. num_positions - 1 for the first `dim` dims of a head (a multiple of 16, at most 256).

    layout: "half" (dim j pairs with j + dim / 2) or "interleaved" (2 j with 2 j + 1); base and scaling as
    rotary_frequencies has them, or the frequencies themselves; magnitude multiplies what is rotated.  The cosines and
    sines are computed once, here, into `table` (fp32 [num_positions, 2, dim / 2]) on the current stream, unless a
    table is given.
    """

    def __init__(self, dim: int, num_positions: int, base: float = 10000.0, layout: str = "half",
                 scaling: tuple | None = None, frequencies=None, magnitude: float = 1.0,
                 table: torch.Tensor | None = None, device="cuda"):
        if layout not in _ROTARY_LAYOUTS:
            raise TQError(TQ_ERR_INVALID_ARG, f"bad rotary layout {layout!r}")
        if dim <= 0 or dim % 16 or dim > 256:
            raise TQError(TQ_ERR_UNSUPPORTED, "the rotated dims must be a multiple of 16, at most 256")
        if num_positions <= 0:
            raise TQError(TQ_ERR_UNSUPPORTED, "the table's positions must be positive")
        self.dim, self.num_positions, self.layout = dim, num_positions, layout
        self._layout, self._lib = _ROTARY_LAYOUTS[layout], lib()
        if table is None:
            if frequencies is None:
                frequencies = rotary_frequencies(dim, base, scaling)
            f = np.ascontiguousarray(frequencies, dtype=np.float64)
            assert f.shape == (dim // 2,)
            table = torch.empty((num_positions, 2, dim // 2), dtype=torch.float32, device=device)
            with torch.cuda.device(table.device):
                _check(self._lib.tq_rotary_table(f.ctypes.data_as(ctypes.c_void_p), dim, float(magnitude), num_positions,
                                                 table.data_ptr(), _stream()))
        assert table.is_cuda and table.dtype is torch.float32 and table.shape == (num_positions, 2, dim // 2)
        assert table.is_contiguous()
        self.table, self._dev = table, table.get_device()

    def apply(self, x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor | None = None, transpose: bool = False,
              status: torch.Tensor | None = None) -> torch.Tensor:
        """x: [T, H, d] (f32/bf16/f16, strided rows on 16-byte boundaries, d a multiple of 16), token t rotated by
        position positions[t] (int32 [T], on the device) -> out, a new contiguous tensor unless given (x itself: in
        place).  transpose: by the transposed matrix, which takes an output's gradient to the input's.  The call records
        no gradient itself."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.apply(x, positions, out, transpose, status)
        dev = self._dev
        T, H, d = x.shape
        if out is None:
            out = torch.empty((T, H, d), dtype=x.dtype, device=x.device)
        else:
            assert out.shape == x.shape and out.dtype is x.dtype and out.get_device() == dev
        xs, os = x.stride(), out.stride()
        assert x.get_device() == dev and (d == 1 or xs[2] == 1 and os[2] == 1)
        assert positions.dtype is torch.int32 and positions.get_device() == dev and positions.is_contiguous()
        assert positions.numel() == T
        assert status is None or status.dtype is torch.int32 and status.get_device() == dev and status.numel() >= 1
        st = self._lib.tq_rotary(x.data_ptr(), _DTYPE_CODES[x.dtype], xs[0] if T > 1 else 0, xs[1] if H > 1 else 0, T, H, d,
                                 positions.data_ptr(), self.table.data_ptr(), self.num_positions, self.dim, self._layout,
                                 int(transpose), out.data_ptr(), os[0] if T > 1 else 0, os[1] if H > 1 else 0, _ptr(status),
                                 torch._C._cuda_getCurrentRawStream(dev))
        if st:
            _check(st)
        return out


class Fp8Cache:
    """An 8-bit paged KV cache on the current CUDA device: e4m3 codes and one
    power-of-two scale for each block, KV head and side (tq_fp8_cache_create).

    pool: uint8 [num_blocks * num_kv_heads * 2 * block_size * d] and scales: fp32
    [num_blocks, num_kv_heads, 2], allocated here unless given.

    A ragged batch is given as cu_tokens int32 [B + 1], start int32 [B] and
    block_table int32 [B, max_blocks], all on the device: rows cu_tokens[b] ..
    cu_tokens[b + 1] - 1 of the packed tensors are positions start[b] .. of
    sequence b.

    Rows of d elements (of K, V and q) are contiguous and start on 16-byte
    boundaries; their token and head strides are free otherwise.  The calls
    record no gradient: their results are detached from q, K and V.
    """

    def __init__(self, num_blocks: int, num_kv_heads: int, block_size: int = 16, d: int = 128,
                 pool: torch.Tensor | None = None, scales: torch.Tensor | None = None, device="cuda"):
        self.num_blocks, self.hkv, self.bs, self.d = num_blocks, num_kv_heads, block_size, d
        if pool is None:
            pool = torch.zeros(num_blocks * num_kv_heads * 2 * block_size * d, dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.ones((num_blocks, num_kv_heads, 2), dtype=torch.float32, device=pool.device)
        assert pool.dtype == torch.uint8 and pool.is_contiguous()
        assert pool.numel() >= num_blocks * num_kv_heads * 2 * block_size * d
        assert scales.dtype == torch.float32 and scales.is_contiguous() and scales.device == pool.device
        assert scales.numel() >= num_blocks * num_kv_heads * 2
        assert pool.is_cuda
        self.pool, self.scales = pool, scales
        self._dev, self._sm_scale = pool.get_device(), 1.0 / math.sqrt(d)
        self._h = ctypes.c_void_p()
        with torch.cuda.device(pool.device):
            _check(lib().tq_fp8_cache_create(_ptr(pool), _ptr(scales), num_blocks, block_size, num_kv_heads, d,
                                             ctypes.byref(self._h)))
        self._ws = {}
        self._lib = lib()
        self._counters_at = int(self._lib.tq_fp8_decode_counters_offset(self._h))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.tq_fp8_cache_free(h)
            self._h = None

    # The checks below run on every call of a serving loop: each reads an attribute once, and the device is only
    # switched where the current one is another.
    def _batch(self, cu, start, table, status):
        """(batch, max_blocks) of a ragged batch's arguments: int32, contiguous, on the cache's device."""
        B, mb = table.shape
        i32, dev = torch.int32, self._dev
        assert cu.dtype is i32 and start.dtype is i32 and table.dtype is i32
        assert cu.get_device() == dev and start.get_device() == dev and table.get_device() == dev
        assert cu.is_contiguous() and start.is_contiguous() and table.is_contiguous()
        assert cu.numel() == B + 1 and start.numel() == B
        assert status is None or self._is_status(status)
        return B, mb

    def _is_status(self, x) -> bool:
        return x.dtype is torch.int32 and x.get_device() == self._dev and x.numel() >= 1

    def _rows(self, x, heads):
        """The token and head strides of rows [T, heads, d] (0 where there is one row only)."""
        T, h, d = x.shape
        st, sh, sd = x.stride()
        assert h == heads and d == self.d and sd == 1 and x.get_device() == self._dev
        return (st if T > 1 else 0), (sh if h > 1 else 0)

    def _new_workspace(self, kind, nbytes) -> torch.Tensor:
        # only a decode's counters have to be zero; a captured call clears them in each replay
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.pool.device)
        if kind == "decode":
            ws[self._counters_at:].zero_()
        return ws

    def _workspace(self, kind, key, stream, nbytes) -> torch.Tensor:
        # one for each stream, so that calls on two streams may overlap; a call
        # that is being captured gets its own
        if torch._C._cuda_isCurrentStreamCapturing():
            return self._new_workspace(kind, nbytes(self._h, *key))
        held = self._ws.get((kind, stream))
        if held is None or held[0] != key:
            need = nbytes(self._h, *key)
            if held is None or held[1].numel() < need:
                held = (key, self._new_workspace(kind, need))
            self._ws[(kind, stream)] = held = (key, held[1])
        return held[1]

    def write(self, K: torch.Tensor, V: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor,
              block_table: torch.Tensor, status: torch.Tensor | None = None) -> None:
        """Quantise K, V ([T, num_kv_heads, d], f32/bf16/f16, strided rows on 16-byte boundaries) into the cache."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.write(K, V, cu_tokens, start, block_table, status)
        B, mb = self._batch(cu_tokens, start, block_table, status)
        ks, vs = self._rows(K, self.hkv), self._rows(V, self.hkv)
        T, dtype = K.shape[0], K.dtype
        assert V.shape[0] == T and V.dtype is dtype
        st = self._lib.tq_fp8_write(self._h, K.data_ptr(), V.data_ptr(), _DTYPE_CODES[dtype], *ks, *vs, T, B,
                                    cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), mb, _ptr(status),
                                    torch._C._cuda_getCurrentRawStream(self._dev))
        if st:
            _check(st)

    def read(self, cu_tokens: torch.Tensor, start: torch.Tensor, block_table: torch.Tensor, num_tokens: int,
             dtype: torch.dtype = torch.bfloat16, out: tuple | None = None, status: torch.Tensor | None = None):
        """The stored keys and values of a ragged batch of positions: two [num_tokens, num_kv_heads, d] tensors
        (`out`, or new ones).  Rows that belong to no sequence are not written."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.read(cu_tokens, start, block_table, num_tokens, dtype, out, status)
        B, mb = self._batch(cu_tokens, start, block_table, status)
        if out is None:
            K = torch.empty((num_tokens, self.hkv, self.d), dtype=dtype, device=self.pool.device)
            V = torch.empty_like(K)
        else:
            K, V = out
            for x in out:
                self._rows(x, self.hkv)
                assert x.shape[0] == num_tokens and x.dtype is dtype and x.is_contiguous()
        st = self._lib.tq_fp8_read(self._h, K.data_ptr(), V.data_ptr(), _DTYPE_CODES[dtype], num_tokens, B,
                                   cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), mb, _ptr(status),
                                   torch._C._cuda_getCurrentRawStream(self._dev))
        if st:
            _check(st)
        return K, V

    def _attend_args(self, q, sm_scale, out):
        T, hq, _ = q.shape
        strides = self._rows(q, hq)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            assert out.get_device() == self._dev and out.dtype is q.dtype and out.shape == q.shape
            assert out.is_contiguous()
        return T, hq, strides, self._sm_scale if sm_scale is None else float(sm_scale), out

    def decode(self, q: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, sm_scale: float | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               status: torch.Tensor | None = None) -> torch.Tensor:
        """q: [B, Hq, d] (bf16/f16, strided rows on 16-byte boundaries); lens: int32 [B] -> out [B, Hq, d]
        of q's type.  A workspace is kept for each stream unless one is given (as tq_fp8_decode_attention wants it:
        its counters zero before the first use)."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.decode(q, block_table, lens, sm_scale, out, workspace, status)
        B, hq, strides, sm_scale, out = self._attend_args(q, sm_scale, out)
        rows, mb = block_table.shape
        assert rows == B and lens.numel() == B and lens.dtype is torch.int32 and block_table.dtype is torch.int32
        assert lens.get_device() == self._dev and block_table.get_device() == self._dev
        assert lens.is_contiguous() and block_table.is_contiguous()
        assert status is None or self._is_status(status)
        stream = torch._C._cuda_getCurrentRawStream(self._dev)
        if workspace is None:
            workspace = self._workspace("decode", (B, hq), stream, self._lib.tq_fp8_decode_workspace_bytes)
        else:
            assert workspace.get_device() == self._dev and workspace.is_contiguous()
        st = self._lib.tq_fp8_decode_attention(self._h, q.data_ptr(), _DTYPE_CODES[q.dtype], *strides, B, hq,
                                               block_table.data_ptr(), mb, lens.data_ptr(), sm_scale, out.data_ptr(),
                                               workspace.data_ptr(), workspace.nbytes, _ptr(status), stream)
        if st:
            _check(st)
        return out

    def prefill(self, q: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor, block_table: torch.Tensor,
                sm_scale: float | None = None, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
        """Causal attention of a ragged batch's new tokens (q: [T, Hq, d]; their keys and values written before)
        -> out [T, Hq, d] of q's type.  Rows that belong to no sequence are not written."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.prefill(q, cu_tokens, start, block_table, sm_scale, out, workspace, status)
        B, mb = self._batch(cu_tokens, start, block_table, status)
        T, hq, strides, sm_scale, out = self._attend_args(q, sm_scale, out)
        stream = torch._C._cuda_getCurrentRawStream(self._dev)
        if workspace is None:
            workspace = self._workspace("prefill", (T, B, hq), stream, self._lib.tq_fp8_prefill_workspace_bytes)
        else:
            assert workspace.get_device() == self._dev and workspace.is_contiguous()
        st = self._lib.tq_fp8_prefill_attention(self._h, q.data_ptr(), _DTYPE_CODES[q.dtype], *strides, T, B, hq,
                                                cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), mb,
                                                sm_scale, out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                                _ptr(status), stream)
        if st:
            _check(st)
        return out

    def append(self, K: torch.Tensor, V: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor,
               block_table: torch.Tensor, rotary: Rotary, positions: torch.Tensor | None = None,
               q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, status: torch.Tensor | None = None):
        """write(), with the keys rotated on the way by their positions: int32 [T], or where they are written.  With q
        ([T, Hq, d] of K's type) its rows are rotated by the same launch -> q_out, a new contiguous tensor unless given
        (q itself: in place); rows that belong to no sequence are not written.  Without q -> None."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.append(K, V, cu_tokens, start, block_table, rotary, positions, q, q_out, status)
        B, mb = self._batch(cu_tokens, start, block_table, status)
        ks, vs = self._rows(K, self.hkv), self._rows(V, self.hkv)
        T, dtype = K.shape[0], K.dtype
        assert V.shape[0] == T and V.dtype is dtype and rotary._dev == self._dev
        if positions is not None:
            assert positions.dtype is torch.int32 and positions.get_device() == self._dev and positions.is_contiguous()
            assert positions.numel() == T
        qs, os, hq = (0, 0), (0, 0), 0
        if q is not None:
            hq = q.shape[1]
            qs = self._rows(q, hq)
            assert q.shape[0] == T and q.dtype is dtype
            if q_out is None:
                q_out = torch.empty((T, hq, self.d), dtype=dtype, device=q.device)
            assert q_out.shape == q.shape and q_out.dtype is dtype
            os = self._rows(q_out, hq)
        else:
            assert q_out is None
        st = self._lib.tq_fp8_append(self._h, K.data_ptr(), V.data_ptr(), _DTYPE_CODES[dtype], *ks, *vs, _ptr(q), *qs, hq,
                                     _ptr(q_out), *os, T, B, cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(),
                                     mb, _ptr(positions), rotary.table.data_ptr(), rotary.num_positions, rotary.dim,
                                     rotary._layout, _ptr(status), torch._C._cuda_getCurrentRawStream(self._dev))
        if st:
            _check(st)
        return q_out

    def tree(self, q: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor, block_table: torch.Tensor,
             mask: torch.Tensor, sm_scale: float | None = None, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of a ragged batch of trees of drafted tokens (q: [T, Hq, d]; their keys and values written before):
        node i of a sequence sees every position before start[b] and the nodes j with bit j % 64 of word j / 64 set in
        its row of mask (int64 [T, words], contiguous) -> out [T, Hq, d] of q's type.  Rows that belong to no sequence
        are not written."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.tree(q, cu_tokens, start, block_table, mask, sm_scale, out, workspace, status)
        B, mb = self._batch(cu_tokens, start, block_table, status)
        T, hq, strides, sm_scale, out = self._attend_args(q, sm_scale, out)
        rows, words = mask.shape
        assert rows == T and mask.dtype is torch.int64 and mask.get_device() == self._dev and mask.is_contiguous()
        stream = torch._C._cuda_getCurrentRawStream(self._dev)
        if workspace is None:
            workspace = self._workspace("tree", (T, B, hq), stream, self._lib.tq_fp8_tree_workspace_bytes)
        else:
            assert workspace.get_device() == self._dev and workspace.is_contiguous()
        st = self._lib.tq_fp8_tree_attention(self._h, q.data_ptr(), _DTYPE_CODES[q.dtype], *strides, T, B, hq,
                                             cu_tokens.data_ptr(), start.data_ptr(), block_table.data_ptr(), mb,
                                             mask.data_ptr(), words, sm_scale, out.data_ptr(), workspace.data_ptr(),
                                             workspace.nbytes, _ptr(status), stream)
        if st:
            _check(st)
        return out

    def keep(self, cu_kept: torch.Tensor, kept: torch.Tensor, start: torch.Tensor, block_table: torch.Tensor,
             status: torch.Tensor | None = None) -> None:
        """Moves the accepted nodes up: position start[b] + r becomes what position start[b] + kept[cu_kept[b] + r] was
        (kept: int32, increasing in every sequence; cu_kept: int32 [B + 1])."""
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self.keep(cu_kept, kept, start, block_table, status)
        B, mb = self._batch(cu_kept, start, block_table, status)
        assert kept.dtype is torch.int32 and kept.get_device() == self._dev and kept.is_contiguous()
        st = self._lib.tq_fp8_keep(self._h, kept.numel(), B, cu_kept.data_ptr(), kept.data_ptr(), start.data_ptr(),
                                   block_table.data_ptr(), mb, _ptr(status), torch._C._cuda_getCurrentRawStream(self._dev))
        if st:
            _check(st)
