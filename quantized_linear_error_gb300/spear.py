"""Thin ctypes binding of ``include/spear.h``.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libspear_gb300.so``. The functions keep the C names; :class:`SpearLinear`
is a convenience owner of one handle that takes torch tensors for device
memory and streams. There is no CPU fallback: loading fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import re
from ctypes import POINTER, byref, c_char_p, c_double, c_float, c_int, c_int32, c_int64, c_void_p
from pathlib import Path
from struct import Struct

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libspear_gb300.so"
HEADER = PKG.parent / "include" / "spear.h"

SPEAR_OK, SPEAR_ERR_INVALID_ARG, SPEAR_ERR_UNSUPPORTED, SPEAR_ERR_OOM, SPEAR_ERR_CUDA, SPEAR_ERR_TIMEOUT = range(6)
SPEAR_GATE_SIGMOID, SPEAR_GATE_ONE, SPEAR_GATE_MLP = 0, 1, 2
SPEAR_BF16, SPEAR_F16, SPEAR_F32 = 0, 1, 2
SPEAR_ACT_SILU, SPEAR_ACT_GELU = 0, 1
DECODE_MAX_TOKENS = 32


class spear_linear_desc_t(ctypes.Structure):
    _fields_ = [("K", c_int32), ("N", c_int32), ("group_size", c_int32),
                ("qweight", c_void_p), ("scales", c_void_p), ("zeros", c_void_p),
                ("rank", c_int32), ("A", c_void_p), ("B", c_void_p),
                ("alpha", c_float), ("gate", c_int), ("max_tokens", c_int32),
                ("gate_hidden", c_int32), ("gate_w1", c_void_p), ("gate_w2", c_void_p)]


class spear_kv_desc_t(ctypes.Structure):
    _fields_ = [("n_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32), ("page_size", c_int32),
                ("n_pages", c_int32), ("pool", c_void_p), ("rope_dim", c_int32), ("rope_interleaved", c_int32),
                ("n_positions", c_int32), ("rope_table", c_void_p)]


class spear_w8_desc_t(ctypes.Structure):
    _fields_ = [("K", c_int32), ("N", c_int32), ("qweight", c_void_p), ("scales", c_void_p), ("qweight_up", c_void_p),
                ("scales_up", c_void_p), ("activation", c_int), ("max_tokens", c_int32), ("workspace", c_void_p),
                ("workspace_bytes", c_int64)]


class SpearError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


_lib = None


def header_functions() -> list[str]:
    """Names of the functions ``include/spear.h`` declares."""
    text = HEADER.read_text()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(spear_\w+)\s*\(", text, re.M)))


def load(path: Path | None = None):
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = Path(path or LIB_PATH)
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build it with quantized_linear_error_gb300.build.build()")
    L = ctypes.CDLL(str(p))
    H = c_void_p  # opaque handle / stream
    L.spear_linear_create.argtypes = [POINTER(spear_linear_desc_t), H, POINTER(c_void_p)]
    L.spear_linear_create_grouped.argtypes = [POINTER(spear_linear_desc_t), c_int32, H, POINTER(c_void_p)]
    L.spear_linear_create_grouped.restype = c_int
    L.spear_linear_forward_decode.argtypes = [H, c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward_prefill.argtypes = [H, c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward.argtypes = [H, c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward_prefill_concurrent.argtypes = [H, c_void_p, c_void_p, c_int32, H, H]
    L.spear_linear_forward_prefill_concurrent.restype = c_int
    L.spear_linear_enable_concurrent_ec.argtypes = [H]
    L.spear_linear_enable_concurrent_ec.restype = c_int
    L.spear_linear_forward_host.argtypes = [H, c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward_host_batch.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward_host_batch.restype = c_int
    L.spear_linear_destroy.argtypes = [H]
    L.spear_linear_dequantize.argtypes = [H, c_int32, c_void_p, H]
    L.spear_linear_check.argtypes = [H, H]
    L.spear_linear_debug_set.argtypes = [H, c_int64, c_int32]
    L.spear_linear_forward_decode_noalloc.argtypes = [POINTER(spear_linear_desc_t), c_void_p, c_void_p, c_int32, H]
    L.spear_linear_forward_decode_noalloc.restype = c_int
    L.spear_sched_create.argtypes = [c_void_p, c_int32, c_void_p, c_int32, c_void_p, POINTER(c_void_p)]
    L.spear_sched_create.restype = c_int
    L.spear_sched_predict.argtypes = [H, c_int32, c_double]
    L.spear_sched_predict.restype = c_double
    L.spear_sched_pick_chunk.argtypes = [H, c_int32, c_double, c_double, c_void_p, c_int32, POINTER(c_int32)]
    L.spear_sched_pick_chunk.restype = c_int
    L.spear_sched_destroy.argtypes = [H]
    L.spear_sched_destroy.restype = c_int
    L.spear_quantize_rtn.argtypes = [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, H]
    L.spear_quantize_rtn.restype = c_int
    L.spear_decode_schedule.argtypes = [c_int32] * 8 + [c_void_p]
    L.spear_decode_schedule.restype = c_int
    L.spear_prefill_schedule.argtypes = [c_int32] * 7 + [c_void_p, c_void_p, c_int32]
    L.spear_prefill_schedule.restype = c_int
    L.spear_kv_create.argtypes = [POINTER(spear_kv_desc_t), H, POINTER(c_void_p)]
    L.spear_kv_append.argtypes = [H, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p,
                                  c_int32, c_void_p, c_int64, H]
    L.spear_kv_read.argtypes = [H, c_void_p, c_int32, c_void_p, c_void_p, H]
    L.spear_kv_attention.argtypes = [H, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32, c_void_p, c_void_p,
                                     c_int32, c_int32, c_int32, c_float, c_int32, H]
    L.spear_kv_check.argtypes = [H, H]
    L.spear_kv_destroy.argtypes = [H]
    L.spear_rms_norm.argtypes = [H, c_int64, c_int, H, c_int64, H, c_int64, c_int, H, c_int, c_float, c_int32, c_int32,
                                 H, c_int64, H, c_int64, H, H]
    L.spear_quantize_rows.argtypes = [H, c_int64, c_int, c_int32, c_int32, H, c_int64, H, H]
    L.spear_dequantize_rows.argtypes = [H, c_int64, H, c_int32, c_int32, H, c_int64, c_int, H]
    L.spear_w8_workspace.argtypes = [POINTER(spear_w8_desc_t), POINTER(c_int64)]
    L.spear_w8_create.argtypes = [POINTER(spear_w8_desc_t), H, POINTER(c_void_p)]
    L.spear_w8_forward.argtypes = [H, H, c_int64, H, H, c_int64, c_int, c_int32, H]
    for name in ("spear_rms_norm_args", "spear_quantize_rows_args", "spear_dequantize_rows_args", "spear_w8_forward_args"):
        getattr(L, name).argtypes = [c_char_p]  # a packed struct
        getattr(L, name).restype = c_int
    L.spear_w8_check.argtypes = [H, H]
    L.spear_w8_destroy.argtypes = [H]
    L.spear_w8_debug_set.argtypes = [H, c_int64, c_int32]
    L.spear_status_string.argtypes = [c_int]
    L.spear_status_string.restype = c_char_p
    for name in ("spear_linear_create", "spear_linear_forward_decode", "spear_linear_forward_prefill",
                 "spear_linear_forward", "spear_linear_forward_host", "spear_linear_destroy",
                 "spear_linear_dequantize", "spear_linear_check", "spear_linear_debug_set",
                 "spear_kv_create", "spear_kv_append", "spear_kv_read", "spear_kv_attention", "spear_kv_check",
                 "spear_kv_destroy", "spear_rms_norm", "spear_quantize_rows", "spear_dequantize_rows",
                 "spear_w8_workspace", "spear_w8_create", "spear_w8_forward", "spear_w8_check", "spear_w8_destroy",
                 "spear_w8_debug_set"):
        getattr(L, name).restype = c_int
    _lib = L
    return L


def status_string(s: int) -> str:
    return load().spear_status_string(s).decode()


def _check(status: int, what: str) -> None:
    if status != SPEAR_OK:
        raise SpearError(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = None  # torch's accessor of the current stream's handle, once torch is loaded


def _stream(stream) -> int:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            # (device index) -> cudaStream_t; current_stream() builds a Stream object, 3 us a call
            get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            torch.cuda.current_stream()  # initialises CUDA
            _raw_stream = (lambda: get(dev())) if get and dev else (lambda: torch.cuda.current_stream().cuda_stream)
        return _raw_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class SpearLinear:
    """Owner of one ``spear_linear_t``.

    ``qweight`` uint8 [N][K/2], ``scales`` bf16 [N][K/G], ``zeros`` uint8
    [N][K/G] or None, ``A`` bf16 [r][K], ``B`` bf16 [N][r] (None when r = 0),
    and for the MLP gate ``W1`` bf16 [h][r], ``W2`` bf16 [r][h]: CUDA tensors
    in the layout ``spear_linear_desc_t`` documents. The library copies them;
    the tensors may be freed after construction.
    """

    def __init__(self, K, N, group_size, qweight, scales, zeros=None, A=None, B=None,
                 alpha=1.0, gate=SPEAR_GATE_SIGMOID, max_tokens=32, stream=None, W1=None, W2=None):
        L = load()
        rank = 0 if A is None else int(A.shape[0])
        hidden = 0 if W1 is None else int(W1.shape[0])
        d = spear_linear_desc_t(int(K), int(N), int(group_size), _ptr(qweight), _ptr(scales), _ptr(zeros),
                                rank, _ptr(A), _ptr(B), float(alpha), int(gate), int(max_tokens),
                                hidden, _ptr(W1), _ptr(W2))
        h = c_void_p()
        _check(L.spear_linear_create(byref(d), _stream(stream), byref(h)), "spear_linear_create")
        self.h = h
        self.K, self.N, self.rank, self.max_tokens = int(K), int(N), rank, int(max_tokens)

    @classmethod
    def grouped(cls, members, max_tokens=32, stream=None):
        """One handle for linears sharing x (spear_linear_create_grouped).
        ``members``: list of dicts with the keyword arguments of the
        constructor (K, N, group_size, qweight, scales, zeros, A, B, alpha,
        gate). y of the handle is [M][sum of the members' N]."""
        L = load()
        n = len(members)
        arr = (spear_linear_desc_t * n)()
        for i, m in enumerate(members):
            A = m.get("A")
            arr[i] = spear_linear_desc_t(int(m["K"]), int(m["N"]), int(m["group_size"]), _ptr(m["qweight"]),
                                         _ptr(m["scales"]), _ptr(m.get("zeros")), 0 if A is None else int(A.shape[0]),
                                         _ptr(A), _ptr(m.get("B")), float(m.get("alpha", 1.0)),
                                         int(m.get("gate", SPEAR_GATE_SIGMOID)), int(max_tokens), 0, None, None)
        h = c_void_p()
        _check(L.spear_linear_create_grouped(arr, n, _stream(stream), byref(h)), "spear_linear_create_grouped")
        self = cls.__new__(cls)
        self.h = h
        self.K = int(members[0]["K"])
        self.N = sum(int(m["N"]) for m in members)
        self.rank = 0 if members[0].get("A") is None else int(members[0]["A"].shape[0]) * n
        self.max_tokens = int(max_tokens)
        return self

    def _io(self, fn, x, y, M, stream, what):
        _check(fn(self.h, _ptr(x), _ptr(y), int(M), _stream(stream)), what)

    def forward_decode(self, x, y, stream=None):
        self._io(load().spear_linear_forward_decode, x, y, x.shape[0], stream, "spear_linear_forward_decode")
        return y

    def forward_prefill(self, x, y, stream=None):
        self._io(load().spear_linear_forward_prefill, x, y, x.shape[0], stream, "spear_linear_forward_prefill")
        return y

    def enable_concurrent_ec(self) -> None:
        _check(load().spear_linear_enable_concurrent_ec(self.h), "spear_linear_enable_concurrent_ec")

    def forward_prefill_concurrent(self, x, y, stream=None, ec_stream=None):
        """Prefill with the compensator pre-kernel on ec_stream (a torch stream)."""
        _check(load().spear_linear_forward_prefill_concurrent(self.h, _ptr(x), _ptr(y), int(x.shape[0]),
                                                              _stream(stream), _stream(ec_stream)),
               "spear_linear_forward_prefill_concurrent")
        return y

    def forward(self, x, y, stream=None):
        self._io(load().spear_linear_forward, x, y, x.shape[0], stream, "spear_linear_forward")
        return y

    def forward_host(self, x_host, y_host, stream=None):
        self._io(load().spear_linear_forward_host, x_host, y_host, x_host.shape[0], stream,
                 "spear_linear_forward_host")
        return y_host

    def dequantize(self, out, path=0, stream=None):
        _check(load().spear_linear_dequantize(self.h, int(path), _ptr(out), _stream(stream)),
               "spear_linear_dequantize")
        return out

    def check(self, stream=None) -> int:
        return load().spear_linear_check(self.h, _stream(stream))

    def debug_set(self, wait_ns: int = 0, skip_arrive: bool = False) -> None:
        _check(load().spear_linear_debug_set(self.h, int(wait_ns), int(bool(skip_arrive))), "spear_linear_debug_set")

    def close(self) -> None:
        if getattr(self, "h", None) and self.h.value:
            load().spear_linear_destroy(self.h)
            self.h = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def forward_host_batch(linears, xs_host, ys_host, stream=None) -> None:
    """spear_linear_forward_host_batch over (SpearLinear, host x, host y)
    triples: the forwards in order on `stream`, the copies on the first
    handle's copy streams overlapping them, one synchronisation at the end."""
    n = len(linears)
    hs = (c_void_p * n)(*[lin.h.value for lin in linears])
    xp = (c_void_p * n)(*[x.data_ptr() for x in xs_host])
    yp = (c_void_p * n)(*[y.data_ptr() for y in ys_host])
    ms = (c_int32 * n)(*[int(x.shape[0]) for x in xs_host])
    _check(load().spear_linear_forward_host_batch(hs, xp, yp, ms, n, _stream(stream)),
           "spear_linear_forward_host_batch")


def from_weights(w, device="cuda", max_tokens=32, alpha=None, gate=None, stream=None) -> SpearLinear:
    """Build a :class:`SpearLinear` from ``workload.LinearWeights`` (host numpy)."""
    import numpy as np
    import torch

    def dev(a, dt):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).view(dt).to(device)

    sp = w.spec
    q = dev(w.q, torch.uint8)
    s = dev(w.s.view(np.int16), torch.bfloat16)
    z = dev(w.z, torch.uint8)
    A = dev(w.A.view(np.int16), torch.bfloat16) if sp.rank else None
    B = dev(w.B.view(np.int16), torch.bfloat16) if sp.rank else None
    W1 = dev(w.W1.view(np.int16), torch.bfloat16) if getattr(w, "W1", None) is not None else None
    W2 = dev(w.W2.view(np.int16), torch.bfloat16) if getattr(w, "W2", None) is not None else None
    lin = SpearLinear(sp.K, sp.N, sp.group_size, q, s, z, A, B,
                      sp.alpha if alpha is None else alpha, sp.gate if gate is None else gate,
                      max_tokens, stream, W1, W2)
    return lin


def grouped_from_weights(ws, device="cuda", max_tokens=32, stream=None) -> SpearLinear:
    """A grouped :class:`SpearLinear` from several ``workload.LinearWeights``
    sharing K (host numpy); member i's outputs are columns
    [N_0 + ... + N_{i-1}, + N_i) of y."""
    import numpy as np
    import torch

    def dev(a, dt):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).view(dt).to(device)

    members, keep = [], []
    for w in ws:
        sp = w.spec
        m = {"K": sp.K, "N": sp.N, "group_size": sp.group_size, "qweight": dev(w.q, torch.uint8),
             "scales": dev(w.s.view(np.int16), torch.bfloat16), "zeros": dev(w.z, torch.uint8),
             "A": dev(w.A.view(np.int16), torch.bfloat16) if sp.rank else None,
             "B": dev(w.B.view(np.int16), torch.bfloat16) if sp.rank else None,
             "alpha": sp.alpha, "gate": sp.gate}
        members.append(m)
    return SpearLinear.grouped(members, max_tokens=max_tokens, stream=stream)


def quantize_rtn(w, group_size=128, stream=None):
    """RTN 4-bit quantisation of a CUDA fp32 tensor w [N][K] by the library's
    kernel: returns (qweight uint8 [N][K/2], scales bf16 [N][K/G], zeros uint8
    [N][K/G]) in the layout :class:`SpearLinear` takes."""
    import torch
    N, K = w.shape
    G = K if group_size == 0 else group_size
    w = w.contiguous()
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // G), dtype=torch.bfloat16, device=w.device)
    z = torch.empty((N, K // G), dtype=torch.uint8, device=w.device)
    _check(load().spear_quantize_rtn(_ptr(w), int(N), int(K), int(group_size), _ptr(q), _ptr(s), _ptr(z),
                                     _stream(stream)), "spear_quantize_rtn")
    return q, s, z


def kv_page_bytes(n_kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of one page of the 4-bit key/value cache."""
    return n_kv_heads * (page_size // 16) * 16 * (head_dim + 8)


def kv_pool(n_pages: int, n_kv_heads: int, head_dim: int, page_size: int, device="cuda"):
    """A zeroed pool for :class:`SpearKVCache`: uint8 [n_pages][n_kv_heads][page bytes of a head]."""
    import torch
    return torch.zeros((n_pages, n_kv_heads, kv_page_bytes(1, head_dim, page_size)), dtype=torch.uint8, device=device)


def rope_table(n_positions: int, rope_dim: int, base: float = 10000.0, device="cuda"):
    """fp32 [n_positions][rope_dim]: the cosines, then the sines, of p * base^(-2 i / rope_dim)."""
    import torch
    inv = base ** (-torch.arange(0, rope_dim, 2, device=device, dtype=torch.float64) / rope_dim)
    a = torch.arange(n_positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


class SpearKVCache:
    """Owner of one ``spear_kv_t``: a paged 4-bit key/value cache with the
    append that fills it and the attention that reads it.

    ``pool`` uint8 [n_pages][n_kv_heads][page_size * (head_dim + 8)] (see
    :func:`kv_pool`) and ``rope_table`` fp32 [n_positions][rope_dim] or None are
    CUDA tensors that the object keeps; layers may share a table, and handles
    over different pools are independent.
    """

    def __init__(self, n_heads, n_kv_heads, head_dim, page_size, pool, rope_table=None, rope_interleaved=False,
                 stream=None):
        import torch
        page = kv_page_bytes(n_kv_heads, head_dim, page_size)
        if pool.dtype != torch.uint8 or not pool.is_cuda or not pool.is_contiguous() or \
                pool.numel() != pool.shape[0] * page:
            raise ValueError(f"pool must be contiguous CUDA uint8 [n_pages][{page} bytes a page]")
        if rope_table is not None and (rope_table.dtype != torch.float32 or rope_table.dim() != 2 or
                                       not rope_table.is_cuda or not rope_table.is_contiguous()):
            raise ValueError("rope_table must be contiguous CUDA fp32 [n_positions][rope_dim]")
        positions, rope_dim = (0, 0) if rope_table is None else rope_table.shape
        d = spear_kv_desc_t(int(n_heads), int(n_kv_heads), int(head_dim), int(page_size), int(pool.shape[0]),
                            _ptr(pool), int(rope_dim), int(bool(rope_interleaved)), int(positions), _ptr(rope_table))
        h = c_void_p()
        L = load()
        _check(L.spear_kv_create(byref(d), _stream(stream), byref(h)), "spear_kv_create")
        self.h, self.pool, self.rope_table = h, pool, rope_table
        self.n_heads, self.n_kv_heads, self.head_dim, self.page_size = n_heads, n_kv_heads, head_dim, page_size
        self._bf16, self._i64, self._i32 = torch.bfloat16, torch.int64, torch.int32
        self._append, self._read, self._attention = L.spear_kv_append, L.spear_kv_read, L.spear_kv_attention
        self._scale = head_dim ** -0.5

    def _bad_rows(self, **xs):
        """Says what is wrong with one of the tensors bf16 [T][heads][D]."""
        for what, (x, T, heads) in xs.items():
            shape = (T, heads, self.head_dim)
            if x.dtype is not self._bf16 or not x.is_cuda or x.shape != shape:
                raise ValueError(f"{what} must be CUDA bf16 {list(shape)}")
            s = x.stride()
            if s[2] != 1 or (s[1] != self.head_dim and heads > 1):
                raise ValueError(f"{what}: the heads of a token must be contiguous")
        raise ValueError("indices must be contiguous CUDA tensors: int64 positions and slots, int32 tables and lengths, "
                         "with an element for every token or sequence")

    def append(self, q, k, v, positions, slots, q_out=None, stream=None):
        """Rotate q [T][n_heads][D] (or None) and k [T][n_kv_heads][D] to the
        int64 ``positions`` and put k and v into the int64 ``slots`` (-1: not
        cached). The rotated queries go to ``q_out`` (default: q in place)."""
        T, H, G, D, bf16, i64 = k.shape[0], self.n_heads, self.n_kv_heads, self.head_dim, self._bf16, self._i64
        qp = op = ldq = ldo = 0
        ldk, k1, k2 = k.stride()
        ldv, v1, v2 = v.stride()
        # one expression for all of them: it is on every step's way
        ok = (k.dtype is bf16 and v.dtype is bf16 and k.shape == (T, G, D) == v.shape and k.is_cuda and v.is_cuda and
              k2 == 1 == v2 and (k1 == D == v1 or G == 1) and
              slots.dtype is i64 and slots.is_cuda and slots.is_contiguous() and slots.numel() >= T)
        if q is not None:
            if q_out is None:
                q_out = q
            ldq, q1, q2 = q.stride()
            ldo, o1, o2 = q_out.stride()
            ok = ok and (q.dtype is bf16 and q_out.dtype is bf16 and q.shape == (T, H, D) == q_out.shape and
                         q.is_cuda and q_out.is_cuda and q2 == 1 == o2 and (q1 == D == o1 or H == 1))
            qp, op = q.data_ptr(), q_out.data_ptr()
        if self.rope_table is not None:
            ok = ok and (positions is not None and positions.dtype is i64 and positions.is_cuda and
                         positions.is_contiguous() and positions.numel() >= T)
        if not ok:
            rows = {"k": (k, T, G), "v": (v, T, G)}
            self._bad_rows(**rows, **({} if q is None else {"q": (q, T, H), "q_out": (q_out, T, H)}))
        pos = 0 if self.rope_table is None else positions.data_ptr()
        if T < 2:  # the stride of a single token means nothing
            ldq, ldo, ldk, ldv = H * D, H * D, G * D, G * D
        st = self._append(self.h, qp, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, pos, slots.data_ptr(), T, op, ldo,
                          _stream(stream))
        if st:
            raise SpearError(st, "spear_kv_append")
        return q_out

    def read(self, slots, k_out, v_out, stream=None):
        """The cached keys and values of ``slots`` as bf16 [T][n_kv_heads][D]."""
        T, G, D, bf16 = slots.shape[0], self.n_kv_heads, self.head_dim, self._bf16
        if not (k_out.dtype is bf16 and v_out.dtype is bf16 and k_out.shape == (T, G, D) == v_out.shape and
                k_out.is_cuda and v_out.is_cuda and k_out.is_contiguous() and v_out.is_contiguous() and
                slots.dtype is self._i64 and slots.is_cuda and slots.is_contiguous()):
            if not (k_out.is_contiguous() and v_out.is_contiguous()):
                raise ValueError("k_out and v_out must be contiguous")
            self._bad_rows(k_out=(k_out, T, G), v_out=(v_out, T, G))
        st = self._read(self.h, slots.data_ptr(), T, k_out.data_ptr(), v_out.data_ptr(), _stream(stream))
        if st:
            raise SpearError(st, "spear_kv_read")
        return k_out, v_out

    def attention(self, q, out, page_table, kv_lens, q_starts, max_q, scale=None, window=0, stream=None):
        """Causal attention of the query rows q [T][n_heads][D] over the cache
        into ``out`` (see spear_kv_attention): int32 ``page_table``
        [n_seqs][max pages], ``kv_lens`` [n_seqs], ``q_starts`` [n_seqs + 1];
        ``scale`` defaults to head_dim ** -0.5, ``window`` 0 means all earlier keys."""
        T, H, D, bf16, i32 = q.shape[0], self.n_heads, self.head_dim, self._bf16, self._i32
        if page_table.dim() != 2:
            raise ValueError("page_table must have two dimensions")
        n, cols = page_table.shape
        ldq, q1, q2 = q.stride()
        ldo, o1, o2 = out.stride()
        if not (q.dtype is bf16 and out.dtype is bf16 and q.shape == (T, H, D) == out.shape and q.is_cuda and
                out.is_cuda and q2 == 1 == o2 and (q1 == D == o1 or H == 1) and
                page_table.dtype is i32 and page_table.is_cuda and page_table.is_contiguous() and
                kv_lens.dtype is i32 and kv_lens.is_cuda and kv_lens.is_contiguous() and kv_lens.numel() >= n and
                q_starts.dtype is i32 and q_starts.is_cuda and q_starts.is_contiguous() and q_starts.numel() > n):
            self._bad_rows(q=(q, T, H), out=(out, T, H))
        if T < 2:  # the stride of a single token means nothing
            ldq = ldo = H * D
        if max_q >> 31 or window >> 31:  # ctypes would cut them to 32 bits; below zero stays refused
            max_q, window = (min(max(x, -1), (1 << 31) - 1) for x in (max_q, window))
        st = self._attention(self.h, q.data_ptr(), ldq, out.data_ptr(), ldo, page_table.data_ptr(), cols,
                             kv_lens.data_ptr(), q_starts.data_ptr(), n, T, max_q,
                             self._scale if scale is None else scale, window, _stream(stream))
        if st:
            raise SpearError(st, "spear_kv_attention")
        return out

    def check(self, stream=None) -> int:
        return load().spear_kv_check(self.h, _stream(stream))

    def close(self) -> None:
        if getattr(self, "h", None) and self.h.value:
            load().spear_kv_destroy(self.h)
            self.h = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Rows:
    """What the calls on rows look up: torch's types, once torch is loaded."""

    def __init__(self):
        import torch
        self.types = {torch.bfloat16: SPEAR_BF16, torch.float16: SPEAR_F16, torch.float32: SPEAR_F32}
        self.i8, self.f32, self.empty = torch.int8, torch.float32, torch.empty
        self.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        # (device index) -> its current stream's handle
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: _stream(None))
        self.cuda = torch.cuda
        L = load()
        self.norm, self.quantize, self.dequantize, self.forward = (
            L.spear_rms_norm_args, L.spear_quantize_rows_args, L.spear_dequantize_rows_args, L.spear_w8_forward_args)
        # their structs: addresses and distances of 64 bits, then sizes and types of 32
        self.norm_args, self.quantize_args = Struct("=QqQqQqQQqQqQQ5if").pack, Struct("=QqQqQQ3i").pack
        self.dequantize_args, self.forward_args = Struct("=QqQQqQ3i").pack, Struct("=QQqQQqQ2i").pack

    def on(self, stream):
        """Context in which tensors are made on `stream` (the current one if None)."""
        if stream is not None and not isinstance(stream, self.cuda.Stream):
            stream = self.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
        return self.cuda.stream(stream)


_rows_ = None


def _rows() -> _Rows:
    global _rows_
    if _rows_ is None:
        _rows_ = _Rows()
    return _rows_


def _not_here(what, device):
    raise ValueError(f"{what}: the tensors have to be on one device, which is the current one (they start on cuda:{device})")


def _int32(what, **sizes):
    for name, n in sizes.items():
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{what}: {name} = {n} is past 32 bits")


def _ld(what, name, x, M, K, *dtypes) -> int:
    """Elements from one row of x to the next, of a CUDA tensor [M][K] with contiguous rows of one of the dtypes."""
    if x.dtype not in dtypes or not x.is_cuda or x.shape != (M, K):
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{what}: {name} must be CUDA {kinds} [{M}][{K}]")
    ld, one = x.stride()
    if one != 1 and K > 1:
        raise ValueError(f"{what}: {name}: the elements of a row must be contiguous")
    return ld if M > 1 else K  # the stride of a single row means nothing


def _vector(what, name, x, n, *dtypes) -> int:
    """Address of a contiguous CUDA tensor [n] of one of the dtypes."""
    if x.dtype not in dtypes or not x.is_cuda or x.shape != (n,) or not x.is_contiguous():
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{what}: {name} must be contiguous CUDA {kinds} [{n}]")
    return x.data_ptr()


def rms_norm(x, weight, eps=1e-5, residual=None, residual_out=None, y=None, q=None, scales=None, stream=None):
    """Root-mean-square norm of the rows of x [M][K] (bf16, f16 or fp32) times ``weight`` [K] (x's type or fp32), in one
    launch. ``residual`` [M][K] (x's type or fp32) is added to x first and the sum goes to ``residual_out`` (default: in
    place). The result goes to ``y`` (x's type), to ``q`` int8 [M][K] with ``scales`` fp32 [M] (8-bit rows, as
    :class:`SpearW8Linear` takes them), or to both. See spear_rms_norm."""
    r = _rows_ or _rows()
    types, f32, shape, xt, wt = r.types, r.f32, x.shape, x.dtype, weight.dtype
    M, K = shape
    # one expression for all of a kind: it is on every step's way
    ld_x, one = x.stride()
    dev = x.get_device()
    ok = (xt in types and (wt is xt or wt is f32) and dev == weight.get_device() and weight.shape == (K,) and
          weight.is_contiguous() and not (M | K) >> 31)
    t, rp, ro, ld_r, ld_ro, rt, yp, ld_y, qp, ld_q, sp = types.get(xt, 0), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0
    if residual is not None:
        if residual_out is None:
            residual_out = residual
        rd = residual.dtype
        (ld_r, one_r), (ld_ro, one_ro) = residual.stride(), residual_out.stride()
        ok = (ok and (rd is xt or rd is f32) and residual_out.dtype is rd and residual.shape == shape == residual_out.shape and
              dev == residual.get_device() == residual_out.get_device() and (one_r == 1 == one_ro or K == 1))
        rt, rp, ro = types.get(rd, 0), residual.data_ptr(), residual_out.data_ptr()
    else:
        ok = ok and residual_out is None
    if y is not None:
        ld_y, one_y = y.stride()
        ok = ok and y.dtype is xt and y.shape == shape and y.get_device() == dev and (one_y == 1 or K == 1)
        yp = y.data_ptr()
    if q is not None and scales is not None:
        ld_q, one_q = q.stride()
        ok = (ok and q.dtype is r.i8 and q.shape == shape and q.get_device() == dev and (one_q == 1 or K == 1) and
              scales.dtype is f32 and scales.shape == (M,) and scales.get_device() == dev and scales.is_contiguous())
        qp, sp = q.data_ptr(), scales.data_ptr()
    else:
        ok = ok and q is None and scales is None and y is not None
    if not ok or dev < 0 or (one != 1 and K > 1) or dev != r.device():
        _bad_norm(r, x, weight, residual, residual_out, y, q, scales)
    if M < 2:  # the stride of a single row means nothing
        ld_x = ld_r = ld_ro = ld_y = ld_q = K
    st = r.norm(r.norm_args(x.data_ptr(), ld_x, rp, ld_r, ro, ld_ro, weight.data_ptr(), yp, ld_y, qp, ld_q, sp,
                            r.stream(dev) if stream is None else _stream(stream), t, rt, types[wt], M, K, eps))
    if st:
        raise SpearError(st, "spear_rms_norm")
    return y if q is None else (q, scales)


def _bad_norm(r, x, weight, residual, residual_out, y, q, scales):
    """Says what is wrong with the arguments of rms_norm."""
    (M, K), xt = x.shape, x.dtype
    _ld("rms_norm", "x", x, M, K, *r.types)
    _vector("rms_norm", "weight", weight, K, xt, r.f32)
    if residual is not None:
        _ld("rms_norm", "residual", residual, M, K, xt, r.f32)
        _ld("rms_norm", "residual_out", residual_out, M, K, residual.dtype)
    elif residual_out is not None:
        raise ValueError("rms_norm: residual_out without residual")
    if y is not None:
        _ld("rms_norm", "y", y, M, K, xt)
    if q is not None and scales is not None:
        _ld("rms_norm", "q", q, M, K, r.i8)
        _vector("rms_norm", "scales", scales, M, r.f32)
    if (q is None) != (scales is None) or (q is None and y is None):
        raise ValueError("rms_norm: give y, or q and scales, or all three")
    _int32("rms_norm", M=M, K=K)
    _not_here("rms_norm", x.get_device())


def quantize_rows(x, q=None, scales=None, stream=None):
    """Rows of x [M][K] (bf16, f16 or fp32) in 8 bits: (q int8 [M][K], scales fp32 [M]), made if not given; activations
    with a scale a token, or weights with a scale an output channel. See spear_quantize_rows."""
    r = _rows_ or _rows()
    shape, xt = x.shape, x.dtype
    M, K = shape
    if q is None or scales is None:
        with r.on(stream):  # of the stream that writes them: memory that another stream has freed may still be in use there
            q = r.empty((M, K), dtype=r.i8, device=x.device) if q is None else q
            scales = r.empty((M,), dtype=r.f32, device=x.device) if scales is None else scales
    (ld_x, one), (ld_q, one_q) = x.stride(), q.stride()
    dev = x.get_device()
    if not (xt in r.types and q.dtype is r.i8 and q.shape == shape and dev == q.get_device() == scales.get_device() and
            (one == 1 == one_q or K == 1) and scales.dtype is r.f32 and scales.shape == (M,) and
            scales.is_contiguous() and not (M | K) >> 31 and dev >= 0 and dev == r.device()):
        _ld("quantize_rows", "x", x, M, K, *r.types)
        _ld("quantize_rows", "q", q, M, K, r.i8)
        _vector("quantize_rows", "scales", scales, M, r.f32)
        _int32("quantize_rows", M=M, K=K)
        _not_here("quantize_rows", dev)
    if M < 2:
        ld_x = ld_q = K
    st = r.quantize(r.quantize_args(x.data_ptr(), ld_x, q.data_ptr(), ld_q, scales.data_ptr(),
                                    r.stream(dev) if stream is None else _stream(stream), r.types[xt], M, K))
    if st:
        raise SpearError(st, "spear_quantize_rows")
    return q, scales


def dequantize_rows(q, scales, out, stream=None):
    """What 8-bit rows stand for, q * scales, into ``out`` [M][K] (bf16, f16 or fp32). See spear_dequantize_rows."""
    r = _rows_ or _rows()
    shape, ot = q.shape, out.dtype
    M, K = shape
    (ld_q, one_q), (ld_o, one) = q.stride(), out.stride()
    dev = q.get_device()
    if not (ot in r.types and q.dtype is r.i8 and out.shape == shape and dev == out.get_device() == scales.get_device() and
            (one == 1 == one_q or K == 1) and scales.dtype is r.f32 and scales.shape == (M,) and
            scales.is_contiguous() and not (M | K) >> 31 and dev >= 0 and dev == r.device()):
        _ld("dequantize_rows", "q", q, M, K, r.i8)
        _ld("dequantize_rows", "out", out, M, K, *r.types)
        _vector("dequantize_rows", "scales", scales, M, r.f32)
        _int32("dequantize_rows", M=M, K=K)
        _not_here("dequantize_rows", dev)
    if M < 2:
        ld_q = ld_o = K
    st = r.dequantize(r.dequantize_args(q.data_ptr(), ld_q, scales.data_ptr(), out.data_ptr(), ld_o,
                                        r.stream(dev) if stream is None else _stream(stream), r.types[ot], M, K))
    if st:
        raise SpearError(st, "spear_dequantize_rows")
    return out


def w8_workspace_bytes(N, K, max_tokens, gated=False) -> int:
    """Bytes of the workspace of a :class:`SpearW8Linear` with weights [N][K]; the largest of several layers serves all."""
    _int32("w8_workspace_bytes", N=int(N), K=int(K), max_tokens=int(max_tokens))
    some = 4096  # any address: nothing is read
    up = some if gated else None
    d = spear_w8_desc_t(int(K), int(N), some, some, up, up, SPEAR_ACT_SILU, int(max_tokens), None, 0)
    n = c_int64()
    _check(load().spear_w8_workspace(byref(d), byref(n)), "spear_w8_workspace")
    return n.value


class SpearW8Linear:
    """Owner of one ``spear_w8_t``: a linear of 8-bit integer weights and activations.

    ``qweight`` int8 [N][K] and ``scales`` fp32 [N] (see :func:`quantize_rows`) are contiguous CUDA tensors; with ``up`` and
    ``up_scales`` of the same shapes the layer is a gated pair, act(x W^T) * (x U^T), ``activation`` "silu" or "gelu" (the
    tanh form). The library copies them; the tensors may be freed after construction. Linears that read the same x (q, k
    and v) are one layer of their weights stacked along N.

    ``workspace`` is a CUDA uint8 tensor of at least :func:`w8_workspace_bytes`, which layers whose calls follow one another
    may share (the object keeps it); without one the layer has its own.
    """

    def __init__(self, qweight, scales, max_tokens=32, up=None, up_scales=None, activation="silu", workspace=None,
                 stream=None):
        r = _rows()
        N, K = qweight.shape
        acts = {"silu": SPEAR_ACT_SILU, "gelu": SPEAR_ACT_GELU}
        if activation not in acts:
            raise ValueError(f"activation must be one of {sorted(acts)}")
        if (up is None) != (up_scales is None):
            raise ValueError("up and up_scales come together")
        for name, w, s in (("qweight", qweight, scales), ("up", up, up_scales)):
            if w is not None:
                if _ld("SpearW8Linear", name, w, N, K, r.i8) != K or not w.is_contiguous():
                    raise ValueError(f"SpearW8Linear: {name} must be contiguous")
                _vector("SpearW8Linear", "the scales of " + name, s, N, r.f32)
        _int32("SpearW8Linear", N=N, K=K, max_tokens=int(max_tokens))
        dev = qweight.get_device()
        if dev != r.device() or any(t is not None and t.get_device() != dev for t in (scales, up, up_scales, workspace)):
            _not_here("SpearW8Linear", dev)
        d = spear_w8_desc_t(K, N, _ptr(qweight), _ptr(scales), _ptr(up), _ptr(up_scales), acts[activation], int(max_tokens),
                            None, 0)
        if workspace is not None:
            if not workspace.is_cuda or not workspace.is_contiguous():
                raise ValueError("SpearW8Linear: workspace must be a contiguous CUDA tensor")
            d.workspace, d.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        h = c_void_p()
        L = load()
        _check(L.spear_w8_create(byref(d), _stream(stream), byref(h)), "spear_w8_create")
        self.h, self.K, self.N, self.gated, self.max_tokens = h, K, N, up is not None, int(max_tokens)
        self.workspace = workspace
        self._forward, self._types, self._i8, self._f32, self._device = r.forward, r.types, r.i8, r.f32, dev
        self._args, self._stream = r.forward_args, r.stream

    def forward(self, q, scales, y, stream=None):
        """y [M][N] (bf16, f16 or fp32) of the 8-bit rows ``q`` int8 [M][K] with ``scales`` fp32 [M]."""
        M, K, N, yt = q.shape[0], self.K, self.N, y.dtype
        (ld_q, one_q), (ld_y, one) = q.stride(), y.stride()
        if not (q.dtype is self._i8 and q.shape == (M, K) and one_q == 1 and yt in self._types and y.shape == (M, N) and
                self._device == q.get_device() == y.get_device() == scales.get_device() and (one == 1 or N == 1) and
                scales.dtype is self._f32 and scales.shape == (M,) and scales.is_contiguous() and not M >> 31):
            _ld("SpearW8Linear", "q", q, M, K, self._i8)
            _ld("SpearW8Linear", "y", y, M, N, *self._types)
            _vector("SpearW8Linear", "scales", scales, M, self._f32)
            _int32("SpearW8Linear", M=M)
            raise ValueError(f"SpearW8Linear: q, scales and y have to be on the layer's device, cuda:{self._device}")
        if M < 2:
            ld_q, ld_y = K, N
        st = self._forward(self._args(self.h.value or 0, q.data_ptr(), ld_q, scales.data_ptr(), y.data_ptr(), ld_y,
                                      self._stream(self._device) if stream is None else _stream(stream), self._types[yt], M))
        if st:
            raise SpearError(st, "spear_w8_forward")
        return y

    def check(self, stream=None) -> int:
        return load().spear_w8_check(self.h, _stream(stream))

    def debug_set(self, wait_ns: int = 0, skip_arrive: bool = False) -> None:
        _check(load().spear_w8_debug_set(self.h, int(wait_ns), int(bool(skip_arrive))), "spear_w8_debug_set")

    def close(self) -> None:
        if getattr(self, "h", None) and self.h.value:
            load().spear_w8_destroy(self.h)
            self.h = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


DECODE_SCHEDULE_FIELDS = ("grid", "P", "NW", "T", "MT", "KW", "KC", "NS", "stage_bytes", "smem", "n_stages",
                          "threads", "bytes_x")


def decode_schedule(N: int, K: int, M: int, sm_count: int, rank_b: int = 0, n_members: int = 1,
                    group_size: int = 128, gate_hidden: int = 0) -> dict:
    """The decode launch plan for a handle of this shape (host only, no GPU):
    the fields of ``DECODE_SCHEDULE_FIELDS``."""
    L = load()
    info = (ctypes.c_int32 * len(DECODE_SCHEDULE_FIELDS))()
    _check(L.spear_decode_schedule(N, K, rank_b, n_members, group_size, gate_hidden, M, sm_count, info),
           "spear_decode_schedule")
    return dict(zip(DECODE_SCHEDULE_FIELDS, list(info)))


PREFILL_SCHEDULE_FIELDS = ("mode", "G", "TN", "kpt", "tail", "units", "pro_items", "pro_d", "NS",
                           "stage_bytes", "smem", "pre_ctas", "tmem_a", "max_contrib")


def prefill_schedule(N: int, K: int, rank: int, M: int, sm_count: int, gate_hidden: int = 0,
                     with_workspace: bool = True) -> dict:
    """The prefill launch plan for a layer of this shape (host only, no GPU):
    the fields of ``PREFILL_SCHEDULE_FIELDS`` plus ``starts``, the first unit
    of each main-kernel CTA's range (G + 1 entries)."""
    L = load()
    info = (ctypes.c_int32 * len(PREFILL_SCHEDULE_FIELDS))()
    _check(L.spear_prefill_schedule(N, K, rank, gate_hidden, M, sm_count, int(with_workspace), info, None, 0),
           "spear_prefill_schedule")
    out = dict(zip(PREFILL_SCHEDULE_FIELDS, list(info)))
    starts = (ctypes.c_uint32 * (out["G"] + 1))()
    _check(L.spear_prefill_schedule(N, K, rank, gate_hidden, M, sm_count, int(with_workspace), info, starts,
                                    out["G"] + 1), "spear_prefill_schedule")
    out["starts"] = list(starts)
    return out


class ChunkScheduler:
    """Owner of one ``spear_sched_t`` (host only): a latency table of measured
    step times over (compensator density, tokens per step)."""

    def __init__(self, densities, tokens, ms):
        import numpy as np
        self._d = np.ascontiguousarray(densities, dtype=np.float64)
        self._t = np.ascontiguousarray(tokens, dtype=np.int32)
        self._ms = np.ascontiguousarray(ms, dtype=np.float64)
        if self._ms.shape != (self._d.size, self._t.size):
            raise ValueError("ms must be [len(densities)][len(tokens)]")
        h = c_void_p()
        _check(load().spear_sched_create(self._d.ctypes.data, self._d.size, self._t.ctypes.data, self._t.size,
                                         self._ms.ctypes.data, byref(h)), "spear_sched_create")
        self.h = h

    def predict(self, M: int, density: float) -> float:
        return load().spear_sched_predict(self.h, int(M), float(density))

    def pick_chunk(self, n_decode: int, density: float, itl_ms: float, candidates) -> int:
        import numpy as np
        c = np.ascontiguousarray(candidates, dtype=np.int32)
        out = c_int32()
        _check(load().spear_sched_pick_chunk(self.h, int(n_decode), float(density), float(itl_ms), c.ctypes.data,
                                             c.size, byref(out)), "spear_sched_pick_chunk")
        return int(out.value)

    def close(self):
        if getattr(self, "h", None) and self.h.value:
            load().spear_sched_destroy(self.h)
            self.h = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
