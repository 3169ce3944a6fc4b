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

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libspear_gb300.so"
HEADER = PKG.parent / "include" / "spear.h"

SPEAR_OK, SPEAR_ERR_INVALID_ARG, SPEAR_ERR_UNSUPPORTED, SPEAR_ERR_OOM, SPEAR_ERR_CUDA, SPEAR_ERR_TIMEOUT = range(6)
SPEAR_GATE_SIGMOID, SPEAR_GATE_ONE, SPEAR_GATE_MLP = 0, 1, 2
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
    L.spear_status_string.argtypes = [c_int]
    L.spear_status_string.restype = c_char_p
    for name in ("spear_linear_create", "spear_linear_forward_decode", "spear_linear_forward_prefill",
                 "spear_linear_forward", "spear_linear_forward_host", "spear_linear_destroy",
                 "spear_linear_dequantize", "spear_linear_check", "spear_linear_debug_set",
                 "spear_kv_create", "spear_kv_append", "spear_kv_read", "spear_kv_attention", "spear_kv_check",
                 "spear_kv_destroy"):
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
