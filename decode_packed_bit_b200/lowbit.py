"""Python binding of liblowbit.so (include/lowbit.h): argument marshalling only.

Every function has the name of the C entry point it calls.  Tensors are
torch CUDA tensors (torch supplies device memory and streams; every step of
the computation runs in the library's own kernels).  fp16/bf16 operands may
be given as float16/bfloat16 tensors or as int16/uint16 bit patterns.  A
non-OK status raises LowbitError.  There is no fallback: if the shared
library is missing, loading fails with an error.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liblowbit.so")

LOWBIT_OK = 0
LOWBIT_ERR_INVALID_ARG = 1
LOWBIT_ERR_MISALIGNED = 2
LOWBIT_ERR_UNSUPPORTED_SHAPE = 3
LOWBIT_ERR_CUDA = 4

LOWBIT_FMT_Q1_G128 = 1
LOWBIT_FMT_Q2 = 2
LOWBIT_FMT_INT4_G64 = 3
LOWBIT_FMT_TERNARY_G128 = 4
FORMATS = {"q1": LOWBIT_FMT_Q1_G128, "q2": LOWBIT_FMT_Q2, "int4": LOWBIT_FMT_INT4_G64, "t3": LOWBIT_FMT_TERNARY_G128}

# (name, restype, argtypes) of every symbol include/lowbit.h declares.
P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
F64 = ctypes.c_double
SYMBOLS = [
    ("lowbit_status_string", ctypes.c_char_p, [I32]),
    ("lowbit_version", I32, []),
    ("lowbit_fault_flags", I32, []),
    ("lowbit_pack", I32, [I32, P, I64, I64, P, P]),
    ("lowbit_unpack", I32, [I32, P, I64, I64, P, P]),
    ("lowbit_quantize", I32, [I32, P, I64, I64, P, P, P]),
    ("lowbit_q1g128_workspace_bytes", SZ, [I32, I32, I32]),
    ("lowbit_q1g128_gemv", I32, [P, P, P, P, I32, I32, I32, P, SZ, P]),
    ("lowbit_q1g128_act_bytes", SZ, [I32, I32]),
    ("lowbit_q1g128_act_workspace_bytes", SZ, [I32, I32, I32, I32]),
    ("lowbit_q1g128_prepare_act", I32, [P, I32, I32, P, SZ, P]),
    ("lowbit_q1g128_gemv_act", I32, [P, P, P, P, I32, I32, I32, P, SZ, P]),
    ("lowbit_q1g128_gemv_act_group", I32, [P, P, P, P, I32, I32, I32, I32, P, SZ, P]),
    ("lowbit_q1g128_group_workspace_bytes", SZ, [I32, I32, I32, I32]),
    ("lowbit_q1g128_gemv_group", I32, [P, P, P, P, I32, I32, I32, I32, P, SZ, P]),
    ("lowbit_q1g128_gemv_noalloc", I32, [P, P, P, P, I32, I32, I32, P]),
    ("lowbit_int4g64_gemm", I32, [P, P, P, P, I32, I32, I32, P]),
    ("lowbit_int4g64_gemm_group", I32, [P, P, P, P, I32, I32, I32, I32, P]),
    ("lowbit_t3g128_gemv", I32, [P, P, P, P, I32, I32, I32, P]),
    ("lowbit_t3g128_gemv_group", I32, [P, P, P, P, I32, I32, I32, I32, P]),
    ("lowbit_q2_mlp_forward", I32, [P, P, I32, P, I32, P, P, P]),
    ("lowbit_z80_generate", I32, [P, P, I32, P, I32, I32, P, I32, P, P, P]),
    ("lowbit_rmsnorm_bf16", I32, [P, P, I32, I32, F32, P, P]),
    ("lowbit_q1g128_stack_workspace_bytes", SZ, [I32, I32, I32]),
    ("lowbit_q1g128_stack_step", I32, [P, P, I32, I32, I32, P, F32, P, SZ, P, P, P]),
    ("lowbit_lora_workspace_bytes", SZ, [I32, I32, I32, I32, I32]),
    ("lowbit_lora_add", I32, [P] * 8 + [I32, I32, I32, I32, I32, P, SZ, P]),
    ("lowbit_lora_add_group", I32, [P] * 8 + [I32, I32, I32, I32, I32, I32, P, SZ, P]),
    ("lowbit_rope_phases", I32, [I32, I32, F64, F64, F64, F64, F64, P]),
    ("lowbit_rope", I32, [P, I64, P, I64, I32, P, I64, P, I64, I32, I32, I32, P, P, I32, I32, I32, I32, F32, P]),
    ("lowbit_kv8_append", I32, [P, P, P, I64, I32, P, I64, I32, P]),
    ("lowbit_kv8_read", I32, [P, P, P, P, I32, P]),
    ("lowbit_kv8_attention_workspace_bytes", SZ, [P, P, I32]),
    ("lowbit_kv8_attention", I32, [P, P, P, I64, I32, F32, P, I64, P, SZ, P]),
    ("lowbit_lora_add_group_args", I32, [P]),
    ("lowbit_rope_args", I32, [P]),
    ("lowbit_kv8_append_args", I32, [P]),
    ("lowbit_kv8_read_args", I32, [P]),
    ("lowbit_kv8_attention_args", I32, [P]),
]

_lib = None


class LowbitError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().lowbit_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m decode_packed_bit_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SYMBOLS:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != LOWBIT_OK:
        raise LowbitError(status, where)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def lowbit_fault_flags() -> int:
    return int(lib().lowbit_fault_flags())


# -- packing ----------------------------------------------------------------------

def lowbit_pack(fmt, codes, packed, stream=None):
    rows, cols = codes.shape
    _check(lib().lowbit_pack(_fmt(fmt), _ptr(codes), rows, cols, _ptr(packed), _stream(stream)),
           "lowbit_pack")


def lowbit_unpack(fmt, packed, codes, stream=None):
    rows, cols = codes.shape
    _check(lib().lowbit_unpack(_fmt(fmt), _ptr(packed), rows, cols, _ptr(codes), _stream(stream)),
           "lowbit_unpack")


def lowbit_quantize(fmt, w, packed, scales, stream=None):
    """float32 weights [rows][cols] -> packed codes and FP16 scale bits ("q1" or "int4")."""
    rows, cols = w.shape
    _check(lib().lowbit_quantize(_fmt(fmt), _ptr(w), rows, cols, _ptr(packed), _ptr(scales), _stream(stream)),
           "lowbit_quantize")


# -- Q1_0_g128 --------------------------------------------------------------------

def lowbit_q1g128_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().lowbit_q1g128_workspace_bytes(M, N, K))


def lowbit_q1g128_act_bytes(M: int, K: int) -> int:
    return int(lib().lowbit_q1g128_act_bytes(M, K))


def lowbit_q1g128_act_workspace_bytes(R: int, M: int, N: int, K: int) -> int:
    return int(lib().lowbit_q1g128_act_workspace_bytes(R, M, N, K))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def lowbit_q1g128_gemv(w_bits, w_scales, x, y, workspace=None, stream=None):
    M, K = x.shape
    N = w_bits.shape[0]
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().lowbit_q1g128_gemv(_ptr(w_bits), _ptr(w_scales), _ptr(x), _ptr(y), M, N, K,
                                    _ptr(workspace), wsb, _stream(stream)), "lowbit_q1g128_gemv")


def lowbit_q1g128_prepare_act(x, act, stream=None):
    M, K = x.shape
    _check(lib().lowbit_q1g128_prepare_act(_ptr(x), M, K, _ptr(act), act.numel() * act.element_size(),
                                           _stream(stream)), "lowbit_q1g128_prepare_act")


def lowbit_q1g128_gemv_act(w_bits, w_scales, act, y, M: int, workspace=None, stream=None):
    """workspace: zero-filled before its first use (calls leave it zeroed)."""
    N = w_bits.shape[0]
    K = w_bits.shape[1] * 8
    _check(lib().lowbit_q1g128_gemv_act(_ptr(w_bits), _ptr(w_scales), _ptr(act), _ptr(y), M, N, K,
                                        _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "lowbit_q1g128_gemv_act")


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])
    return ctypes.cast(arr, ctypes.c_void_p), arr


def lowbit_q1g128_gemv_act_group(w_bits, w_scales, act, ys, M: int, workspace=None, stream=None):
    """w_bits, w_scales, ys: equal-length lists of tensors (one per matrix)."""
    R = len(w_bits)
    N = w_bits[0].shape[0]
    K = w_bits[0].shape[1] * 8
    pb, kb = _ptr_array(w_bits)
    ps, ks = _ptr_array(w_scales)
    py, ky = _ptr_array(ys)
    _check(lib().lowbit_q1g128_gemv_act_group(pb, ps, _ptr(act), py, R, M, N, K, _ptr(workspace),
                                              _nbytes(workspace), _stream(stream)),
           "lowbit_q1g128_gemv_act_group")


def lowbit_q1g128_group_workspace_bytes(R: int, M: int, N: int, K: int) -> int:
    return lib().lowbit_q1g128_group_workspace_bytes(R, M, N, K)


def lowbit_q1g128_gemv_group(w_bits, w_scales, x, ys, workspace=None, stream=None):
    """y_r = W_r x for equal-length lists of weight tensors and outputs; x [M][K]
    bf16 bits.  workspace: lowbit_q1g128_group_workspace_bytes(R, M, N, K)
    bytes (None when that is 0)."""
    R = len(w_bits)
    M, K = x.shape
    N = w_bits[0].shape[0]
    pb, kb = _ptr_array(w_bits)
    ps, ks = _ptr_array(w_scales)
    py, ky = _ptr_array(ys)
    _check(lib().lowbit_q1g128_gemv_group(pb, ps, _ptr(x), py, R, M, N, K, _ptr(workspace), _nbytes(workspace),
                                          _stream(stream)),
           "lowbit_q1g128_gemv_group")


def lowbit_q1g128_gemv_noalloc(w_bits, w_scales, x, y, stream=None):
    """The product without a workspace (scratch in the library's own fixed
    device array; K <= 32768 at M = 1; calls must not overlap on the GPU)."""
    M, K = x.shape
    N = w_bits.shape[0]
    _check(lib().lowbit_q1g128_gemv_noalloc(_ptr(w_bits), _ptr(w_scales), _ptr(x), _ptr(y), M, N, K,
                                            _stream(stream)), "lowbit_q1g128_gemv_noalloc")


# -- INT4_G64 ---------------------------------------------------------------------

def lowbit_int4g64_gemm(w_q, w_scales, x, y, stream=None):
    M, K = x.shape
    N = w_q.shape[0]
    _check(lib().lowbit_int4g64_gemm(_ptr(w_q), _ptr(w_scales), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "lowbit_int4g64_gemm")


def lowbit_int4g64_gemm_group(w_q, w_scales, x, ys, stream=None):
    """y_r = W_r x for equal-length lists of INT4_G64 weights (uint8 [N][K/2],
    fp16 bits [N][K/64]) and fp32 outputs [M][N]; x [M][K] bf16 bits."""
    R = len(w_q)
    M, K = x.shape
    N = w_q[0].shape[0]
    pq, kq = _ptr_array(w_q)
    ps, ks = _ptr_array(w_scales)
    py, ky = _ptr_array(ys)
    _check(lib().lowbit_int4g64_gemm_group(pq, ps, _ptr(x), py, R, M, N, K, _stream(stream)),
           "lowbit_int4g64_gemm_group")


# -- ternary, FP16 scale per 128 ---------------------------------------------------

def lowbit_t3g128_gemv(w, w_scales, x, y, stream=None):
    """w uint8 [N][26 K/128], w_scales fp16 bits [N][K/128], x bf16 [M][K], y fp32 [M][N]."""
    M, K = x.shape
    N = w.shape[0]
    _check(lib().lowbit_t3g128_gemv(_ptr(w), _ptr(w_scales), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "lowbit_t3g128_gemv")


def lowbit_t3g128_gemv_group(w, w_scales, x, ys, stream=None):
    R = len(w)
    M, K = x.shape
    N = w[0].shape[0]
    pw, kw = _ptr_array(w)
    ps, ks = _ptr_array(w_scales)
    py, ky = _ptr_array(ys)
    _check(lib().lowbit_t3g128_gemv_group(pw, ps, _ptr(x), py, R, M, N, K, _stream(stream)),
           "lowbit_t3g128_gemv_group")


# -- Q2 MLP -----------------------------------------------------------------------

def lowbit_q2_mlp_forward(w_packed, dims, x, logits, argmax=None, stream=None):
    n_layers = len(w_packed)
    ptrs = (ctypes.c_void_p * n_layers)(*[w.data_ptr() for w in w_packed])
    dims_c = (ctypes.c_int32 * (n_layers + 1))(*[int(d) for d in dims])
    _check(lib().lowbit_q2_mlp_forward(ctypes.cast(ptrs, ctypes.c_void_p), ctypes.cast(dims_c, ctypes.c_void_p),
                                       n_layers, _ptr(x), x.shape[0], _ptr(logits), _ptr(argmax),
                                       _stream(stream)), "lowbit_q2_mlp_forward")


def lowbit_z80_generate(w_packed, dims, queries, charset, reply, reply_len, stream=None):
    """Autoregressive replies: queries uint8 [batch][qlen] (0-padded text),
    charset: bytes or a uint8 sequence of dims[-1] entries (0 = end of reply),
    reply uint8 [batch][max_new], reply_len int32 [batch]."""
    n_layers = len(w_packed)
    ptrs = (ctypes.c_void_p * n_layers)(*[w.data_ptr() for w in w_packed])
    dims_c = (ctypes.c_int32 * (n_layers + 1))(*[int(d) for d in dims])
    cs = bytes(bytearray(int(c) for c in charset))
    cs_c = ctypes.create_string_buffer(cs, len(cs))
    batch, qlen = queries.shape
    max_new = reply.shape[1]
    _check(lib().lowbit_z80_generate(ctypes.cast(ptrs, ctypes.c_void_p), ctypes.cast(dims_c, ctypes.c_void_p),
                                     n_layers, _ptr(queries), batch, qlen, ctypes.cast(cs_c, ctypes.c_void_p),
                                     max_new, _ptr(reply), _ptr(reply_len), _stream(stream)),
           "lowbit_z80_generate")


# -- glue -------------------------------------------------------------------------

def lowbit_rmsnorm_bf16(a, b, out, eps=1e-6, stream=None):
    M, D = a.shape
    _check(lib().lowbit_rmsnorm_bf16(_ptr(a), _ptr(b), M, D, float(eps), _ptr(out), _stream(stream)),
           "lowbit_rmsnorm_bf16")


# -- the fused decode step of a Q1 stack ------------------------------------------

def lowbit_q1g128_stack_workspace_bytes(n_layers: int, hidden: int, ffn: int) -> int:
    return int(lib().lowbit_q1g128_stack_workspace_bytes(n_layers, hidden, ffn))


def lowbit_q1g128_stack_step(w_bits, w_scales, x, hidden, ffn, workspace, eps=1e-6, record_inputs=None,
                             record_outputs=None, stream=None):
    """w_bits / w_scales: lists of 7 * n_layers device tensors (q, k, v, o, gate, up, down per layer)."""
    n = len(w_bits)
    bits, bits_keep = _ptr_array(w_bits)
    scales, scales_keep = _ptr_array(w_scales)
    wsb = workspace.numel() * workspace.element_size()
    _check(lib().lowbit_q1g128_stack_step(bits, scales, n // 7, hidden, ffn, _ptr(x), float(eps), _ptr(workspace), wsb,
                                          _ptr(record_inputs), _ptr(record_outputs), _stream(stream)),
           "lowbit_q1g128_stack_step")



# -- low-rank adapters of many requests ---------------------------------------------
#
# The operands of these and of the following calls are checked here as far as the C
# side cannot see them: element types, shapes, strides and the device.  A decode step
# makes many such calls in a row, so the checks are kept to what a tensor answers
# without building objects, and plain integers go to ctypes.

LOWBIT_F32 = 0
LOWBIT_BF16 = 1
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}
_types = {}  # torch dtypes of the operands that may be either -> lowbit_dtype
_float32 = _bfloat16 = _int32 = _int64 = _int8 = None  # torch's, set on the first call (torch is imported late)
_halves = None  # bf16 values, as such or as int16 bit patterns
_dense = _rows = _scratch = _call = None  # csrc/marshal.cpp's: the checks of operands, and the call with a block of words
_LORA = _ROPE = _APPEND = _READ = _ATTENTION = 0  # addresses of the entry points that take a block


def _first_call():
    import torch
    try:
        from . import _marshal
    except ImportError as e:
        raise RuntimeError(f"{os.path.join(PKG, '_marshal.so')} is missing or for another torch: build it with "
                           "`python -m decode_packed_bit_b200.build` (it needs g++)") from e
    global _float32, _bfloat16, _int32, _int64, _int8, _halves, _dense, _rows, _scratch, _call
    global _LORA, _ROPE, _APPEND, _READ, _ATTENTION, _device, _current_stream
    torch.cuda.init()
    _float32, _bfloat16 = torch.float32, torch.bfloat16
    _int32, _int64, _int8, _halves = torch.int32, torch.int64, torch.int8, (torch.bfloat16, torch.int16)
    _dense, _rows, _scratch, _call = _marshal.dense, _marshal.rows, _marshal.scratch, _marshal.call
    _LORA, _ROPE, _APPEND, _READ, _ATTENTION = (
        ctypes.cast(getattr(lib(), f"lowbit_{name}_args"), P).value
        for name in ("lora_add_group", "rope", "kv8_append", "kv8_read", "kv8_attention"))
    _types.update({_float32: LOWBIT_F32, _bfloat16: LOWBIT_BF16})
    # _device last: from then on another thread takes all of these as set
    _current_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    return _device()


_device = _first_call  # the current CUDA device; every operand has to be there
_current_stream = None


def _raw_stream(stream, dev):
    if stream is None:
        return _current_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _either(t, what):
    found = _types.get(t.dtype)
    if found is None:
        raise ValueError(f"{what}: expected float32 or bfloat16, got {t.dtype}")
    return found


def lowbit_lora_workspace_bytes(R: int, M: int, N: int, K: int, rank: int) -> int:
    return int(lib().lowbit_lora_workspace_bytes(R, M, N, K, rank))


def lowbit_lora_add_group(x, ids, a, b, base, ys, ranks=None, scales=None, workspace=None, stream=None):
    """y_r[m] = base_r[m] + scales[i] B_r,i (A_r,i x[m]) with i = ids[m] (any i outside the pool: y_r[m] = base_r[m]).

    x bf16 [M][K], ids int32 [M]; a, b, base, ys: equal-length lists of bf16 [L][rank][K], bf16 [L][N][rank],
    fp32 [M][N] and fp32 [M][N] (base_r may be y_r itself); ranks int32 [L] and scales fp32 [L], or None.
    workspace: lowbit_lora_workspace_bytes(R, M, N, K, rank) bytes."""
    dev = _device()
    R = len(a)
    if not 1 <= R == len(b) == len(base) == len(ys) <= 16:
        raise ValueError("lowbit_lora_add_group: expected lists of one length, 1 to 16")
    M, K = x.shape
    L, rank, _ = a[0].shape
    _, N, _ = b[0].shape
    sa, sb, sy, sl = (L, rank, K), (L, N, rank), (M, N), (L,)
    ws, ws_bytes = _scratch(workspace, dev)
    _check(_call(
        _LORA, _dense(x, _halves, (M, K), "x", dev), _dense(ids, _int32, (M,), "ids", dev),
        0 if ranks is None else _dense(ranks, _int32, sl, "ranks", dev),
        0 if scales is None else _dense(scales, _float32, sl, "scales", dev),
        R, M, N, K, rank, L, ws, ws_bytes, _raw_stream(stream, dev),
        *[_dense(t, _halves, sa, "a", dev) for t in a], *[_dense(t, _halves, sb, "b", dev) for t in b],
        *[_dense(t, _float32, sy, "base", dev) for t in base], *[_dense(t, _float32, sy, "y", dev) for t in ys]),
        "lowbit_lora_add_group")


def lowbit_lora_add(x, ids, a, b, base, y, ranks=None, scales=None, workspace=None, stream=None):
    """One projection's adapters: see lowbit_lora_add_group."""
    lowbit_lora_add_group(x, ids, [a], [b], [base], [y], ranks, scales, workspace, stream)


# -- rotary positions ---------------------------------------------------------------

def lowbit_rope_phases(rot: int, base: float = 10000.0, scaling="plain", factor: float = 1.0,
                       trained_length: float = 0.0, slow: float = 1.0, fast: float = 32.0):
    """The rot/2 phases (2^-64 turns per position) as an int64 CPU tensor; scaling "plain", "linear", "base" or "bands"."""
    import torch
    phases = torch.empty(max(rot, 0) // 2, dtype=torch.int64)
    _check(lib().lowbit_rope_phases(ROPE_SCALINGS[scaling], rot, base, factor, trained_length, slow, fast,
                                    _ptr(phases)), "lowbit_rope_phases")
    return phases


def lowbit_rope(q, q_out, k, k_out, positions, phases, interleaved=False, magnitude=1.0, stream=None):
    """q [M][q_heads][D] -> q_out and k [M][kv_heads][D] -> k_out (either pair may be None), fp32 or bf16, rows dense
    and any stride (a multiple of 8) apart; positions int32 [M]; phases int64 [rot / 2].  In place where types match."""
    dev = _device()
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or q is k is None:
        raise ValueError("lowbit_rope: expected q with q_out, k with k_out, or both")
    ref, ref_out = (q, q_out) if q is not None else (k, k_out)
    M, _, D = ref.shape
    half = phases.shape[0]
    ti, to = _either(ref, "input"), _either(ref_out, "output")
    qp = qo = kp = ko = qs = qos = qh = ks = kos = kh = 0
    if q is not None:
        qh = q.shape[1]
        qp, qs = _rows(q, ref.dtype, (M, qh, D), "q", dev)
        qo, qos = _rows(q_out, ref_out.dtype, (M, qh, D), "q_out", dev)
    if k is not None:
        kh = k.shape[1]
        kp, ks = _rows(k, ref.dtype, (M, kh, D), "k", dev)
        ko, kos = _rows(k_out, ref_out.dtype, (M, kh, D), "k_out", dev)
    _check(_call(_ROPE, qp, qs, qo, qos, qh, kp, ks, ko, kos, kh, ti, to, _dense(positions, _int32, (M,), "positions", dev),
                 _dense(phases, _int64, (half,), "phases", dev), M, D, 2 * half, 1 if interleaved else 0, float(magnitude),
                 _raw_stream(stream, dev)), "lowbit_rope")


# -- KV8 cache ----------------------------------------------------------------------

class _KV8CacheC(ctypes.Structure):
    _fields_ = [("k", P), ("k_scales", P), ("v", P), ("v_scales", P), ("n_pages", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _KV8BatchC(ctypes.Structure):
    _fields_ = [("kv_len", P), ("page_table", P), ("row_start", P), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_rows", ctypes.c_int32)]


class KV8Cache:
    """The buffers of a KV8 cache: int8 codes k, v [n_pages][n_heads][page_tokens][head_dim] and fp32 scales
    [n_pages][n_heads].  Holds them alive; a call reads or writes them in place."""

    def __init__(self, k, k_scales, v, v_scales):
        dev = _device()
        n_pages, heads, page, dim = k.shape
        self._c = _KV8CacheC(_dense(k, _int8, (n_pages, heads, page, dim), "k", dev),
                             _dense(k_scales, _float32, (n_pages, heads), "k_scales", dev),
                             _dense(v, _int8, (n_pages, heads, page, dim), "v", dev),
                             _dense(v_scales, _float32, (n_pages, heads), "v_scales", dev), n_pages, heads, page,
                             dim)
        self._at = ctypes.addressof(self._c)
        self.k, self.k_scales, self.v, self.v_scales = k, k_scales, v, v_scales
        self.n_pages, self.n_heads, self.page_tokens, self.head_dim, self.device = n_pages, heads, page, dim, dev

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, page_tokens: int, head_dim: int, device="cuda"):
        """A cache of zeros."""
        import torch
        shape = (n_pages, n_heads, page_tokens, head_dim)

        def zeros(s, dtype):
            return torch.zeros(s, dtype=dtype, device=device)

        return cls(zeros(shape, torch.int8), zeros(shape[:2], torch.float32), zeros(shape, torch.int8),
                   zeros(shape[:2], torch.float32))


def _kv8_batch(cache, page_table, kv_len, row_start, rows, dev):
    i32 = _int32
    B, width = page_table.shape
    if cache.device != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    return (_dense(kv_len, i32, (B,), "kv_len", dev), _dense(page_table, i32, (B, width), "page_table", dev),
            0 if row_start is None else _dense(row_start, i32, (B + 1,), "row_start", dev), B, width, rows)


def lowbit_kv8_append(cache: KV8Cache, page_table, kv_len, k, v, row_start=None, stream=None):
    """Write k, v [rows][n_heads][head_dim] (fp32 or bf16 each, rows dense and any stride apart) as the sequences' last
    tokens.  page_table int32 [B][max_pages], kv_len int32 [B] (the new tokens included), row_start int32 [B + 1], or
    None for one row per sequence."""
    dev = _device()
    rows = k.shape[0]
    shape = (rows, cache.n_heads, cache.head_dim)
    batch = _kv8_batch(cache, page_table, kv_len, row_start, rows, dev)
    tk, tv = _either(k, "k"), _either(v, "v")
    kp, ks = _rows(k, k.dtype, shape, "k", dev)
    vp, vs = _rows(v, v.dtype, shape, "v", dev)
    _check(_call(_APPEND, cache._at, *batch, kp, ks, tk, vp, vs, tv, _raw_stream(stream, dev)), "lowbit_kv8_append")


def lowbit_kv8_read(cache: KV8Cache, page_table, kv_len, k_out, v_out, row_start=None, stream=None):
    """The values of the sequences' last tokens back from the cache: k_out, v_out [rows][n_heads][head_dim] (dense, one
    type, fp32 or bf16; either may be None)."""
    dev = _device()
    ref = k_out if k_out is not None else v_out
    if ref is None:  # nothing is asked for
        return
    rows = ref.shape[0]
    shape = (rows, cache.n_heads, cache.head_dim)
    batch = _kv8_batch(cache, page_table, kv_len, row_start, rows, dev)
    _check(_call(_READ, cache._at, *batch, 0 if k_out is None else _dense(k_out, ref.dtype, shape, "k_out", dev),
                 0 if v_out is None else _dense(v_out, ref.dtype, shape, "v_out", dev), _either(ref, "output"),
                 _raw_stream(stream, dev)), "lowbit_kv8_read")


def lowbit_kv8_attention_workspace_bytes(cache: KV8Cache, n_seqs: int, n_rows: int, q_heads: int) -> int:
    """Bytes for calls with this many sequences and rows (zero-fill them once)."""
    batch = _KV8BatchC(16, 16, 16, n_seqs, 1, n_rows)
    return int(lib().lowbit_kv8_attention_workspace_bytes(cache._at, ctypes.byref(batch), q_heads))


def lowbit_kv8_attention(cache: KV8Cache, page_table, kv_len, q, out, scale, row_start=None, workspace=None,
                         stream=None):
    """out = softmax(scale q k^T) v of each row over its sequence's tokens up to the row's own position.

    q, out bf16 [rows][q_heads][head_dim], rows dense and any stride (a multiple of 8) apart; page_table, kv_len and
    row_start as for lowbit_kv8_append.  workspace: lowbit_kv8_attention_workspace_bytes(...) bytes, zero-filled before
    their first use."""
    dev = _device()
    rows, heads, _ = q.shape
    shape = (rows, heads, cache.head_dim)
    batch = _kv8_batch(cache, page_table, kv_len, row_start, rows, dev)
    qp, qs = _rows(q, _bfloat16, shape, "q", dev)
    op, os_ = _rows(out, _bfloat16, shape, "out", dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _check(_call(_ATTENTION, cache._at, *batch, qp, qs, heads, float(scale), op, os_, ws, ws_bytes,
                 _raw_stream(stream, dev)), "lowbit_kv8_attention")
