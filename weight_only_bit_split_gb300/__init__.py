"""weight_only_bit_split_gb300 -- weight-only low-bit decode GEMV for GB300.

A thin Python binding over the C ABI of ``libwobs.so`` (declared in
``include/wobs.h``).  Each function here has the name of the C entry point
it calls and only marshals arguments: it checks tensor devices, dtypes and
shapes, passes raw pointers and the current CUDA stream, and turns a
negative status into ``WobsError``.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU fallback.

PyTorch supplies device memory and streams only.
"""
import ctypes

import torch

from . import _lib

OP_GEMV_F16 = 1
OP_GEMV_BF16 = 2
OP_GEMV_Q4_0_Q8_1 = 3
OP_GEMV_NF4 = 4
OP_ARGCMP = 5
OP_GEMV_Q8_0_Q8_1 = 6
OP_GEMV_Q4_0_F32 = 7
OP_GEMV_Q8_0_F32 = 8
OP_ATTN_KV4 = 9
ERR_DEVICE_TIMEOUT = -7
DEVICE_CACHE_INDEX = 4      # wobs_error_word: a length or page index outside a Kv4Cache
# leading workspace bytes that hold counters and keys: zero between calls
WS_ZERO_BYTES = 262408
DTYPE_CODES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 3}
MAX_M = 32
Q8_1_BLOCK_BYTES = 36

STATUS = {0: "OK", -1: "INVALID_ARG", -2: "MISALIGNED", -3: "UNSUPPORTED_SHAPE",
          -4: "WORKSPACE_TOO_SMALL", -5: "LAUNCH_FAILED", -6: "CUDA", -7: "DEVICE_TIMEOUT"}


class WobsError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code


def _check(rc, lib):
    if rc != 0:
        raise WobsError(rc, lib.wobs_last_error().decode(errors="replace"))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype=None, ndim=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the library has no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: {t.dim()} dims, expected {ndim}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dim() >= 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")


def _rows(t):
    """Row pitch in elements of a 2-D tensor with a contiguous last dim."""
    return t.stride(0) if t.dim() == 2 else t.shape[-1]


def _codebook(cb):
    vals = [float(v) for v in (cb.tolist() if hasattr(cb, "tolist") else cb)]
    if len(vals) != 16:
        raise ValueError("codebook: 16 levels expected")
    return (ctypes.c_float * 16)(*vals)


# ----------------------------------------------------------- step graph

class StepGraph:
    """A fixed sequence of library calls, replayed as one CUDA graph.

    Decode loops make the same calls with the same shapes and buffers for
    every token.  ``fn`` (any mix of ``wobs_*`` calls and tensor copies) runs
    once eagerly on ``stream``, which also sizes the cached workspaces, and is
    then captured; ``replay()`` launches the whole sequence with one graph
    launch on the current stream.  Every buffer the calls touch must stay
    alive and in place while the graph is used; host buffers of copies must
    be pinned.
    """

    def __init__(self, fn, stream=None):
        self.stream = stream if stream is not None else torch.cuda.Stream()
        with torch.cuda.stream(self.stream):
            fn()
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            fn()

    def replay(self):
        self.graph.replay()


# ------------------------------------------------------------ workspace

_ws_cache = {}
_ws_replaced = []     # outgrown ones: captured graphs may hold their addresses

# Workspace bytes of the argmax state alone (counter, keys, alignment).  A
# larger wobs_workspace_size() means the call splits K and needs the
# workspace even without an argmax.
_WS_HEADER_BYTES = 512


def _auto_ws(op, M, N, K, device, argmax):
    if argmax is None and wobs_workspace_size(op, M, N, K) <= _WS_HEADER_BYTES:
        return None
    return workspace(op, M, N, K, device)


def workspace(op, M, N, K, device=None):
    """A zero-filled workspace for (op, M, N, K) on the current stream.

    Cached per (device, stream) and grown as needed, twofold at least; an
    outgrown one is kept, since a captured graph may still use it.  The
    library leaves its counter region (the first WS_ZERO_BYTES bytes) zero
    after every successful call and overwrites partials before reading them,
    so it is reused as is.  Calls that may overlap on the GPU should run on
    different streams.
    """
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = wobs_workspace_size(op, M, N, K)
    if need == 0:
        return None
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        size = max(need, 4096)
        if buf is not None:
            _ws_replaced.append(buf)
            size = max(size, 2 * buf.numel())
        buf = torch.zeros(size, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def wobs_workspace_size(op, M, N, K):
    lib = _lib.get()
    return int(lib.wobs_workspace_size(int(op), int(M), int(N), int(K)))


def wobs_version():
    return int(_lib.get().wobs_version())


def wobs_last_error():
    return _lib.get().wobs_last_error().decode(errors="replace")


# ------------------------------------------------------------ entry points

def wobs_bw_probe(buf, grid=0, variant=1, xor_out=None):
    """Streaming read of ``buf`` (uint8 CUDA tensor); returns the uint32 XOR tensor."""
    lib = _lib.get()
    _need(buf, "buf")
    if xor_out is None:
        xor_out = torch.zeros(1, dtype=torch.int32, device=buf.device)
    rc = lib.wobs_bw_probe(_ptr(buf), buf.numel() * buf.element_size(), int(grid), int(variant),
                           _ptr(xor_out), _stream(buf.device))
    _check(rc, lib)
    return xor_out


def wobs_gemv_f16(W, X, Y=None, ws=None):
    """Y[M, N] (fp16) = X[M, K] @ W[N, K]^T with fp32 accumulation."""
    lib = _lib.get()
    _need(W, "W", torch.float16, 2)
    X2 = X if X.dim() == 2 else X.view(1, -1)
    _need(X2, "X", torch.float16, 2, W.device)
    M, K = X2.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W and X disagree on K")
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float16, device=W.device)
    _need(Y, "Y", torch.float16, None, W.device)
    if ws is None:
        ws = _auto_ws(OP_GEMV_F16, M, N, K, W.device, None)
    rc = lib.wobs_gemv_f16(_ptr(W), _rows(W), _ptr(X2), _rows(X2), M, _ptr(Y), N, K, _ptr(ws),
                           ws.numel() if ws is not None else 0, _stream(W.device))
    _check(rc, lib)
    return Y


def wobs_gemv_bf16(W, X, logits=None, argmax=None, want_argmax=False, ws=None):
    """logits[M, N] (fp32) = X[M, K] @ W[N, K]^T; optional fused argmax[M] (int64)."""
    lib = _lib.get()
    _need(W, "W", torch.bfloat16, 2)
    X2 = X if X.dim() == 2 else X.view(1, -1)
    _need(X2, "X", torch.bfloat16, 2, W.device)
    M, K = X2.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W and X disagree on K")
    if logits is None:
        logits = torch.empty(M, N, dtype=torch.float32, device=W.device)
    _need(logits, "logits", torch.float32, None, W.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(M, dtype=torch.int64, device=W.device)
    if ws is None:
        ws = _auto_ws(OP_GEMV_BF16, M, N, K, W.device, argmax)
    rc = lib.wobs_gemv_bf16(_ptr(W), _rows(W), _ptr(X2), _rows(X2), M, _ptr(logits), _ptr(argmax),
                            N, K, _ptr(ws), ws.numel() if ws is not None else 0, _stream(W.device))
    _check(rc, lib)
    return logits, argmax


def wobs_gemv_bf16_noalloc(W, X, logits=None, argmax=None, want_argmax=False):
    """wobs_gemv_bf16 with the library's fixed scratch in place of a workspace.

    For callers that may not allocate device memory at call time (an engine
    that reserved its memory budget up front and owns every allocation, a
    plugin whose host process accounts all device memory).  Pass
    preallocated ``logits`` / ``argmax`` to allocate nothing here either.
    Calls that may overlap on the GPU share the scratch and must not be issued.
    """
    lib = _lib.get()
    _need(W, "W", torch.bfloat16, 2)
    X2 = X if X.dim() == 2 else X.view(1, -1)
    _need(X2, "X", torch.bfloat16, 2, W.device)
    M, K = X2.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W and X disagree on K")
    if logits is None:
        logits = torch.empty(M, N, dtype=torch.float32, device=W.device)
    _need(logits, "logits", torch.float32, None, W.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(M, dtype=torch.int64, device=W.device)
    rc = lib.wobs_gemv_bf16_noalloc(_ptr(W), _rows(W), _ptr(X2), _rows(X2), M, _ptr(logits),
                                    _ptr(argmax), N, K, _stream(W.device))
    _check(rc, lib)
    return logits, argmax


def wobs_quantize_q8_1(X, xq=None):
    """Q8_1 blocks of fp32 activations X[M, K]: uint8 [M, K/32*36]."""
    lib = _lib.get()
    X2 = X if X.dim() == 2 else X.view(1, -1)
    _need(X2, "X", torch.float32, 2)
    M, K = X2.shape
    if xq is None:
        xq = torch.empty(M, (K // 32) * Q8_1_BLOCK_BYTES, dtype=torch.uint8, device=X2.device)
    _need(xq, "xq", torch.uint8, None, X2.device)
    rc = lib.wobs_quantize_q8_1(_ptr(X2), _rows(X2), M, K, _ptr(xq), _stream(X2.device))
    _check(rc, lib)
    return xq


def wobs_quantize_q4_0(W, qs=None, d=None):
    """Q4_0 planes of fp32 weights W[N, K]: (qs uint8 [N, K/2], d fp16 [N, K/32])."""
    lib = _lib.get()
    _need(W, "W", torch.float32, 2)
    N, K = W.shape
    if qs is None:
        qs = torch.empty(N, K // 2, dtype=torch.uint8, device=W.device)
    if d is None:
        d = torch.empty(N, K // 32, dtype=torch.float16, device=W.device)
    _need(qs, "qs", torch.uint8, 2, W.device)
    _need(d, "d", torch.float16, 2, W.device)
    rc = lib.wobs_quantize_q4_0(_ptr(W), _rows(W), N, K, _ptr(qs), _ptr(d), _stream(W.device))
    _check(rc, lib)
    return qs, d


def wobs_quantize_nf4(W, codebook, qs=None, absmax=None):
    """NF4 planes of bf16 weights W[N, K]: (qs uint8 [N, K/2], absmax fp32 [N, K/64])."""
    lib = _lib.get()
    _need(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if qs is None:
        qs = torch.empty(N, K // 2, dtype=torch.uint8, device=W.device)
    if absmax is None:
        absmax = torch.empty(N, K // 64, dtype=torch.float32, device=W.device)
    _need(qs, "qs", torch.uint8, 2, W.device)
    _need(absmax, "absmax", torch.float32, 2, W.device)
    rc = lib.wobs_quantize_nf4(_ptr(W), _rows(W), N, K, _codebook(codebook), _ptr(qs),
                               _ptr(absmax), _stream(W.device))
    _check(rc, lib)
    return qs, absmax


def wobs_gemv_q4_0_q8_1(qs, d, xq, y=None, argmax=None, want_argmax=False, ws=None):
    """y[M, N] (fp32) from Q4_0 planes (qs [N, K/2], d [N, K/32]) and Q8_1 blocks xq [M, ...]."""
    lib = _lib.get()
    _need(qs, "qs", torch.uint8, 2)
    _need(d, "d", torch.float16, 2, qs.device)
    xq2 = xq if xq.dim() == 2 else xq.view(1, -1)
    _need(xq2, "xq", torch.uint8, 2, qs.device)
    N, K = qs.shape[0], qs.shape[1] * 2
    M = xq2.shape[0]
    if xq2.shape[1] != (K // 32) * Q8_1_BLOCK_BYTES or not xq2.is_contiguous():
        raise ValueError("xq must be contiguous [M, K/32*36]")
    if not (qs.is_contiguous() and d.is_contiguous()) or d.shape != (N, K // 32):
        raise ValueError("qs/d must be contiguous planes [N, K/2] and [N, K/32]")
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=qs.device)
    _need(y, "y", torch.float32, None, qs.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(M, dtype=torch.int64, device=qs.device)
    if ws is None:
        ws = _auto_ws(OP_GEMV_Q4_0_Q8_1, M, N, K, qs.device, argmax)
    rc = lib.wobs_gemv_q4_0_q8_1(_ptr(qs), _ptr(d), _ptr(xq2), M, _ptr(y), _ptr(argmax), N, K,
                                 _ptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(qs.device))
    _check(rc, lib)
    return y, argmax


def wobs_gemv_q4_0_f32(qs, d, x, y=None, argmax=None, want_argmax=False, ws=None, xq_out=None):
    """y[1, N] (fp32) from Q4_0 planes and one fp32 activation vector x [K] (or [1, K]),
    quantised to Q8_1 inside the GEMV kernel; the Q8_1 blocks are also written to
    ``xq_out`` (uint8, K/32*36 bytes) when it is given."""
    lib = _lib.get()
    _need(qs, "qs", torch.uint8, 2)
    _need(d, "d", torch.float16, 2, qs.device)
    x1 = x.reshape(-1) if x.dim() == 2 and x.shape[0] == 1 else x
    _need(x1, "x", torch.float32, 1, qs.device)
    N, K = qs.shape[0], qs.shape[1] * 2
    if x1.shape[0] != K or not x1.is_contiguous():
        raise ValueError("x must be a contiguous fp32 vector of K elements")
    if not (qs.is_contiguous() and d.is_contiguous()) or d.shape != (N, K // 32):
        raise ValueError("qs/d must be contiguous planes [N, K/2] and [N, K/32]")
    if y is None:
        y = torch.empty(1, N, dtype=torch.float32, device=qs.device)
    _need(y, "y", torch.float32, None, qs.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(1, dtype=torch.int64, device=qs.device)
    if xq_out is not None:
        _need(xq_out, "xq_out", torch.uint8, None, qs.device)
        if xq_out.numel() < (K // 32) * Q8_1_BLOCK_BYTES or not xq_out.is_contiguous():
            raise ValueError("xq_out must be a contiguous uint8 buffer of K/32*36 bytes")
    if ws is None:
        ws = _auto_ws(OP_GEMV_Q4_0_F32, 1, N, K, qs.device, argmax)
    rc = lib.wobs_gemv_q4_0_f32(_ptr(qs), _ptr(d), _ptr(x1), _ptr(xq_out), _ptr(y), _ptr(argmax), N, K,
                                _ptr(ws), ws.numel() if ws is not None else 0, _stream(qs.device))
    _check(rc, lib)
    return y, argmax


def wobs_quantize_q8_0(W, qs=None, d=None):
    """Q8_0 planes of fp32 weights W[N, K]: (qs int8 [N, K], d fp16 [N, K/32])."""
    lib = _lib.get()
    _need(W, "W", torch.float32, 2)
    N, K = W.shape
    if qs is None:
        qs = torch.empty(N, K, dtype=torch.int8, device=W.device)
    if d is None:
        d = torch.empty(N, K // 32, dtype=torch.float16, device=W.device)
    _need(qs, "qs", torch.int8, 2, W.device)
    _need(d, "d", torch.float16, 2, W.device)
    rc = lib.wobs_quantize_q8_0(_ptr(W), _rows(W), N, K, _ptr(qs), _ptr(d), _stream(W.device))
    _check(rc, lib)
    return qs, d


def wobs_gemv_q8_0_q8_1(qs, d, xq, y=None, argmax=None, want_argmax=False, ws=None):
    """y[M, N] (fp32) from Q8_0 planes (qs int8 [N, K], d [N, K/32]) and Q8_1 blocks xq [M, ...]."""
    lib = _lib.get()
    _need(qs, "qs", torch.int8, 2)
    _need(d, "d", torch.float16, 2, qs.device)
    xq2 = xq if xq.dim() == 2 else xq.view(1, -1)
    _need(xq2, "xq", torch.uint8, 2, qs.device)
    N, K = qs.shape
    M = xq2.shape[0]
    if xq2.shape[1] != (K // 32) * Q8_1_BLOCK_BYTES or not xq2.is_contiguous():
        raise ValueError("xq must be contiguous [M, K/32*36]")
    if not (qs.is_contiguous() and d.is_contiguous()) or d.shape != (N, K // 32):
        raise ValueError("qs/d must be contiguous planes [N, K] and [N, K/32]")
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=qs.device)
    _need(y, "y", torch.float32, None, qs.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(M, dtype=torch.int64, device=qs.device)
    if ws is None:
        ws = _auto_ws(OP_GEMV_Q8_0_Q8_1, M, N, K, qs.device, argmax)
    rc = lib.wobs_gemv_q8_0_q8_1(_ptr(qs), _ptr(d), _ptr(xq2), M, _ptr(y), _ptr(argmax), N, K,
                                 _ptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(qs.device))
    _check(rc, lib)
    return y, argmax


def wobs_gemv_q8_0_f32(qs, d, x, y=None, argmax=None, want_argmax=False, ws=None, xq_out=None):
    """y[1, N] (fp32) from Q8_0 planes (qs int8 [N, K], d [N, K/32]) and one fp32 activation
    vector x [K] (or [1, K]), quantised to Q8_1 inside the GEMV kernel; the Q8_1 blocks are
    also written to ``xq_out`` (uint8, K/32*36 bytes) when it is given."""
    lib = _lib.get()
    _need(qs, "qs", torch.int8, 2)
    _need(d, "d", torch.float16, 2, qs.device)
    x1 = x.reshape(-1) if x.dim() == 2 and x.shape[0] == 1 else x
    _need(x1, "x", torch.float32, 1, qs.device)
    N, K = qs.shape
    if x1.shape[0] != K or not x1.is_contiguous():
        raise ValueError("x must be a contiguous fp32 vector of K elements")
    if not (qs.is_contiguous() and d.is_contiguous()) or d.shape != (N, K // 32):
        raise ValueError("qs/d must be contiguous planes [N, K] and [N, K/32]")
    if y is None:
        y = torch.empty(1, N, dtype=torch.float32, device=qs.device)
    _need(y, "y", torch.float32, None, qs.device)
    if argmax is None and want_argmax:
        argmax = torch.empty(1, dtype=torch.int64, device=qs.device)
    if xq_out is not None:
        _need(xq_out, "xq_out", torch.uint8, None, qs.device)
        if xq_out.numel() < (K // 32) * Q8_1_BLOCK_BYTES or not xq_out.is_contiguous():
            raise ValueError("xq_out must be a contiguous uint8 buffer of K/32*36 bytes")
    if ws is None:
        ws = _auto_ws(OP_GEMV_Q8_0_F32, 1, N, K, qs.device, argmax)
    rc = lib.wobs_gemv_q8_0_f32(_ptr(qs), _ptr(d), _ptr(x1), _ptr(xq_out), _ptr(y), _ptr(argmax), N, K,
                                _ptr(ws), ws.numel() if ws is not None else 0, _stream(qs.device))
    _check(rc, lib)
    return y, argmax


def wobs_gemv_nf4(qs, absmax, codebook, x, y=None, argmax=None, want_argmax=False, ws=None):
    """NF4 GEMV: bf16 y from NF4 planes (qs [N, K/2], absmax [N, K/64]).

    ``x`` is bf16 [K] (one column; y is [N]) or [M, K] (M columns, 1 <= M <=
    32; y is [M, N]); ``argmax`` is int64 [M].
    """
    lib = _lib.get()
    _need(qs, "qs", torch.uint8, 2)
    _need(absmax, "absmax", torch.float32, 2, qs.device)
    one = x.dim() == 1
    X2 = x.view(1, -1) if one else x
    _need(X2, "x", torch.bfloat16, 2, qs.device)
    N, K = qs.shape[0], qs.shape[1] * 2
    M = X2.shape[0]
    if X2.shape[1] != K or not (qs.is_contiguous() and absmax.is_contiguous()):
        raise ValueError("x must have K elements per column; planes must be contiguous")
    if y is None:
        y = torch.empty((N,) if one else (M, N), dtype=torch.bfloat16, device=qs.device)
    _need(y, "y", torch.bfloat16, None, qs.device)
    if y.numel() != M * N or not y.is_contiguous():
        raise ValueError("y must be a contiguous [M, N] bf16 tensor")
    if argmax is None and want_argmax:
        argmax = torch.empty(M, dtype=torch.int64, device=qs.device)
    if ws is None:
        ws = _auto_ws(OP_GEMV_NF4, M, N, K, qs.device, argmax)
    rc = lib.wobs_gemv_nf4(_ptr(qs), _ptr(absmax), _codebook(codebook), _ptr(X2), _rows(X2), M,
                           _ptr(y), _ptr(argmax), N, K, _ptr(ws), ws.numel() if ws is not None else 0,
                           _stream(qs.device))
    _check(rc, lib)
    return y, argmax


def wobs_dequantize_nf4(qs, absmax, codebook, W=None):
    """bf16 W [N, K] = absmax * codebook[code] (fp32 product, rounded to bf16)."""
    lib = _lib.get()
    _need(qs, "qs", torch.uint8, 2)
    _need(absmax, "absmax", torch.float32, 2, qs.device)
    N, K = qs.shape[0], qs.shape[1] * 2
    if not (qs.is_contiguous() and absmax.is_contiguous()):
        raise ValueError("planes must be contiguous")
    if W is None:
        W = torch.empty(N, K, dtype=torch.bfloat16, device=qs.device)
    _need(W, "W", torch.bfloat16, 2, qs.device)
    rc = lib.wobs_dequantize_nf4(_ptr(qs), _ptr(absmax), _codebook(codebook), N, K, _ptr(W), _rows(W),
                                 _stream(qs.device))
    _check(rc, lib)
    return W


def nf4_dequant_gemm(qs, absmax, codebook, X, W=None, logits=None):
    """The dequantise-then-GEMM path: wobs_dequantize_nf4 into ``W`` (bf16
    [N, K], allocated if not given), then the dense bf16 GEMV
    (wobs_gemv_bf16) over the columns of X (bf16 [M, K]) in calls of at most
    32 columns.  Returns fp32 logits [M, N] and W."""
    W = wobs_dequantize_nf4(qs, absmax, codebook, W)
    X2 = X.view(1, -1) if X.dim() == 1 else X
    _need(X2, "X", torch.bfloat16, 2, qs.device)
    M = X2.shape[0]
    N = W.shape[0]
    if logits is None:
        logits = torch.empty(M, N, dtype=torch.float32, device=qs.device)
    for m0 in range(0, M, MAX_M):
        m1 = min(M, m0 + MAX_M)
        wobs_gemv_bf16(W, X2[m0:m1], logits=logits[m0:m1])
    return logits, W


def _argcmp(name, X, out, ws):
    lib = _lib.get()
    X2 = X if X.dim() == 2 else X.view(1, -1)
    _need(X2, "X", None, 2)
    if X2.dtype not in DTYPE_CODES:
        raise TypeError(f"X: dtype {X2.dtype}, expected float16, bfloat16 or float32")
    M, N = X2.shape
    if out is None:
        out = torch.empty(M, dtype=torch.int64, device=X2.device)
    _need(out, "out", torch.int64, None, X2.device)
    if ws is None:
        need = wobs_workspace_size(OP_ARGCMP, M, N, X2.element_size())
        ws = workspace(OP_ARGCMP, M, N, X2.element_size(), X2.device) if need else None
    rc = getattr(lib, name)(DTYPE_CODES[X2.dtype], _ptr(X2), _rows(X2), M, N, _ptr(out), _ptr(ws),
                            ws.numel() if ws is not None else 0, _stream(X2.device))
    _check(rc, lib)
    return out


def wobs_argmax(X, out=None, ws=None):
    """int64 [M]: index of the largest element of each row of X [M, N] (lowest on ties)."""
    return _argcmp("wobs_argmax", X, out, ws)


def wobs_argmin(X, out=None, ws=None):
    """int64 [M]: index of the smallest element of each row of X [M, N] (lowest on ties)."""
    return _argcmp("wobs_argmin", X, out, ws)


# ------------------------------------- the decode step around the products
#
# A decode step makes these calls once a layer, so their checks are written
# for the common case: one condition that holds for good arguments, and
# _need's messages only where it does not.  Element types go to the library
# as codes; one that it does not know is 0, which it refuses.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_code = DTYPE_CODES.get


def _pitch(t, name, index):
    """Row pitch of a 2-D tensor on CUDA device ``index`` (-1: any) whose last dim is contiguous."""
    _need(t, name, None, 2, None if index < 0 else torch.device("cuda", index))
    return t.stride(0)


def _vector(t, name, dtype, n, index):
    """Checks a vector of n elements; its address."""
    if t.dtype is dtype and t.get_device() == index and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype, 1, torch.device("cuda", index))
    raise ValueError(f"{name}: {t.shape[0]} values, expected {n}")


def wobs_rmsnorm_q8_1(x, weight, eps=1e-5, residual=None, residual_out=None, xq=None, want_xq=True, y=None):
    """Residual addition, RMS norm and Q8_1 quantisation of rows x [M, K] (or [K]) in one kernel.

    h = x + residual, rounded to the residual's dtype and stored to ``residual_out`` (default: to
    ``residual`` itself); y = h / sqrt(mean(h^2) + eps) * weight in float32.  Returns (xq, h): the
    Q8_1 blocks of y (uint8 [M, K/32*36], None with ``want_xq=False``) and the stored sum (x itself
    without a residual).  ``y`` (float16, bfloat16 or float32 [M, K]) also receives y when given, for
    products that take plain activations (as their activations: a copy or another kernel must stand
    between y or h and a product that takes them as weights).
    """
    lib = _lib.get()
    X2 = x if x.dim() == 2 else x.view(1, -1)
    M, K = shape = X2.shape
    dev = X2.get_device()
    x_pitch = K if dev >= 0 and X2.is_contiguous() else _pitch(X2, "x", -1)
    w_type = weight.dtype
    w_ptr = _vector(weight, "weight", w_type, K, dev)
    r_code = r_ptr = r_pitch = h_ptr = h_pitch = y_code = y_ptr = y_pitch = 0
    if residual is not None:
        if residual_out is None:
            residual_out = residual
        r2 = residual if residual.dim() == 2 else residual.view(1, -1)
        h2 = residual_out if residual_out.dim() == 2 else residual_out.view(1, -1)
        if r2.shape != shape or h2.shape != shape:
            raise ValueError("x, residual and residual_out must have the same shape")
        r_type = r2.dtype
        if h2.dtype is not r_type:
            raise TypeError(f"residual_out: dtype {h2.dtype}, expected {r_type}")
        r_code, r_ptr, h_ptr = _code(r_type, 0), r2.data_ptr(), h2.data_ptr()
        r_pitch = K if r2.get_device() == dev and r2.is_contiguous() else _pitch(r2, "residual", dev)
        h_pitch = K if h2.get_device() == dev and h2.is_contiguous() else _pitch(h2, "residual_out", dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if y is not None:
        y2 = y if y.dim() == 2 else y.view(1, -1)
        if y2.shape != shape:
            raise ValueError("x and y must have the same shape")
        y_pitch = K if y2.get_device() == dev and y2.is_contiguous() else _pitch(y2, "y", dev)
        y_code, y_ptr = _code(y2.dtype, 0), y2.data_ptr()
    if not want_xq:
        xq = None
    elif xq is None:
        xq = X2.new_empty((M, K // 32 * Q8_1_BLOCK_BYTES), dtype=torch.uint8)
    else:
        _need(xq, "xq", torch.uint8, None, X2.device)
        if xq.numel() != M * (K // 32) * Q8_1_BLOCK_BYTES or not xq.is_contiguous():
            raise ValueError("xq must be contiguous [M, K/32*36]")
    rc = lib.wobs_rmsnorm_q8_1(_code(X2.dtype, 0), X2.data_ptr(), x_pitch, r_code, r_ptr, r_pitch, h_ptr, h_pitch,
                               _code(w_type, 0), w_ptr, eps, M, K, 0 if xq is None else xq.data_ptr(), y_code, y_ptr,
                               y_pitch, _raw_stream(dev))
    if rc:
        _check(rc, lib)
    return xq, (x if residual is None else residual_out)


def wobs_dequantize_q8_1(xq, dtype=torch.float32, out=None):
    """The values [M, K] (q * d, rounded once to ``dtype``) of Q8_1 blocks xq [M, K/32*36]."""
    lib = _lib.get()
    xq2 = xq if xq.dim() == 2 else xq.view(1, -1)
    M, width = xq2.shape
    dev = xq2.get_device()
    if xq2.dtype is not torch.uint8 or dev < 0:
        _need(xq2, "xq", torch.uint8, 2)
    if width % Q8_1_BLOCK_BYTES or not xq2.is_contiguous():
        raise ValueError("xq must be contiguous [M, K/32*36]")
    K = width // Q8_1_BLOCK_BYTES * 32
    if out is None:
        out = xq2.new_empty((M, K), dtype=dtype)
    else:
        _need(out, "out", dtype, None, xq2.device)
        if out.numel() != M * K or not out.is_contiguous():
            raise ValueError("out must be contiguous [M, K]")
    rc = lib.wobs_dequantize_q8_1(xq2.data_ptr(), M, K, _code(out.dtype, 0), out.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc, lib)
    return out


class Kv4Cache:
    """A paged key/value cache held in 4 bits (Q4_0 blocks of 32 along each token's head).

    ``kq``, ``vq``: uint8 [pages, heads, page_size, dim/2]; ``kd``, ``vd``: float16
    [pages, heads, page_size, dim/32]; all contiguous.  The calls below also take ``table``, int32
    [B, max_pages] (the pages of each sequence, in order; entries past its last page are not read),
    and ``lens``, int32 [B] (tokens held of each sequence, the newest of the call included).
    """

    def __init__(self, kq, kd, vq, vd):
        for t, name, dt in ((kq, "kq", torch.uint8), (kd, "kd", torch.float16), (vq, "vq", torch.uint8),
                            (vd, "vd", torch.float16)):
            _need(t, name, dt, 4, kq.device)
            if not t.is_contiguous():
                raise ValueError(f"{name}: must be contiguous")
        if vq.shape != kq.shape or kd.shape != vd.shape or kd.shape[:3] != kq.shape[:3] \
                or kq.shape[3] != 16 * kd.shape[3]:
            raise ValueError("planes must be [pages, heads, page_size, dim/2] and [pages, heads, page_size, dim/32]")
        self.kq, self.kd, self.vq, self.vd = kq, kd, vq, vd
        self.pages, self.heads, self.page_size = kq.shape[:3]
        self.dim = 2 * kq.shape[3]
        self.device = kq.device
        self._index = kq.get_device()
        self._c = _lib.Kv4CacheStruct(kq.data_ptr(), kd.data_ptr(), vq.data_ptr(), vd.data_ptr(), self.pages,
                                      self.page_size, self.heads, self.dim)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages, page_size, heads, dim, device=None):
        """A cache of that many pages; its contents are undefined until tokens are appended."""
        device = torch.device("cuda") if device is None else device
        plane = lambda width, dt: torch.empty(pages, heads, page_size, width, dtype=dt, device=device)  # noqa: E731
        return cls(plane(dim // 2, torch.uint8), plane(dim // 32, torch.float16), plane(dim // 2, torch.uint8),
                   plane(dim // 32, torch.float16))


def _sequences(cache, table, lens):
    """Checks a block table and its lengths: (device index, batch, table address and pitch, pages a sequence,
    lengths' address)."""
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache: expected a Kv4Cache")
    index = cache._index
    B, P = table.shape if table.dim() == 2 else (0, 0)
    if table.dtype is torch.int32 and table.get_device() == index and table.is_contiguous():
        pitch = P
    else:
        pitch = _pitch(table, "table", index)
        _need(table, "table", torch.int32)
    return index, B, table.data_ptr(), pitch, P, _vector(lens, "lens", torch.int32, B, index)


_Strides = ctypes.c_int64 * 3


def _tokens(t, name, B, dim, index, heads=0):
    """Checks [B, L, heads, dim] (a missing L is 1): (L, heads, dtype code, address, strides as a C array)."""
    shape, s = t.shape, t.stride()
    if len(shape) == 3:
        shape, s = (shape[0], 1, shape[1], shape[2]), (s[0], 0, s[1], s[2])
    if len(shape) != 4 or shape[0] != B or shape[3] != dim or (heads and shape[2] != heads):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{B}, L, {heads or 'heads'}, {dim}]")
    if t.get_device() != index or s[3] != 1:
        _need(t, name, None, None, torch.device("cuda", index))
    return shape[1], shape[2], _code(t.dtype, 0), t.data_ptr(), _Strides(s[0], s[1], s[2])


def wobs_kv4_append(cache, k, v, table, lens):
    """Writes the newest tokens k, v [B, L, heads, dim] (or [B, heads, dim]) at positions lens - L .. lens - 1.

    float16, bfloat16 or float32; any strides with a contiguous last axis (slices of a fused
    projection).  Codes and scales equal wobs_quantize_q4_0 of the float32 values.
    """
    lib = _lib.get()
    index, B, table_ptr, pitch, P, lens_ptr = _sequences(cache, table, lens)
    L, _, code, k_ptr, ks = _tokens(k, "k", B, cache.dim, index, cache.heads)
    Lv, _, v_code, v_ptr, vs = _tokens(v, "v", B, cache.dim, index, cache.heads)
    if Lv != L or v_code != code:
        raise ValueError("k and v must have the same shape and dtype")
    rc = lib.wobs_kv4_append(cache._ref, code, k_ptr, ks, v_ptr, vs, B, L, table_ptr, pitch, P, lens_ptr, _raw_stream(index))
    if rc:
        _check(rc, lib)


def wobs_kv4_read(cache, table, lens, count, dtype=torch.float32, k=None, v=None):
    """The values (k, v), each [B, count, heads, dim] of ``dtype``, of the newest ``count`` tokens (zeros before
    a sequence's first token)."""
    lib = _lib.get()
    index, B, table_ptr, pitch, P, lens_ptr = _sequences(cache, table, lens)
    shape = (B, count, cache.heads, cache.dim)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _need(t, name, dtype, 4, cache.device)
            if t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name}: must be contiguous {shape}")
    if k is None:
        k = table.new_empty(shape, dtype=dtype)
    if v is None:
        v = table.new_empty(shape, dtype=dtype)
    rc = lib.wobs_kv4_read(cache._ref, table_ptr, pitch, P, lens_ptr, B, count, _code(dtype, 0), k.data_ptr(),
                           v.data_ptr(), _raw_stream(index))
    if rc:
        _check(rc, lib)
    return k, v


_attn_bytes = {}      # workspace bytes of wobs_attn_kv4 by (device, dim): they depend on nothing else


def wobs_attn_kv4(cache, q, table, lens, scale=None, out=None, out_dtype=None, ws=None):
    """Attention of the newest L <= 32 tokens q [B, L, q_heads, dim] (or [B, q_heads, dim]) over the cache.

    Causal: query i sees positions up to lens - L + i; one that sees none gives zeros.  q_heads is a
    multiple of the cache's heads (grouped heads).  ``scale`` defaults to dim ** -0.5.  Returns a
    contiguous tensor of q's shape, of q's dtype or float32 (``out_dtype``); as with every activation,
    a copy or another kernel must stand between it and a product that takes it as weights.
    """
    lib = _lib.get()
    index, B, table_ptr, pitch, P, lens_ptr = _sequences(cache, table, lens)
    dim = cache.dim
    L, heads, code, q_ptr, qs = _tokens(q, "q", B, dim, index)
    if out is None:
        out = q.new_empty(q.shape, dtype=out_dtype)
    else:
        _need(out, "out", out_dtype, None, cache.device)
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous, of q's shape")
    stream = _raw_stream(index)
    if ws is None:
        need = _attn_bytes.get((index, dim))
        if need is None:
            need = _attn_bytes[(index, dim)] = wobs_workspace_size(OP_ATTN_KV4, 1, 1, dim)
        ws = _ws_cache.get((index, stream))
        if ws is None or ws.numel() < need:
            ws = workspace(OP_ATTN_KV4, B * L, heads, dim, cache.device)
    ws_ptr, ws_bytes = (0, 0) if ws is None else (ws.data_ptr(), ws.numel())
    rc = lib.wobs_attn_kv4(cache._ref, code, q_ptr, qs, B, L, heads, dim ** -0.5 if scale is None else scale, table_ptr,
                           pitch, P, lens_ptr, _code(out.dtype, 0), out.data_ptr(), ws_ptr, ws_bytes, stream)
    if rc:
        _check(rc, lib)
    return out


def wobs_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None):
    """One token a row of logits [M, N] (or [N]) from the random numbers u [M] in [0, 1).

    ``temperature``, ``top_p``, ``min_p`` (float32 [M]) and ``top_k`` (int32 [M]) are optional device
    tensors; values that switch a row's filter off: top_k <= 0, top_p >= 1, min_p <= 0, and a
    temperature <= 0 takes the largest logit.  Returns (tokens int64 [M], probs float32 [M]): the
    token and its probability among those kept; (-1, 0) where a row holds only -infinity and NaN.
    """
    lib = _lib.get()
    X2 = logits if logits.dim() == 2 else logits.view(1, -1)
    M, N = X2.shape
    dev = X2.get_device()
    pitch = N if dev >= 0 and X2.is_contiguous() else _pitch(X2, "logits", -1)
    f32 = torch.float32
    u_ptr = _vector(u, "u", f32, M, dev)
    t_ptr = 0 if temperature is None else _vector(temperature, "temperature", f32, M, dev)
    k_ptr = 0 if top_k is None else _vector(top_k, "top_k", torch.int32, M, dev)
    p_ptr = 0 if top_p is None else _vector(top_p, "top_p", f32, M, dev)
    m_ptr = 0 if min_p is None else _vector(min_p, "min_p", f32, M, dev)
    if tokens is None:
        tokens = X2.new_empty(M, dtype=torch.int64)
        token_ptr = tokens.data_ptr()
    else:
        token_ptr = _vector(tokens, "tokens", torch.int64, M, dev)
    if probs is None:
        probs = X2.new_empty(M, dtype=f32)
        prob_ptr = probs.data_ptr()
    else:
        prob_ptr = _vector(probs, "probs", f32, M, dev)
    rc = lib.wobs_sample(_code(X2.dtype, 0), X2.data_ptr(), pitch, M, N, u_ptr, t_ptr, k_ptr, p_ptr, m_ptr, token_ptr, prob_ptr,
                         _raw_stream(dev))
    if rc:
        _check(rc, lib)
    return tokens, probs


def wobs_q4_0_q8_1_blockdots(qs, xq):
    """Exact int32 block dots [M, N, K/32] (test export)."""
    lib = _lib.get()
    _need(qs, "qs", torch.uint8, 2)
    xq2 = xq if xq.dim() == 2 else xq.view(1, -1)
    _need(xq2, "xq", torch.uint8, 2, qs.device)
    N, K = qs.shape[0], qs.shape[1] * 2
    M = xq2.shape[0]
    out = torch.empty(M, N, K // 32, dtype=torch.int32, device=qs.device)
    rc = lib.wobs_q4_0_q8_1_blockdots(_ptr(qs), _ptr(xq2), M, N, K, _ptr(out), _stream(qs.device))
    _check(rc, lib)
    return out


def wobs_selftest_wait_timeout(limit_cycles=1_000_000, device=None):
    """Launch the failure-path self test (a wait that gives up); returns nothing."""
    lib = _lib.get()
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    _check(lib.wobs_selftest_wait_timeout(int(limit_cycles), _stream(device)), lib)


def wobs_error_word(device=None):
    """Read and clear the device error word (synchronises the current stream)."""
    lib = _lib.get()
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    v = ctypes.c_int(0)
    rc = lib.wobs_error_word(_stream(device), ctypes.byref(v))
    if v.value == 0:                   # a recorded code is the value asked for
        _check(rc, lib)
    return v.value
