"""Python binding of libqspec.so (the C ABI in include/qspec.h).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of the library.  Importing this module loads the library and raises
if it is missing; there is no fallback implementation.

Functions take CUDA torch tensors (contiguous, on the current device) and
launch on the current torch stream unless `stream` is given.  Outputs that are
not given are memory of the stream that the call runs on; the caller orders
the streams (inputs ready before, outputs read after) and keeps the inputs
until the call is done, as with any torch operation on another stream.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqspec.so")

OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported device", 3: "CUDA error",
                4: "workspace too small", 5: "timeout", 6: "bad input"}
OP_QUANTIZE_WEIGHTS, OP_QUANT_ACT, OP_GEMM_W4A4, OP_GEMM_W4A16, OP_SPEC_ACCEPT, OP_GEMM_W4A8 = range(6)

EXPORTED = ("qspec_quantize_weights", "qspec_quant_act", "qspec_cast_bf16", "qspec_gemm_w4a4",
            "qspec_gemm_w4a8",
            "qspec_gemm_w4a16",
            "qspec_spec_accept", "qspec_spec_accept_greedy", "qspec_workspace_size",
            "qspec_workspace_status",
            "qspec_status_string", "qspec_gemm_w4a16_noalloc", "qspec_gemm_w4a16_noalloc_status",
            "qspec_kv_append", "qspec_attn_decode", "qspec_attn_workspace_size", "qspec_kv_commit",
            "qspec_rope_table", "qspec_qkv_rope_append", "qspec_attn_prefill",
            "qspec_attn_prefill_workspace_size", "qspec_attn_prefix",
            "qspec_attn_prefix_workspace_size", "qspec_call", "qspec_abi_version")
ABI_VERSION = 5
_raw_stream = torch._C._cuda_getCurrentRawStream     # the current stream of a device, as a plain handle
HEAD_DIM = 128           # the KV-cache calls' head dimension
ROPE_INTERLEAVED, ROPE_Q_FP32 = 1, 2
GEMM_WEIGHTS_READY = 1   # flag: wq/ws are not written by work still in flight
GEMM_TEST_STALL = 0x100  # test hook: the GEMM's first wait runs out (QSPEC_GEMM_TEST_STALL)
CALL_TEST_STALL = 0x100  # test hook: the prompt attention's waits run out (QSPEC_CALL_TEST_STALL)
GEMM_FUSED_QUANT = 0x2   # drafting modes, m <= 32: activations quantized inside the GEMM kernel


class QSpecError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} (status {status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"libqspec.so not found at {_LIB_PATH}; build it with "
            "`python -m quantized_speculative_decoding_packed_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, U32, SZ, F32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32,
                                 ctypes.c_size_t, ctypes.c_float)
    lib.qspec_quantize_weights.argtypes = [P, I64, I64, I32, P, P, P]
    lib.qspec_quant_act.argtypes = [P, I64, I64, P, P, P]
    lib.qspec_cast_bf16.argtypes = [P, I64, I64, I64, P, P]
    lib.qspec_gemm_w4a4.argtypes = [P, I64, I64, P, P, I64, I32, P, P, SZ, P, U32, P]
    lib.qspec_gemm_w4a8.argtypes = [P, I64, I64, P, P, I64, I32, P, P, SZ, P, U32, P]
    lib.qspec_gemm_w4a4_f32in.argtypes = [P, I64, I64, I64, P, P, I64, I32, P, P, SZ, P, U32, P]
    lib.qspec_gemm_w4a8_f32in.argtypes = [P, I64, I64, I64, P, P, I64, I32, P, P, SZ, P, U32, P]
    lib.qspec_gemm_w4a16.argtypes = [P, I64, I64, P, P, I64, I32, P, P, SZ, U32, P]
    lib.qspec_gemm_w4a16_noalloc.argtypes = [P, I64, I64, P, P, I64, I32, P, U32, P]
    lib.qspec_gemm_w4a16_noalloc_status.argtypes = [P]
    lib.qspec_abi_version.argtypes = []
    lib.qspec_abi_version.restype = I32
    lib.qspec_spec_accept.argtypes = [P, P, P, P, P, I32, I32, I32, P, P, P, SZ, P]
    lib.qspec_spec_accept_greedy.argtypes = [P, P, I32, I32, I32, P, P, P, SZ, P]
    lib.qspec_workspace_size.argtypes = [I32, I64, I64, I64, I32, I32, I32, I32]
    lib.qspec_workspace_size.restype = SZ
    lib.qspec_workspace_status.argtypes = [P, P]
    lib.qspec_kv_append.argtypes = [P, I64, I32, I32, I32, I32, I32, P, I32, P, P, I32, P, SZ, P]
    lib.qspec_attn_decode.argtypes = [P, I64, I32, I32, I32, I32, I32, P, I32, P, P, I32, I32, P,
                                      I64, P, SZ, P]
    lib.qspec_attn_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32]
    lib.qspec_attn_workspace_size.restype = SZ
    lib.qspec_kv_commit.argtypes = [P, P, I32, I32, P, SZ, P]
    lib.qspec_rope_table.argtypes = [P, I32, I64, P, P]
    lib.qspec_qkv_rope_append.argtypes = [P, I64, I64, I32, P, I32, I32, I32, P, P, F32, P, I64, I32, P, P,
                                          I32, P, P, I32, P, I64, U32, P, SZ, P]
    lib.qspec_attn_prefill.argtypes = [P, I64, I64, I32, P, I32, I32, I32, P, P, P, I32, P, I64, P, SZ, P]
    lib.qspec_attn_prefix.argtypes = [P, I64, I64, I32, P, I32, I32, I32, P, I32, P, P, I32, P, P, I32, P,
                                      P, I64, P, SZ, P]
    lib.qspec_call.argtypes = [I32, ctypes.c_char_p, I32, P]
    lib.qspec_attn_prefill_workspace_size.argtypes = []
    lib.qspec_attn_prefill_workspace_size.restype = SZ
    lib.qspec_attn_prefix_workspace_size.argtypes = [I64, I32, I32, I32]
    lib.qspec_attn_prefix_workspace_size.restype = SZ
    lib.qspec_status_string.argtypes = [I32]
    lib.qspec_status_string.restype = ctypes.c_char_p
    for name in ("qspec_quantize_weights", "qspec_quant_act", "qspec_cast_bf16", "qspec_gemm_w4a4",
                 "qspec_gemm_w4a8", "qspec_gemm_w4a4_f32in", "qspec_gemm_w4a8_f32in",
                 "qspec_gemm_w4a16", "qspec_spec_accept", "qspec_spec_accept_greedy",
                 "qspec_workspace_status",
                 "qspec_gemm_w4a16_noalloc", "qspec_gemm_w4a16_noalloc_status",
                 "qspec_kv_append", "qspec_attn_decode", "qspec_kv_commit", "qspec_rope_table",
                 "qspec_qkv_rope_append", "qspec_attn_prefill", "qspec_attn_prefix", "qspec_call"):
        getattr(lib, name).restype = ctypes.c_int
    if lib.qspec_abi_version() != ABI_VERSION:
        raise ImportError(f"{_LIB_PATH} has ABI version {lib.qspec_abi_version()}, "
                          f"this binding needs {ABI_VERSION}; rebuild the library")
    return lib


LIB = _load()
LIB_PATH = _LIB_PATH


def _check(status: int, what: str) -> None:
    if status != OK:
        raise QSpecError(status, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _empty(stream, shape, dtype, device) -> torch.Tensor:
    """An output that is not given: memory of the stream that writes it.

    A block that the current stream has freed may still be in use by work queued there, for which
    another stream does not wait; and this one is kept until the current stream is done with it too.
    """
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


_WS_CACHE: dict = {}


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-initialised per-device scratch buffer of at least `nbytes` bytes.

    The library leaves it ready for reuse after every call that completes.
    Calls that run concurrently on different streams, or come from different
    host threads, need separate buffers.
    """
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    cur = _WS_CACHE.get(dev)
    if cur is None or cur.numel() < nbytes:
        cur = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _WS_CACHE[dev] = cur
    return cur


def workspace_size(op: int, m: int = 0, n: int = 0, k: int = 0, group: int = 128,
                   batch: int = 0, gamma: int = 0, vocab: int = 0) -> int:
    return int(LIB.qspec_workspace_size(op, m, n, k, group, batch, gamma, vocab))


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    return int(LIB.qspec_workspace_status(_ptr(ws), _stream(stream)))


def scale_row_stride(k: int, group: int) -> int:
    """Entries per row of the scale matrix: k/group rounded up to a multiple of 8."""
    return (k // group + 7) // 8 * 8


def quantize_weights(w: torch.Tensor, group: int = 128, wq: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None):
    """fp32 [N][K] -> (wq uint8 [N][K/2], ws fp16 [N][scale_row_stride(K, group)]).

    ws[:, :K/group] holds the group scales; the padding columns are zero.
    """
    _need(w, torch.float32, "w")
    n, k = w.shape
    if wq is None:
        wq = _empty(stream, (n, k // 2), torch.uint8, w.device)
    if ws is None:
        ws = _empty(stream, (n, scale_row_stride(k, group)), torch.float16, w.device)
    _check(LIB.qspec_quantize_weights(_ptr(w), n, k, group, _ptr(wq), _ptr(ws), _stream(stream)),
           "qspec_quantize_weights")
    return wq, ws


def quant_act(x: torch.Tensor, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None,
              stream=None):
    """bf16 [M][K] -> (xq uint8 [M][K/2] packed INT4, xs fp32 [M] per-token scales)."""
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    if xq is None:
        xq = _empty(stream, (m, k // 2), torch.uint8, x.device)
    if xs is None:
        xs = _empty(stream, (m,), torch.float32, x.device)
    _check(LIB.qspec_quant_act(_ptr(x), m, k, _ptr(xq), _ptr(xs), _stream(stream)),
           "qspec_quant_act")
    return xq, xs


def _flags(weights_ready: bool, flags: int) -> int:
    return (GEMM_WEIGHTS_READY if weights_ready else 0) | flags


def cast_bf16(y: torch.Tensor, k: int | None = None, x: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """fp32 [M][N] -> bf16 [M][k]: the first k columns rounded to nearest even."""
    _need(y, torch.float32, "y")
    m, n = y.shape
    k = n if k is None else k
    if x is None:
        x = _empty(stream, (m, k), torch.bfloat16, y.device)
    _check(LIB.qspec_cast_bf16(_ptr(y), m, n, k, _ptr(x), _stream(stream)), "qspec_cast_bf16")
    return x


def linear_chain(x0: torch.Tensor, layers, mode: str = "w4a4", group: int = 128,
                 ys=None, xs=None, work: torch.Tensor | None = None, stream=None,
                 weights_ready: bool = False):
    """Runs linear layers back to back on one token batch: layer j's input is
    the first K_j columns of layer j-1's fp32 output, rounded to bf16 (by the
    drafting GEMMs' quantizer as it reads them, or by qspec_cast_bf16 for the
    verifying GEMM).  layers: [(wq, ws)]; mode: w4a4 | w4a8 | w4a16.  ys/xs:
    optional preallocated outputs / intermediate inputs (for CUDA-graph
    capture).  Returns the list of fp32 outputs."""
    gemm = {"w4a4": gemm_w4a4, "w4a8": gemm_w4a8, "w4a16": gemm_w4a16}[mode]
    m = x0.shape[0]
    outs = []
    x = x0
    for j, (wq, ws) in enumerate(layers):
        n, k = wq.shape[0], wq.shape[1] * 2
        if j and mode != "w4a16":
            x = outs[-1][:, :k]
        elif j:
            x = cast_bf16(outs[-1], k, x=None if xs is None else xs[j], stream=stream)
        y = None if ys is None else ys[j]
        outs.append(gemm(x, wq, ws, group, y=y, work=work, stream=stream, weights_ready=weights_ready))
    return outs


def gemm_w4a4(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, group: int = 128,
              y: torch.Tensor | None = None, work: torch.Tensor | None = None,
              dbg_acc: torch.Tensor | None = None, stream=None,
              weights_ready: bool = False, flags: int = 0) -> torch.Tensor:
    """W4A4 drafting GEMM: y[M][N] fp32 = quant(x) . deq(wq, ws)^T.

    weights_ready: wq/ws are not being written by work that may still be
    running (sets QSPEC_GEMM_WEIGHTS_READY; the weights then stream while the
    preceding kernel finishes).  flags: further QSPEC_GEMM_* bits.
    """
    return _drafting("w4a4", x, wq, ws, group, y, work, dbg_acc, stream, weights_ready, flags)


def gemm_w4a8(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, group: int = 128,
              y: torch.Tensor | None = None, work: torch.Tensor | None = None,
              dbg_acc: torch.Tensor | None = None, stream=None,
              weights_ready: bool = False, flags: int = 0) -> torch.Tensor:
    """W4A8 drafting variant: y[M][N] fp32 = quant8(x) . deq(wq, ws)^T (arguments as gemm_w4a4)."""
    return _drafting("w4a8", x, wq, ws, group, y, work, dbg_acc, stream, weights_ready, flags)


def _drafting(mode, x, wq, ws, group, y, work, dbg_acc, stream, weights_ready, flags):
    """The drafting GEMMs: x bf16 [M][K] (contiguous), or fp32 [M][K] with unit column
    stride (e.g. the first K columns of a layer's output), rounded to bf16 as it is
    quantized (qspec_gemm_*_f32in)."""
    m, k = x.shape
    n = wq.shape[0]
    op = OP_GEMM_W4A4 if mode == "w4a4" else OP_GEMM_W4A8
    if y is None:
        y = _empty(stream, (m, n), torch.float32, x.device)
    need = workspace_size(op, m, n, k, group)
    if work is None:
        work = workspace(need, x.device)
    fl = _flags(weights_ready, flags)
    if x.dtype == torch.float32:
        if not x.is_cuda or x.stride(1) != 1:
            raise ValueError("fp32 x must be a CUDA tensor with unit column stride")
        fn = LIB.qspec_gemm_w4a4_f32in if mode == "w4a4" else LIB.qspec_gemm_w4a8_f32in
        _check(fn(_ptr(x), x.stride(0), m, k, _ptr(wq), _ptr(ws), n, group, _ptr(y), _ptr(work),
                  work.numel(), _ptr(dbg_acc), fl, _stream(stream)), f"qspec_gemm_{mode}_f32in")
        return y
    _need(x, torch.bfloat16, "x")
    fn = LIB.qspec_gemm_w4a4 if mode == "w4a4" else LIB.qspec_gemm_w4a8
    _check(fn(_ptr(x), m, k, _ptr(wq), _ptr(ws), n, group, _ptr(y), _ptr(work), work.numel(),
              _ptr(dbg_acc), fl, _stream(stream)), f"qspec_gemm_{mode}")
    return y


def gemm_w4a16(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, group: int = 128,
               y: torch.Tensor | None = None, work: torch.Tensor | None = None,
               stream=None, weights_ready: bool = False, flags: int = 0) -> torch.Tensor:
    """W4A16 verifying GEMM: y[M][N] fp32 = x . deq(wq, ws)^T (weights_ready, flags: as gemm_w4a4)."""
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    n = wq.shape[0]
    if y is None:
        y = _empty(stream, (m, n), torch.float32, x.device)
    need = workspace_size(OP_GEMM_W4A16, m, n, k, group)
    if work is None:
        work = workspace(need, x.device)
    _check(LIB.qspec_gemm_w4a16(_ptr(x), m, k, _ptr(wq), _ptr(ws), n, group, _ptr(y), _ptr(work),
                                work.numel(), _flags(weights_ready, flags),
                                _stream(stream)), "qspec_gemm_w4a16")
    return y


def gemm_w4a16_noalloc(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, group: int = 128,
                       y: torch.Tensor | None = None, stream=None,
                       weights_ready: bool = False) -> torch.Tensor:
    """W4A16 verifying GEMM using the library's built-in scratch (no workspace).

    For callers that cannot allocate device memory where they call; the
    output buffer is still the caller's.  Calls must not overlap on the GPU.
    """
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    n = wq.shape[0]
    if y is None:
        y = _empty(stream, (m, n), torch.float32, x.device)
    _check(LIB.qspec_gemm_w4a16_noalloc(_ptr(x), m, k, _ptr(wq), _ptr(ws), n, group, _ptr(y),
                                        GEMM_WEIGHTS_READY if weights_ready else 0,
                                        _stream(stream)), "qspec_gemm_w4a16_noalloc")
    return y


def noalloc_status(stream=None) -> int:
    """Device status of gemm_w4a16_noalloc on the current device (read and cleared)."""
    return int(LIB.qspec_gemm_w4a16_noalloc_status(_stream(stream)))


def spec_accept(p: torch.Tensor, q: torch.Tensor, draft: torch.Tensor, u_acc: torch.Tensor,
                u_res: torch.Tensor, n_accepted: torch.Tensor | None = None,
                tokens: torch.Tensor | None = None, work: torch.Tensor | None = None,
                stream=None):
    """Speculative accept / residual resample -> (n_accepted int32 [B], tokens int32 [B][gamma+1])."""
    _need(p, torch.float32, "p")
    _need(q, torch.float32, "q")
    _need(draft, torch.int32, "draft")
    _need(u_acc, torch.float32, "u_acc")
    _need(u_res, torch.float32, "u_res")
    b, g1, v = p.shape
    gamma = g1 - 1
    if n_accepted is None:
        n_accepted = _empty(stream, (b,), torch.int32, p.device)
    if tokens is None:
        tokens = _empty(stream, (b, gamma + 1), torch.int32, p.device)
    nbytes = 0 if work is None else work.numel()
    _check(LIB.qspec_spec_accept(_ptr(p), _ptr(q), _ptr(draft), _ptr(u_acc), _ptr(u_res), b, gamma,
                                 v, _ptr(n_accepted), _ptr(tokens), _ptr(work), nbytes,
                                 _stream(stream)), "qspec_spec_accept")
    return n_accepted, tokens


def spec_accept_greedy(p: torch.Tensor, draft: torch.Tensor, n_accepted: torch.Tensor | None = None,
                       tokens: torch.Tensor | None = None, work: torch.Tensor | None = None,
                       stream=None):
    """Greedy verification -> (n_accepted int32 [B], tokens int32 [B][gamma+1])."""
    _need(p, torch.float32, "p")
    _need(draft, torch.int32, "draft")
    b, g1, v = p.shape
    gamma = g1 - 1
    if n_accepted is None:
        n_accepted = _empty(stream, (b,), torch.int32, p.device)
    if tokens is None:
        tokens = _empty(stream, (b, gamma + 1), torch.int32, p.device)
    nbytes = 0 if work is None else work.numel()
    _check(LIB.qspec_spec_accept_greedy(_ptr(p), _ptr(draft), b, gamma, v, _ptr(n_accepted),
                                        _ptr(tokens), _ptr(work), nbytes, _stream(stream)),
           "qspec_spec_accept_greedy")
    return n_accepted, tokens


# ---------------------------------------------------------------- shared KV cache
def _kv_cache_check(k_cache: torch.Tensor, v_cache: torch.Tensor):
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor [B][H_kv][L_max][128]")
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != HEAD_DIM:
        raise ValueError("k_cache and v_cache must both be [B][H_kv][L_max][128]")
    b, h_kv, l_max, _ = k_cache.shape
    return b, h_kv, l_max


def _qkv_check(qkv: torch.Tensor):
    if not qkv.is_cuda or qkv.dtype != torch.float32 or qkv.dim() != 2 or qkv.stride(1) != 1:
        raise ValueError("qkv must be a CUDA fp32 [B*T][N] tensor with unit column stride")


def _tokens_per_sequence(qkv: torch.Tensor, batch: int) -> int:
    if qkv.shape[0] % batch != 0 or qkv.shape[0] == 0:
        raise ValueError(f"qkv has {qkv.shape[0]} rows, not a positive multiple of the batch {batch}")
    return qkv.shape[0] // batch


def attn_workspace_size(batch: int, t_new: int, h_q: int, h_kv: int, ctx_max: int) -> int:
    return int(LIB.qspec_attn_workspace_size(batch, t_new, h_q, h_kv, HEAD_DIM, ctx_max))


class _StreamBuffers(threading.local):
    """Default workspaces of one host thread, by device and stream.  Work of two streams may overlap; and what
    two threads enqueue on one stream may interleave between the kernels of a call."""

    def __init__(self):
        self.of = {}
        self.retired = []        # what has become too small, for who asked for it may still use it


# attn_decode's own: [buffer, bytes from its start that are zero between calls].  The partial results lie
# behind a call's arrival counters, where the GEMMs keep their split-tile tickets, and where a call with
# more counters has counters; so the buffer is not the GEMMs', and those that a call with fewer counters
# has written over are cleared before they count again.
_ATTN_WS = _StreamBuffers()


def _attn_workspace(nbytes: int, dev: int, counters: int, stream=None) -> torch.Tensor:
    if stream is not None:
        # it decides whether a graph is captured, owns the memory and clears it
        with torch.cuda.stream(stream):
            return _attn_workspace(nbytes, dev, counters)
    handle = _raw_stream(dev)
    head = 256 + 4 * counters
    if torch.cuda.is_current_stream_capturing():
        # the graph's alone, and cleared in it: an eager call could run before the graph, and would outgrow it
        ws = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
        ws[:head].zero_()
        return ws
    cur = _ATTN_WS.of.get((dev, handle))
    if cur is None or cur[0].numel() < nbytes:
        cur = [torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}"), 0]
        _ATTN_WS.of[dev, handle] = cur
    ws, clear = cur
    if head > clear:
        ws[clear:head].zero_()
    cur[1] = head
    return ws


def attn_workspace(device=None, stream=None) -> torch.Tensor:
    """The buffer that attn_decode of this thread takes where `work` is not given, on one stream: workspace_status
    of it tells what the calls have reported.  (A captured call has one of the graph's: pass it `work`.)"""
    dev = torch.cuda.current_device() if device is None else torch.device(device).index
    return _attn_workspace(256, torch.cuda.current_device() if dev is None else dev, 0, stream)


def kv_append(qkv: torch.Tensor, lens: torch.Tensor, offset: int, k_cache: torch.Tensor,
              v_cache: torch.Tensor, h_q: int, work: torch.Tensor | None = None, stream=None):
    """Write the new tokens' keys and values (rows b*T + t of the fused QKV output)
    into the caches at positions lens[b] + offset + t."""
    _qkv_check(qkv)
    _need(lens, torch.int32, "lens")
    b, h_kv, l_max = _kv_cache_check(k_cache, v_cache)
    t_new = _tokens_per_sequence(qkv, b)
    nbytes = 0 if work is None else work.numel()
    _check(LIB.qspec_kv_append(_ptr(qkv), qkv.stride(0), b, t_new, h_q, h_kv, HEAD_DIM, _ptr(lens),
                               offset, _ptr(k_cache), _ptr(v_cache), l_max, _ptr(work), nbytes,
                               _stream(stream)), "qspec_kv_append")


def attn_decode(qkv: torch.Tensor, lens: torch.Tensor, offset: int, k_cache: torch.Tensor,
                v_cache: torch.Tensor, h_q: int, ctx_max: int, out: torch.Tensor | None = None,
                work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode attention of the new tokens over the shared cache -> fp32 [B*T][H*128].

    Without `work` the call takes a buffer of this thread and stream; under capture one of the graph's own, which
    the graph clears before each call (pass `work`, zeroed once, to capture the kernel alone).
    """
    _qkv_check(qkv)
    _need(lens, torch.int32, "lens")
    b, h_kv, l_max = _kv_cache_check(k_cache, v_cache)
    t_new = _tokens_per_sequence(qkv, b)
    if out is None:
        out = _empty(stream, (b * t_new, h_q * HEAD_DIM), torch.float32, qkv.device)
    if work is None:
        need = attn_workspace_size(b, t_new, h_q, h_kv, ctx_max)
        if need == 0:
            raise QSpecError(1, "qspec_attn_decode")
        work = _attn_workspace(need, qkv.get_device(), b * h_kv, stream)
    _check(LIB.qspec_attn_decode(_ptr(qkv), qkv.stride(0), b, t_new, h_q, h_kv, HEAD_DIM,
                                 _ptr(lens), offset, _ptr(k_cache), _ptr(v_cache), l_max, ctx_max,
                                 _ptr(out), out.stride(0), _ptr(work), work.numel(),
                                 _stream(stream)), "qspec_attn_decode")
    return out


def kv_commit(lens: torch.Tensor, n_accepted: torch.Tensor, l_max: int,
              work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """lens += n_accepted + 1 on the device (the round's accepted drafts plus one)."""
    _need(lens, torch.int32, "lens")
    _need(n_accepted, torch.int32, "n_accepted")
    nbytes = 0 if work is None else work.numel()
    _check(LIB.qspec_kv_commit(_ptr(lens), _ptr(n_accepted), lens.numel(), l_max, _ptr(work),
                               nbytes, _stream(stream)), "qspec_kv_commit")
    return lens


# ---------------------------------------------------------------- the prompt path
# These calls run thousands of times a second for single tokens, so what they do on the host
# is kept short: the current stream is asked for as a plain handle (3 us less than the Stream
# object), and the arguments go to the library in one block (qspec_call; 25 arguments of a
# ctypes call take 3 us).
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_ROPE_ARGS, _PREFILL_ARGS, _PREFIX_ARGS = (struct.Struct(f) for f in ("10qd14q", "16q", "21q"))


def _on(t: torch.Tensor, dtype, dev: int, name: str) -> int:
    """The address of a contiguous tensor of `dtype` on CUDA device `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}, "
                         f"not {t.dtype} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, dtype, dev: int, rows: int, columns: int, name: str):
    """(address, row stride) of a [rows][>= columns] tensor with unit column stride."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{dev}, not {t.dtype} on {t.device}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < columns:
        raise ValueError(f"{name} must be [{rows}][{columns}], not {list(shape)}")
    if t.is_contiguous():
        # one row has no stride of its own: a slice of a wider one counts as contiguous
        return t.data_ptr(), shape[1] if rows > 1 else columns
    ld, step = t.stride()
    if step != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld


def _current_device(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


_PROMPT_WS = _StreamBuffers()        # the prompt attention's


def _new_prompt_workspace(nbytes: int, dev: int) -> torch.Tensor:
    ws = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
    ws[:PROMPT_WORKSPACE_ZERO].zero_()
    return ws


PROMPT_WORKSPACE_ZERO = 256       # bytes of a prompt attention workspace that start as zeros


def prompt_workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """The scratch buffer, of at least `nbytes` bytes, that the prompt attention calls of this thread take
    where `work` is not given, on one stream: workspace_status of it tells what they have reported.

    Under stream capture the buffer is a new one that belongs to the graph alone; to read the status of
    captured calls, pass them a buffer as `work`.  Graphs that share one must not run at the same time, and
    neither must calls of two threads.
    """
    dev = torch.device(device).index if torch.device(device).index is not None else torch.cuda.current_device()
    return _prompt_workspace(nbytes, dev, stream)


def _prompt_workspace(nbytes: int, dev: int, stream=None) -> torch.Tensor:
    if stream is not None:
        # it decides whether a graph is captured, owns the memory and clears it
        with torch.cuda.stream(stream):
            return _prompt_workspace(nbytes, dev)
    if torch.cuda.is_current_stream_capturing():
        return _new_prompt_workspace(nbytes, dev)
    key = dev, _raw_stream(dev)
    cur = _PROMPT_WS.of.get(key)
    if cur is None or cur.numel() < nbytes:
        if cur is not None:
            _PROMPT_WS.retired.append(cur)
            nbytes = max(nbytes, 2 * cur.numel())
        cur = _new_prompt_workspace(nbytes, dev)
        _PROMPT_WS.of[key] = cur
    return cur


def attn_prefill_workspace_size() -> int:
    """Bytes that attn_prefill needs on the current device (0 where it does not run)."""
    return int(LIB.qspec_attn_prefill_workspace_size())


def attn_prefix_workspace_size(n_tokens: int, batch: int, h_q: int, h_kv: int) -> int:
    """Bytes that attn_prefix needs on the current device (0: invalid shape, or it does not run).

    Fewer tokens can need more: the size falls where the prefix goes ahead of each sequence's own keys
    (n_tokens // batch * (h_q // h_kv) >= 96); the largest below is for batch * ceil(96 / (h_q // h_kv)) - 1.
    """
    return int(LIB.qspec_attn_prefix_workspace_size(n_tokens, batch, h_q, h_kv))


@functools.lru_cache(maxsize=256)
def _prompt_workspace_size(dev: int, *shape) -> int:
    """One of the sizes above, for the device `dev`, which is current."""
    return attn_prefix_workspace_size(*shape) if shape else attn_prefill_workspace_size()


def _cache_on(k_cache: torch.Tensor, v_cache: torch.Tensor, dev: int):
    """(addresses, batch, KV heads, positions) of a cache pair."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[3] != HEAD_DIM:
        raise ValueError("k_cache and v_cache must both be [B][H_kv][L_max][128]")
    b, h_kv, l_max, _ = k_cache.shape
    return _on(k_cache, _BF16, dev, "k_cache"), _on(v_cache, _BF16, dev, "v_cache"), b, h_kv, l_max


def _packed_on(cu, lens: torch.Tensor, batch: int, n_tokens: int, dev: int):
    """Addresses of lens and cu (None: the same number of tokens for every sequence)."""
    if lens.numel() != batch:
        raise ValueError(f"lens has {lens.numel()} entries for a cache of {batch} sequences")
    if cu is None:
        if n_tokens == 0 or n_tokens % batch != 0:
            raise ValueError(f"{n_tokens} rows are not a positive multiple of the batch {batch}")
        return _on(lens, _I32, dev, "lens"), 0
    if cu.numel() != batch + 1:
        raise ValueError(f"cu has {cu.numel()} entries, {batch + 1} are needed")
    return _on(lens, _I32, dev, "lens"), _on(cu, _I32, dev, "cu")


def _one(t: torch.Tensor, dev: int) -> int:
    if t.numel() != 1:
        raise ValueError("prefix_len must have one element")
    return _on(t, _I32, dev, "prefix_len")


def rope_table(inv_freq: torch.Tensor, positions: int, table: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Angles of `positions` positions for qkv_rope_append: inv_freq fp64 [rot/2] -> fp32 [positions][rot],
    cosines, then sines (computed in 64 bits)."""
    dev = _current_device(inv_freq)
    rot = 2 * inv_freq.numel()
    freq = _on(inv_freq, torch.float64, dev, "inv_freq")
    if table is None:
        table = _empty(stream, (positions, rot), _F32, inv_freq.device)
    if tuple(table.shape) != (positions, rot):
        raise ValueError(f"table must be [{positions}][{rot}]")
    _check(LIB.qspec_rope_table(freq, rot, positions, _on(table, _F32, dev, "table"),
                                _raw_stream(dev) if stream is None else stream.cuda_stream), "qspec_rope_table")
    return table


def qkv_rope_append(qkv: torch.Tensor, lens: torch.Tensor, offset: int, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    h_q: int, table: torch.Tensor | None, cu: torch.Tensor | None = None,
                    prefix_len: torch.Tensor | None = None, q_gamma: torch.Tensor | None = None,
                    k_gamma: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                    q_out: torch.Tensor | None = None, work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Norms and rotation of the queries and keys of packed tokens; keys and values into the caches.

    qkv fp32 [tokens][(h_q + 2 h_kv) * 128]; the queries are returned in q_out: bf16 (the default, for
    attn_prefill and attn_prefix) or fp32, which may be qkv[:, :h_q * 128] itself (for attn_decode on qkv).
    table: rope_table's, or None for no rotation.  cu: int32 [batch + 1] starts of the sequences' tokens
    (None: the same number for each).
    """
    dev = _current_device(qkv)
    kc, vc, b, h_kv, l_max = _cache_on(k_cache, v_cache, dev)
    n = qkv.shape[0]
    x, ld_qkv = _rows(qkv, _F32, dev, n, (h_q + 2 * h_kv) * HEAD_DIM, "qkv")
    lens_p, cu_p = _packed_on(cu, lens, b, n, dev)
    rot = positions = 0
    angles = 0
    if table is not None:
        positions, rot = table.shape
        angles = _on(table, _F32, dev, "table")
    gammas = [0, 0]
    for i, gamma in enumerate((q_gamma, k_gamma)):
        if gamma is not None:
            if gamma.numel() != HEAD_DIM:
                raise ValueError(f"q_gamma and k_gamma must have {HEAD_DIM} entries")
            gammas[i] = _on(gamma, _F32, dev, "q_gamma" if i == 0 else "k_gamma")
    if q_out is None:
        q_out = _empty(stream, (n, h_q * HEAD_DIM), _BF16, qkv.device)
    if q_out.dtype is not _BF16 and q_out.dtype is not _F32:
        raise ValueError("q_out must be bf16 or fp32")
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_Q_FP32 if q_out.dtype is _F32 else 0)
    q_p, ld_q = _rows(q_out, q_out.dtype, dev, n, h_q * HEAD_DIM, "q_out")
    args = _ROPE_ARGS.pack(
        x, ld_qkv, n, b, cu_p, h_q, h_kv, HEAD_DIM, gammas[0], gammas[1], eps, angles, positions, rot,
        0 if prefix_len is None else _one(prefix_len, dev), lens_p, offset, kc, vc, l_max,
        q_p, ld_q, flags,
        0 if work is None else _on(work, torch.uint8, dev, "work"), 0 if work is None else work.numel())
    _check(LIB.qspec_call(0, args, 25, _raw_stream(dev) if stream is None else stream.cuda_stream),
           "qspec_qkv_rope_append")
    return q_out


def attn_prefill(q: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 h_q: int, out: torch.Tensor | None = None, work: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Causal attention of packed prompts over the cache: bf16 [tokens][h_q * 128] -> bf16 of the same shape.

    Token i of sequence b (rows cu[b] .. cu[b + 1] - 1 of q) sees positions 0 .. lens[b] + i.  Rows behind the
    last sequence are not written.
    """
    dev = _current_device(q)
    if cu is None:
        raise ValueError("cu is needed")
    kc, vc, b, h_kv, l_max = _cache_on(k_cache, v_cache, dev)
    n, cols = q.shape[0], h_q * HEAD_DIM
    lens_p, cu_p = _packed_on(cu, lens, b, n, dev)
    if out is None:
        out = _empty(stream, (n, cols), _BF16, q.device)
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if work is None:
        work = _prompt_workspace(_prompt_workspace_size(dev), dev, stream)
    q_p, ld_q = _rows(q, _BF16, dev, n, cols, "q")
    out_p, ld_out = _rows(out, _BF16, dev, n, cols, "out")
    args = _PREFILL_ARGS.pack(q_p, ld_q, n, b, cu_p, h_q, h_kv, HEAD_DIM, lens_p, kc, vc, l_max, out_p, ld_out,
                              _on(work, torch.uint8, dev, "work"), work.numel())
    _check(LIB.qspec_call(1, args, 16, handle), "qspec_attn_prefill")
    return out


def attn_prefix(q: torch.Tensor, lens: torch.Tensor, offset: int, k_cache: torch.Tensor, v_cache: torch.Tensor,
                h_q: int, prefix_k: torch.Tensor, prefix_v: torch.Tensor, prefix_len: torch.Tensor,
                cu: torch.Tensor | None = None, out: torch.Tensor | None = None, work: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Attention of a batch behind one shared prefix: bf16 [tokens][h_q * 128] -> bf16 of the same shape.

    Token t of sequence b sees prefix_len positions of prefix_k, prefix_v (bf16 [h_kv][prefix_max][128]) and
    positions 0 .. lens[b] + offset + t of its own cache.  cu None: the same number of tokens for each sequence
    (drafting and verifying passes); else packed prompts.
    """
    dev = _current_device(q)
    kc, vc, b, h_kv, l_max = _cache_on(k_cache, v_cache, dev)
    n, cols = q.shape[0], h_q * HEAD_DIM
    lens_p, cu_p = _packed_on(cu, lens, b, n, dev)
    if prefix_k.dim() != 3 or prefix_k.shape != prefix_v.shape or prefix_k.shape[0] != h_kv or prefix_k.shape[2] != HEAD_DIM:
        raise ValueError(f"prefix_k and prefix_v must both be [{h_kv}][positions][{HEAD_DIM}]")
    if out is None:
        out = _empty(stream, (n, cols), _BF16, q.device)
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if work is None:
        work = _prompt_workspace(_prompt_workspace_size(dev, n, b, h_q, h_kv), dev, stream)
    q_p, ld_q = _rows(q, _BF16, dev, n, cols, "q")
    out_p, ld_out = _rows(out, _BF16, dev, n, cols, "out")
    args = _PREFIX_ARGS.pack(q_p, ld_q, n, b, cu_p, h_q, h_kv, HEAD_DIM, lens_p, offset, kc, vc, l_max,
                             _on(prefix_k, _BF16, dev, "prefix_k"), _on(prefix_v, _BF16, dev, "prefix_v"),
                             prefix_k.shape[1], _one(prefix_len, dev), out_p, ld_out,
                             _on(work, torch.uint8, dev, "work"), work.numel())
    _check(LIB.qspec_call(2, args, 21, handle), "qspec_attn_prefix")
    return out
