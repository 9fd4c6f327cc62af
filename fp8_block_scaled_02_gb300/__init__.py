"""fp8_block_scaled_02_gb300 -- block-scaled FP8 / MXFP8 / per-row FP8 W8A16 on GB300.

A thin Python binding over the C ABI in ``include/fp8bs.h`` (``libfp8bs.so``,
built from ``csrc/`` for sm_103a).  Every function here only marshals
arguments -- device pointers, sizes and the current CUDA stream -- and calls
the library; all computation runs in the library's kernels.  There is no CPU
fallback: if the shared library has not been built, or a tensor is not on a
CUDA device, the call raises.

Functions (names follow the C entry points):
    quantize(w)            -> (codes u8 [N,K], scales f32 [ceil(N/128), ceil(K/128)])
    gemv(x, codes, scales) -> y bf16 [M,N]
    mx_quantize(w)         -> (codes u8 [N,K], e8m0 u8 [N, ceil(K/32)])
    mx_gemv(x, codes, e8m0)-> y bf16 [M,N]
    gemv_ws(x, codes, scales, workspace) -> y bf16 [M,N]        (fp8bs_gemv_ws)
    gemv_batch([(x, codes, scales[, y]), ...]) -> [y, ...]   (fp8bs_gemv_batch)
    GemvBatch(ops)() -> [y, ...]                  (fp8bs_gemv_batch, op table built once)
    mx_gemv_batch([(x, codes, e8m0[, y]), ...]) -> [y, ...]  (mxfp8_gemv_batch)
    row_quantize(w)        -> (codes u8 [N,K], scales f32 [N])       (fp8row_*)
    tensor_quantize(w)     -> (codes u8 [N,K], scale f32 [1])        (fp8tensor_*)
    row_gemv(x, codes, s)  -> y bf16 [M,N]; s is [N] (per row) or [1] (per tensor)
    act_quantize(x)        -> (x codes u8 [M,K], scale f32 [1])      (fp8act_quantize)
    w8a8_gemm(xq, sx, wq, sw) -> y bf16 [M,N]                        (w8a8_gemm)
    w8a8_linear(x, wq, sw) -> y bf16 [M,N]: act_quantize then w8a8_gemm
    moe_gemv(x, ids, codes, scales) -> y bf16 [M, topk, N]            (fp8bs_moe_gemv)
    moe_gemv_ws(x, ids, codes, scales, workspace) -> y                (fp8bs_moe_gemv_ws)
        codes [E,N,K], scales [E, ceil(N/128), ceil(K/128)], ids int32 [M, topk]
    moe_route(logits, topk) -> (ids int32 [M, topk], weights f32 [M, topk])   (fp8bs_moe_route)
    moe_combine(y, weights) -> out bf16 [M, N]: sum over topk of weights * y [M, topk, N]   (fp8bs_moe_combine)
    kv_append(x, slots, scale, cache)    FP8 KV cache append (fp8kv_append), in place
    kv_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                        max_seq_len, sm_scale) -> o bf16 [B, Hq, 128]   (fp8kv_decode_attention)
    kv_plan(ctx_lens, new_lens, block_table, free_blocks, free_head, page_size, num_blocks, num_tokens)
                           -> KvPlan: the step's cache blocks and slot map from request lengths (fp8bs_kv_plan)
    kv4_append(k, v, slots, k_scale, v_scale, k_cache, v_cache)   4-bit KV cache append, in place (fp4kv_append)
    kv4_gather(k_cache, v_cache, slots, k_scale, v_scale) -> k, v bf16 [T, Hkv, D]   (fp4kv_gather)
    kv4_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                         max_seq_len, sm_scale, workspace) -> o bf16 [T, Hq, D]   (fp4kv_decode_attention)
        4-bit caches are uint8 of kv4_cache_shape(num_blocks, page_size, kv_heads, head_dim)
    kv_rope_append(q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache) -> q bf16 [T, Hq, D]
    kv4_rope_append(...)   norm and rotation of q and k, q out, k and v into the FP8 / 4-bit cache
                           (fp8kv_rope_append, fp4kv_rope_append)
    token_logprobs(logits, targets, top) -> TokenLogprobs: log probabilities of given tokens, entropy,
                           top alternatives   (fp8bs_token_logprobs)
    sample_tokens(logits, u, temperature, top_k, top_p, min_p) -> SampledTokens: the next token of each row and
                           its log probability, from given random numbers   (fp8bs_sample_tokens)
    check_device_error()   -> the kernels' error word (synchronises; reading clears it)
    select_path(m, n, k)   -> the kernel path an AUTO call takes (host only)
    debug_wait_expiry(), debug_encode_f32(first_bits, count)   test hooks (fp8bs_debug_*)
"""
from __future__ import annotations

import collections
import ctypes
import os
import threading


class _OnFirstUse:
    """torch, imported when a call first needs it: building and the calls that
    only ask the library need none.  The module then takes this name."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _OnFirstUse()

PATH_AUTO, PATH_DECODE, PATH_PREFILL, PATH_GENERIC = 0, 1, 2, 3
PATH_NAMES = {PATH_AUTO: "auto", PATH_DECODE: "decode", PATH_PREFILL: "prefill", PATH_GENERIC: "generic"}

STATUS = {0: "FP8BS_OK", -1: "FP8BS_ERR_NULL", -2: "FP8BS_ERR_SHAPE", -3: "FP8BS_ERR_BLOCK",
          -4: "FP8BS_ERR_ALIGN", -5: "FP8BS_ERR_CUDA", -6: "FP8BS_ERR_DEVICE", -7: "FP8BS_ERR_PATH"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfp8bs.so")
_lock = threading.Lock()
_lib = None


class GemvOp(ctypes.Structure):
    """fp8bs_gemv_op: one GEMV of a batch (device pointers, sizes)."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("y_bf16", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class Fp8bsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({strerror(status)})")


def lib() -> ctypes.CDLL:
    """The loaded libfp8bs.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "or `python fp8_block_scaled_02_gb300/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        L.fp8bs_quantize.argtypes = [p, i64, i64, i32, p, p, p]
        L.fp8bs_gemv.argtypes = [p, i64, p, p, i64, i64, p, p]
        L.fp8bs_gemv_ex.argtypes = [p, i64, p, p, i64, i64, p, i32, p]
        L.fp8bs_gemv_ws_bytes.argtypes = [i64, i64]
        L.fp8bs_gemv_ws_bytes.restype = i64
        L.fp8bs_gemv_ws.argtypes = [p, i64, p, p, i64, i64, p, p, i64, p]
        L.fp8bs_gemv_batch.argtypes = [p, i64, i64, p]
        L.fp8bs_gemv_batch_ex.argtypes = [p, i64, i64, i32, p]
        L.mxfp8_gemv_batch.argtypes = [p, i64, i64, p]
        L.mxfp8_gemv_batch_ex.argtypes = [p, i64, i64, i32, p]
        L.mxfp8_quantize.argtypes = [p, i64, i64, p, p, p]
        L.mxfp8_gemv.argtypes = [p, i64, p, p, i64, i64, p, p]
        L.mxfp8_gemv_ex.argtypes = [p, i64, p, p, i64, i64, p, i32, p]
        L.fp8row_quantize.argtypes = [p, i64, i64, p, p, p]
        L.fp8tensor_quantize.argtypes = [p, i64, i64, p, p, p]
        L.fp8row_gemv.argtypes = [p, i64, p, p, i64, i64, p, p]
        L.fp8row_gemv_ex.argtypes = [p, i64, p, p, i64, i64, p, i32, p]
        L.fp8tensor_gemv.argtypes = [p, i64, p, p, i64, i64, p, p]
        L.fp8tensor_gemv_ex.argtypes = [p, i64, p, p, i64, i64, p, i32, p]
        L.fp8act_quantize.argtypes = [p, i64, i64, p, p, p]
        L.fp8bs_moe_gemv.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, p, p]
        L.fp8bs_moe_gemv_ws.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, p, p, i64, p]
        L.fp8bs_moe_gemv_ws_bytes.argtypes = [i64, i64, i64, i64]
        L.fp8bs_moe_gemv_ws_bytes.restype = i64
        L.fp8kv_append.argtypes = [p, i64, i64, i64, p, p, p, i64, p]
        L.fp8kv_decode_attention.argtypes = [p, p, p, p, p, p, i64, p, i64, i64, i64, i64, i64, i64, i64,
                                             ctypes.c_float, p, p]
        L.fp8bs_kv_plan.argtypes = [p, p, i64, p, i64, p, i64, p, i64, i64, i64, p, p, p, p, p, p, p]
        L.fp4kv_append.argtypes = [p, i64, p, i64, i64, i64, i64, p, p, p, p, p, i64, i64, p]
        L.fp4kv_gather.argtypes = [p, p, p, i64, i64, i64, i64, i64, p, p, p, p, p]
        L.fp4kv_attention_ws_bytes.argtypes = [i64]
        L.fp4kv_attention_ws_bytes.restype = i64
        L.fp4kv_decode_attention.argtypes = [p, i64, p, i64, i64, p, p, p, p, p, i64, p, i64, i64, i64, i64, i64, i64,
                                             i64, i64, ctypes.c_float, p, p, p, i64, p]
        rope = [p, i64, p, i64, p, i64, i64, i64, i64, i64, p, p, p, i64, i64, i32, p, p, ctypes.c_float, p, p, p, p, p]
        L.fp8kv_rope_append.argtypes = rope + [i64, p]
        L.fp4kv_rope_append.argtypes = rope + [i64, i64, p]
        L.fp8bs_moe_route.argtypes = [p, i32, i64, i64, i64, i64, i32, p, i64, i64, i64, i32, ctypes.c_float, p, p, p]
        L.fp8bs_moe_combine.argtypes = [p, p, p, i64, p, i64, i64, i64, p, p]
        L.fp8bs_token_logprobs.argtypes = [p, i32, i64, i64, i64, p, i64, p, p, p, p, p]
        L.fp8bs_sample_tokens.argtypes = [p, i32, i64, i64, i64, p, p, p, p, p, p, p, p]
        L.w8a8_gemm.argtypes = [p, i64, p, p, p, i64, i64, p, p]
        L.w8a8_gemm_ex.argtypes = [p, i64, p, p, p, i64, i64, p, i32, p]
        L.fp8bs_select_path.argtypes = [i64, i64, i64, p, p, i32]
        L.fp8bs_strerror.argtypes = [i32]
        L.fp8bs_strerror.restype = ctypes.c_char_p
        L.fp8bs_check_device_error.argtypes = [p, ctypes.POINTER(ctypes.c_uint32)]
        L.fp8bs_debug_wait_expiry.argtypes = [p]
        L.fp8bs_debug_encode_f32.argtypes = [ctypes.c_uint32, i64, p, p]
        L.fp8bs_version.argtypes = []
        for f in ("fp8bs_quantize", "fp8bs_gemv", "fp8bs_gemv_ex", "fp8bs_gemv_ws", "fp8bs_gemv_batch",
                  "fp8bs_gemv_batch_ex",
                  "mxfp8_gemv_batch", "mxfp8_gemv_batch_ex", "mxfp8_quantize", "mxfp8_gemv",
                  "mxfp8_gemv_ex", "fp8row_quantize", "fp8tensor_quantize", "fp8row_gemv", "fp8row_gemv_ex",
                  "fp8tensor_gemv", "fp8tensor_gemv_ex", "fp8act_quantize", "w8a8_gemm", "w8a8_gemm_ex",
                  "fp8bs_moe_gemv", "fp8bs_moe_gemv_ws", "fp8kv_append", "fp8kv_decode_attention",
                  "fp8bs_kv_plan", "fp4kv_append", "fp4kv_gather", "fp4kv_decode_attention", "fp8bs_token_logprobs",
                  "fp8kv_rope_append", "fp4kv_rope_append", "fp8bs_moe_route", "fp8bs_moe_combine",
                  "fp8bs_sample_tokens",
                  "fp8bs_select_path", "fp8bs_check_device_error", "fp8bs_debug_wait_expiry",
                  "fp8bs_debug_encode_f32", "fp8bs_version"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
        return L


def strerror(status: int) -> str:
    try:
        return lib().fp8bs_strerror(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(status: int, what: str):
    if status != 0:
        raise Fp8bsError(status, what)


def _stream(stream, device=None):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def cdiv(a: int, b: int) -> int:
    return (a + b - 1) // b


class _Args:
    """Checks one call's tensors before anything is launched.

    ``need(name, t, dtype, numel=..., shape=...)`` records a tensor; sizes
    are checked first (ValueError, for any device), then that every tensor
    sits on the device of the first one (ValueError), then CUDA, dtype and
    contiguity (TypeError / ValueError; with ``rows`` only the dimensions
    after the first have to be contiguous).  ``ptr(name)`` gives the device
    address once ``check()`` has passed; ``device`` is where the call runs."""

    def __init__(self):
        self.items = []

    def need(self, name, t, dtype, numel=None, shape=None, rows=False):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if shape is not None and t.shape != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
        self.items.append((name, t, dtype, rows))
        return self

    def check(self):
        first = self.items[0][1].device
        good = first.type == "cuda"
        for _, t, dtype, _ in self.items:
            if t.device != first or t.dtype != dtype or not t.is_contiguous():
                good = False
                break
        if not good:
            self._refuse(first)
        self.device = first
        self.ptrs = {name: t.data_ptr() for name, t, _, _ in self.items}
        return self

    def _refuse(self, first):
        """Raise for the first tensor that does not fit (none may: rows)."""
        for name, t, _, _ in self.items:
            if t.device != first:
                raise ValueError(f"{name} is on {t.device}, the call's tensors on {first}")
        for name, t, dtype, rows in self.items:
            if t.device.type != "cuda":
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if not (t.is_contiguous() or (rows and t.numel() and t[0].is_contiguous())):
                raise ValueError(f"{name} must be contiguous" + (" in all but its first dimension" if rows else ""))

    def ptr(self, name):
        return self.ptrs[name]


def _rows_contiguous(t):
    """Whether every t[i] is contiguous."""
    if t.dim() == 3:
        (_, h, d), (_, by_head, by_element) = t.shape, t.stride()
        return (by_element == 1 or d == 1) and (by_head == d or h == 1)
    n = 1
    for size, stride in zip(t.shape[:0:-1], t.stride()[:0:-1]):
        if size != 1 and stride != n:
            return False
        n *= size
    return True


def _checked(*specs):
    """_Args' checks of (name, tensor, dtype, numel or shape or None, rows) in
    one quick pass; raises what _Args raises.  Returns the call's device."""
    try:
        first = specs[0][1]
        index = first.get_device()  # -1: not a GPU
        if index >= 0:
            for _, t, dtype, numel, rows in specs:
                if (t.dtype is not dtype or t.get_device() != index
                        or (numel is not None and (t.shape if numel.__class__ is tuple else t.numel()) != numel)
                        or not (t.is_contiguous() or (rows and _rows_contiguous(t)))):
                    break
            else:
                return first.device
    except (AttributeError, RuntimeError):  # not a tensor, or of a kind that is on no device
        pass
    a = _Args()
    for name, t, dtype, numel, rows in specs:
        a.need(name, t, dtype, **{"shape" if isinstance(numel, tuple) else "numel": numel}, rows=rows)
    return a.check().device


def _raw_stream(stream, device):
    """The cudaStream_t a call on `device` runs on."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _call(device, what, fn, call_args, stream=None):
    """fn(*call_args, stream) with `device` current."""
    raw = _raw_stream(stream, device)
    if torch.cuda.current_device() == device.index:
        status = fn(*call_args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*call_args, raw)
    if status != 0:
        _check(status, what)


def _run(args: _Args, what: str, fn, *call_args, stream=None):
    """Call the library on the device of the call's tensors, on that
    device's current stream unless one is given."""
    _call(args.device, what, fn, call_args, stream)


def _shape2(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    return t.shape


def _new(t, shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device) if t is None else t


def quantize(w, block: int = 128, codes=None, scales=None, stream=None):
    """Block-FP8 load-time quantization of a bf16 [N, K] CUDA tensor."""
    n, k = _shape2(w, "w")
    codes = _new(codes, (n, k), torch.uint8, w)
    scales = _new(scales, (cdiv(n, 128), cdiv(k, 128)), torch.float32, w)
    a = _Args().need("w", w, torch.bfloat16).need("codes", codes, torch.uint8, numel=n * k) \
        .need("scales", scales, torch.float32, numel=cdiv(n, 128) * cdiv(k, 128)).check()
    _run(a, "fp8bs_quantize", lib().fp8bs_quantize, a.ptr("w"), n, k, int(block), a.ptr("codes"), a.ptr("scales"),
         stream=stream)
    return codes, scales


def _gemv_args(x, codes, y, scales, sdtype, snumel, check=True):
    m, k = _shape2(x, "x")
    n, k2 = _shape2(codes, "codes")
    if k2 != k:
        raise ValueError("codes and x disagree on K")
    y = _new(y, (m, n), torch.bfloat16, x)
    a = _Args().need("x", x, torch.bfloat16).need("codes", codes, torch.uint8) \
        .need("scales", scales, sdtype, numel=snumel(n, k)).need("y", y, torch.bfloat16, numel=m * n)
    return (a.check() if check else a), m, n, k, y


def _block_numel(n, k):
    return cdiv(n, 128) * cdiv(k, 128)


def gemv(x, codes, scales, y=None, path: int = PATH_AUTO, stream=None):
    """y[M, N] = x[M, K] . dequant(codes, scales)^T (bf16 out, fp32 accumulate)."""
    a, m, n, k, y = _gemv_args(x, codes, y, scales, torch.float32, _block_numel)
    _run(a, "fp8bs_gemv", lib().fp8bs_gemv_ex, a.ptr("x"), m, a.ptr("codes"), a.ptr("scales"), n, k, a.ptr("y"),
         int(path), stream=stream)
    return y


def gemv_ws_bytes(m: int, k: int) -> int:
    """Bytes of device workspace gemv_ws needs (fp8bs_gemv_ws_bytes)."""
    v = lib().fp8bs_gemv_ws_bytes(m, k)
    if v < 0:
        raise Fp8bsError(int(v), "fp8bs_gemv_ws_bytes")
    return int(v)


def gemv_ws(x, codes, scales, workspace, y=None, stream=None):
    """gemv with caller-provided device scratch (fp8bs_gemv_ws): x is
    converted once per call to f16 in `workspace` (a uint8 CUDA tensor of at
    least gemv_ws_bytes(M, K) bytes) and the decode kernel reads that copy."""
    a, m, n, k, y = _gemv_args(x, codes, y, scales, torch.float32, _block_numel, check=False)
    a.need("workspace", workspace, torch.uint8).check()
    _run(a, "fp8bs_gemv_ws", lib().fp8bs_gemv_ws, a.ptr("x"), m, a.ptr("codes"), a.ptr("scales"), n, k, a.ptr("y"),
         a.ptr("workspace"), workspace.numel(), stream=stream)
    return y


def _batch_ops(ops, mx):
    arr = (GemvOp * max(1, len(ops)))()
    if not ops:
        return arr, 0, [], None
    m = _shape2(ops[0][0], "x")[0]
    sdtype = torch.uint8 if mx else torch.float32
    snumel = (lambda n, k: n * cdiv(k, 32)) if mx else _block_numel
    # every op's sizes first (nothing about devices), then devices and dtypes
    for i, op in enumerate(ops):
        if _shape2(op[0], f"op {i} x")[0] != m:
            raise ValueError("every op of a batch has the same M")
        if len(op) > 3 and op[3] is not None:
            _gemv_args(op[0], op[1], op[3], op[2], sdtype, snumel, check=False)
        else:
            n = _shape2(op[1], f"op {i} codes")[0]
            _Args().need("scales", op[2], sdtype, numel=snumel(n, op[0].shape[1]))
    first = ops[0][0].device
    for i, op in enumerate(ops):
        for name, tt in zip(("x", "codes", "scales", "y"), op):
            if tt is not None and tt.device != first:
                raise ValueError(f"op {i} {name} is on {tt.device}, the batch on {first}")
    ys = []
    device = None
    for i, op in enumerate(ops):
        y = op[3] if len(op) > 3 else None
        a, _, n, k, y = _gemv_args(op[0], op[1], y, op[2], sdtype, snumel)
        if device is None:
            device = a.device
        elif a.device != device:
            raise ValueError(f"op {i} is on {a.device}, the batch on {device}")
        ys.append(y)
        arr[i] = GemvOp(a.ptr("x"), a.ptr("codes"), a.ptr("scales"), a.ptr("y"), n, k)
    return arr, m, ys, device


def _run_batch(fn, what, ops, mx, path, stream):
    arr, m, ys, device = _batch_ops(ops, mx)
    if not ops:
        return ys
    with torch.cuda.device(device):
        _check(fn(ctypes.cast(arr, ctypes.c_void_p), len(ops), m, int(path), _stream(stream, device)), what)
    return ys


def gemv_batch(ops, path: int = PATH_AUTO, stream=None):
    """A sequence of block-FP8 GEMVs (fp8bs_gemv_batch): ops is a list of
    (x [M,K], codes, scales[, y]) with one M; returns the list of y.  Same
    results as calling gemv on each op in order."""
    return _run_batch(lib().fp8bs_gemv_batch_ex, "fp8bs_gemv_batch", ops, False, path, stream)


class GemvBatch:
    """A prepared sequence of block-FP8 GEMVs (fp8bs_gemv_batch): the op
    table is built once, so calling it only enqueues the launches.  ops as
    for gemv_batch."""

    def __init__(self, ops, path: int = PATH_AUTO):
        self.arr, self.m, self.ys, self.device = _batch_ops(ops, False)
        self.count = len(ops)
        self.path = path
        self.ops = ops  # keeps the tensors alive

    def __call__(self, stream=None):
        if not self.count:
            return self.ys
        with torch.cuda.device(self.device):
            _check(lib().fp8bs_gemv_batch_ex(ctypes.cast(self.arr, ctypes.c_void_p), self.count, self.m,
                                             int(self.path), _stream(stream, self.device)), "fp8bs_gemv_batch")
        return self.ys


def mx_gemv_batch(ops, path: int = PATH_AUTO, stream=None):
    """A sequence of MXFP8 GEMVs (mxfp8_gemv_batch): ops is a list of
    (x [M,K], codes, e8m0[, y]) with one M; returns the list of y."""
    return _run_batch(lib().mxfp8_gemv_batch_ex, "mxfp8_gemv_batch", ops, True, path, stream)


def mx_quantize(w, codes=None, e8m0=None, stream=None):
    """MXFP8 load-time quantization of a bf16 [N, K] CUDA tensor."""
    n, k = _shape2(w, "w")
    codes = _new(codes, (n, k), torch.uint8, w)
    e8m0 = _new(e8m0, (n, cdiv(k, 32)), torch.uint8, w)
    a = _Args().need("w", w, torch.bfloat16).need("codes", codes, torch.uint8, numel=n * k) \
        .need("e8m0", e8m0, torch.uint8, numel=n * cdiv(k, 32)).check()
    _run(a, "mxfp8_quantize", lib().mxfp8_quantize, a.ptr("w"), n, k, a.ptr("codes"), a.ptr("e8m0"), stream=stream)
    return codes, e8m0


def mx_gemv(x, codes, e8m0, y=None, path: int = PATH_AUTO, stream=None):
    """y[M, N] = x[M, K] . dequant_mx(codes, e8m0)^T."""
    a, m, n, k, y = _gemv_args(x, codes, y, e8m0, torch.uint8, lambda n, k: n * cdiv(k, 32))
    _run(a, "mxfp8_gemv", lib().mxfp8_gemv_ex, a.ptr("x"), m, a.ptr("codes"), a.ptr("scales"), n, k, a.ptr("y"),
         int(path), stream=stream)
    return y


def _rowwise_quantize(fn, what, w, codes, scales, count, stream):
    n, k = _shape2(w, "w")
    codes = _new(codes, (n, k), torch.uint8, w)
    scales = _new(scales, (count(n),), torch.float32, w)
    a = _Args().need("w", w, torch.bfloat16).need("codes", codes, torch.uint8, numel=n * k) \
        .need("scales", scales, torch.float32, numel=count(n)).check()
    _run(a, what, fn, a.ptr("w"), n, k, a.ptr("codes"), a.ptr("scales"), stream=stream)
    return codes, scales


def row_quantize(w, codes=None, scales=None, stream=None):
    """Per-row FP8 load-time quantization: one fp32 scale per row of w."""
    return _rowwise_quantize(lib().fp8row_quantize, "fp8row_quantize", w, codes, scales, lambda n: n, stream)


def tensor_quantize(w, codes=None, scale=None, stream=None):
    """Per-tensor FP8 load-time quantization: one fp32 scale for all of w."""
    return _rowwise_quantize(lib().fp8tensor_quantize, "fp8tensor_quantize", w, codes, scale, lambda n: 1, stream)


def row_gemv(x, codes, scales, y=None, path: int = PATH_AUTO, stream=None):
    """y[M, N] = x[M, K] . (dec(codes) * s_row)^T.  ``scales`` of shape [N]
    calls fp8row_gemv, of shape [1] fp8tensor_gemv."""
    n = _shape2(codes, "codes")[0]
    per_row = tuple(scales.shape) == (n,) and n > 1
    if not per_row and tuple(scales.shape) not in ((1,), ()):
        raise ValueError("scales must have shape [N] (per row) or [1] (per tensor)")
    a, m, n, k, y = _gemv_args(x, codes, y, scales, torch.float32, lambda n, k: n if per_row else 1)
    fn = lib().fp8row_gemv_ex if per_row else lib().fp8tensor_gemv_ex
    _run(a, "fp8row_gemv" if per_row else "fp8tensor_gemv", fn, a.ptr("x"), m, a.ptr("codes"), a.ptr("scales"), n,
         k, a.ptr("y"), int(path), stream=stream)
    return y


def _moe_args(x, ids, codes, scales, y):
    m, k = _shape2(x, "x")
    if codes.dim() != 3:
        raise ValueError("codes must be [E, N, K]")
    e, n, k2 = codes.shape
    topk = _shape2(ids, "ids")[1]
    if k2 != k or ids.shape[0] != m:
        raise ValueError("x, ids and codes disagree on M or K")
    y = _new(y, (m, topk, n), torch.bfloat16, x)
    a = _Args().need("x", x, torch.bfloat16).need("ids", ids, torch.int32) \
        .need("codes", codes, torch.uint8) \
        .need("scales", scales, torch.float32, numel=e * cdiv(n, 128) * cdiv(k, 128)) \
        .need("y", y, torch.bfloat16, numel=m * topk * n)
    return a, m, topk, e, n, k, y


def moe_gemv(x, ids, codes, scales, y=None, stream=None):
    """Grouped block-FP8 GEMV over routed experts: y[t, j] = x[t] . dequant(W[ids[t, j]])^T."""
    a, m, topk, e, n, k, y = _moe_args(x, ids, codes, scales, y)
    a.check()
    _run(a, "fp8bs_moe_gemv", lib().fp8bs_moe_gemv, a.ptr("x"), m, a.ptr("ids"), topk, a.ptr("codes"),
         a.ptr("scales"), e, n, k, a.ptr("y"), stream=stream)
    return y


def moe_gemv_ws_bytes(m: int, topk: int, num_experts: int, k: int) -> int:
    """Bytes of device workspace moe_gemv_ws needs (fp8bs_moe_gemv_ws_bytes)."""
    v = lib().fp8bs_moe_gemv_ws_bytes(m, topk, num_experts, k)
    if v < 0:
        raise Fp8bsError(int(v), "fp8bs_moe_gemv_ws_bytes")
    return int(v)


def moe_gemv_ws(x, ids, codes, scales, workspace, y=None, stream=None):
    """moe_gemv with caller-provided device scratch (fp8bs_moe_gemv_ws): more
    than 32 tokens run as one grouped tensor-core GEMM over the routed
    experts; `workspace` is a uint8 CUDA tensor of at least
    moe_gemv_ws_bytes(M, topk, E, K) bytes."""
    a, m, topk, e, n, k, y = _moe_args(x, ids, codes, scales, y)
    a.need("workspace", workspace, torch.uint8).check()
    _run(a, "fp8bs_moe_gemv_ws", lib().fp8bs_moe_gemv_ws, a.ptr("x"), m, a.ptr("ids"), topk, a.ptr("codes"),
         a.ptr("scales"), e, n, k, a.ptr("y"), a.ptr("workspace"), workspace.numel(), stream=stream)
    return y


def kv_append(x, slots, scale, cache, stream=None):
    """Quantize new keys or values x [T, Hkv, 128] bf16 into the e4m3 cache
    [num_blocks, page_size, Hkv, 128] at flat token slots (in place)."""
    if x.dim() != 3 or cache.dim() != 4:
        raise ValueError("x must be [T, Hkv, 128] and cache [num_blocks, page_size, Hkv, 128]")
    t, hkv, d = x.shape
    nb, page, hkv2, d2 = cache.shape
    if (hkv2, d2) != (hkv, d):
        raise ValueError("x and cache disagree on kv heads or head_dim")
    a = _Args().need("x", x, torch.bfloat16).need("slots", slots, torch.int32, numel=t) \
        .need("scale", scale, torch.float32, numel=1).need("cache", cache, torch.uint8).check()
    _run(a, "fp8kv_append", lib().fp8kv_append, a.ptr("x"), t, hkv, d, a.ptr("slots"), a.ptr("scale"),
         a.ptr("cache"), nb * page, stream=stream)
    return cache


def kv_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_seq_len: int,
                        sm_scale: float, out=None, stream=None):
    """Paged decode attention over the FP8 KV cache: q [B, Hq, 128] bf16."""
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, 128] and the caches [num_blocks, page_size, Hkv, 128]")
    b, hq, d = q.shape
    nb, page, hkv, d2 = k_cache.shape
    bt_rows, max_blocks = _shape2(block_table, "block_table")
    if d2 != d or tuple(v_cache.shape) != tuple(k_cache.shape) or bt_rows != b:
        raise ValueError("q, caches and block table disagree")
    out = _new(out, (b, hq, d), torch.bfloat16, q)
    a = _Args().need("q", q, torch.bfloat16).need("k_cache", k_cache, torch.uint8) \
        .need("v_cache", v_cache, torch.uint8).need("k_scale", k_scale, torch.float32, numel=1) \
        .need("v_scale", v_scale, torch.float32, numel=1).need("block_table", block_table, torch.int32) \
        .need("seq_lens", seq_lens, torch.int32, numel=b).need("out", out, torch.bfloat16, numel=b * hq * d).check()
    _run(a, "fp8kv_decode_attention", lib().fp8kv_decode_attention, a.ptr("q"), a.ptr("k_cache"),
         a.ptr("v_cache"), a.ptr("k_scale"), a.ptr("v_scale"), a.ptr("block_table"), max_blocks,
         a.ptr("seq_lens"), b, hq, hkv, d, page, nb, int(max_seq_len), float(sm_scale), a.ptr("out"), stream=stream)
    return out


_SCORING = {"softmax": 0, "sigmoid": 1}


def moe_route(logits, topk: int, scoring: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """The experts of each token and their weights from the router's logits
    [M, E], bf16 or fp32 (fp8bs_moe_route): the topk of softmax or sigmoid
    scores plus `bias` [E] fp32, in the topk_groups best of `groups` groups,
    each scored by its group_top best experts.  Returns ids int32 [M, topk]
    (what moe_gemv takes) and weights fp32 [M, topk] (what moe_combine takes)."""
    m, e = _shape2(logits, "logits")
    topk = int(topk)
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    if not 1 <= topk <= e:
        raise ValueError(f"topk is {topk}, the experts are {e}")
    stride = logits.stride(0) if m > 1 else e
    if 0 < stride < e:
        raise ValueError(f"the rows of logits overlap: they are {stride} elements apart and {e} long")
    i32, f32 = torch.int32, torch.float32
    is_f32 = logits.dtype == f32
    specs = [("logits", logits, f32 if is_f32 else torch.bfloat16, None, True)]
    if bias is not None:
        specs.append(("bias", bias, f32, e, False))
    if ids is not None:
        specs.append(("ids", ids, i32, (m, topk), False))
    if weights is not None:
        specs.append(("weights", weights, f32, (m, topk), False))
    device = _checked(*specs)
    if ids is None:
        ids = _empty(stream, device, (m, topk), i32)
    if weights is None:
        weights = _empty(stream, device, (m, topk), f32)
    _call(device, "fp8bs_moe_route", lib().fp8bs_moe_route,
          (logits.data_ptr(), int(is_f32), stride, m, e, topk, _SCORING[scoring],
           bias.data_ptr() if bias is not None else None, int(groups), int(topk_groups), int(group_top),
           int(bool(renormalize)), float(scale), ids.data_ptr(), weights.data_ptr()), stream)
    return ids, weights


def moe_combine(y, weights, ids=None, num_experts: int = 0, residual=None, out=None, stream=None):
    """The weighted sum of the experts' outputs y [M, topk, N] bf16
    (fp8bs_moe_combine): out [M, N] bf16 = residual + sum_j weights[:, j] y[:, j].
    With ids (int32 [M, topk]) and num_experts a slot whose id is outside
    [0, num_experts) adds nothing.  out may be residual."""
    if y.dim() != 3:
        raise ValueError("y must be [M, topk, N]")
    m, topk, n = y.shape
    if ids is not None and num_experts < 1:
        raise ValueError("ids need num_experts: a slot whose id is outside [0, num_experts) adds nothing")
    bf16 = torch.bfloat16
    specs = [("y", y, bf16, None, False), ("weights", weights, torch.float32, (m, topk), False)]
    if ids is not None:
        specs.append(("ids", ids, torch.int32, (m, topk), False))
    if residual is not None:
        specs.append(("residual", residual, bf16, (m, n), False))
    if out is not None:
        specs.append(("out", out, bf16, (m, n), False))
    device = _checked(*specs)
    if out is None:
        out = _empty(stream, device, (m, n), bf16)
    _call(device, "fp8bs_moe_combine", lib().fp8bs_moe_combine,
          (y.data_ptr(), weights.data_ptr(), ids.data_ptr() if ids is not None else None, int(num_experts),
           residual.data_ptr() if residual is not None else None, m, topk, n, out.data_ptr()), stream)
    return out


KvPlan = collections.namedtuple("KvPlan", "seq_lens cu_new slots positions requests free_head")
TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprobs entropy top_ids top_logprobs")


def _empty(stream, device, shape, dtype):
    """A call's own output: in the memory pool of the stream the call runs on,
    so that its memory is not handed out again while it runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_stride(t):
    """Elements from one row of the first dimension to the next."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1:].numel() if t.shape[0] else 0


def kv_plan(ctx_lens, new_lens, block_table, free_blocks, free_head, page_size: int, num_blocks: int,
            num_tokens: int, seq_lens=None, cu_new=None, slots=None, positions=None, requests=None,
            free_head_out=None, stream=None):
    """The paging plan of one step from request lengths (fp8bs_kv_plan): new
    blocks of each request from the free list (written into block_table),
    the slot, position and request of each of the step's num_tokens tokens
    (-1 past the last and where a request is refused).  Returns a KvPlan;
    seq_lens may be ctx_lens and free_head_out may be free_head."""
    b = ctx_lens.numel()
    rows, max_blocks = _shape2(block_table, "block_table")
    if rows != b:
        raise ValueError("block_table and ctx_lens disagree on the number of requests")
    num_tokens = int(num_tokens)
    if num_tokens < 0:
        raise ValueError("num_tokens must not be negative")
    i32 = torch.int32
    outs = (slots, positions, requests, seq_lens, cu_new, free_head_out)
    sizes = (num_tokens, num_tokens, num_tokens, b, b + 1, 1)
    given = ()
    if any(t is not None for t in outs):
        given = [(name, t, i32, n, False) for name, t, n in
                 zip(("slots", "positions", "requests", "seq_lens", "cu_new", "free_head_out"), outs, sizes)
                 if t is not None]
    device = _checked(("ctx_lens", ctx_lens, i32, None, False), ("new_lens", new_lens, i32, b, False),
                      ("block_table", block_table, i32, None, False), ("free_blocks", free_blocks, i32, None, False),
                      ("free_head", free_head, i32, 1, False), *given)
    # one allocation holds every output the caller did not give
    if given:
        sizes = [n if t is None else 0 for t, n in zip(outs, sizes)]
    own = torch.split_with_sizes(_empty(stream, device, (sum(sizes),), i32), sizes)
    if given:
        own = [o if t is None else t for t, o in zip(outs, own)]
    slots, positions, requests, seq_lens, cu_new, free_head_out = own
    _call(device, "fp8bs_kv_plan", lib().fp8bs_kv_plan,
          (ctx_lens.data_ptr(), new_lens.data_ptr(), b, block_table.data_ptr(), max_blocks, free_blocks.data_ptr(),
           free_blocks.numel(), free_head.data_ptr(), int(page_size), int(num_blocks), num_tokens, seq_lens.data_ptr(),
           cu_new.data_ptr(), slots.data_ptr(), positions.data_ptr(), requests.data_ptr(), free_head_out.data_ptr()),
          stream)
    return KvPlan(seq_lens, cu_new, slots, positions, requests, free_head_out)


def kv4_cache_shape(num_blocks: int, page_size: int, num_kv_heads: int, head_dim: int):
    """Shape of one 4-bit cache (K or V), uint8: tiles of 16 tokens of one kv head."""
    if page_size % 16 != 0:
        raise ValueError("page_size must be a multiple of 16")
    return num_blocks, num_kv_heads, page_size // 16, 9 * head_dim


def _kv4_specs(k_cache, v_cache, k_scale, v_scale, hkv, d):
    """What _checked has to see of a pair of 4-bit caches and their scales, num_blocks and page_size."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] != hkv or shape[3] != 9 * d:
        raise ValueError(f"k_cache has shape {tuple(shape)}, expected [num_blocks, {hkv}, page_size / 16, {9 * d}]")
    if v_cache.shape != shape:
        raise ValueError(f"v_cache has shape {tuple(v_cache.shape)}, expected {tuple(shape)}")
    u8, f32 = torch.uint8, torch.float32
    return (("k_cache", k_cache, u8, None, False), ("v_cache", v_cache, u8, None, False),
            ("k_scale", k_scale, f32, 1, False), ("v_scale", v_scale, f32, 1, False)), shape[0], shape[2] * 16


def kv4_append(k, v, slots, k_scale, v_scale, k_cache, v_cache, stream=None):
    """Quantize new keys and values [T, Hkv, D] bf16 into 4-bit caches at flat
    token slots, in place (fp4kv_append).  k and v may be slices of a fused
    projection: only the rows of one token have to be contiguous."""
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, D]")
    t, hkv, d = k.shape
    specs, nb, page = _kv4_specs(k_cache, v_cache, k_scale, v_scale, hkv, d)
    device = _checked(*specs, ("slots", slots, torch.int32, t, False), ("k", k, torch.bfloat16, None, True),
                      ("v", v, torch.bfloat16, None, True))
    _call(device, "fp4kv_append", lib().fp4kv_append,
          (k.data_ptr(), _row_stride(k), v.data_ptr(), _row_stride(v), t, hkv, d, slots.data_ptr(),
           k_scale.data_ptr(), v_scale.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page, nb), stream)
    return k_cache, v_cache


def kv4_gather(k_cache, v_cache, slots, k_scale, v_scale, k=None, v=None, stream=None):
    """The cached tokens at flat slots in bf16 [T, Hkv, D] (fp4kv_gather)."""
    if k_cache.dim() != 4 or k_cache.shape[3] % 9 != 0:
        raise ValueError("k_cache must be [num_blocks, Hkv, page_size / 16, 9 * D]")
    t, hkv, d = slots.numel(), k_cache.shape[1], k_cache.shape[3] // 9
    specs, nb, page = _kv4_specs(k_cache, v_cache, k_scale, v_scale, hkv, d)
    given = [(name, x, torch.bfloat16, t * hkv * d, False) for name, x in (("k", k), ("v", v)) if x is not None]
    device = _checked(*specs, ("slots", slots, torch.int32, None, False), *given)
    k = _empty(stream, device, (t, hkv, d), torch.bfloat16) if k is None else k
    v = _empty(stream, device, (t, hkv, d), torch.bfloat16) if v is None else v
    _call(device, "fp4kv_gather", lib().fp4kv_gather,
          (k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr(), t, hkv, d, page, nb, k_scale.data_ptr(),
           v_scale.data_ptr(), k.data_ptr(), v.data_ptr()), stream)
    return k, v


def kv4_workspace_bytes(head_dim: int) -> int:
    """Bytes of device workspace kv4_decode_attention needs (fp4kv_attention_ws_bytes)."""
    v = lib().fp4kv_attention_ws_bytes(head_dim)
    if v < 0:
        raise Fp8bsError(int(v), "fp4kv_attention_ws_bytes")
    return int(v)


def kv4_workspace(head_dim: int, device="cuda"):
    """A workspace for kv4_decode_attention (zeroed once, here): one serves
    every shape of a head size, but only one call at a time."""
    return torch.zeros(kv4_workspace_bytes(head_dim), dtype=torch.uint8, device=device)


def kv4_decode_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_seq_len: int,
                         sm_scale: float, workspace, cu_q=None, max_q: int = 1, window: int = 0, out=None, lse=None,
                         return_lse: bool = False, stream=None):
    """Attention of the newest tokens of each sequence over its 4-bit cache
    (fp4kv_decode_attention): q [T, Hq, D] bf16 (a slice of a fused projection
    will do), one token per sequence, or sequence b's tokens cu_q[b] ..
    cu_q[b + 1] - 1, at most max_q.  Returns o [T, Hq, D], with return_lse
    (o, lse [T, Hq] fp32)."""
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    t, hq, d = q.shape
    b = seq_lens.numel()
    bt_rows, max_blocks = _shape2(block_table, "block_table")
    if bt_rows != b or (cu_q is None and t != b):
        raise ValueError("q, block_table and seq_lens disagree on the number of sequences")
    hkv = k_cache.shape[1] if k_cache.dim() == 4 else 0
    specs, nb, page = _kv4_specs(k_cache, v_cache, k_scale, v_scale, hkv, d)
    given = [spec for spec in (("cu_q", cu_q, torch.int32, b + 1, False), ("out", out, torch.bfloat16, t * hq * d, False),
                               ("lse", lse, torch.float32, t * hq, False)) if spec[1] is not None]
    device = _checked(*specs, ("block_table", block_table, torch.int32, None, False),
                      ("seq_lens", seq_lens, torch.int32, None, False), ("workspace", workspace, torch.uint8, None, False),
                      *given, ("q", q, torch.bfloat16, None, True))
    if out is None:
        out = _empty(stream, device, (t, hq, d), torch.bfloat16)
    if lse is None and return_lse:
        lse = _empty(stream, device, (t, hq), torch.float32)
    _call(device, "fp4kv_decode_attention", lib().fp4kv_decode_attention,
          (q.data_ptr(), _row_stride(q), cu_q.data_ptr() if cu_q is not None else None, t, int(max_q), k_cache.data_ptr(),
           v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), max_blocks,
           seq_lens.data_ptr(), b, hq, hkv, d, page, nb, int(max_seq_len), int(window), float(sm_scale), out.data_ptr(),
           lse.data_ptr() if lse is not None else None, workspace.data_ptr(), workspace.numel()), stream)
    return (out, lse) if return_lse else out


def _rope_append(four_bit, q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache, q_norm, k_norm, eps,
                 interleaved, out, stream):
    try:
        (t, hq, d), (tk, hkv, dk) = q.shape, k.shape
    except ValueError:
        t, tk = -1, -2
    if t != tk or d != dk or v.shape != k.shape:
        raise ValueError("q must be [T, Hq, D], k and v [T, Hkv, D]")
    max_pos, rot = _shape2(cos_sin, "cos_sin")
    bf16, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    L = lib()
    if four_bit:
        caches, nb, page = _kv4_specs(k_cache, v_cache, k_scale, v_scale, hkv, d)
        what, fn, places = "fp4kv_rope_append", L.fp4kv_rope_append, (page, nb)
    else:
        shape = k_cache.shape
        if len(shape) != 4 or shape[2] != hkv or shape[3] != d:
            raise ValueError(f"k_cache has shape {tuple(shape)}, expected [num_blocks, page_size, Hkv, D] of k")
        if v_cache.shape != shape:
            raise ValueError(f"v_cache has shape {tuple(v_cache.shape)}, expected {tuple(shape)}")
        caches = (("k_cache", k_cache, u8, None, False), ("v_cache", v_cache, u8, None, False),
                  ("k_scale", k_scale, f32, 1, False), ("v_scale", v_scale, f32, 1, False))
        what, fn, places = "fp8kv_rope_append", L.fp8kv_rope_append, (shape[0] * shape[1],)
    given = ()
    if q_norm is not None:
        given = (("q_norm", q_norm, bf16, d, False),)
    if k_norm is not None:
        given += (("k_norm", k_norm, bf16, d, False),)
    if out is not None:
        given += (("out", out, bf16, (t, hq, d), False),)
    device = _checked(*caches, ("positions", positions, i32, t, False), ("slots", slots, i32, t, False),
                      ("cos_sin", cos_sin, f32, None, False), ("q", q, bf16, None, True), ("k", k, bf16, None, True),
                      ("v", v, bf16, None, True), *given)
    if out is None:
        out = _empty(stream, device, (t, hq, d), bf16)
    q_stride, k_stride, v_stride = (q.stride(0), k.stride(0), v.stride(0)) if t > 1 else (hq * d, hkv * d, hkv * d)
    _call(device, what, fn,
          (q.data_ptr(), q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, t, hq, hkv, d, positions.data_ptr(),
           slots.data_ptr(), cos_sin.data_ptr(), max_pos, rot, int(interleaved),
           q_norm.data_ptr() if q_norm is not None else None, k_norm.data_ptr() if k_norm is not None else None, float(eps),
           out.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *places), stream)
    return out


def kv_rope_append(q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache, q_norm=None, k_norm=None,
                   eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """Norm (RMS, per head, with the weights q_norm and k_norm [D] bf16 where
    they are given) and rotate q and k [T, H, 128] bf16 by their positions,
    then write k and v into the FP8 caches [num_blocks, page_size, Hkv, 128]
    at flat token slots (fp8kv_rope_append).  cos_sin [max_pos, rot_dim] fp32
    holds cos of a position's pairs, then sin.  q, k and v may be slices of a
    fused projection.  Returns q [T, Hq, 128]; rows at position -1 are left as
    they were."""
    return _rope_append(False, q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache, q_norm, k_norm, eps,
                        interleaved, out, stream)


def kv4_rope_append(q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache, q_norm=None, k_norm=None,
                    eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """kv_rope_append into 4-bit caches (fp4kv_rope_append); head size 64 or 128."""
    return _rope_append(True, q, k, v, positions, slots, cos_sin, k_scale, v_scale, k_cache, v_cache, q_norm, k_norm, eps,
                        interleaved, out, stream)


def token_logprobs(logits, targets, top: int = 0, logprobs=None, entropy=None, top_ids=None, top_logprobs=None,
                   stream=None):
    """Log probabilities of the targets [M] under logits [M, V] (bf16 or fp32,
    rows may be padded, or one row expanded to M), each row's entropy and its
    `top` best tokens (fp8bs_token_logprobs).  Returns a TokenLogprobs."""
    m, v = _shape2(logits, "logits")
    stride = logits.stride(0) if m > 1 else v
    if 0 < stride < v:
        raise ValueError(f"the rows of logits overlap: they are {stride} elements apart and {v} long")
    top = int(top)
    f32 = logits.dtype == torch.float32
    given = [spec for spec in (("logprobs", logprobs, torch.float32, m, False), ("entropy", entropy, torch.float32, m, False),
                               ("top_ids", top_ids, torch.int32, m * top, False),
                               ("top_logprobs", top_logprobs, torch.float32, m * top, False)) if spec[1] is not None]
    device = _checked(("logits", logits, torch.float32 if f32 else torch.bfloat16, None, True),
                      ("targets", targets, torch.int32, m, False), *given)
    if logprobs is None:
        logprobs = _empty(stream, device, (m,), torch.float32)
    if entropy is None:
        entropy = _empty(stream, device, (m,), torch.float32)
    if top_ids is None:
        top_ids = _empty(stream, device, (m, top), torch.int32)
    if top_logprobs is None:
        top_logprobs = _empty(stream, device, (m, top), torch.float32)
    _call(device, "fp8bs_token_logprobs", lib().fp8bs_token_logprobs,
          (logits.data_ptr(), int(f32), stride, m, v, targets.data_ptr(), top,
           logprobs.data_ptr(), entropy.data_ptr(), top_ids.data_ptr(), top_logprobs.data_ptr()), stream)
    return TokenLogprobs(logprobs, entropy, top_ids, top_logprobs)


SampledTokens = collections.namedtuple("SampledTokens", "tokens logprobs")


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprobs=None,
                  stream=None):
    """The next token of each row of logits [M, V] (bf16 or fp32, rows may be
    padded, or one row expanded to M), drawn with u [M, 2] fp32 from what
    temperature, top_k (int32), top_p and min_p ([M] each, None: off) leave
    (fp8bs_sample_tokens).  Returns a SampledTokens: int32 tokens [M], -1 for
    a row that has none, and their log probabilities."""
    m, v = _shape2(logits, "logits")
    if u.shape[-1:] != (2,):
        raise ValueError(f"u has shape {tuple(u.shape)}, expected ({m}, 2)")
    stride = logits.stride(0) if m > 1 else v
    if 0 < stride < v:
        raise ValueError(f"the rows of logits overlap: they are {stride} elements apart and {v} long")
    f32, i32 = torch.float32, torch.int32
    is_f32 = logits.dtype == f32
    specs = [("logits", logits, f32 if is_f32 else torch.bfloat16, None, True), ("u", u, f32, (m, 2), False)]
    if temperature is not None:
        specs.append(("temperature", temperature, f32, m, False))
    if top_k is not None:
        specs.append(("top_k", top_k, i32, m, False))
    if top_p is not None:
        specs.append(("top_p", top_p, f32, m, False))
    if min_p is not None:
        specs.append(("min_p", min_p, f32, m, False))
    if tokens is not None:
        specs.append(("tokens", tokens, i32, m, False))
    if logprobs is not None:
        specs.append(("logprobs", logprobs, f32, m, False))
    device = _checked(*specs)
    if tokens is None:
        tokens = _empty(stream, device, (m,), i32)
    if logprobs is None:
        logprobs = _empty(stream, device, (m,), f32)
    _call(device, "fp8bs_sample_tokens", lib().fp8bs_sample_tokens,
          (logits.data_ptr(), int(is_f32), stride, m, v, u.data_ptr(),
           temperature.data_ptr() if temperature is not None else None, top_k.data_ptr() if top_k is not None else None,
           top_p.data_ptr() if top_p is not None else None, min_p.data_ptr() if min_p is not None else None,
           tokens.data_ptr(), logprobs.data_ptr()), stream)
    return SampledTokens(tokens, logprobs)


def act_quantize(x, codes=None, scale=None, stream=None):
    """Dynamic per-tensor e4m3 quantization of bf16 activations [M, K]."""
    m, k = _shape2(x, "x")
    codes = _new(codes, (m, k), torch.uint8, x)
    scale = _new(scale, (1,), torch.float32, x)
    a = _Args().need("x", x, torch.bfloat16).need("codes", codes, torch.uint8, numel=m * k) \
        .need("scale", scale, torch.float32, numel=1).check()
    _run(a, "fp8act_quantize", lib().fp8act_quantize, a.ptr("x"), m, k, a.ptr("codes"), a.ptr("scale"),
         stream=stream)
    return codes, scale


def w8a8_gemm(xq, sx, wq, sw, y=None, path: int = PATH_AUTO, stream=None):
    """y[M, N] = sx * sw * dec(xq) . dec(wq)^T (e4m3 x e4m3, fp32 accumulate, bf16 out)."""
    m, k = _shape2(xq, "xq")
    n, k2 = _shape2(wq, "wq")
    if k2 != k:
        raise ValueError("x codes and weight codes disagree on K")
    y = _new(y, (m, n), torch.bfloat16, xq)
    a = _Args().need("xq", xq, torch.uint8).need("sx", sx, torch.float32, numel=1).need("wq", wq, torch.uint8) \
        .need("sw", sw, torch.float32, numel=1).need("y", y, torch.bfloat16, numel=m * n).check()
    _run(a, "w8a8_gemm", lib().w8a8_gemm_ex, a.ptr("xq"), m, a.ptr("sx"), a.ptr("wq"), a.ptr("sw"), n, k,
         a.ptr("y"), int(path), stream=stream)
    return y


def w8a8_linear(x, wq, sw, y=None, xq=None, sx=None, path: int = PATH_AUTO, stream=None):
    """The W8A8 route end to end: quantize x per tensor, then w8a8_gemm."""
    xq, sx = act_quantize(x, codes=xq, scale=sx, stream=stream)
    return w8a8_gemm(xq, sx, wq, sw, y=y, path=path, stream=stream)


def select_path(m: int, n: int, k: int, x_ptr: int = 0, codes_ptr: int = 0, mx: bool = False) -> int:
    """Path the AUTO dispatch would take (host-only; pointers only matter for alignment)."""
    return lib().fp8bs_select_path(m, n, k, ctypes.c_void_p(x_ptr), ctypes.c_void_p(codes_ptr), int(mx))


def debug_wait_expiry(stream=None) -> None:
    """Launch the library's wait-expiry probe (fp8bs_debug_wait_expiry): one
    thread gives up a bounded wait after about 2 s and sets the error word."""
    _check(lib().fp8bs_debug_wait_expiry(_stream(stream)), "fp8bs_debug_wait_expiry")


def debug_encode_f32(first_bits: int, count: int, out=None, stream=None):
    """The quantizers' e4m3 encode step on the binary32 bit patterns
    first_bits .. first_bits + count - 1 (fp8bs_debug_encode_f32); returns
    uint8 codes on the device."""
    if out is None:
        out = torch.empty(count, dtype=torch.uint8, device="cuda")
    if out.numel() < count:
        raise ValueError("out holds fewer than count bytes")
    a = _Args().need("out", out, torch.uint8).check()
    _run(a, "fp8bs_debug_encode_f32", lib().fp8bs_debug_encode_f32, first_bits, count, a.ptr("out"), stream=stream)
    return out


def check_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the kernels' error word."""
    word = ctypes.c_uint32(0)
    st = lib().fp8bs_check_device_error(_stream(stream), ctypes.byref(word))
    if st not in (0, -6):
        raise Fp8bsError(st, "fp8bs_check_device_error")
    return int(word.value)
