"""skinny_gemm_qlin_amd -- weight-quantized decode GEMV for MI355X (gfx950).

Thin torch-facing binding of the C ABI in include/qlin.h (libqlin.so).  The
functions carry the C names and only marshal arguments: they check dtype,
device and that the innermost dimension is contiguous, pass data pointers,
row pitches and torch's current HIP stream, and raise QlinError on a non-zero
status.  Outputs that are not supplied are allocated with torch (device
memory plumbing only), in memory of the stream that the call runs on.  Every
arithmetic step runs in the HIP kernels.

Storage conventions: bf16 tensors are torch.bfloat16; int8 codes are
torch.int8; E4M3 codes, UE8M0 scale bytes and packed E2M1 nibbles are
torch.uint8 (a torch.float8_e4m3fn tensor may be passed for E4M3 codes).
"""
from __future__ import annotations

import torch

from ._lib import (QLIN_ACT_GELU_TANH, QLIN_ACT_SILU, QLIN_DT_BF16, QLIN_DT_FP16, QLIN_ERR_SHAPE,  # noqa: F401
                   QLIN_FMT_E4M3, QLIN_FMT_E5M2, QLIN_ROUTE_ALL, QLIN_ROUTE_SELECTED, QlinError, check, load, status_str)

__all__ = [
    "QlinError", "qlin_act_quant_i8", "qlin_gemv_i8", "qlin_linear_i8", "qlin_gemv_fp8", "qlin_gemv_fp8_blk",
    "qlin_act_quant_fp8", "qlin_gemv_fp8_w8a8", "QLIN_FMT_E4M3", "QLIN_FMT_E5M2", "qlin_gemv_fp8_blk_ex",
    "qlin_moe_mxfp4", "qlin_moe_mxfp4_workspace_bytes", "qlin_moe_mxfp4_noalloc", "status_str",
    "qlin_gemv_w4", "qlin_gemv_w4_bwd", "qlin_gemv_w4_bwd_workspace_bytes", "qlin_glu_w4", "qlin_glu_w4_bwd",
    "QLIN_DT_BF16", "QLIN_DT_FP16", "QLIN_ACT_SILU", "QLIN_ACT_GELU_TANH",
    "qlin_glu_i8", "qlin_moe_ffn_i8", "qlin_moe_ffn_i8_workspace_bytes", "QLIN_ROUTE_SELECTED", "QLIN_ROUTE_ALL",
]


def _stream(t: torch.Tensor, stream):
    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _need(t: torch.Tensor, name: str, dtypes, dims: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor, got {t.device}")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dims, got shape {tuple(t.shape)}")
    if dims >= 1 and t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}: innermost dimension must be contiguous (stride {t.stride(-1)})")
    return t


def _own(name, shape, dtype, like, stream):
    """Memory of the call's own on the stream that its kernels run on: a torch.cuda.Stream or a raw handle, None
    for the current one.

    A block belongs to the stream it was allocated on: taken from the current one it may still be written by work
    queued there, and once dropped it is handed out there again, while the kernels on `stream` are using it.  The
    caller meets the result on the current stream, so that one is recorded, too.  `name`, if given, is what the
    caller has to supply along with a raw handle that is not the current stream's; without a name torch keeps
    memory for the handle as it does for an external stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    here = torch.cuda.current_stream(like.device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = getattr(stream, "cuda_stream", stream)
        if raw == here.cuda_stream:
            return torch.empty(shape, dtype=dtype, device=like.device)
        if name:
            raise ValueError(f"a raw stream that is not the current one needs {name} along with it, {tuple(shape)}")
        stream = (torch.cuda.ExternalStream(raw, device=like.device) if raw
                  else torch.cuda.default_stream(like.device))
    elif stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {like.device}")
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    if stream != here:
        t.record_stream(here)
    return t


_U8 = (torch.uint8, torch.float8_e4m3fn)


def qlin_act_quant_i8(x, xq=None, xs=None, stream=None):
    """Per-token INT8 quantisation of bf16 x [M, K] -> (xq int8 [M, K], xs fp32 [M])."""
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    if xq is None:
        xq = _own(None, (M, K), torch.int8, x, stream)
    if xs is None:
        xs = _own(None, (M,), torch.float32, x, stream)
    _need(xq, "xq", (torch.int8,), 2)
    _need(xs, "xs", (torch.float32,), 1)
    check(load().qlin_act_quant_i8(x.data_ptr(), x.stride(0), M, K, xq.data_ptr(), xq.stride(0),
                                   xs.data_ptr(), _stream(x, stream)), "qlin_act_quant_i8")
    return xq, xs


def qlin_gemv_i8(xq, xs, w, ws, bias=None, y=None, out_kind=0, stream=None):
    """W8A8 GEMV: xq int8 [M, K], xs fp32 [M] or [1], w int8 [N, K] (row pitch
    w.stride(0)), ws fp32 [N] or [1], bias bf16 [N] or None.  out_kind 0 ->
    y bf16 [M, N]; out_kind 1 -> y int32 [M, N] holding the raw accumulators."""
    _need(xq, "xq", (torch.int8,), 2)
    _need(w, "w", (torch.int8,), 2)
    M, K = xq.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w has K={w.shape[1]}, xq has K={K}")
    _need(xs, "xs", (torch.float32,), 1)
    _need(ws, "ws", (torch.float32,), 1)
    if bias is not None:
        _need(bias, "bias", (torch.bfloat16,), 1)
    if y is None:
        y = _own(None, (M, N), torch.int32 if out_kind == 1 else torch.bfloat16, xq, stream)
    _need(y, "y", (torch.int32,) if out_kind == 1 else (torch.bfloat16,), 2)
    check(load().qlin_gemv_i8(xq.data_ptr(), xq.stride(0), xs.data_ptr(), int(xs.numel() > 1), M, K,
                              w.data_ptr(), w.stride(0), N, ws.data_ptr(), int(ws.numel() > 1),
                              None if bias is None else bias.data_ptr(), y.data_ptr(), y.stride(0),
                              int(out_kind), _stream(xq, stream)), "qlin_gemv_i8")
    return y


def qlin_linear_i8(x, w, ws, bias=None, xq=None, xs=None, y=None, stream=None):
    """The whole INT8 decode linear layer in one call: per-token quantisation of
    bf16 x [M, K] (codes and scales into xq int8 [M, K] / xs fp32 [M]) and the
    W8A8 GEMV with its bf16 epilogue.  One kernel for one token.
    Returns (y bf16 [M, N], xq, xs)."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", (torch.int8,), 2)
    _need(ws, "ws", (torch.float32,), 1)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w has K={w.shape[1]}, x has K={K}")
    if bias is not None:
        _need(bias, "bias", (torch.bfloat16,), 1)
    if xq is None:
        xq = _own(None, (M, K), torch.int8, x, stream)
    if xs is None:
        xs = _own(None, (M,), torch.float32, x, stream)
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, x, stream)
    _need(xq, "xq", (torch.int8,), 2)
    _need(xs, "xs", (torch.float32,), 1)
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_linear_i8(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), w.stride(0), N, ws.data_ptr(),
                                int(ws.numel() > 1), None if bias is None else bias.data_ptr(), xq.data_ptr(),
                                xq.stride(0), xs.data_ptr(), y.data_ptr(), y.stride(0), _stream(x, stream)),
          "qlin_linear_i8")
    return y, xq, xs


def qlin_gemv_fp8(x, w, ws, y=None, stream=None):
    """E4M3 weight-only GEMV: x bf16 [M, K], w E4M3 codes [N, K], ws fp32 [N] or [1]."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", _U8, 2)
    _need(ws, "ws", (torch.float32,), 1)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w has K={w.shape[1]}, x has K={K}")
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, x, stream)
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_gemv_fp8(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), w.stride(0), N,
                               ws.data_ptr(), int(ws.numel() > 1), y.data_ptr(), y.stride(0),
                               _stream(x, stream)), "qlin_gemv_fp8")
    return y


_FP8_DT = {QLIN_FMT_E4M3: torch.float8_e4m3fn, QLIN_FMT_E5M2: torch.float8_e5m2}


def _codes(t: torch.Tensor, name: str, fmt: int) -> torch.Tensor:
    """FP8 codes as stored: torch.uint8, or the float8 dtype of the format."""
    if fmt not in _FP8_DT:
        raise ValueError(f"{name}: unknown FP8 format {fmt}")
    _need(t, name, (torch.uint8, _FP8_DT[fmt]), 2)
    return t


def qlin_act_quant_fp8(x, fmt=QLIN_FMT_E4M3, per_token=True, xq=None, xs=None, stream=None):
    """Dynamic FP8 quantisation of bf16 x [M, K] -> (xq uint8 codes [M, K] of
    format fmt, xs fp32 [M] (per_token) or [1])."""
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    if xq is None:
        xq = _own(None, (M, K), torch.uint8, x, stream)
    if xs is None:
        xs = _own(None, (M if per_token else 1,), torch.float32, x, stream)
    _codes(xq, "xq", fmt)
    _need(xs, "xs", (torch.float32,), 1)
    if xs.numel() < (M if per_token else 1):
        raise ValueError(f"xs holds {xs.numel()} scales, needs {M if per_token else 1}")
    check(load().qlin_act_quant_fp8(x.data_ptr(), x.stride(0), M, K, int(fmt), int(bool(per_token)),
                                    xq.data_ptr(), xq.stride(0), xs.data_ptr(), _stream(x, stream)),
          "qlin_act_quant_fp8")
    return xq, xs


def qlin_gemv_fp8_w8a8(xq, xs, w, ws, x_fmt=QLIN_FMT_E4M3, w_fmt=QLIN_FMT_E4M3, y=None, stream=None):
    """FP8 W8A8 GEMV: xq codes [M, K] (format x_fmt), xs fp32 [M] or [1], w codes
    [N, K] (format w_fmt, row pitch w.stride(0)), ws fp32 [N] or [1] -> y bf16 [M, N]."""
    _codes(xq, "xq", x_fmt)
    _codes(w, "w", w_fmt)
    _need(xs, "xs", (torch.float32,), 1)
    _need(ws, "ws", (torch.float32,), 1)
    M, K = xq.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w has K={w.shape[1]}, xq has K={K}")
    if xs.numel() not in (1, M) or ws.numel() not in (1, N):
        raise ValueError(f"xs must hold 1 or M={M} scales, ws 1 or N={N}")
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, xq, stream)
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_gemv_fp8_w8a8(xq.data_ptr(), xq.stride(0), xs.data_ptr(), int(xs.numel() > 1),
                                    int(x_fmt), M, K, w.data_ptr(), w.stride(0), N, ws.data_ptr(),
                                    int(ws.numel() > 1), int(w_fmt), y.data_ptr(), y.stride(0),
                                    _stream(xq, stream)), "qlin_gemv_fp8_w8a8")
    return y


def qlin_gemv_fp8_blk(x, w, ws, xq=None, xs=None, y=None, stream=None, export=True):
    """Block-scaled FP8: x bf16 [M, K], w E4M3 [N, K], ws UE8M0 [ceil(N/128), K/128].
    Returns (y bf16 [M, N], xq E4M3 [M, K], xs UE8M0 [M, K/128]).  export=False
    passes NULL code / scale buffers (accepted for one token, K <= 32768) and
    returns (y, None, None)."""
    if not export:
        _need(x, "x", (torch.bfloat16,), 2)
        if y is None:
            y = _own(None, (x.shape[0], w.shape[0]), torch.bfloat16, x, stream)
        check(load().qlin_gemv_fp8_blk(x.data_ptr(), x.stride(0), x.shape[0], x.shape[1], w.data_ptr(),
                                       w.stride(0), w.shape[0], ws.data_ptr(), None, None, y.data_ptr(),
                                       y.stride(0), _stream(x, stream)), "qlin_gemv_fp8_blk")
        return y, None, None
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", _U8, 2)
    _need(ws, "ws", (torch.uint8,), 2)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w has K={w.shape[1]}, x has K={K}")
    if tuple(ws.shape) != ((N + 127) // 128, K // 128) or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous [{(N + 127) // 128}, {K // 128}], got {tuple(ws.shape)}")
    if xq is None:
        xq = _own(None, (M, K), torch.uint8, x, stream)
    if xs is None:
        xs = _own(None, (M, K // 128), torch.uint8, x, stream)
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, x, stream)
    if not xq.is_contiguous() or not xs.is_contiguous():
        raise ValueError("xq / xs must be contiguous")
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_gemv_fp8_blk(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), w.stride(0), N,
                                   ws.data_ptr(), xq.data_ptr(), xs.data_ptr(), y.data_ptr(),
                                   y.stride(0), _stream(x, stream)), "qlin_gemv_fp8_blk")
    return y, xq, xs


def qlin_gemv_fp8_blk_ex(x, w, ws, block_n, block_k, xq=None, xs=None, y=None, stream=None):
    """Block-scaled FP8 at any block shape: x bf16 [M, K], w E4M3 [N, K], ws UE8M0
    [ceil(N/block_n), K/block_k].  Returns (y bf16 [M, N], xq E4M3 [M, K], xs UE8M0 [M, K/block_k])."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", _U8, 2)
    _need(ws, "ws", (torch.uint8,), 2)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or K % block_k:
        raise ValueError(f"w has K={w.shape[1]}, x has K={K}, block_k={block_k}")
    if tuple(ws.shape) != ((N + block_n - 1) // block_n, K // block_k) or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous [{(N + block_n - 1) // block_n}, {K // block_k}], got {tuple(ws.shape)}")
    if xq is None:
        xq = _own(None, (M, K), torch.uint8, x, stream)
    if xs is None:
        xs = _own(None, (M, K // block_k), torch.uint8, x, stream)
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, x, stream)
    if not xq.is_contiguous() or not xs.is_contiguous():
        raise ValueError("xq / xs must be contiguous")
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_gemv_fp8_blk_ex(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), w.stride(0), N,
                                      ws.data_ptr(), int(block_n), int(block_k), xq.data_ptr(), xs.data_ptr(),
                                      y.data_ptr(), y.stride(0), _stream(x, stream)), "qlin_gemv_fp8_blk_ex")
    return y, xq, xs


def qlin_moe_mxfp4_workspace_bytes(M: int, N: int, topk: int, E: int) -> int:
    return int(load().qlin_moe_mxfp4_workspace_bytes(M, N, topk, E))


def qlin_moe_mxfp4(x, w, s, topk_ids, topk_w, y=None, workspace=None, stream=None):
    """Top-k MXFP4 expert GEMV: x bf16 [M, K]; w uint8 [E, N, K/2] (element 2i in
    the low nibble); s UE8M0 [E, N, K/32]; topk_ids int32 [M, topk]; topk_w fp32
    [M, topk].  Returns y bf16 [M, N]."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", (torch.uint8,), 3)
    _need(s, "s", (torch.uint8,), 3)
    _need(topk_ids, "topk_ids", (torch.int32,), 2)
    _need(topk_w, "topk_w", (torch.float32,), 2)
    M, K = x.shape
    E, N, Kh = w.shape
    topk = topk_ids.shape[1]
    if Kh * 2 != K or tuple(s.shape) != (E, N, K // 32):
        raise ValueError(f"w {tuple(w.shape)} / s {tuple(s.shape)} do not match K={K}")
    if not (w.is_contiguous() and s.is_contiguous() and topk_ids.is_contiguous() and topk_w.is_contiguous()):
        raise ValueError("w, s, topk_ids, topk_w must be contiguous")
    if tuple(topk_ids.shape) != (M, topk) or tuple(topk_w.shape) != (M, topk):
        raise ValueError("topk_ids / topk_w must be [M, topk]")
    need = qlin_moe_mxfp4_workspace_bytes(M, N, topk, E)
    if workspace is None:
        workspace = _own(None, (max(need, 1),), torch.uint8, x, stream)
    if y is None:
        y = _own(None, (M, N), torch.bfloat16, x, stream)
    _need(y, "y", (torch.bfloat16,), 2)
    check(load().qlin_moe_mxfp4(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), s.data_ptr(), E, N,
                                topk_ids.data_ptr(), topk_w.data_ptr(), topk, y.data_ptr(), y.stride(0),
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream(x, stream)), "qlin_moe_mxfp4")
    return y


QLIN_NOALLOC_SCRATCH_BYTES = 4 << 20  # the library's per-GPU scratch array behind qlin_moe_mxfp4_noalloc


def qlin_moe_mxfp4_noalloc(x, w, s, topk_ids, topk_w, y, stream=None):
    """qlin_moe_mxfp4 with the library's own per-GPU scratch array as its
    workspace: the call allocates nothing (y, the output, is the caller's).
    Calls that can overlap on one GPU share that array and must be serialised."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(w, "w", (torch.uint8,), 3)
    _need(s, "s", (torch.uint8,), 3)
    _need(topk_ids, "topk_ids", (torch.int32,), 2)
    _need(topk_w, "topk_w", (torch.float32,), 2)
    _need(y, "y", (torch.bfloat16,), 2)
    M, K = x.shape
    E, N, Kh = w.shape
    topk = topk_ids.shape[1]
    if Kh * 2 != K or tuple(s.shape) != (E, N, K // 32):
        raise ValueError(f"w {tuple(w.shape)} / s {tuple(s.shape)} do not match K={K}")
    if not (w.is_contiguous() and s.is_contiguous() and topk_ids.is_contiguous() and topk_w.is_contiguous()):
        raise ValueError("w, s, topk_ids, topk_w must be contiguous")
    if tuple(topk_ids.shape) != (M, topk) or tuple(topk_w.shape) != (M, topk) or tuple(y.shape) != (M, N):
        raise ValueError("topk_ids / topk_w must be [M, topk] and y [M, N]")
    check(load().qlin_moe_mxfp4_noalloc(x.data_ptr(), x.stride(0), M, K, w.data_ptr(), s.data_ptr(), E, N,
                                        topk_ids.data_ptr(), topk_w.data_ptr(), topk, y.data_ptr(), y.stride(0),
                                        _stream(x, stream)), "qlin_moe_mxfp4_noalloc")
    return y


def qlin_moe_ffn_mxfp4_workspace_bytes(M: int, H: int, I: int, topk: int, E: int) -> int:
    return int(load().qlin_moe_ffn_mxfp4_workspace_bytes(M, H, I, topk, E))


def _round256(b: int) -> int:
    return (b + 255) // 256 * 256


def qlin_moe_ffn_mxfp4(x, wr, w13, s13, w2, s2, topk, alpha=1.0, limit=10.0, y=None, workspace=None,
                       stream=None, return_internals=False, ids=None, gw=None):
    """Routed MXFP4 expert FFN with on-device routing.  x bf16 [M, H]; wr bf16
    [E, H]; w13 uint8 [E, 2I, H/2] (gate rows then up rows); s13 [E, 2I, H/32];
    w2 uint8 [E, H, I/2]; s2 [E, H, I/32].  Returns (y bf16 [M, H], topk_ids
    int32 [M, topk], topk_w fp32 [M, topk]); with return_internals also the
    router logits fp32 [M, E] and the activations bf16 [M*topk, I] read back
    from the workspace (valid once the stream has run the call)."""
    _need(x, "x", (torch.bfloat16,), 2)
    _need(wr, "wr", (torch.bfloat16,), 2)
    for name, t in (("w13", w13), ("s13", s13), ("w2", w2), ("s2", s2)):
        _need(t, name, (torch.uint8,), 3)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not wr.is_contiguous():
        raise ValueError("wr must be contiguous")
    M, H = x.shape
    E = wr.shape[0]
    I = w13.shape[1] // 2
    if (tuple(wr.shape) != (E, H) or tuple(w13.shape) != (E, 2 * I, H // 2) or tuple(s13.shape) != (E, 2 * I, H // 32)
            or tuple(w2.shape) != (E, H, I // 2) or tuple(s2.shape) != (E, H, I // 32)):
        raise ValueError("router / expert tensor shapes do not match x")
    need = qlin_moe_ffn_mxfp4_workspace_bytes(M, H, I, topk, E)
    if workspace is None:
        workspace = _own(None, (max(need, 1),), torch.uint8, x, stream)
    if y is None:
        y = _own(None, (M, H), torch.bfloat16, x, stream)
    _need(y, "y", (torch.bfloat16,), 2)
    if ids is None:
        ids = _own(None, (M, topk), torch.int32, x, stream)
    if gw is None:
        gw = _own(None, (M, topk), torch.float32, x, stream)
    _need(ids, "ids", (torch.int32,), 2)
    _need(gw, "gw", (torch.float32,), 2)
    if tuple(ids.shape) != (M, topk) or tuple(gw.shape) != (M, topk) or not (ids.is_contiguous() and gw.is_contiguous()):
        raise ValueError("ids / gw must be contiguous [M, topk]")
    check(load().qlin_moe_ffn_mxfp4(x.data_ptr(), x.stride(0), M, H, wr.data_ptr(), E, topk,
                                    w13.data_ptr(), s13.data_ptr(), I, w2.data_ptr(), s2.data_ptr(),
                                    float(alpha), float(limit), ids.data_ptr(), gw.data_ptr(),
                                    y.data_ptr(), y.stride(0), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _stream(x, stream)),
          "qlin_moe_ffn_mxfp4")
    if not return_internals:
        return y, ids, gw
    o_act = _round256(M * E * 4)
    logits = workspace[:M * E * 4].view(torch.float32).view(M, E)
    act = workspace[o_act:o_act + M * topk * I * 2].view(torch.bfloat16).view(M * topk, I)
    return y, ids, gw, logits, act


# ----------------------------------------------------------------------------- 4-bit weights with group scales
# One token through a small layer is a few microseconds on the GPU, so these calls look at each tensor
# only as often as the checks need; _w4_weight says what was wrong once a check has failed.
# `stream`: a torch.cuda.Stream (results and workspaces that are not supplied come from its memory) or a raw
# handle (every one of them is supplied, unless the handle is the current stream's).

_DT16 = {torch.bfloat16: QLIN_DT_BF16, torch.float16: QLIN_DT_FP16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_U8_ONLY = torch.uint8


def _w4_weight(a, name, w, ws, wz):
    """Checks a 4-bit weight against the 16-bit operand `a`; returns (N, K, group, dtype flag, device index)."""
    try:
        dt = _DT16.get(a.dtype)
        if dt is not None and w.dim() == 2 and ws.dim() == 2 and a.dim() == 2:
            N, Kh = w.shape
            rows, groups = ws.shape
            K, dev = 2 * Kh, a.get_device()
            if (rows == N and groups > 0 and K % groups == 0 and w.dtype is _U8_ONLY and ws.dtype is a.dtype
                    and ws.is_contiguous() and w.get_device() == dev == ws.get_device() and dev >= 0
                    and (w.stride(1) == 1 or Kh == 1) and (a.stride(1) == 1 or a.shape[1] == 1)
                    and (wz is None or (wz.dtype is _U8_ONLY and wz.shape == ws.shape and wz.is_contiguous()
                                        and wz.get_device() == dev))):
                return N, K, K // groups, dt, dev
    except AttributeError:  # something here is no tensor
        pass
    # something is wrong: say what
    _need(a, name, tuple(_DT16), 2)
    _need(w, "w", (torch.uint8,), 2)
    _need(ws, "ws", (a.dtype,), 2)
    N, Kh = w.shape
    if ws.shape[0] != N or ws.shape[1] < 1 or (2 * Kh) % ws.shape[1] or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous [{N}, K / group], got {tuple(ws.shape)}")
    if wz is not None:
        _need(wz, "wz", (torch.uint8,), 2)
        if wz.shape != ws.shape or not wz.is_contiguous():
            raise ValueError(f"wz must be contiguous {tuple(ws.shape)}, got {tuple(wz.shape)}")
    raise ValueError(f"w, ws and wz must be on {name}'s device, {a.device}")


def _out16(t, name, like, rows, cols, stream=None):
    """An operand or output of `like`'s type and device: allocated if None, or checked."""
    if t is None:
        return _own(name, (rows, cols), like.dtype, like, stream)
    if (isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.dim() == 2
            and t.shape[0] == rows and t.shape[1] == cols and (t.stride(1) == 1 or cols == 1)
            and t.get_device() == like.get_device()):
        return t
    _need(t, name, (like.dtype,), 2)
    raise ValueError(f"{name} must be [{rows}, {cols}] on {like.device}, got {tuple(t.shape)} on {t.device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pitch(t, rows, cols):
    """Row pitch in elements; a single row has none of its own: its length, rounded up to 8."""
    return t.stride(0) if rows > 1 else (cols + 7) // 8 * 8


def _wpitch(w):
    return w.stride(0) if w.shape[0] > 1 else w.shape[1]


def _launch(fn, where, dev, stream, *args):
    """fn(*args, stream) with `dev` current: kernels are launched on the current device."""
    st = _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)
    if dev == torch.cuda.current_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc != 0:
        check(rc, where)


def qlin_gemv_w4(x, w, ws, wz=None, bias=None, y=None, stream=None):
    """Linear layer on 4-bit weights with group scales: x bf16 or fp16 [M, K]; w
    uint8 [N, K/2] (element 2i in the low nibble, any row pitch that is a
    multiple of 16); ws [N, K/group] of x's dtype; wz uint8 [N, K/group] or None
    (zero point 8); bias [N] of x's dtype or None.  Returns y [M, N]."""
    N, K, group, dt, dev = _w4_weight(x, "x", w, ws, wz)
    M, Kx = x.shape
    if Kx != K:
        raise ValueError(f"w has K={K}, x has K={Kx}")
    if bias is not None:
        _need(bias, "bias", (x.dtype,), 1)
        if bias.shape[0] != N or bias.get_device() != dev:
            raise ValueError(f"bias must be [{N}] on {x.device}")
    y = _out16(y, "y", x, M, N, stream)
    _launch(load().qlin_gemv_w4, "qlin_gemv_w4", dev, stream, x.data_ptr(), _pitch(x, M, K), M, K, dt, w.data_ptr(),
            _wpitch(w), N, ws.data_ptr(), _ptr(wz), group, _ptr(bias), y.data_ptr(), _pitch(y, M, N))
    return y


def qlin_gemv_w4_bwd_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().qlin_gemv_w4_bwd_workspace_bytes(M, N, K))


def _w4_workspace(workspace, M, N, K, like, stream):
    """The caller's workspace, or one allocated for the stream that the call runs on."""
    need = qlin_gemv_w4_bwd_workspace_bytes(M, N, K)
    if workspace is None:
        if not need:
            return None, 0
        workspace = _own("a workspace", (need,), torch.uint8, like, stream)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {like.device}")
    return workspace, workspace.numel() * workspace.element_size()


def qlin_gemv_w4_bwd(dy, w, ws, wz=None, dx=None, workspace=None, stream=None):
    """Input gradient of qlin_gemv_w4: dy [M, N] (row pitch a multiple of 8) and
    the weight -> dx [M, K]."""
    N, K, group, dt, dev = _w4_weight(dy, "dy", w, ws, wz)
    M, Ny = dy.shape
    if Ny != N:
        raise ValueError(f"w has N={N}, dy has N={Ny}")
    dx = _out16(dx, "dx", dy, M, K, stream)
    buf, size = _w4_workspace(workspace, M, N, K, dy, stream)
    _launch(load().qlin_gemv_w4_bwd, "qlin_gemv_w4_bwd", dev, stream, dy.data_ptr(), _pitch(dy, M, N), M, N, dt,
            w.data_ptr(), _wpitch(w), K, ws.data_ptr(), _ptr(wz), group, dx.data_ptr(), _pitch(dx, M, K), _ptr(buf), size)
    return dx


def qlin_glu_w4(x, w13, s13, z13=None, act=QLIN_ACT_SILU, y=None, gu=None, stream=None):
    """Gated feed-forward front on 4-bit weights: w13 uint8 [2I, K/2] (gate rows,
    then up rows), s13 / z13 as ws / wz of qlin_gemv_w4.  Returns
    y = act(x Wg^T) * (x Wu^T) [M, I]; gu [M, 2I], if given, receives gate and up."""
    N, K, group, dt, dev = _w4_weight(x, "x", w13, s13, z13)
    M, Kx = x.shape
    I = N // 2
    if Kx != K or N != 2 * I:
        raise ValueError(f"w13 is [{N}, {K}], x has K={Kx}: rows must be 2I, K equal")
    y = _out16(y, "y", x, M, I, stream)
    if gu is not None:
        _out16(gu, "gu", x, M, N)
    _launch(load().qlin_glu_w4, "qlin_glu_w4", dev, stream, x.data_ptr(), _pitch(x, M, K), M, K, dt, w13.data_ptr(),
            _wpitch(w13), I, s13.data_ptr(), _ptr(z13), group, act, y.data_ptr(), _pitch(y, M, I), _ptr(gu),
            0 if gu is None else _pitch(gu, M, N))
    return y


def qlin_glu_w4_bwd(dy, w13, s13, z13=None, act=QLIN_ACT_SILU, x=None, gu=None, dgu=None, dx=None, workspace=None,
                    need_dx=True, stream=None):
    """Backward of qlin_glu_w4 from dy [M, I] and either the kept gu [M, 2I] or x
    [M, K] (gate and up are then recomputed).  Returns (dx [M, K], dgu [M, 2I]);
    need_dx=False skips the input gradient and returns (None, dgu)."""
    N, K, group, dt, dev = _w4_weight(dy, "dy", w13, s13, z13)
    M, I = dy.shape
    if I * 2 != N:
        raise ValueError(f"w13 has {N} rows, dy has I={I}")
    if x is None and gu is None:
        raise ValueError("either x or gu is needed")
    if x is not None:
        _out16(x, "x", dy, M, K)
    if gu is not None:
        _out16(gu, "gu", dy, M, N)
    if dgu is None:  # row pitch a multiple of 8, as the second product reads it
        dgu = _own("dgu", (M, (N + 7) // 8 * 8), dy.dtype, dy, stream)[:, :N]
    else:
        _out16(dgu, "dgu", dy, M, N)
    buf, size = None, 0
    if need_dx:
        dx = _out16(dx, "dx", dy, M, K, stream)
        buf, size = _w4_workspace(workspace, M, N, K, dy, stream)
    else:
        dx = None
    _launch(load().qlin_glu_w4_bwd, "qlin_glu_w4_bwd", dev, stream, dy.data_ptr(), _pitch(dy, M, I), M, I, dt, act,
            _ptr(x), 0 if x is None else _pitch(x, M, K), _ptr(gu), 0 if gu is None else _pitch(gu, M, N),
            w13.data_ptr(), _wpitch(w13), K, s13.data_ptr(), _ptr(z13), group, dgu.data_ptr(), _pitch(dgu, M, N),
            _ptr(dx), 0 if dx is None else _pitch(dx, M, K), _ptr(buf), size)
    return dx, dgu


# ----------------------------------------------------------------------------- INT8 feed-forward
# As with the 4-bit calls, each tensor is looked at once; the functions named _..._wrong say what a failed check saw.

def _operand(t, name, dtype, shape, dev, dense=True):
    """Raises unless t has this type, shape and device, and contiguous rows (dense: is contiguous)."""
    _need(t, name, (dtype,), len(shape))
    if tuple(t.shape) != tuple(shape) or t.get_device() != dev or not (t.is_contiguous() or not dense):
        raise ValueError(f"{name} must be {'contiguous ' if dense else ''}{tuple(shape)} on cuda:{dev}, got "
                         f"{tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _glu_i8_wrong(x, w13, s13, xq, xs, y):
    _need(x, "x", tuple(_DT16), 2)
    M, K = x.shape
    dev = x.get_device()
    _need(w13, "w13", (torch.int8,), 2)
    N = w13.shape[0]
    _operand(w13, "w13", torch.int8, (N, K), dev, False)
    if N % 2:
        raise ValueError(f"w13 has {N} rows: 2I are needed")
    _need(s13, "s13", (torch.float32,), 1)
    _operand(s13, "s13", torch.float32, (1,) if s13.numel() == 1 else (N,), dev)
    if xq is not None:
        _operand(xq, "xq", torch.int8, (M, K), dev, False)
    if xs is not None:
        _operand(xs, "xs", torch.float32, (M,), dev)
    if y is not None:
        _operand(y, "y", x.dtype, (M, N // 2), dev, False)
    raise ValueError("qlin_glu_i8: operands that are no plain strided tensors")


def qlin_glu_i8(x, w13, s13, act=QLIN_ACT_SILU, xq=None, xs=None, y=None, stream=None):
    """Gated feed-forward front on INT8 weights: x bf16 or fp16 [M, K]; w13 int8
    [2I, K] (gate rows, then up rows; any row pitch that is a multiple of 16); s13
    fp32 [2I] or [1].  x is quantised per token (codes and scales into xq int8 [M, K]
    / xs fp32 [M]).  Returns (y [M, I] of x's dtype, xq, xs).  The down projection of a
    bf16 y is qlin_linear_i8; an fp16 block is qlin_moe_ffn_i8 with one expert."""
    try:
        dt, dtype, dev = _DT16.get(x.dtype), x.dtype, x.get_device()
        M, K = x.shape
        N, Kw = w13.shape
        ns, = s13.shape
        I = N // 2
        ok = (dt is not None and dev >= 0 and Kw == K and 2 * I == N and (ns == N or ns == 1)
              and w13.dtype is torch.int8 and s13.dtype is torch.float32
              and w13.get_device() == dev == s13.get_device() and s13.is_contiguous()
              and (x.stride(1) == 1 or K == 1) and (w13.stride(1) == 1 or K == 1)
              and (xq is None or (xq.dtype is torch.int8 and xq.shape == x.shape and xq.get_device() == dev
                                  and (xq.stride(1) == 1 or K == 1)))
              and (xs is None or (xs.dtype is torch.float32 and xs.shape == (M,) and xs.get_device() == dev
                                  and xs.is_contiguous()))
              and (y is None or (y.dtype is dtype and y.shape == (M, I) and y.get_device() == dev
                                 and (y.stride(1) == 1 or I == 1))))
    except (AttributeError, ValueError, TypeError, IndexError, RuntimeError):  # something here is no such tensor
        ok = False
    if not ok:
        _glu_i8_wrong(x, w13, s13, xq, xs, y)
    if xq is None:
        xq = _own(None, (M, K), torch.int8, x, stream)
    if xs is None:
        xs = _own(None, (M,), torch.float32, x, stream)
    if y is None:
        y = _own(None, (M, I), dtype, x, stream)
    _launch(load().qlin_glu_i8, "qlin_glu_i8", dev, stream, x.data_ptr(), x.stride(0) if M > 1 else (K + 7) // 8 * 8, M, K,
            dt, w13.data_ptr(), w13.stride(0) if N > 1 else K, I, s13.data_ptr(), 1 if ns > 1 else 0, act, xq.data_ptr(),
            xq.stride(0) if M > 1 else K, xs.data_ptr(), y.data_ptr(), y.stride(0) if M > 1 else I)
    return y, xq, xs


def qlin_moe_ffn_i8_workspace_bytes(M: int, H: int, I: int, topk: int, E: int) -> int:
    return int(load().qlin_moe_ffn_i8_workspace_bytes(M, H, I, topk, E))


def _expert_pitch(w):
    """Row pitch of expert matrices [E, rows, cols] that lie one behind the other, else None."""
    E, rows, cols = w.shape
    s0, s1, s2 = w.stride()
    if s2 != 1 and cols > 1:
        return None
    if rows == 1:
        s1 = s0 if E > 1 else cols
    return s1 if E == 1 or s0 == rows * s1 else None


def _moe_i8_wrong(x, w13, s13, w2, s2, logits, topk, ids, gw, y, workspace):
    _need(x, "x", tuple(_DT16), 2)
    M, H = x.shape
    dev = x.get_device()
    _need(w13, "w13", (torch.int8,), 3)
    _need(w2, "w2", (torch.int8,), 3)
    E, I = w13.shape[0], w2.shape[2]
    for name, w, rows, cols in (("w13", w13, 2 * I, H), ("w2", w2, H, I)):
        _operand(w, name, torch.int8, (E, rows, cols), dev, False)
        if _expert_pitch(w) is None:
            raise ValueError(f"{name}: rows must be contiguous and the experts lie one behind the other, strides {w.stride()}")
    _operand(s13, "s13", torch.float32, (E, 2 * I), dev)
    _operand(s2, "s2", torch.float32, (E, H), dev)
    if logits is None:
        if ids is None or gw is None:
            raise ValueError("either logits or ids and gw are needed")
        _need(ids, "ids", (torch.int32,), 2)
        topk = ids.shape[1] if topk is None else topk
    else:
        if not isinstance(topk, int):
            raise ValueError("topk, an int, is needed along with logits")
        _operand(logits, "logits", torch.float32, (M, E), dev, False)
    for name, t, dtype in (("ids", ids, torch.int32), ("gw", gw, torch.float32)):
        if t is not None:
            _operand(t, name, dtype, (M, topk), dev)
    if y is not None:
        _operand(y, "y", x.dtype, (M, H), dev, False)
    if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.get_device() == dev
                                      and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {x.device}")
    raise ValueError("qlin_moe_ffn_i8: operands that are no plain strided tensors")


def qlin_moe_ffn_i8(x, w13, s13, w2, s2, logits=None, topk=None, route=QLIN_ROUTE_SELECTED, act=QLIN_ACT_SILU, ids=None,
                    gw=None, y=None, workspace=None, stream=None):
    """Mixture-of-experts layer on INT8 experts: x bf16 or fp16 [M, H]; w13 int8
    [E, 2I, H] (gate rows, then up rows), s13 fp32 [E, 2I]; w2 int8 [E, H, I], s2 fp32
    [E, H].  logits fp32 [M, E]: the router's; topk experts of each token are selected
    on the device (NaN and -inf mask an expert) and written to ids int32 [M, topk] / gw
    fp32 [M, topk].  Without logits ids and gw are inputs; an id outside the experts
    contributes nothing.  Returns (y [M, H] of x's dtype, ids, gw)."""
    try:
        dt, dtype, dev = _DT16.get(x.dtype), x.dtype, x.get_device()
        M, H = x.shape
        E, N, Hw = w13.shape
        E2, H2, I = w2.shape
        if logits is None and topk is None:
            topk = ids.shape[1]
        p13, p2, slots = _expert_pitch(w13), _expert_pitch(w2), (M, topk)
        ok = (dt is not None and dev >= 0 and Hw == H == H2 and E2 == E and N == 2 * I
              and p13 is not None and p2 is not None and (x.stride(1) == 1 or H == 1)
              and w13.dtype is torch.int8 and w2.dtype is torch.int8 and s13.dtype is torch.float32
              and s2.dtype is torch.float32 and s13.shape == (E, N) and s2.shape == (E, H)
              and w13.get_device() == dev == w2.get_device() and s13.get_device() == dev == s2.get_device()
              and s13.is_contiguous() and s2.is_contiguous()
              and (logits is not None or (ids is not None and gw is not None))
              and (logits is None or (logits.dtype is torch.float32 and logits.shape == (M, E)
                                      and logits.get_device() == dev and (logits.stride(1) == 1 or E == 1)
                                      and isinstance(topk, int)))
              and (ids is None or (ids.dtype is torch.int32 and ids.shape == slots and ids.get_device() == dev
                                   and ids.is_contiguous()))
              and (gw is None or (gw.dtype is torch.float32 and gw.shape == slots and gw.get_device() == dev
                                  and gw.is_contiguous()))
              and (y is None or (y.dtype is dtype and y.shape == (M, H) and y.get_device() == dev
                                 and (y.stride(1) == 1 or H == 1)))
              and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous())))
    except (AttributeError, ValueError, TypeError, IndexError, RuntimeError):  # something here is no such tensor
        ok = False
    if not ok:
        _moe_i8_wrong(x, w13, s13, w2, s2, logits, topk, ids, gw, y, workspace)
    if logits is not None and not 0 < topk <= E:  # nothing is allocated for it
        check(QLIN_ERR_SHAPE, "qlin_moe_ffn_i8")
    lib = load()
    if workspace is None:
        workspace = _own(None, (max(lib.qlin_moe_ffn_i8_workspace_bytes(M, H, I, topk, E), 1),), torch.uint8, x, stream)
    if ids is None:
        ids = _own(None, slots, torch.int32, x, stream)
    if gw is None:
        gw = _own(None, slots, torch.float32, x, stream)
    if y is None:
        y = _own(None, (M, H), dtype, x, stream)
    _launch(lib.qlin_moe_ffn_i8, "qlin_moe_ffn_i8", dev, stream, x.data_ptr(), x.stride(0) if M > 1 else (H + 7) // 8 * 8, M,
            H, dt, None if logits is None else logits.data_ptr(), E if logits is None or M == 1 else logits.stride(0), E,
            topk, route, w13.data_ptr(), p13, s13.data_ptr(), I, w2.data_ptr(), p2, s2.data_ptr(), act, ids.data_ptr(),
            gw.data_ptr(), y.data_ptr(), y.stride(0) if M > 1 else H, workspace.data_ptr(), workspace.nbytes)
    return y, ids, gw
