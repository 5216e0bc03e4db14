"""Torch-tensor wrappers over the C ABI: argument marshalling only.

Every function checks devices, dtypes, shapes and contiguity, allocates its
outputs with torch (device memory and the current stream are torch's), and
calls the HIP library; a non-OK status raises RuntimeError with the
library's message.  There is no fallback: without the built library on a
GPU, ``load()`` raises ImportError.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import MoeAux, load

_DT = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16,
       torch.float8_e4m3fn: _lib.MOE_FP8_E4M3}
_EL = (torch.float32, torch.bfloat16)
_EPI = {"none": _lib.MOE_EPI_NONE, "silu_mul": _lib.MOE_EPI_SILU_MUL}


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(status: int) -> None:
    if status != _lib.MOE_OK:
        lib = load()
        raise RuntimeError(f"{lib.status_string(status).decode()}: {lib.last_error().decode()}")


def _a(t: Optional[torch.Tensor]):
    """A tensor's address, as ctypes takes it for a pointer argument."""
    return None if t is None else t.data_ptr()


def _run(fn, device: torch.device, *args) -> None:
    """Calls the library with ``device`` current and its current stream, the last argument, added.

    The stream's handle comes straight from torch's C side: torch.cuda.current_stream makes an
    object first, 1.7 us of the 8 us that a small call takes on the host.
    """
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != _lib.MOE_OK:
        _check(status)


def _need(t: torch.Tensor, name: str, dtype=None, shape=None, device=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def route_topk(logits: torch.Tensor, k: int, num_valid_rows: int = -1, renormalize: bool = True):
    """logits f32 [T, E] -> (topk_ids int32 [T, k], topk_weights f32 [T, k])."""
    _need(logits, "logits", torch.float32)
    T, E = logits.shape
    ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _check(load().route_topk(_p(logits), T, E, k, num_valid_rows, int(bool(renormalize)),
                             _p(ids), _p(w), _stream(logits)))
    return ids, w


def build_offsets(topk_ids: torch.Tensor, E: int):
    """flat ids int32 [R] -> (offsets int32 [E+1], sorted_rows int32 [R], row_pos int32 [R])."""
    _need(topk_ids, "topk_ids", torch.int32)
    ids = topk_ids.reshape(-1)
    R = ids.numel()
    dev = ids.device
    lib = load()
    ws = torch.empty(max(1, lib.build_offsets_workspace(R, E)), dtype=torch.uint8, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_rows = torch.empty(R, dtype=torch.int32, device=dev)
    row_pos = torch.empty(R, dtype=torch.int32, device=dev)
    _check(lib.build_offsets(_p(ids), R, E, _p(offsets), _p(sorted_rows), _p(row_pos), _p(ws),
                             ws.numel(), _stream(ids)))
    return offsets, sorted_rows, row_pos


def build_offsets_noalloc(topk_ids: torch.Tensor, E: int, offsets: torch.Tensor, sorted_rows: torch.Tensor,
                          row_pos: torch.Tensor):
    """build_offsets into caller-provided outputs, with no workspace (the library's static scratch):
    flat ids int32 [R] -> offsets int32 [E+1], sorted_rows int32 [R], row_pos int32 [R]."""
    _need(topk_ids, "topk_ids", torch.int32)
    ids = topk_ids.reshape(-1)
    R = ids.numel()
    dev = ids.device
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _need(sorted_rows, "sorted_rows", torch.int32, (R,), dev)
    _need(row_pos, "row_pos", torch.int32, (R,), dev)
    _check(load().build_offsets_noalloc(_p(ids), R, E, _p(offsets), _p(sorted_rows), _p(row_pos), _stream(ids)))
    return offsets, sorted_rows, row_pos


def permute(x: torch.Tensor, sorted_rows: torch.Tensor, offsets: torch.Tensor, k: int,
            out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
            out_scales: Optional[torch.Tensor] = None):
    """x [T, H] -> x_perm [R, H] (rows >= offsets[E] untouched); fp8 also returns scales [H/128, R]."""
    _need(x, "x", (torch.float32, torch.bfloat16))
    T, H = x.shape
    R = sorted_rows.numel()
    E = offsets.numel() - 1
    out_dtype = out_dtype or x.dtype
    _need(sorted_rows, "sorted_rows", torch.int32, device=x.device)
    _need(offsets, "offsets", torch.int32, device=x.device)
    if out is None:
        out = torch.empty(R, H, dtype=out_dtype, device=x.device)
    _need(out, "out", out_dtype, (R, H), x.device)
    fp8 = out_dtype == torch.float8_e4m3fn
    if fp8 and out_scales is None:
        out_scales = torch.empty(H // 128, R, dtype=torch.float32, device=x.device)
    _check(load().permute(_p(x), _DT[x.dtype], T, H, k, _p(sorted_rows), _p(offsets), E, R,
                          _p(out), _DT[out_dtype], _p(out_scales) if fp8 else None, _stream(x)))
    return (out, out_scales) if fp8 else out


def _gemm(a, b, offsets, epilogue, a_scales, b_scales, out_dtype, out, out_scales, gather):
    _need(a, "a", tuple(_DT))
    A_rows, K = a.shape
    E, N, K2 = b.shape
    if K2 != K:
        raise ValueError(f"K mismatch: a has {K}, b has {K2}")
    _need(b, "b", a.dtype, device=a.device)
    _need(offsets, "offsets", torch.int32, (E + 1,), a.device)
    if gather is not None:
        rows, div = gather
        _need(rows, "gather_rows", torch.int32, device=a.device)
        M = rows.numel()
    else:
        M = A_rows
    fp8 = a.dtype == torch.float8_e4m3fn
    if fp8:
        _need(a_scales, "a_scales", torch.float32, (K // 128, A_rows), a.device)
        _need(b_scales, "b_scales", torch.float32, (E, N // 128, K // 128), a.device)
    n_out = N // 2 if epilogue == "silu_mul" else N
    out_dtype = out_dtype or (torch.bfloat16 if fp8 else a.dtype)
    if out is None:
        out = torch.empty(M, n_out, dtype=out_dtype, device=a.device)
    _need(out, "out", out_dtype, (M, n_out), a.device)
    fp8_out = out_dtype == torch.float8_e4m3fn
    if fp8_out and out_scales is None:
        out_scales = torch.empty(n_out // 128, M, dtype=torch.float32, device=a.device)
    common = (_p(b), _p(b_scales) if fp8 else None, _DT[a.dtype], _p(offsets), E, M, N, K, _EPI[epilogue],
              _p(out), _DT[out_dtype], _p(out_scales) if fp8_out else None, _stream(a))
    if gather is None:
        _check(load().grouped_gemm(_p(a), _p(a_scales) if fp8 else None, *common))
    else:
        _check(load().grouped_gemm_gather(_p(a), _p(a_scales) if fp8 else None, A_rows, _p(rows), int(div),
                                          *common))
    return (out, out_scales) if fp8_out else out


def grouped_gemm(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, epilogue: str = "none",
                 a_scales: Optional[torch.Tensor] = None, b_scales: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                 out_scales: Optional[torch.Tensor] = None):
    """a [M, K] x b [E, N, K] over segments of offsets -> c [M, N or N/2] (+ scales for fp8 out).

    fp8 activation scales (a_scales, and the returned scales) are block-major:
    [K/128, M] and [N_out/128, M].
    """
    return _gemm(a, b, offsets, epilogue, a_scales, b_scales, out_dtype, out, out_scales, None)


def grouped_gemm_gather(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, gather_rows: torch.Tensor,
                        gather_div: int, epilogue: str = "none", a_scales: Optional[torch.Tensor] = None,
                        b_scales: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None):
    """grouped_gemm with product row p reading a[gather_rows[p] // gather_div]; c has gather_rows.numel() rows.

    a [A_rows, K] holds token rows (a_scales [K/128, A_rows] for fp8); gather_rows is
    sorted_rows of build_offsets and gather_div is k.
    """
    return _gemm(a, b, offsets, epilogue, a_scales, b_scales, out_dtype, out, out_scales,
                 (gather_rows, gather_div))


def quantize_rows(x: torch.Tensor):
    """bf16 x [T, H] -> (e4m3 codes [T, H], f32 scales [H/128, T]), per row and 128 channels."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    xq = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=x.device)
    xs = torch.empty(H // 128, T, dtype=torch.float32, device=x.device)
    _check(load().quantize_rows(_p(x), T, H, _p(xq), _p(xs), _stream(x)))
    return xq, xs


def grouped_gemm_tile_shape(dtype: torch.dtype, epilogue: str, M_rows: int, E: int,
                            out_dtype: Optional[torch.dtype] = None):
    """(tile rows, tile weight rows, K elements per slice) of moe_grouped_gemm for a dtype, epilogue,
    launch size (M_rows product rows over E experts) and output dtype (default: bf16 for fp8
    operands, else the operand dtype)."""
    out_dtype = out_dtype or (torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype)
    m, n, k = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().grouped_gemm_tile_shape(_DT[dtype], _EPI[epilogue], _DT[out_dtype], M_rows, E,
                                          ctypes.byref(m), ctypes.byref(n), ctypes.byref(k)))
    return m.value, n.value, k.value


def unpermute_combine(y: torch.Tensor, row_pos: torch.Tensor, topk_weights: torch.Tensor,
                      offsets: torch.Tensor, k: int, out_dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None):
    """y [R, H] -> out [T, H] = weighted sum of each token's valid rows."""
    _need(y, "y", (torch.float32, torch.bfloat16))
    R, H = y.shape
    T = R // k
    E = offsets.numel() - 1
    _need(row_pos, "row_pos", torch.int32, device=y.device)
    _need(topk_weights, "topk_weights", torch.float32, device=y.device)
    _need(offsets, "offsets", torch.int32, device=y.device)
    out_dtype = out_dtype or y.dtype
    if out is None:
        out = torch.empty(T, H, dtype=out_dtype, device=y.device)
    _need(out, "out", out_dtype, (T, H), y.device)
    _check(load().unpermute_combine(_p(y), _DT[y.dtype], _p(row_pos), _p(topk_weights), _p(offsets),
                                    E, T, H, k, _p(out), _DT[out_dtype], _stream(y)))
    return out


@dataclass
class ForwardAux:
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    offsets: torch.Tensor
    sorted_rows: torch.Tensor
    row_pos: torch.Tensor


def forward_workspace_bytes(T: int, H: int, I: int, E: int, k: int, w_dtype: torch.dtype) -> int:
    return load().forward_workspace(T, H, I, E, k, _DT[w_dtype])


def forward(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, k: int,
            num_valid_rows: int = -1, renormalize: bool = True,
            w13_scale: Optional[torch.Tensor] = None, w2_scale: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, return_aux: bool = False,
            stage_events=None):
    """The whole layer: x [T, H], logits f32 [T, E], w13 [E, 2I, H], w2 [E, H, I] -> out [T, H].

    ``stage_events``: optional sequence of 7 hipEvent_t handles (ints) that the
    library records before the first stage and after each of the six stages.
    """
    _need(x, "x", (torch.float32, torch.bfloat16))
    T, H = x.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    dev = x.device
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(w13, "w13", tuple(_DT), (E, 2 * I, H), dev)
    _need(w2, "w2", w13.dtype, (E, H, I), dev)
    fp8 = w13.dtype == torch.float8_e4m3fn
    if fp8:
        _need(w13_scale, "w13_scale", torch.float32, (E, 2 * I // 128, H // 128), dev)
        _need(w2_scale, "w2_scale", torch.float32, (E, H // 128, I // 128), dev)
    out_dtype = out_dtype or (torch.float32 if w13.dtype == torch.float32 else torch.bfloat16)
    if out is None:
        out = torch.empty(T, H, dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, (T, H), dev)
    lib = load()
    need = lib.forward_workspace(T, H, I, E, k, _DT[w13.dtype])
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    aux_t = None
    aux_c = None
    ev_arr = None
    if stage_events is not None:
        if len(stage_events) != len(_lib.FORWARD_STAGES) + 1:
            raise ValueError("stage_events needs one event per stage boundary (7)")
        ev_arr = (ctypes.c_void_p * len(stage_events))(*stage_events)
        aux_c = MoeAux()
        aux_c.stage_events = ctypes.cast(ev_arr, ctypes.POINTER(ctypes.c_void_p))
    if return_aux:
        R = T * k
        aux_t = ForwardAux(torch.empty(T, k, dtype=torch.int32, device=dev),
                           torch.empty(T, k, dtype=torch.float32, device=dev),
                           torch.empty(E + 1, dtype=torch.int32, device=dev),
                           torch.empty(R, dtype=torch.int32, device=dev),
                           torch.empty(R, dtype=torch.int32, device=dev))
        aux_c = aux_c or MoeAux()
        aux_c.topk_ids = aux_t.topk_ids.data_ptr()
        aux_c.topk_weights = aux_t.topk_weights.data_ptr()
        aux_c.offsets = aux_t.offsets.data_ptr()
        aux_c.sorted_rows = aux_t.sorted_rows.data_ptr()
        aux_c.row_pos = aux_t.row_pos.data_ptr()
    _check(lib.forward(_p(x), _DT[x.dtype], _p(logits), _p(w13), _p(w13_scale) if fp8 else None,
                       _p(w2), _p(w2_scale) if fp8 else None, _DT[w13.dtype], T, H, I, E, k,
                       num_valid_rows, int(bool(renormalize)), _p(out), _DT[out_dtype],
                       ctypes.byref(aux_c) if aux_c is not None else None, _p(workspace),
                       workspace.numel(), _stream(x)))
    return (out, aux_t) if return_aux else out


@dataclass
class Gradients:
    dx: torch.Tensor              # [T, H]
    dw13: torch.Tensor            # [E, 2I, H]
    dw2: torch.Tensor             # [E, H, I]
    dtopk_weights: torch.Tensor   # f32 [T, k]


def backward_workspace_bytes(T: int, H: int, I: int, E: int, k: int, w_dtype: torch.dtype = torch.bfloat16) -> int:
    return load().backward_workspace(T, H, I, E, k, _DT[w_dtype])


def backward(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, dout: torch.Tensor,
             topk_weights: torch.Tensor, offsets: torch.Tensor, sorted_rows: torch.Tensor,
             row_pos: torch.Tensor, grad_dtype: torch.dtype = torch.float32,
             workspace: Optional[torch.Tensor] = None, w13_scale: Optional[torch.Tensor] = None,
             w2_scale: Optional[torch.Tensor] = None) -> Gradients:
    """Gradients of the layer for the routing ``forward`` chose (its aux outputs):
    x, dout bf16 [T, H]; w13 [E, 2I, H]; w2 [E, H, I] (bf16, or e4m3 with block scales
    w13_scale [E, 2I/128, H/128] and w2_scale [E, H/128, I/128]) -> dx, dw13, dw2
    (grad_dtype), dtopk_weights (f32)."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    k = topk_weights.shape[1] if topk_weights.dim() == 2 else 1
    dev = x.device
    _need(w13, "w13", (torch.bfloat16, torch.float8_e4m3fn), (E, 2 * I, H), dev)
    _need(w2, "w2", w13.dtype, (E, H, I), dev)
    fp8 = w13.dtype == torch.float8_e4m3fn
    if fp8:
        _need(w13_scale, "w13_scale", torch.float32, (E, 2 * I // 128, H // 128), dev)
        _need(w2_scale, "w2_scale", torch.float32, (E, H // 128, I // 128), dev)
    _need(dout, "dout", torch.bfloat16, (T, H), dev)
    _need(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _need(sorted_rows, "sorted_rows", torch.int32, device=dev)
    _need(row_pos, "row_pos", torch.int32, device=dev)
    if sorted_rows.numel() != T * k or row_pos.numel() != T * k:
        raise ValueError("sorted_rows and row_pos need T*k entries")
    g = Gradients(torch.empty(T, H, dtype=grad_dtype, device=dev),
                  torch.empty(E, 2 * I, H, dtype=grad_dtype, device=dev),
                  torch.empty(E, H, I, dtype=grad_dtype, device=dev),
                  torch.empty(T, k, dtype=torch.float32, device=dev))
    lib = load()
    need = lib.backward_workspace(T, H, I, E, k, _DT[w13.dtype])
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    _check(lib.backward(_p(x), _p(w13), _p(w13_scale) if fp8 else None, _p(w2), _p(w2_scale) if fp8 else None,
                        _DT[w13.dtype], T, H, I, E, k, _p(topk_weights), _p(offsets), _p(sorted_rows), _p(row_pos),
                        _p(dout), _p(g.dx), _p(g.dw13), _p(g.dw2), _DT[grad_dtype], _p(g.dtopk_weights),
                        _p(workspace), workspace.numel(), _stream(x)))
    return g


def _fourbit(codes: torch.Tensor, scales: torch.Tensor, device, what: str):
    """Checks 4-bit codes [E, N, K/2] and their scales; returns (E, N, K, format, group).

    uint8 scales are the e8m0 bytes of mxfp4, float32 scales those of int4.
    """
    _need(codes, f"{what}codes", torch.uint8, device=device)
    _need(scales, f"{what}scales", (torch.uint8, torch.float32), device=device)
    if codes.dim() != 3 or scales.dim() != 3 or scales.shape[:2] != codes.shape[:2]:
        raise ValueError(f"{what}codes must be [E, N, K/2] and {what}scales [E, N, K/group]")
    E, N, half = codes.shape
    groups = scales.shape[2]
    if groups == 0 or (2 * half) % groups != 0:
        raise ValueError(f"{what}scales has {groups} groups for K = {2 * half}")
    fmt = _lib.MOE_MXFP4 if scales.dtype == torch.uint8 else _lib.MOE_INT4
    return E, N, 2 * half, fmt, 2 * half // groups


def quantize_fourbit(w: torch.Tensor, format: str = "int4", group: Optional[int] = None):
    """w [E, N, K] (f32 or bf16) -> (codes uint8 [E, N, K/2], scales [E, N, K/group]).

    ``format``: "int4" (codes - 8 times f32 scales; group 32, 64 or 128, default 128) or
    "mxfp4" (e2m1 codes, e8m0 scale bytes; group 32).  The even channel is in the low nibble.
    """
    _need(w, "w", _EL)
    if w.dim() != 3:
        raise ValueError(f"w must be [E, N, K], not {tuple(w.shape)}")
    if format not in ("int4", "mxfp4"):
        raise ValueError(f"format must be 'int4' or 'mxfp4', not {format!r}")
    fp = format == "mxfp4"
    group = group or (32 if fp else 128)
    E, N, K = w.shape
    if K % 2 or K % group:
        raise ValueError(f"K = {K} is not a multiple of group = {group}")
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, N, K // group, dtype=torch.uint8 if fp else torch.float32, device=w.device)
    _run(load().quantize_fourbit, w.device, _a(w), _DT[w.dtype], E, N, K,
         _lib.MOE_MXFP4 if fp else _lib.MOE_INT4, group, _a(codes), _a(scales))
    return codes, scales


def grouped_matvec_fourbit(a: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                           epilogue: str = "none", gather_rows: Optional[torch.Tensor] = None,
                           gather_div: int = 1, out_dtype: Optional[torch.dtype] = None,
                           out: Optional[torch.Tensor] = None):
    """grouped_gemm on 4-bit weights for few rows per expert: a bf16 [A_rows, K] x codes
    [E, N, K/2] over segments of offsets -> c [M, N or N/2] (bf16 or f32).

    With ``gather_rows`` product row p reads a[gather_rows[p] // gather_div], as in
    grouped_gemm_gather.  uint8 scales are mxfp4's, float32 scales int4's.
    """
    _need(a, "a", torch.bfloat16)
    dev = a.device
    A_rows, K = a.shape
    E, N, K2, fmt, group = _fourbit(codes, scales, dev, "")
    if K2 != K:
        raise ValueError(f"K mismatch: a has {K}, codes have {K2}")
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    M = A_rows
    if gather_rows is not None:
        _need(gather_rows, "gather_rows", torch.int32, device=dev)
        M = gather_rows.numel()
    n_out = N // 2 if epilogue == "silu_mul" else N
    if out is None:
        out = a.new_empty(M, n_out, dtype=out_dtype or torch.bfloat16)
    _need(out, "out", out_dtype or _EL, (M, n_out), dev)
    _run(load().grouped_matvec_fourbit, dev, _a(a), A_rows, _a(gather_rows), int(gather_div), _a(codes), _a(scales),
         fmt, group, _a(offsets), E, M, N, K, _EPI[epilogue], _a(out), _DT[out.dtype])
    return out


def forward_fourbit_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return load().forward_fourbit_workspace(T, H, I, E, k)


def forward_fourbit(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
                    w2: torch.Tensor, w2_scale: torch.Tensor, k: int, num_valid_rows: int = -1,
                    renormalize: bool = True, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    return_aux: bool = False):
    """The whole layer on 4-bit weights, for decode sizes: x bf16 [T, H], logits f32 [T, E],
    codes w13 [E, 2I, H/2] and w2 [E, H, I/2] with their scales (quantize_fourbit's formats)
    -> out [T, H] (bf16 or f32)."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    dev = x.device
    E, I2, H2, fmt, group = _fourbit(w13, w13_scale, dev, "w13 ")
    E2, Hn, I, fmt2, group2 = _fourbit(w2, w2_scale, dev, "w2 ")
    if (E2, Hn, 2 * I, H2) != (E, H, I2, H):
        raise ValueError(f"w13 [{E}, {I2}, {H2}] and w2 [{E2}, {Hn}, {I}] do not fit x [{T}, {H}]")
    if (fmt, group) != (fmt2, group2):
        raise ValueError("w13 and w2 must have one format and group")
    _need(logits, "logits", torch.float32, (T, E), dev)
    if out is None:
        out = torch.empty(T, H, dtype=out_dtype or torch.bfloat16, device=dev)
    _need(out, "out", out_dtype or _EL, (T, H), dev)
    lib = load()
    if workspace is None:
        workspace = torch.empty(max(lib.forward_fourbit_workspace(T, H, I, E, k), 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    aux_t = aux_c = None
    if return_aux:
        i32 = lambda *shape: torch.empty(*shape, dtype=torch.int32, device=dev)
        aux_t = ForwardAux(i32(T, k), torch.empty(T, k, dtype=torch.float32, device=dev), i32(E + 1), i32(T * k),
                           i32(T * k))
        aux_c = MoeAux(aux_t.topk_ids.data_ptr(), aux_t.topk_weights.data_ptr(), aux_t.offsets.data_ptr(),
                       aux_t.sorted_rows.data_ptr(), aux_t.row_pos.data_ptr())
    _run(lib.forward_fourbit, dev, _a(x), _a(logits), _a(w13), _a(w13_scale), _a(w2), _a(w2_scale), fmt, group, T, H,
         I, E, k, num_valid_rows, int(bool(renormalize)), _a(out), _DT[out.dtype],
         ctypes.byref(aux_c) if aux_c is not None else None, _a(workspace), workspace.numel())
    return (out, aux_t) if return_aux else out


@dataclass
class NormStats:
    mean: Optional[torch.Tensor]  # f32 [T]; None in the root-mean-square form
    rstd: torch.Tensor            # f32 [T]


@dataclass
class NormGradients:
    dx: torch.Tensor                   # [T, H]
    dweight: Optional[torch.Tensor]    # [H]; None without a weight
    dbias: Optional[torch.Tensor]      # [H]; None unless asked for


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, rms: bool = False, return_stats: bool = False,
               out: Optional[torch.Tensor] = None):
    """Layer norm of token rows x [T, H] (f32 or bf16, any H up to 32768) -> y of x's shape and dtype.

    ``rms``: the root-mean-square form (no mean is subtracted).  weight and bias [H], f32 or
    bf16 (one dtype), may be None.  ``return_stats`` also returns what layer_norm_backward needs.
    """
    _need(x, "x", _EL)
    T, H = x.shape
    dev = x.device
    if weight is not None:
        _need(weight, "weight", _EL, (H,), dev)
    if bias is not None:
        _need(bias, "bias", _EL if weight is None else weight.dtype, (H,), dev)
    params = weight if weight is not None else bias
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (T, H), dev)
    stats = None
    if return_stats:
        stats = NormStats(None if rms else x.new_empty(T, dtype=torch.float32), x.new_empty(T, dtype=torch.float32))
    _run(load().layer_norm, dev, _a(x), _DT[x.dtype], T, H, _a(weight), _a(bias),
         _lib.MOE_F32 if params is None else _DT[params.dtype], eps, int(bool(rms)), _a(out),
         _a(stats.mean) if stats else None, _a(stats.rstd) if stats else None)
    return (out, stats) if return_stats else out


def layer_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return load().layer_norm_backward_workspace(T, H)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: NormStats, weight: Optional[torch.Tensor] = None,
                        bias_grad: bool = False, grad_dtype: torch.dtype = torch.float32,
                        dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> NormGradients:
    """Gradients of layer_norm: dy, x [T, H] and the statistics of the forward (stats.mean None:
    the root-mean-square form) -> dx (x's dtype), dweight and dbias (grad_dtype) [H]."""
    _need(x, "x", _EL)
    T, H = x.shape
    dev = x.device
    _need(dy, "dy", x.dtype, (T, H), dev)
    _need(stats.rstd, "stats.rstd", torch.float32, (T,), dev)
    if stats.mean is not None:
        _need(stats.mean, "stats.mean", torch.float32, (T,), dev)
    if weight is not None:
        _need(weight, "weight", _EL, (H,), dev)
    if grad_dtype not in _EL:
        raise ValueError(f"grad_dtype must be float32 or bfloat16, not {grad_dtype}")
    if dx is None:
        dx = torch.empty_like(x)
    _need(dx, "dx", x.dtype, (T, H), dev)
    new = lambda wanted: x.new_empty(H, dtype=grad_dtype) if wanted else None
    g = NormGradients(dx, new(weight is not None), new(bias_grad))
    lib = load()
    if workspace is None and (g.dweight is not None or g.dbias is not None):
        workspace = x.new_empty(max(lib.layer_norm_backward_workspace(T, H), 1), dtype=torch.uint8)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, device=dev)
    _run(lib.layer_norm_backward, dev, _a(dy), _a(x), _DT[x.dtype], T, H, _a(weight),
         _lib.MOE_F32 if weight is None else _DT[weight.dtype], _a(stats.mean), _a(stats.rstd),
         int(stats.mean is None), _a(dx), _a(g.dweight), _a(g.dbias), _DT[grad_dtype], _a(workspace),
         0 if workspace is None else workspace.numel())
    return g


def dropout_counters(n: int) -> int:
    """Counters that a dropout call over n elements uses: what to add to rng[1] between calls."""
    return (n + 7) // 8


def _need_rng(rng: torch.Tensor, device) -> None:
    _need(rng, "rng", (torch.int64, torch.uint64), (2,), device)


def dropout_add(x: torch.Tensor, rng: torch.Tensor, p: float, residual: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None):
    """residual + dropout(x), or dropout(x) alone; x (f32 or bf16) of any shape.

    ``rng``: GPU int64 (or uint64) [2] holding seed and offset; the mask is a function of them, p
    and the element's index, so dropout_add_backward with the same rng draws it again.  Advance
    rng[1] by dropout_counters(x.numel()) between calls.  out (default: the residual's dtype, else
    x's) may be x or residual.
    """
    _need(x, "x", _EL)
    dev = x.device
    _need_rng(rng, dev)
    if residual is not None:
        _need(residual, "residual", _EL, x.shape, dev)
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype or (x.dtype if residual is None else residual.dtype))
    _need(out, "out", out_dtype or _EL, x.shape, dev)
    _run(load().dropout_add, dev, _a(x), _DT[x.dtype], _a(residual),
         _lib.MOE_F32 if residual is None else _DT[residual.dtype], x.numel(), p, _a(rng), _a(out), _DT[out.dtype])
    return out


def dropout_add_backward(dout: torch.Tensor, rng: torch.Tensor, p: float, dx_dtype: Optional[torch.dtype] = None,
                         dx: Optional[torch.Tensor] = None):
    """Gradient of dropout_add (or unpermute_combine_dropout) with respect to what it dropped, for
    the same rng and p; the residual's gradient is dout itself."""
    return dropout_add(dout, rng, p, None, dx_dtype, dx)


def unpermute_combine_dropout(y: torch.Tensor, row_pos: torch.Tensor, topk_weights: torch.Tensor,
                              offsets: torch.Tensor, k: int, rng: torch.Tensor, p: float,
                              residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                              out: Optional[torch.Tensor] = None):
    """residual + dropout(unpermute_combine(y, ...)) in one pass: y [R, H] -> out [T, H].

    The mask is dropout_add's for an array [T, H].  out (default: the residual's dtype, else
    y's) must not overlap residual.
    """
    _need(y, "y", _EL)
    R, H = y.shape
    T = R // k
    E = offsets.numel() - 1
    dev = y.device
    _need(row_pos, "row_pos", torch.int32, device=dev)
    _need(topk_weights, "topk_weights", torch.float32, device=dev)
    _need(offsets, "offsets", torch.int32, device=dev)
    if row_pos.numel() < T * k or topk_weights.numel() < T * k:
        raise ValueError("row_pos and topk_weights need T*k entries")
    _need_rng(rng, dev)
    if residual is not None:
        _need(residual, "residual", _EL, (T, H), dev)
    if out is None:
        out = y.new_empty(T, H, dtype=out_dtype or (y.dtype if residual is None else residual.dtype))
    _need(out, "out", out_dtype or _EL, (T, H), dev)
    _run(load().unpermute_combine_dropout, dev, _a(y), _DT[y.dtype], _a(row_pos), _a(topk_weights), _a(offsets), E, T,
         H, k, _a(residual), _lib.MOE_F32 if residual is None else _DT[residual.dtype], p, _a(rng), _a(out),
         _DT[out.dtype])
    return out
