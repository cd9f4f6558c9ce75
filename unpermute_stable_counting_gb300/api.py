"""PyTorch-facing binding of the C ABI (include/moe_reorder.h).

Argument marshalling only: shapes, dtypes and device pointers of torch CUDA
tensors go to the library; every step of every operation runs in the
library's CUDA kernels. PyTorch supplies device memory (outputs and the
workspace, when the caller does not pass them) and the current stream.
A call with stream= runs as a whole with that stream current.
"""
from __future__ import annotations

import ctypes
import functools
import inspect

import torch

from ._native import int64_array, lib

DT_F16, DT_BF16, DT_INT8, DT_F32 = 0, 1, 2, 3
_TORCH_TO_DT = {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float32: DT_F32}
_DT_TO_TORCH = {DT_F16: torch.float16, DT_BF16: torch.bfloat16, DT_INT8: torch.int8,
                DT_F32: torch.float32}

MR_OK = 0
MR_BATCHING_FULL_TAIL = 1


class MoeReorderError(RuntimeError):
    def __init__(self, status: int, where: str):
        text = lib().mr_status_string(status).decode()
        super().__init__(f"{where} failed with status {status}: {text}")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != MR_OK:
        raise MoeReorderError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_current_device(name, index):
    """The library launches on the current device, whose streams the handles name."""
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{index}, which is not the current device "
                         f"(cuda:{torch._C._cuda_getDevice()})")


def _require_cuda(name, t, dtype=None, strided=False):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    _on_current_device(name, t.get_device())
    if not strided and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _as_stream(stream):
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _cuda_tensors(values):
    return [t for t in values if isinstance(t, torch.Tensor) and t.is_cuda]


def _on_stream(f):
    """f with an argument more: stream, a torch.cuda.Stream or a cudaStream_t (None: the
    current stream). f runs with that stream current, so that the memory it allocates
    comes from that stream's pool. Memory of the current stream's pool may have been freed
    on the host with its last kernel still in flight, and nothing orders the other stream
    behind that kernel. Tensors that the caller gave are kept until the stream is done with
    them, and tensors that the call made until the caller's stream is."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        here, stream = torch.cuda.current_stream(), _as_stream(stream)
        if stream == here:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            result = f(*args, **kw)
        for t in _cuda_tensors((*args, *kw.values(), *(kw.get("out") or {}).values())):
            t.record_stream(stream)
        for t in _cuda_tensors(result.values()):
            t.record_stream(here)
        return result

    signature = inspect.signature(f)
    argument = inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)
    call.__signature__ = signature.replace(parameters=[*signature.parameters.values(), argument])
    return call


# ---------------------------------------------------------------------------
# FFN-worker batching
# ---------------------------------------------------------------------------

def batching_workspace_size(expert_num: int, max_out_shape, token_dtype: int, layer_num: int,
                            need_schedule: int = 0) -> int:
    ws = ctypes.c_uint64(0)
    shape = int64_array(max_out_shape)
    _check(lib().ffnwb_batching_get_workspace_size(expert_num, shape, token_dtype, need_schedule,
                                                   layer_num, ctypes.byref(ws)),
           "ffnwb_batching_get_workspace_size")
    return int(ws.value)


def batching_outputs(Y: int, H: int, expert_num: int, token_dtype: int, device,
                     with_sorted_indices: bool = False) -> dict:
    """Allocate the output tensors of one batching call."""
    i32 = dict(dtype=torch.int32, device=device)
    return dict(
        y=torch.empty((Y, H), dtype=_DT_TO_TORCH[token_dtype], device=device),
        groupList=torch.empty((expert_num, 2), dtype=torch.int64, device=device),
        sessionIds=torch.empty(Y, **i32), microBatchIds=torch.empty(Y, **i32),
        tokenIds=torch.empty(Y, **i32), expertOffsets=torch.empty(Y, **i32),
        dynamicScale=torch.empty(Y, dtype=torch.float32, device=device) if token_dtype == DT_INT8 else None,
        actualTokenNum=torch.empty(1, dtype=torch.int64, device=device),
        sortedIndices=torch.empty(Y, **i32) if with_sorted_indices else None)


@_on_stream
def ffnwb_batching(expert_ids, token_data, session_ids, micro_batch_ids, *, expert_num: int,
                   max_out_shape, token_dtype: int, layer_num: int = 1, layer_id: int = 0,
                   token_ids=None, scales=None, scale_stride: int = 4, token_row_stride=None,
                   need_schedule: int = 0, with_sorted_indices: bool = False, out: dict | None = None,
                   workspace=None, full_tail: bool = False) -> dict:
    """Run the batching on the current CUDA stream.

    token_data: CUDA tensor whose first dimension is the Y slots; row s starts
    at token_row_stride bytes * s (default: the tensor's own row stride).
    full_tail: also gather the rows (and ids) of the masked slots.
    Returns the output dict (see batching_outputs)."""
    A, BS, K1, H = (int(v) for v in max_out_shape)
    Y = A * BS * K1
    for name, t in (("expert_ids", expert_ids), ("session_ids", session_ids),
                    ("micro_batch_ids", micro_batch_ids), ("token_ids", token_ids)):
        _require_cuda(name, t, torch.int32)
    _require_cuda("token_data", token_data)
    _require_cuda("scales", scales, strided=True)
    if token_row_stride is None:
        token_row_stride = token_data.stride(0) * token_data.element_size()
    dev = token_data.device
    if out is None:
        out = batching_outputs(Y, H, expert_num, token_dtype, dev, with_sorted_indices)
    if workspace is None:
        ws = batching_workspace_size(expert_num, max_out_shape, token_dtype, layer_num, need_schedule)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    shape = int64_array(max_out_shape)
    args = [_ptr(expert_ids), int(layer_id), _ptr(token_data), int(token_row_stride), _ptr(scales),
            int(scale_stride), _ptr(session_ids), _ptr(micro_batch_ids), _ptr(token_ids),
            int(expert_num), shape, int(token_dtype), int(need_schedule), int(layer_num),
            _ptr(out["y"]), _ptr(out["groupList"]), _ptr(out["sessionIds"]),
            _ptr(out["microBatchIds"]), _ptr(out["tokenIds"]), _ptr(out["expertOffsets"]),
            _ptr(out.get("dynamicScale")), _ptr(out["actualTokenNum"]), _ptr(out.get("sortedIndices"))]
    tail = [_ptr(workspace), int(workspace.numel()), _stream(dev)]
    if full_tail:
        st = lib().ffnwb_batching_ex(*args, MR_BATCHING_FULL_TAIL, *tail)
    else:
        st = lib().ffnwb_batching(*args, *tail)
    _check(st, "ffnwb_batching")
    return out


def batching_context_workspace_size(expert_num: int, max_out_shape, token_dtype: int,
                                    layer_num: int, need_schedule: int = 0) -> int:
    ws = ctypes.c_uint64(0)
    _check(lib().ffnwb_batching_context_get_workspace_size(
        expert_num, int64_array(max_out_shape), token_dtype, need_schedule, layer_num,
        ctypes.byref(ws)), "ffnwb_batching_context_get_workspace_size")
    return int(ws.value)


@_on_stream
def ffnwb_batching_context(schedule_context, *, expert_num: int, max_out_shape, token_dtype: int,
                           layer_num: int = 1, need_schedule: int = 0,
                           wait_timeout_us: int = 1_000_000, out: dict | None = None,
                           workspace=None, full_tail: bool = False) -> dict:
    """Batching from a ScheduleContext (a CUDA tensor of its 1024 bytes) on the
    current stream. Returns the batching outputs plus scheduleStatus (int32 [1]):
    blocks not ready with need_schedule = 1, or -1 for a context that does not fit.
    full_tail: also gather the rows (and ids) of the context's masked slots."""
    _require_cuda("schedule_context", schedule_context)
    if schedule_context.numel() * schedule_context.element_size() < 1024:
        raise ValueError("schedule_context must hold 1024 bytes")
    A, BS, K1, H = (int(v) for v in max_out_shape)
    dev = schedule_context.device
    if out is None:
        out = batching_outputs(A * BS * K1, H, expert_num, token_dtype, dev)
    if out.get("scheduleStatus") is None:
        out["scheduleStatus"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        ws = batching_context_workspace_size(expert_num, max_out_shape, token_dtype, layer_num,
                                             need_schedule)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    args = [_ptr(schedule_context), int(expert_num), int64_array(max_out_shape), int(token_dtype),
            int(need_schedule), int(layer_num), int(wait_timeout_us), _ptr(out["y"]),
            _ptr(out["groupList"]), _ptr(out["sessionIds"]), _ptr(out["microBatchIds"]),
            _ptr(out["tokenIds"]), _ptr(out["expertOffsets"]), _ptr(out.get("dynamicScale")),
            _ptr(out["actualTokenNum"]), _ptr(out["scheduleStatus"])]
    tail = [_ptr(workspace), int(workspace.numel()), _stream(dev)]
    if full_tail:
        st = lib().ffnwb_batching_context_ex(*args, MR_BATCHING_FULL_TAIL, *tail)
    else:
        st = lib().ffnwb_batching_context(*args, *tail)
    _check(st, "ffnwb_batching_context")
    return out


# ---------------------------------------------------------------------------
# Routing-map unpermute
# ---------------------------------------------------------------------------

def _unpermute_shapes(permuted_tokens, sorted_indices, probs, padded_mode, restore_shape):
    tdt = _TORCH_TO_DT.get(permuted_tokens.dtype)
    if tdt is None:
        raise TypeError(f"permuted_tokens dtype {permuted_tokens.dtype} is not f16/bf16/f32")
    rows, H = int(permuted_tokens.shape[0]), int(permuted_tokens.shape[1])
    n = int(sorted_indices.numel())
    if probs is not None:
        pdt = _TORCH_TO_DT.get(probs.dtype)
        if pdt is None:
            raise TypeError(f"probs dtype {probs.dtype} is not f16/bf16/f32")
        T, Eu = int(probs.shape[0]), int(probs.shape[1])
    else:
        pdt, Eu = tdt, 0
        if restore_shape is None:
            raise ValueError("restore_shape is required without probs")
        T = int(restore_shape[0])
    return tdt, pdt, rows, H, n, T, Eu


def unpermute_workspace_size(rows: int, H: int, token_dtype: int, n: int, has_probs: bool,
                             probs_dtype: int, T: int, Eu: int, padded_mode: bool,
                             restore_shape=None) -> int:
    ws = ctypes.c_uint64(0)
    rs = int64_array(restore_shape) if restore_shape is not None else None
    _check(lib().moe_unpermute_get_workspace_size(rows, H, token_dtype, n, int(has_probs),
                                                  probs_dtype, T, Eu, int(padded_mode), rs,
                                                  ctypes.byref(ws)),
           "moe_unpermute_get_workspace_size")
    return int(ws.value)


def unpermute_outputs(T: int, H: int, n: int, token_dtype: int, probs_dtype: int | None, device) -> dict:
    return dict(
        unpermutedTokens=torch.empty((T, H), dtype=_DT_TO_TORCH[token_dtype], device=device),
        outIndex=torch.empty(n, dtype=torch.int32, device=device),
        permuteTokenId=torch.empty(n, dtype=torch.int32, device=device),
        permuteProbs=(torch.empty(n, dtype=_DT_TO_TORCH[probs_dtype], device=device)
                      if probs_dtype is not None else None))


@_on_stream
def moe_unpermute(permuted_tokens, sorted_indices, routing_map=None, probs=None, *,
                  padded_mode: bool = False, restore_shape=None, out: dict | None = None,
                  workspace=None) -> dict:
    """Run the unpermute on the current CUDA stream. Returns unpermutedTokens,
    outIndex, permuteTokenId and permuteProbs (None without probs)."""
    _require_cuda("permuted_tokens", permuted_tokens)
    _require_cuda("sorted_indices", sorted_indices, torch.int32)
    _require_cuda("routing_map", routing_map, (torch.int8, torch.bool, torch.uint8))
    _require_cuda("probs", probs)
    tdt, pdt, rows, H, n, T, Eu = _unpermute_shapes(permuted_tokens, sorted_indices, probs,
                                                     padded_mode, restore_shape)
    dev = permuted_tokens.device
    if out is None:
        out = unpermute_outputs(T, H, n, tdt, pdt if probs is not None else None, dev)
    if workspace is None:
        ws = unpermute_workspace_size(rows, H, tdt, n, probs is not None, pdt, T, Eu, padded_mode,
                                      restore_shape)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    rs = int64_array(restore_shape) if restore_shape is not None else None
    st = lib().moe_unpermute(
        _ptr(permuted_tokens), _ptr(sorted_indices), _ptr(routing_map), _ptr(probs), rows, H, tdt,
        n, pdt, T, Eu, int(bool(padded_mode)), rs, _ptr(out["unpermutedTokens"]),
        _ptr(out["outIndex"]), _ptr(out["permuteTokenId"]), _ptr(out.get("permuteProbs")),
        _ptr(workspace), int(workspace.numel()), _stream(dev))
    _check(st, "moe_unpermute")
    return out


def permute_workspace_size(T: int, H: int, token_dtype: int, Eu: int, topk: int = 0,
                           padded_mode: bool = False, capacity: int = 0) -> int:
    ws = ctypes.c_uint64(0)
    _check(lib().moe_permute_get_workspace_size(T, H, token_dtype, Eu, topk, int(padded_mode),
                                                capacity, ctypes.byref(ws)),
           "moe_permute_get_workspace_size")
    return int(ws.value)


@_on_stream
def moe_permute(tokens, routing_map, *, topk: int = 0, padded_mode: bool = False, capacity: int = 0,
                out: dict | None = None, workspace=None) -> dict:
    """Permute tokens [T, H] by routing_map [T, Eu] on the current stream.
    Returns permutedTokens, sortedIndices and permutedRows (int32 [1])."""
    _require_cuda("tokens", tokens)
    _require_cuda("routing_map", routing_map, (torch.int8, torch.bool, torch.uint8))
    tdt = _TORCH_TO_DT.get(tokens.dtype)
    if tdt is None:
        raise TypeError(f"tokens dtype {tokens.dtype} is not f16/bf16/f32")
    T, H = int(tokens.shape[0]), int(tokens.shape[1])
    Eu = int(routing_map.shape[1])
    rows = Eu * capacity if padded_mode else T * topk
    dev = tokens.device
    if out is None:
        out = dict(permutedTokens=torch.empty((rows, H), dtype=tokens.dtype, device=dev),
                   sortedIndices=torch.empty(rows, dtype=torch.int32, device=dev),
                   permutedRows=torch.zeros(1, dtype=torch.int32, device=dev))
    if workspace is None:
        ws = permute_workspace_size(T, H, tdt, Eu, topk, padded_mode, capacity)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    st = lib().moe_permute(_ptr(tokens), _ptr(routing_map), T, H, tdt, Eu, int(topk),
                           int(bool(padded_mode)), int(capacity), _ptr(out["permutedTokens"]),
                           _ptr(out["sortedIndices"]), _ptr(out.get("permutedRows")),
                           _ptr(workspace), int(workspace.numel()), _stream(dev))
    _check(st, "moe_permute")
    return out


_ID_TO_DT = {torch.int32: 4, torch.int64: 5}


@_on_stream
def moe_update_expert(expert_ids, eplb_table, *, local_rank: int = 0, world_size: int,
                      balance_mode: int = 0, scales=None, threshold=None, active=None,
                      out: dict | None = None) -> dict:
    """Map expert_ids [BS, K] (int32/int64) to physical instances through
    eplb_table [E, F] int32 and, with scales [BS, K] and threshold [K] (or
    [1, K]), prune them. Strided views are passed by their strides (no copy).
    Returns balancedExpertIds and balancedActiveMask (None without scales)."""
    _require_cuda("expert_ids", expert_ids, (torch.int32, torch.int64), strided=True)
    _require_cuda("eplb_table", eplb_table, (torch.int32,), strided=True)
    BS, K = int(expert_ids.shape[0]), int(expert_ids.shape[1])
    E, F = int(eplb_table.shape[0]), int(eplb_table.shape[1])
    dev = expert_ids.device
    sdt = 3
    if scales is not None:
        _require_cuda("scales", scales, strided=True)
        sdt = _TORCH_TO_DT.get(scales.dtype)
        if sdt is None:
            raise TypeError(f"scales dtype {scales.dtype} is not f16/bf16/f32")
    if threshold is not None:
        _require_cuda("threshold", threshold, (torch.float32,), strided=True)
    if active is not None:
        _require_cuda("active", active, (torch.bool, torch.uint8), strided=True)
    if out is None:
        out = dict(balancedExpertIds=torch.empty((BS, K), dtype=expert_ids.dtype, device=dev),
                   balancedActiveMask=(torch.empty((BS, K), dtype=torch.bool, device=dev)
                                       if scales is not None else None))
    bal, msk = out["balancedExpertIds"], out.get("balancedActiveMask")
    z = (0, 0)
    strides = (tuple(expert_ids.stride()) + tuple(eplb_table.stride())
               + (tuple(scales.stride()) if scales is not None else z)
               + ((threshold.stride(-1),) if threshold is not None else (0,))
               + ((active.stride(0),) if active is not None else (0,))
               + tuple(bal.stride()) + (tuple(msk.stride()) if msk is not None else (1, 1)))
    st = lib().moe_update_expert(_ptr(expert_ids), _ID_TO_DT[expert_ids.dtype], _ptr(eplb_table),
                                 _ptr(scales), sdt, _ptr(threshold), _ptr(active), BS, K, E, F,
                                 int(local_rank), int(world_size), int(balance_mode),
                                 int64_array(strides), _ptr(bal), _ptr(msk), _stream(dev))
    _check(st, "moe_update_expert")
    return out


# ---------------------------------------------------------------------------
# Expert products
# ---------------------------------------------------------------------------

DT_E4M3 = 6
_E4M3 = torch.float8_e4m3fn
_FLOAT_OR_E4M3 = {**_TORCH_TO_DT, _E4M3: DT_E4M3}
_BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // _BLOCK)


# The expert products are called per layer of a decode step: what a call costs on
# the host is part of its latency. So their checks read each tensor's attributes
# once, pointers go to ctypes as plain ints, pairs of strides as arrays of one
# type, and workspace sizes (functions of the sizes, the layer's also of the device)
# are kept.
_Pair = ctypes.c_int64 * 2


@functools.lru_cache(maxsize=64)
def _device(index):
    return torch.device("cuda", index)


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _float_dt(name, t, table=_TORCH_TO_DT):
    dt = table.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} dtype {t.dtype} is not f16/bf16/f32" + ("/e4m3" if DT_E4M3 in table.values() else ""))
    return dt


def _rows_of(name, t, dims):
    """Shape and strides of a CUDA tensor of `dims` dimensions whose rows have
    adjacent elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    shape, strides = t.shape, t.stride()
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(shape)}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have adjacent elements in a row")
    return shape, strides


def _row_stride(shape, strides):
    return strides[-2] if shape[-2] > 1 else max(strides[-2], shape[-1])


def _matrix_strides(name, shape, strides, size=1):
    """{row, matrix} byte strides of weights [..., rows, cols] with evenly spaced matrices."""
    row = _row_stride(shape, strides)
    matrix = shape[-2] * row  # of a single matrix, whose stride says nothing
    if shape[-3] > 1:
        matrix = strides[-3]
        if len(shape) == 4 and shape[0] > 1 and strides[0] != shape[1] * matrix:
            raise ValueError(f"{name} must have evenly spaced matrices")
    elif len(shape) == 4 and shape[0] > 1:
        matrix = strides[0]
    return _Pair(row * size, matrix * size)


def _vector(name, t, dtype, index, shape=None):
    """The address of a contiguous tensor (None: no tensor)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    _same_device(name, t, index)
    return t.data_ptr()


def _same_device(name, t, index):
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


def _workspace(workspace, size, index):
    if workspace is None:
        return torch.empty(max(size, 1), dtype=torch.uint8, device=_device(index))
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a CUDA tensor of uint8")
    if not workspace.is_contiguous():  # its length in bytes is passed on, whatever lies behind it
        raise ValueError("workspace must be contiguous")
    _same_device("workspace", workspace, index)
    return workspace


def _wide_rows(lead, cols, index):
    """e4m3 [*lead, cols] whose rows start on 16 bytes."""
    wide = -(-cols // 16) * 16
    if wide == cols:
        return torch.empty((*lead, cols), dtype=_E4M3, device=_device(index))
    strides = [1]  # one tensor, not a slice of a wider one: that costs a small call 4 us more
    for n in (wide, *lead[:0:-1]):
        strides.append(strides[-1] * max(n, 1))
    return torch.empty_strided((*lead, cols), strides[::-1], dtype=_E4M3, device=_device(index))


def quantize_outputs(shape, device, block_rows: int = 1) -> dict:
    """Allocate the output tensors of one moe_quantize call for x of `shape`:
    rows start on 16 bytes, as the expert products take them."""
    *lead, rows, cols = (int(v) for v in shape)
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    return dict(values=_wide_rows((*lead, rows), cols, index),
                scales=torch.empty((*lead, rows if block_rows == 1 else _blocks(rows), _blocks(cols)),
                                   dtype=torch.float32, device=_device(index)))


@_on_stream
def moe_quantize(x, *, block_rows: int = 1, num_rows=None, out: dict | None = None) -> dict:
    """Quantize x (f16/bf16/f32) to e4m3 blocks on the current stream. Returns
    values and scales.

    block_rows 1: x [rows, cols], a scale per row and 128 columns. block_rows
    128: weights x [..., rows, cols], a scale per 128 x 128 block. num_rows
    (int64 [1] on the device): rows at or past it are not written."""
    if block_rows not in (1, _BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    dims = 2 if block_rows == 1 else x.dim()
    shape, strides = _rows_of("x", x, dims)
    if not 2 <= dims <= 4:
        raise ValueError("x must have 2 to 4 dimensions")
    dt, index = _float_dt("x", x), x.get_device()
    _on_current_device("x", index)
    rows, cols = shape[-2], shape[-1]
    sshape = (*shape[:-2], rows if block_rows == 1 else _blocks(rows), _blocks(cols))
    num_rows = _vector("num_rows", num_rows, torch.int64, index)
    if out is None:
        values = _wide_rows(shape[:-1], cols, index)
        scales = torch.empty(sshape, dtype=torch.float32, device=_device(index))
        out = dict(values=values, scales=scales)
        if block_rows == 1:
            st = lib().moe_quantize(x.data_ptr(), dt, 1, rows, cols, _Pair(0, _row_stride(shape, strides)), 1, num_rows,
                                    values.data_ptr(), _Pair(0, -(-cols // 16) * 16), scales.data_ptr(), None,
                                    _raw_stream(index))
            if st:
                _check(st, "moe_quantize")
            return out
    else:
        values, scales = out["values"], out["scales"]
    vshape, vstrides = _rows_of("values", values, dims)
    if values.dtype != _E4M3 or vshape != shape:
        raise ValueError("values must be e4m3 of x's shape")
    _same_device("values", values, index)
    ss = None
    if block_rows == 1:
        if not scales.is_cuda or scales.dtype != torch.float32 or scales.shape != sshape:
            raise ValueError(f"scales must be float32 {list(sshape)}")
        _same_device("scales", scales, index)
        for n, step in zip(sshape, scales.stride()):
            if n > 1 and step < 1:  # an expanded tensor has fewer elements than it shows
                raise ValueError("scales must have an element of their own for each scale")
        s0, s1 = scales.stride()
        ss = _Pair(max(1, s0), max(1, s1))
        saddr = scales.data_ptr()
        xs, vs = _Pair(0, _row_stride(shape, strides)), _Pair(0, _row_stride(vshape, vstrides))
        batch = 1
    else:
        saddr = _vector("scales", scales, torch.float32, index, sshape)
        if x.numel() == 0 and rows and cols:  # no matrices
            return out
        batch = x.numel() // max(1, rows * cols)
        if dims == 2:
            xs, vs = _Pair(0, _row_stride(shape, strides)), _Pair(0, _row_stride(vshape, vstrides))
        else:
            xs, vs = _matrix_strides("x", shape, strides), _matrix_strides("values", vshape, vstrides)
            xs[0], xs[1] = xs[1], xs[0]
            vs[0], vs[1] = vs[1], vs[0]
    st = lib().moe_quantize(x.data_ptr(), dt, max(1, batch), rows, cols, xs, block_rows,
                            num_rows, values.data_ptr(), vs, saddr, ss, _raw_stream(index))
    _check(st, "moe_quantize")
    return out


@functools.lru_cache(maxsize=1024)
def grouped_matmul_workspace_size(rows: int, cols: int, x_dtype: int) -> int:
    ws = ctypes.c_uint64(0)
    _check(lib().moe_grouped_matmul_get_workspace_size(rows, cols, x_dtype, ctypes.byref(ws)),
           "moe_grouped_matmul_get_workspace_size")
    return int(ws.value)


def _expert_rows(x, x_scales, group_list):
    """Checks of the rows and groups that both products take."""
    shape, strides = _rows_of("x", x, 2)
    dt, index = _float_dt("x", x, _FLOAT_OR_E4M3), x.get_device()
    _on_current_device("x", index)
    sa = ss = None
    if dt == DT_E4M3:
        if x_scales is None:
            raise ValueError("e4m3 rows need x_scales")
        if not isinstance(x_scales, torch.Tensor) or not x_scales.is_cuda or x_scales.dtype != torch.float32:
            raise TypeError("x_scales must be a CUDA tensor of float32")
        if x_scales.shape != (shape[0], _blocks(shape[1])):
            raise ValueError("x_scales must be [rows, ceil(cols/128)]")
        _same_device("x_scales", x_scales, index)
        sa, ss = x_scales.data_ptr(), _Pair(*x_scales.stride())
    elif x_scales is not None:
        raise ValueError("x_scales belong to e4m3 rows")
    ga, groups = _vector("group_list", group_list, torch.int64, index), -1
    if group_list is not None:
        if group_list.dim() != 2 or group_list.shape[1] != 2:
            raise ValueError("group_list must be [groups, 2]")
        groups = group_list.shape[0]
    return dt, index, shape, _row_stride(shape, strides), sa, ss, ga, groups


def _expert_weights(name, w, scales, shape, index):
    """Address and strides of e4m3 weights of `shape`, address of their scales."""
    wshape, strides = _rows_of(name, w, len(shape))
    if w.dtype != _E4M3:
        raise TypeError(f"{name} must have dtype {_E4M3}, got {w.dtype}")
    if wshape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(wshape)}")
    _same_device(name, w, index)
    if scales is None:
        raise ValueError(f"{name} needs its scales")
    sa = _vector(name + "_scales", scales, torch.float32, index, (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1])))
    return w.data_ptr(), _matrix_strides(name, wshape, strides), sa


def _out_rows(out, rows, cols, dtype, index):
    if out is None:
        dt = _TORCH_TO_DT.get(dtype)
        if dt is None:
            raise TypeError(f"y dtype {dtype} is not f16/bf16/f32")
        y = torch.empty((rows, cols), dtype=dtype, device=_device(index))
        return dict(y=y), y.data_ptr(), dt, cols
    y = out["y"]
    shape, strides = _rows_of("y", y, 2)
    if shape != (rows, cols):
        raise ValueError(f"y must be [{rows}, {cols}]")
    _same_device("y", y, index)
    return out, y.data_ptr(), _float_dt("y", y), _row_stride(shape, strides)


@_on_stream
def moe_grouped_matmul(x, weights, weight_scales, group_list=None, *, x_scales=None, num_rows=None,
                       expert_base: int = 0, out_dtype=torch.bfloat16, out: dict | None = None,
                       workspace=None) -> dict:
    """Product of each group's rows with its expert's e4m3 weights [experts,
    out_cols, cols] on the current stream. Returns y [rows, out_cols].

    x: e4m3 rows with x_scales, or f16/bf16/f32 rows, which the call quantizes.
    group_list: int64 [groups, 2] of (expert, rows) on the device (the
    batching's groupList); None: all rows with expert 0. num_rows: the
    batching's actualTokenNum. expert_base: the list's id of weights[0]."""
    dt, index, (rows, K), xst, xsa, xss, ga, groups = _expert_rows(x, x_scales, group_list)
    if weights.dim() != 3 or weights.shape[2] != K:
        raise ValueError("weights must be [experts, out_cols, cols]")
    E, N = weights.shape[0], weights.shape[1]
    wa, wst, wsa = _expert_weights("weights", weights, weight_scales, (E, N, K), index)
    out, ya, ydt, yst = _out_rows(out, rows, N, out_dtype, index)
    wsp, size = None, 0
    if dt != DT_E4M3 or workspace is not None:
        workspace = _workspace(workspace, grouped_matmul_workspace_size(rows, K, dt), index)
        wsp, size = workspace.data_ptr(), workspace.numel()
    st = lib().moe_grouped_matmul(x.data_ptr(), dt, xst, xsa, xss, wa, wst, wsa, ga, groups,
                                  _vector("num_rows", num_rows, torch.int64, index), int(expert_base), rows, E, N, K, ya,
                                  ydt, yst, wsp, size, _raw_stream(index))
    _check(st, "moe_grouped_matmul")
    return out


@functools.lru_cache(maxsize=1024)
def expert_ffn_workspace_size(rows: int, hidden: int, inter: int) -> int:
    ws = ctypes.c_uint64(0)
    _check(lib().moe_expert_ffn_get_workspace_size(rows, hidden, inter, ctypes.byref(ws)),
           "moe_expert_ffn_get_workspace_size")
    return int(ws.value)


@_on_stream
def moe_expert_ffn(x, w13, w13_scales, w2, w2_scales, group_list=None, *, x_scales=None, num_rows=None,
                   expert_base: int = 0, out_dtype=None, out: dict | None = None, workspace=None) -> dict:
    """The experts' network, y = quantized(silu(x W1^T) * (x W3^T)) W2^T, for
    each group's rows on the current stream. Returns y [rows, hidden].

    w13: e4m3 [experts, 2, inter, hidden]; w2: e4m3 [experts, hidden, inter].
    out_dtype: x's by default (bf16 for e4m3 rows). The other arguments are
    moe_grouped_matmul's."""
    dt, index, (rows, H), xst, xsa, xss, ga, groups = _expert_rows(x, x_scales, group_list)
    if w13.dim() != 4 or w13.shape[1] != 2 or w13.shape[3] != H:
        raise ValueError("w13 must be [experts, 2, inter, hidden]")
    E, inter = w13.shape[0], w13.shape[2]
    a13, st13, s13 = _expert_weights("w13", w13, w13_scales, (E, 2, inter, H), index)
    a2, st2, s2 = _expert_weights("w2", w2, w2_scales, (E, H, inter), index)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if dt == DT_E4M3 else x.dtype
    out, ya, ydt, yst = _out_rows(out, rows, H, out_dtype, index)
    workspace = _workspace(workspace, expert_ffn_workspace_size(rows, H, inter), index)
    st = lib().moe_expert_ffn(x.data_ptr(), dt, xst, xsa, xss, a13, st13, s13, a2, st2, s2, ga, groups,
                              _vector("num_rows", num_rows, torch.int64, index), int(expert_base), rows, E, H, inter, ya,
                              ydt, yst, workspace.data_ptr(), workspace.numel(), _raw_stream(index))
    _check(st, "moe_expert_ffn")
    return out


MR_LAYER_SIGMOID, MR_LAYER_KEEP_WEIGHTS = 1, 2


def layer_workspace_size(tokens: int, hidden: int, inter: int, experts: int, topk: int, weight_dtype: int) -> int:
    index = torch.cuda.current_device() if torch.cuda.is_available() else -1
    return _layer_workspace_size(index, tokens, hidden, inter, experts, topk, weight_dtype)


@functools.lru_cache(maxsize=1024)
def _layer_workspace_size(index, tokens, hidden, inter, experts, topk, weight_dtype):
    """Of the current device, whose index is `index`: the shares of the second product go by its SMs."""
    ws = ctypes.c_uint64(0)
    _check(lib().moe_layer_get_workspace_size(tokens, hidden, inter, experts, topk, weight_dtype, ctypes.byref(ws)),
           "moe_layer_get_workspace_size")
    return int(ws.value)


@_on_stream
def moe_layer(x, router, w13, w2, *, topk: int, w13_scales=None, w2_scales=None, score: str = "softmax",
              renormalize: bool = True, routed_scale: float = 1.0, select_bias=None, out: dict | None = None,
              workspace=None) -> dict:
    """A whole mixture-of-experts layer for up to 64 tokens, in one launch on the
    current stream. Returns y [tokens, hidden], expertIds and expertWeights
    [tokens, topk].

    router [experts, hidden]; w13 [experts, 2, inter, hidden] and w2 [experts,
    hidden, inter], e4m3 with their scales or of x's 16-bit dtype. score:
    "softmax" (over all experts) or "sigmoid"; renormalize: a token's weights
    sum to routed_scale. select_bias float32 [experts]: experts are chosen by
    score + select_bias."""
    if score not in ("softmax", "sigmoid"):
        raise ValueError("score must be softmax or sigmoid")
    topk = int(topk)
    (T, H), xstrides = _rows_of("x", x, 2)
    rshape, rstrides = _rows_of("router", router, 2)
    xdt, rdt, index = _float_dt("x", x), _float_dt("router", router), x.get_device()
    _on_current_device("x", index)
    E = rshape[0]
    if rshape[1] != H or w13.dim() != 4 or w13.shape[1] != 2:
        raise ValueError("router must be [experts, hidden], w13 [experts, 2, inter, hidden]")
    _same_device("router", router, index)
    inter = w13.shape[2]
    if w13.dtype == _E4M3:
        wdt = DT_E4M3
        a13, st13, s13 = _expert_weights("w13", w13, w13_scales, (E, 2, inter, H), index)
        a2, st2, s2 = _expert_weights("w2", w2, w2_scales, (E, H, inter), index)
    else:
        wdt = _float_dt("w13", w13)
        if w13.dtype != x.dtype or w2.dtype != x.dtype:
            raise TypeError("16-bit weights must have x's dtype")
        if w13_scales is not None or w2_scales is not None:
            raise ValueError("scales belong to e4m3 weights")
        shape13, strides13 = _rows_of("w13", w13, 4)
        shape2, strides2 = _rows_of("w2", w2, 3)
        if shape13 != (E, 2, inter, H) or shape2 != (E, H, inter):
            raise ValueError("w13 must be [experts, 2, inter, hidden], w2 [experts, hidden, inter]")
        _same_device("w13", w13, index)
        _same_device("w2", w2, index)
        size = w13.element_size()
        st13, st2 = _matrix_strides("w13", shape13, strides13, size), _matrix_strides("w2", shape2, strides2, size)
        a13, a2, s13, s2 = w13.data_ptr(), w2.data_ptr(), None, None
    bias = _vector("select_bias", select_bias, torch.float32, index, (E,))
    # (the size call refuses what the layer does not take before anything is allocated)
    size = _layer_workspace_size(index, T, H, inter, E, topk, wdt)
    if out is None:
        dev = _device(index)
        out = dict(y=torch.empty((T, H), dtype=x.dtype, device=dev),
                   expertIds=torch.empty((T, topk), dtype=torch.int32, device=dev),
                   expertWeights=torch.empty((T, topk), dtype=torch.float32, device=dev))
    y = out["y"]
    yshape, ystrides = _rows_of("y", y, 2)
    if yshape != (T, H) or y.dtype != x.dtype:
        raise ValueError("y must be [tokens, hidden] of x's dtype")
    _same_device("y", y, index)
    ids = _vector("expertIds", out["expertIds"], torch.int32, index, (T, topk))
    weights = _vector("expertWeights", out["expertWeights"], torch.float32, index, (T, topk))
    workspace = _workspace(workspace, size, index)
    flags = (MR_LAYER_SIGMOID if score == "sigmoid" else 0) | (0 if renormalize else MR_LAYER_KEEP_WEIGHTS)
    st = lib().moe_layer(x.data_ptr(), xdt, _row_stride((T, H), xstrides), router.data_ptr(), rdt,
                         _row_stride(rshape, rstrides), bias, a13, wdt, st13, s13, a2, st2, s2, T, H, inter, E, topk,
                         flags, routed_scale, y.data_ptr(), _row_stride(yshape, ystrides), ids, weights,
                         workspace.data_ptr(), workspace.numel(), _raw_stream(index))
    _check(st, "moe_layer")
    return out


def waits_out(reset: bool = False) -> int:
    """Blocks of the expert operators on the current device that gave up a wait, and so left
    results unwritten, since the last reset: 0 on a working device. Waits for the device."""
    n = ctypes.c_uint32(0)
    _check(lib().mr_waits_out(ctypes.byref(n), 1 if reset else 0), "mr_waits_out")
    return int(n.value)


def profile_set_events(events) -> None:
    """Attach cudaEvents (torch.cuda.Event, created with enable_timing) to the
    library's phase markers for this thread; None to detach."""
    if not events:
        _check(lib().mr_profile_set_events(None, 0), "mr_profile_set_events")
        return
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().mr_profile_set_events(arr, len(events)), "mr_profile_set_events")
