"""The paged latent cache's own operators on torch tensors: ``append`` writes rows into a
block-scaled e4m3 cache, ``evict`` keeps the keys with the largest accumulated weight.

Both only check shapes, dtypes and devices and pass raw pointers through to
``mla_cache_append`` / ``mla_cache_evict``; what they compute is stated in
include/mla_decode.h. They enqueue on ``stream`` (default: torch's current stream of the
tensors' device) and do not synchronise, so they can be captured in a CUDA graph; what scratch
``evict`` needs comes from torch's allocator, call by call. Device-side faults (lengths that do not
fit, pages out of range) are OR-ed into ``status``, an int32 tensor, as ``binding.MLA_DEVICE_*``
bits.
"""
from __future__ import annotations

import torch

from . import binding

PAGE_SIZE = 64
D_QK = 576
ROW = (PAGE_SIZE, D_QK)
E4M3 = (torch.uint8, torch.float8_e4m3fn)  # a cache of e4m3 codes comes as either


def stream_handle(index: int, stream: torch.cuda.Stream | None) -> int:
    """The cudaStream_t of ``stream``, or of torch's current stream of device ``index``."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def on_device(index: int, call, *args) -> None:
    """A library call, which launches on the current device, with device ``index`` current."""
    if torch.cuda.current_device() == index:
        call(*args)
    else:
        with torch.cuda.device(index):
            call(*args)


def scratch_bytes(count: int, index: int, stream: torch.cuda.Stream | None) -> torch.Tensor:
    """Scratch for one call on ``stream`` from torch's allocator, which hands it out again only to
    later work of that stream (or, in a capture, of that graph): no two calls share any."""
    if stream is None:
        return torch.empty(count, dtype=torch.uint8, device=index)
    with torch.cuda.stream(stream):
        return torch.empty(count, dtype=torch.uint8, device=index)


def check_tensor(name: str, t: torch.Tensor, dtype, shape, index: int) -> None:
    """A contiguous tensor of this dtype (or one of these) and shape on CUDA device ``index``. (A
    call checks up to a dozen tensors, so the case that all is well is one test.)"""
    if (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)) and t.shape == shape \
            and t.get_device() == index and t.is_contiguous():
        return
    if t.shape != shape or not (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, the device of the call's tensors")
    raise ValueError(f"{name} must be contiguous")


def check_scales(name: str, scales: torch.Tensor, pages: int, index: int) -> int:
    """Scales [pages, 64 / block_tokens] of a cache; returns block_tokens."""
    check_tensor(name, scales, torch.float32, (pages, *scales.shape[1:2]), index)
    per_page = scales.shape[1] if scales.dim() == 2 else 0
    if per_page < 1 or PAGE_SIZE % per_page:
        raise ValueError(f"{name} must hold 1, 2, 4, .. 64 scales a page, got {list(scales.shape)}")
    return PAGE_SIZE // per_page


def check_table(name: str, table: torch.Tensor, batch: int, index: int) -> int:
    """A page table [batch, stride] int32; returns its stride."""
    if table.dim() != 2:
        raise ValueError(f"{name} must be int32 [batch, stride], got {list(table.shape)}")
    stride = table.shape[1]
    check_tensor(name, table, torch.int32, (batch, stride), index)
    return stride


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _cuda_index(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("the cache operators run on CUDA tensors")
    return index


def append(rows: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
           seq_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int, status: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None) -> None:
    """Quantise ``rows`` [total, 576] bf16 into the paged e4m3 cache ``codes`` [pages, 64, 576]
    (uint8 or float8_e4m3fn) with ``scales`` [pages, 64 / block_tokens] fp32, both in place.

    Request b's rows are rows[cu_new[b]:cu_new[b + 1]] (int32, device) and become its last
    tokens: its length with them is seq_lens[b] (int32, device). ``max_new`` is at least the
    largest number of new rows of a request; with 0 the call does nothing.

    A block's scale never shrinks while it holds older tokens, so the scale that a rejected draft
    asked for stays with the older tokens of its block. Where key weights are added up, the
    caller zeroes the places of the new tokens.
    """
    index = _cuda_index(rows)
    check_tensor("rows", rows, torch.bfloat16, rows.shape[:1] + (D_QK,), index)
    pages = codes.shape[0] if codes.dim() else 0
    check_tensor("codes", codes, E4M3, (pages, *ROW), index)
    block = check_scales("scales", scales, pages, index)
    batch = page_table.shape[0] if page_table.dim() else 0
    stride = check_table("page_table", page_table, batch, index)
    check_tensor("seq_lens", seq_lens, torch.int32, (batch,), index)
    check_tensor("cu_new", cu_new, torch.int32, (batch + 1,), index)
    if status is not None:
        check_tensor("status", status, torch.int32, (1,), index)
    on_device(index, binding.cache_append, rows.data_ptr(), rows.shape[0], cu_new.data_ptr(), seq_lens.data_ptr(), batch,
              max_new, codes.data_ptr(), scales.data_ptr(), block, page_table.data_ptr(), stride, pages, _ptr(status),
              stream_handle(index, stream))


def evict(weights: torch.Tensor, seq_lens: torch.Tensor, budget: int, n_first: int, n_last: int, kv: torch.Tensor,
          page_table: torch.Tensor, kv_dst: torch.Tensor, page_table_dst: torch.Tensor, kept: torch.Tensor,
          seq_lens_dst: torch.Tensor, weights_dst: torch.Tensor | None = None, scales: torch.Tensor | None = None,
          scales_dst: torch.Tensor | None = None, max_seq: int | None = None, status: torch.Tensor | None = None,
          stream: torch.cuda.Stream | None = None) -> None:
    """Shorten every request to at most ``budget`` keys: its first ``n_first``, its last
    ``n_last`` and those with the largest ``weights`` [batch, >= max_seq] (fp32); move them in
    order from the pages of ``page_table`` in ``kv`` [pages, 64, 576] (bf16, or e4m3 as uint8 or
    float8_e4m3fn, with ``scales`` if block-scaled) to those of ``page_table_dst`` in ``kv_dst``.

    Written: ``kept`` [batch, budget] int32 (indices in order, then -1), ``seq_lens_dst``
    [batch] int32, ``weights_dst`` [batch, >= new length] fp32 if given, and the new pages.
    ``kv_dst`` may be ``kv`` itself and ``seq_lens_dst`` may be ``seq_lens``; ``weights_dst`` must
    not overlap ``weights``, and the new pages must not be among the old ones. A request that is
    short enough already moves to its new pages too. Entries of ``weights_dst`` behind the new
    length are left as they are; zero them before tokens are appended there. ``max_seq``
    (default: what ``weights`` and ``page_table`` have room for) is at least the longest length.
    """
    index = _cuda_index(weights)
    if weights.dim() != 2:
        raise ValueError(f"weights must be fp32 [batch, stride], got {list(weights.shape)}")
    batch, w_stride = weights.shape
    check_tensor("weights", weights, torch.float32, (batch, w_stride), index)
    bf16 = kv.dtype == torch.bfloat16
    kind = torch.bfloat16 if bf16 else E4M3
    pages, pages_dst = kv.shape[0] if kv.dim() else 0, kv_dst.shape[0] if kv_dst.dim() else 0
    check_tensor("kv", kv, kind, (pages, *ROW), index)
    check_tensor("kv_dst", kv_dst, kind, (pages_dst, *ROW), index)
    block = 0
    if scales is not None and scales_dst is not None:
        block = check_scales("scales", scales, pages, index)
        if check_scales("scales_dst", scales_dst, pages_dst, index) != block:
            raise ValueError("scales and scales_dst must have the same block_tokens")
    elif scales is not None or scales_dst is not None:
        raise ValueError("scales and scales_dst must both be given, or neither")
    stride = check_table("page_table", page_table, batch, index)
    stride_dst = check_table("page_table_dst", page_table_dst, batch, index)
    check_tensor("seq_lens", seq_lens, torch.int32, (batch,), index)
    check_tensor("seq_lens_dst", seq_lens_dst, torch.int32, (batch,), index)
    check_tensor("kept", kept, torch.int32, (batch, budget), index)
    wd_stride = 0
    if weights_dst is not None:
        wd_stride = weights_dst.shape[1] if weights_dst.dim() == 2 else 0
        check_tensor("weights_dst", weights_dst, torch.float32, (batch, wd_stride), index)
    if status is not None:
        check_tensor("status", status, torch.int32, (1,), index)
    if max_seq is None:
        max_seq = min(w_stride, PAGE_SIZE * stride)
    need = binding.cache_evict_workspace(batch, max_seq)
    scratch = scratch_bytes(need, index, stream) if need else None
    on_device(index, binding.cache_evict, weights.data_ptr(), w_stride, seq_lens.data_ptr(), batch, max_seq, budget,
              n_first, n_last, binding.MLA_KV_BF16 if bf16 else binding.MLA_KV_FP8_E4M3, kv.data_ptr(), _ptr(scales),
              block, page_table.data_ptr(), stride, pages, kv_dst.data_ptr(), _ptr(scales_dst),
              page_table_dst.data_ptr(), stride_dst, pages_dst, kept.data_ptr(), seq_lens_dst.data_ptr(),
              _ptr(weights_dst), wd_stride, _ptr(scratch), need, _ptr(status), stream_handle(index, stream))
