"""The paged latent cache's own operators on torch tensors: ``append`` writes rows into a
block-scaled e4m3 cache, ``evict`` keeps the keys with the largest accumulated weight.

Both only check shapes, dtypes and devices and pass raw pointers through to
``mla_cache_append`` / ``mla_cache_evict``; what they compute is stated in
include/mla_decode.h. They enqueue on ``stream`` (default: torch's current stream of the
tensors' device), allocate nothing and do not synchronise, so they can be captured in a CUDA
graph. Device-side faults (lengths that do not fit, pages out of range) are OR-ed into
``status``, an int32 tensor, as ``binding.MLA_DEVICE_*`` bits.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding

PAGE_SIZE = 64
D_QK = 576
_NO_GUARD = contextlib.nullcontext()


def device_guard(device: torch.device):
    """Makes ``device`` current for a library call, which launches on the current device."""
    return _NO_GUARD if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def check_tensor(name: str, t: torch.Tensor, dtype, shape, device) -> None:
    """A contiguous tensor of this dtype (or one of these), shape (None: any) and device."""
    ok = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
    if not ok or t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {dtype} {['any' if s is None else s for s in shape]}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, the device of the call's tensors")


def check_scales(name: str, scales: torch.Tensor, pages: int, device) -> int:
    """Scales [pages, 64 / block_tokens] of a cache; returns block_tokens."""
    check_tensor(name, scales, torch.float32, (pages, None), device)
    per_page = scales.shape[1]
    if per_page < 1 or per_page > PAGE_SIZE or PAGE_SIZE % per_page:
        raise ValueError(f"{name} must hold 1, 2, 4, .. 64 scales a page, got {per_page}")
    return PAGE_SIZE // per_page


def check_status(status: torch.Tensor | None, device) -> None:
    if status is not None:
        check_tensor("status", status, torch.int32, (1,), device)


def _cuda_device(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("the cache operators run on CUDA tensors")
    return t.device


def append(rows: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
           seq_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int, status: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None) -> None:
    """Quantise ``rows`` [total, 576] bf16 into the paged e4m3 cache ``codes`` [pages, 64, 576]
    (uint8 or float8_e4m3fn) with ``scales`` [pages, 64 / block_tokens] fp32, both in place.

    Request b's rows are rows[cu_new[b]:cu_new[b + 1]] (int32, device) and become its last
    tokens: its length with them is seq_lens[b] (int32, device). ``max_new`` is at least the
    largest number of new rows of a request.
    """
    device = _cuda_device(rows)
    check_tensor("rows", rows, torch.bfloat16, (None, D_QK), device)
    check_tensor("codes", codes, (torch.uint8, torch.float8_e4m3fn), (None, PAGE_SIZE, D_QK), device)
    block = check_scales("scales", scales, codes.shape[0], device)
    check_tensor("page_table", page_table, torch.int32, (None, None), device)
    batch = page_table.shape[0]
    check_tensor("seq_lens", seq_lens, torch.int32, (batch,), device)
    check_tensor("cu_new", cu_new, torch.int32, (batch + 1,), device)
    check_status(status, device)
    st = stream if stream is not None else torch.cuda.current_stream(device)
    with device_guard(device):
        binding.cache_append(rows.data_ptr(), rows.shape[0], cu_new.data_ptr(), seq_lens.data_ptr(), batch, max_new,
                             codes.data_ptr(), scales.data_ptr(), block, page_table.data_ptr(), page_table.shape[1],
                             codes.shape[0], None if status is None else status.data_ptr(), st.cuda_stream)


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
    ``kv_dst`` may be ``kv`` itself; the new pages must not be among the old ones. ``max_seq``
    (default: what ``weights`` and ``page_table`` have room for) is at least the longest length.
    """
    device = _cuda_device(weights)
    check_tensor("weights", weights, torch.float32, (None, None), device)
    batch = weights.shape[0]
    if kv.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise ValueError("kv must be bf16, or e4m3 codes as uint8 or float8_e4m3fn")
    bf16 = kv.dtype == torch.bfloat16
    check_tensor("kv", kv, kv.dtype, (None, PAGE_SIZE, D_QK), device)
    check_tensor("kv_dst", kv_dst, torch.bfloat16 if bf16 else (torch.uint8, torch.float8_e4m3fn),
                 (None, PAGE_SIZE, D_QK), device)
    if (scales is None) != (scales_dst is None):
        raise ValueError("scales and scales_dst must both be given, or neither")
    block = 0
    if scales is not None:
        block = check_scales("scales", scales, kv.shape[0], device)
        if check_scales("scales_dst", scales_dst, kv_dst.shape[0], device) != block:
            raise ValueError("scales and scales_dst must have the same block_tokens")
    check_tensor("page_table", page_table, torch.int32, (batch, None), device)
    check_tensor("page_table_dst", page_table_dst, torch.int32, (batch, None), device)
    check_tensor("seq_lens", seq_lens, torch.int32, (batch,), device)
    check_tensor("seq_lens_dst", seq_lens_dst, torch.int32, (batch,), device)
    check_tensor("kept", kept, torch.int32, (batch, budget), device)
    if weights_dst is not None:
        check_tensor("weights_dst", weights_dst, torch.float32, (batch, None), device)
    check_status(status, device)
    if max_seq is None:
        max_seq = min(weights.shape[1], PAGE_SIZE * page_table.shape[1])
    st = stream if stream is not None else torch.cuda.current_stream(device)
    with device_guard(device):
        binding.cache_evict(weights.data_ptr(), weights.shape[1], seq_lens.data_ptr(), batch,
                            max_seq, budget, n_first, n_last,
                            binding.MLA_KV_BF16 if bf16 else binding.MLA_KV_FP8_E4M3, kv.data_ptr(),
                            None if scales is None else scales.data_ptr(), block, page_table.data_ptr(),
                            page_table.shape[1], kv.shape[0], kv_dst.data_ptr(),
                            None if scales_dst is None else scales_dst.data_ptr(), page_table_dst.data_ptr(),
                            page_table_dst.shape[1], kv_dst.shape[0], kept.data_ptr(), seq_lens_dst.data_ptr(),
                            None if weights_dst is None else weights_dst.data_ptr(),
                            0 if weights_dst is None else weights_dst.shape[1],
                            None if status is None else status.data_ptr(), st.cuda_stream)
