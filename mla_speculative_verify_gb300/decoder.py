"""Torch-facing convenience wrapper around the C entry points.

``VerifyDecoder`` plans once for a batch shape (seq_lens, q_lens, H, cache dtype),
keeps the plan bytes on the device together with the split-KV workspace, and
enqueues ``mla_decode_run`` on torch device tensors. It only checks shapes,
dtypes and devices and passes raw pointers through; the decode itself runs in the
library's kernels.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import binding
from .cache import E4M3, check_scales, check_table, check_tensor, on_device, scratch_bytes, stream_handle

KV_DTYPES = {"bf16": binding.MLA_KV_BF16, "fp8": binding.MLA_KV_FP8_E4M3}
SM_SCALE = 1.0 / math.sqrt(192.0)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


class VerifyDecoder:
    def __init__(self, seq_lens, q_lens, num_heads: int, kv_dtype: str, device="cuda", num_sms: int | None = None,
                 options: binding.PlanOptions | None = None, tree: bool = False):
        """``tree``: plan for trees of verify tokens (``run`` with ``tree_masks``), whose sizes need
        no handy divisors; such a decoder runs chains as well."""
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        if kv_dtype not in KV_DTYPES:
            raise ValueError(f"kv_dtype must be one of {list(KV_DTYPES)}")
        self.kv_dtype = kv_dtype
        self.num_heads = int(num_heads)
        self.seq_lens = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
        self.q_lens = np.ascontiguousarray(np.asarray(q_lens, dtype=np.int32))
        if num_sms is None:
            num_sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.num_sms = int(num_sms)
        if self.device.type == "cuda":
            # clusters of two CTAs the device runs at once, for plans that use them
            opts = binding.PlanOptions() if options is None else options
            if opts.pair_slots == 0 and (kv_dtype == "bf16" or tree):
                opts = binding.PlanOptions.from_buffer_copy(opts)
                opts.pair_slots = binding.device_pair_slots(self.device.index)
            options = opts
        self.plan_host, self.workspace_bytes = binding.plan(self.seq_lens, self.q_lens, self.num_heads,
                                                            KV_DTYPES[kv_dtype], self.num_sms, options, tree=tree)
        self.info = binding.plan_info(self.plan_host)
        self._plan_host_ptr = self.plan_host.ctypes.data
        self.weights_workspace_bytes = binding.key_weights_workspace(self.plan_host)
        # the plan runs on clusters of two CTAs (PlanHeader.cta_pair, the int32 at byte 64)
        self.cta_pair = bool(int(self.plan_host[64:68].view(np.int32)[0]))
        self.plan_dev = torch.from_numpy(self.plan_host).to(self.device)
        self.workspace = (torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
                          if self.workspace_bytes else None)
        self.seq_lens_dev = torch.from_numpy(self.seq_lens).to(self.device)
        self.q_lens_dev = torch.from_numpy(self.q_lens).to(self.device)
        self.total_q = int(self.q_lens.sum())
        self._last_run_saw_tree = False

    def run(self, q: torch.Tensor, kv_cache: torch.Tensor, page_table: torch.Tensor, out: torch.Tensor,
            lse: torch.Tensor | None = None, sm_scale: float = SM_SCALE, kv_scale: float = 1.0,
            status: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
            seq_lens_dev: torch.Tensor | None = None, q_lens_dev: torch.Tensor | None = None,
            kv_scales: torch.Tensor | None = None, tree_masks: torch.Tensor | None = None) -> None:
        """The verify decode. With ``kv_scales`` [pages, 64 / block_tokens] fp32 the e4m3 cache
        is block-scaled: code * scale of its block (``kv_scale`` is then not used). A decoder's
        calls share its workspace: those that may overlap (on two streams, or in two graphs that
        are replayed at once) need a decoder each. ``tree_masks`` [total_q, words] int32, as
        ``tree.masks`` writes them: verify token i sees the keys before the request's verify tokens,
        and of those the ones whose bit is set (a row that sees none gets zeros)."""
        if tree_masks is not None:
            self._run_tree(q, kv_cache, page_table, out, lse, sm_scale, kv_scale, status, stream, seq_lens_dev, q_lens_dev,
                           kv_scales, tree_masks)
            return
        H = self.num_heads
        want_kv = torch.bfloat16 if self.kv_dtype == "bf16" else torch.uint8
        if q.dtype != torch.bfloat16 or tuple(q.shape) != (self.total_q, H, 576) or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous bf16 tensor of shape {(self.total_q, H, 576)}")
        if kv_cache.dtype not in (want_kv, torch.float8_e4m3fn) or kv_cache.shape[-1] != 576 or not kv_cache.is_contiguous():
            raise ValueError(f"kv_cache must be contiguous {want_kv} [..., 576]")
        if self.kv_dtype == "bf16" and kv_cache.dtype != torch.bfloat16:
            raise ValueError("a bf16 plan needs a bf16 cache")
        rows = kv_cache.numel() // 576
        if rows % 64:
            raise ValueError("kv_cache must hold whole 64-row pages")
        if out.dtype != torch.bfloat16 or tuple(out.shape) != (self.total_q, H, 512) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bf16 tensor of shape {(self.total_q, H, 512)}")
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (self.total_q, H)):
            raise ValueError("lse must be float32 [total_q, H]")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 [batch, stride] tensor")
        for t in (q, kv_cache, out, page_table, lse, status):
            if t is not None and t.device != self.device:
                raise ValueError("all tensors must be on the decoder's device")
        if kv_scales is not None:
            if self.kv_dtype != "fp8":
                raise ValueError("block scales belong to an fp8 cache")
            index = self.device.index
            block = check_scales("kv_scales", kv_scales, rows // 64, index)
            check_table("page_table", page_table, self.seq_lens.shape[0], index)
            on_device(index, binding.run_scaled, self.plan_dev.data_ptr(), self._plan_host_ptr, self.plan_host.nbytes,
                      q.data_ptr(), kv_cache.data_ptr(), kv_scales.data_ptr(), block, page_table.data_ptr(),
                      page_table.shape[1], rows // 64,
                      (seq_lens_dev if seq_lens_dev is not None else self.seq_lens_dev).data_ptr(),
                      (q_lens_dev if q_lens_dev is not None else self.q_lens_dev).data_ptr(),
                      sm_scale, out.data_ptr(), _ptr(lse), _ptr(self.workspace), self.workspace_bytes,
                      _ptr(status), stream_handle(index, stream))
            self._last_run_saw_tree = False
            return
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        binding.run(self.plan_dev.data_ptr(), self.plan_host, q.data_ptr(), kv_cache.data_ptr(), page_table.data_ptr(),
                    page_table.shape[1], rows // 64,
                    (seq_lens_dev if seq_lens_dev is not None else self.seq_lens_dev).data_ptr(),
                    (q_lens_dev if q_lens_dev is not None else self.q_lens_dev).data_ptr(),
                    sm_scale, kv_scale, out.data_ptr(), _ptr(lse), _ptr(self.workspace), self.workspace_bytes,
                    _ptr(status), st.cuda_stream)
        self._last_run_saw_tree = False

    def _run_tree(self, q, kv_cache, page_table, out, lse, sm_scale, kv_scale, status, stream, seq_lens_dev, q_lens_dev,
                  kv_scales, tree_masks) -> None:
        """``run`` with ``tree_masks``."""
        H, index, batch, total = self.num_heads, self.device.index, self.seq_lens.shape[0], self.total_q
        check_tensor("q", q, torch.bfloat16, (total, H, 576), index)
        shape = kv_cache.shape
        if shape[-1:] != (576,) or kv_cache.numel() % (64 * 576):
            raise ValueError("kv_cache must hold whole 64-row pages [..., 576]")
        pages = kv_cache.numel() // (64 * 576)
        check_tensor("kv_cache", kv_cache, torch.bfloat16 if self.kv_dtype == "bf16" else E4M3, shape, index)
        check_tensor("out", out, torch.bfloat16, (total, H, 512), index)
        if lse is not None:
            check_tensor("lse", lse, torch.float32, (total, H), index)
        block = 0
        if kv_scales is not None:
            if self.kv_dtype != "fp8":
                raise ValueError("block scales belong to an fp8 cache")
            block = check_scales("kv_scales", kv_scales, pages, index)
        stride = check_table("page_table", page_table, batch, index)
        words = tree_masks.shape[1] if tree_masks.dim() == 2 else 0
        check_tensor("tree_masks", tree_masks, torch.int32, (total, words), index)
        if status is not None:
            check_tensor("status", status, torch.int32, (1,), index)
        if seq_lens_dev is None:
            seq_lens_dev = self.seq_lens_dev
        else:
            check_tensor("seq_lens_dev", seq_lens_dev, torch.int32, (batch,), index)
        if q_lens_dev is None:
            q_lens_dev = self.q_lens_dev
        else:
            check_tensor("q_lens_dev", q_lens_dev, torch.int32, (batch,), index)
        on_device(index, binding.run_tree, self.plan_dev.data_ptr(), self._plan_host_ptr, self.plan_host.nbytes, q.data_ptr(),
                  kv_cache.data_ptr(), _ptr(kv_scales), block, page_table.data_ptr(), stride, pages,
                  seq_lens_dev.data_ptr(), q_lens_dev.data_ptr(), tree_masks.data_ptr(), words, sm_scale, kv_scale,
                  out.data_ptr(), _ptr(lse), _ptr(self.workspace), self.workspace_bytes, _ptr(status),
                  stream_handle(index, stream))
        self._last_run_saw_tree = True

    def key_weights(self, q: torch.Tensor, kv_cache: torch.Tensor, page_table: torch.Tensor, lse: torch.Tensor,
                    weights: torch.Tensor, decay: float = 1.0, counted: torch.Tensor | None = None,
                    sm_scale: float = SM_SCALE, kv_scale: float = 1.0, kv_scales: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> None:
        """After ``run``: add to ``weights`` [batch, >= longest request] fp32 what every cached
        key received, weights = decay * weights + sum over rows of exp(score - lse), with the
        ``lse`` that ``run`` wrote. ``counted`` [batch] int32: only the first so many verify
        tokens of a request count (the accepted ones). A new token's sum starts from what
        ``weights`` holds in its place, so zero the places that an append fills. Its scratch comes from torch's allocator,
        call by call, so calls on several streams or captured in several graphs share none.

        The rows count as a chain: row i gives weight to every key up to its own place. So it is
        refused after a ``run`` with ``tree_masks``, whose ``lse`` does not hold the other branches
        of a tree. The weights of a tree's accepted path are those of the committed chain:
        after ``cache.commit`` a decoder of the new lengths and the accepted counts takes the
        accepted nodes' rows of q and of the tree's ``lse`` (see ``tree``)."""
        if self.device.type != "cuda":
            raise ValueError("key_weights runs on a CUDA device")
        if self._last_run_saw_tree:
            raise ValueError("the last run took tree_masks: its lse holds what a tree's rows see, and key_weights counts a chain's "
                             "rows; call it on the committed chain")
        H, batch, index = self.num_heads, self.seq_lens.shape[0], self.device.index
        check_tensor("q", q, torch.bfloat16, (self.total_q, H, 576), index)
        if kv_cache.shape[-1:] != (576,) or kv_cache.numel() % (64 * 576):
            raise ValueError("kv_cache must hold whole 64-row pages [..., 576]")
        pages = kv_cache.numel() // (64 * 576)
        check_tensor("kv_cache", kv_cache, torch.bfloat16 if self.kv_dtype == "bf16" else E4M3, kv_cache.shape, index)
        block = 0 if kv_scales is None else check_scales("kv_scales", kv_scales, pages, index)
        stride = check_table("page_table", page_table, batch, index)
        check_tensor("lse", lse, torch.float32, (self.total_q, H), index)
        w_stride = weights.shape[1] if weights.dim() == 2 else 0
        check_tensor("weights", weights, torch.float32, (batch, w_stride), index)
        if counted is not None:
            check_tensor("counted", counted, torch.int32, (batch,), index)
        if status is not None:
            check_tensor("status", status, torch.int32, (1,), index)
        need = self.weights_workspace_bytes
        scratch = scratch_bytes(need, index, stream) if need else None
        on_device(index, binding.key_weights, self.plan_dev.data_ptr(), self._plan_host_ptr, self.plan_host.nbytes,
                  q.data_ptr(), kv_cache.data_ptr(), _ptr(kv_scales), block, page_table.data_ptr(), stride, pages,
                  lse.data_ptr(), _ptr(counted), sm_scale, kv_scale, decay, weights.data_ptr(), w_stride, _ptr(scratch),
                  need, _ptr(status), stream_handle(index, stream))
