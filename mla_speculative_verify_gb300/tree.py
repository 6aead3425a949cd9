"""Trees of drafted tokens on torch tensors: ``masks`` turns parents into what the decode of a tree
reads, ``verify`` walks the trees down as far as the target model's distribution accepts them.

Both only check shapes, dtypes and devices and pass raw pointers through to ``mla_tree_masks`` /
``mla_tree_verify``; what they compute is stated in include/mla_decode.h. They enqueue on
``stream`` (default: torch's current stream of the tensors' device) and do not synchronise, so
they can be captured in a CUDA graph. A step of a server:

    tree.masks(parents, cu_nodes, masks, depths, max_nodes)
    decoder = VerifyDecoder(seq_lens, q_lens, num_heads, kv_dtype, tree=True)
    for each layer: cache.append(...); decoder.run(..., tree_masks=masks)
    tree.verify(logits, tokens, parents, cu_nodes, path, out_tokens, accepted, ...)
    cache.commit(kv_of_all_layers, page_table, seq_lens, cu_nodes, path, accepted, new_lens, scales)

A plan is made on the host (0.06 to 2.4 ms, by the batch) for exact lengths: a decoder serves all layers of a
step, the next step needs a new one, and a captured step is good for its lengths alone. Lengths after a
commit are on the device, so a copy to the host comes before the plan.

The keys' weights, where an eviction goes by them, are taken after the commit: ``VerifyDecoder(new_lens,
accepted, ..).key_weights`` with the accepted nodes' rows of q and of the tree's lse, each layer.

Device-side faults (a parent that is not before its node, nodes that do not fit) are OR-ed into
``status``, an int32 tensor, as ``binding.MLA_DEVICE_*`` bits.
"""
from __future__ import annotations

import torch

from . import binding
from .cache import _cuda_index, _ptr, check_tensor, on_device, stream_handle

LOGITS = {torch.bfloat16: binding.MLA_LOGITS_BF16, torch.float32: binding.MLA_LOGITS_FP32}


def _check_rows(name: str, t: torch.Tensor, dtype, rows: int, cols: int, index: int) -> int:
    """A matrix [rows, cols] whose rows are contiguous, at any distance; returns that distance."""
    if t.dim() != 2 or t.shape != (rows, cols) or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} {[rows, cols]}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, the device of the call's tensors")
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or stride < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return stride


def masks(parents: torch.Tensor, cu_nodes: torch.Tensor, out: torch.Tensor, depths: torch.Tensor | None = None,
          max_nodes: int | None = None, status: torch.Tensor | None = None,
          stream: torch.cuda.Stream | None = None) -> None:
    """Visibility words of trees: ``out`` [total, words] int32, bit a of a node's row (bit a % 32
    of word a / 32) set where a is the node or one of its ancestors, and ``depths`` [total] int32,
    its number of ancestors.

    ``parents`` [total] int32 are indices within the request, each before its own node; a negative
    one is a root. Request b's nodes are cu_nodes[b] .. cu_nodes[b + 1] - 1. ``max_nodes`` (default:
    what a row of ``out`` has room for) is at least the largest number of nodes of a request.
    """
    index = _cuda_index(parents)
    total = parents.shape[0] if parents.dim() else 0
    check_tensor("parents", parents, torch.int32, (total,), index)
    batch = cu_nodes.shape[0] - 1 if cu_nodes.dim() else 0
    check_tensor("cu_nodes", cu_nodes, torch.int32, (batch + 1,), index)
    words = out.shape[1] if out.dim() == 2 else 0
    check_tensor("out", out, torch.int32, (total, words), index)
    if total and not words:
        raise ValueError("out must have room for a bit for each node of a request")
    if depths is not None:
        check_tensor("depths", depths, torch.int32, (total,), index)
    if status is not None:
        check_tensor("status", status, torch.int32, (1,), index)
    if max_nodes is None:
        max_nodes = min(32 * words, binding.MLA_TREE_MAX_NODES)
    on_device(index, binding.tree_masks, parents.data_ptr(), cu_nodes.data_ptr(), batch, total, max_nodes,
              out.data_ptr(), words, _ptr(depths), _ptr(status), stream_handle(index, stream))


def verify(logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, cu_nodes: torch.Tensor,
           path: torch.Tensor, out_tokens: torch.Tensor, accepted: torch.Tensor, temperature: torch.Tensor | None = None,
           uniforms: torch.Tensor | None = None, noise: torch.Tensor | None = None,
           draft_logits: torch.Tensor | None = None, max_nodes: int | None = None, status: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None) -> None:
    """Walk each request's tree from its root as far as the target's distribution accepts the
    drafted tokens, and draw the token that follows.

    ``logits`` [total, vocab] bf16 or fp32 (rows may be further apart than vocab) are the target's
    at each node, ``tokens`` [total] int32 the nodes' tokens, ``parents`` and ``cu_nodes`` as in
    ``masks``. ``draft_logits`` (as ``logits``): row u is the distribution that the children of u
    were drawn from; without it the draft counts as certain. ``temperature`` [batch] fp32 (default
    1) divides both; 0 is greedy. ``uniforms`` [total] in [0, 1) decide on the nodes, ``noise``
    [batch, vocab], exponentially distributed, draws the next token; without both all requests are
    greedy. Rows of ``logits`` and ``draft_logits`` are best equally far apart: where they start
    differently between 16-byte boundaries, verification takes up to 1.7 times as long.

    Written: ``path`` [batch, width] int32, the accepted nodes from the root on, then -1;
    ``out_tokens`` [batch, width], the token behind each of them, the new one last, then -1;
    ``accepted`` [batch], nodes on the path, which is also the number of tokens that came out. A
    walk whose path is full ends there. ``max_nodes`` (default: as many as allowed) is at least the
    largest number of nodes of a request.
    """
    index = _cuda_index(logits)
    kind = LOGITS.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise ValueError(f"logits must be bf16 or fp32 [total, vocab], got {logits.dtype} {list(logits.shape)}")
    total, vocab = logits.shape
    stride = _check_rows("logits", logits, logits.dtype, total, vocab, index)
    check_tensor("tokens", tokens, torch.int32, (total,), index)
    check_tensor("parents", parents, torch.int32, (total,), index)
    batch = cu_nodes.shape[0] - 1 if cu_nodes.dim() else 0
    check_tensor("cu_nodes", cu_nodes, torch.int32, (batch + 1,), index)
    width = path.shape[1] if path.dim() == 2 else 0
    check_tensor("path", path, torch.int32, (batch, width), index)
    check_tensor("out_tokens", out_tokens, torch.int32, (batch, width), index)
    check_tensor("accepted", accepted, torch.int32, (batch,), index)
    if temperature is not None:
        check_tensor("temperature", temperature, torch.float32, (batch,), index)
    noise_stride = draft_stride = 0
    if uniforms is not None:
        check_tensor("uniforms", uniforms, torch.float32, (total,), index)
    if noise is not None:
        noise_stride = _check_rows("noise", noise, torch.float32, batch, vocab, index)
    if draft_logits is not None:
        draft_stride = _check_rows("draft_logits", draft_logits, logits.dtype, total, vocab, index)
    if status is not None:
        check_tensor("status", status, torch.int32, (1,), index)
    if max_nodes is None:
        max_nodes = min(total, binding.MLA_TREE_MAX_NODES)
    on_device(index, binding.tree_verify, kind, logits.data_ptr(), stride, _ptr(draft_logits), draft_stride, vocab,
              tokens.data_ptr(), parents.data_ptr(), cu_nodes.data_ptr(), batch, total, max_nodes, _ptr(temperature),
              _ptr(uniforms), _ptr(noise), noise_stride, path.data_ptr(), out_tokens.data_ptr(), width,
              accepted.data_ptr(), _ptr(status), stream_handle(index, stream))
