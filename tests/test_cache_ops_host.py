"""Refusals of the cache operators: every argument is checked on the host before the CUDA runtime
is touched, so no GPU is needed. A case changes one argument of a call that is in order."""
import ctypes

import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref

P = 1 << 20  # a device pointer in all its alignments; nothing is read through it
INVALID, UNSUPPORTED, BUFFER, PLAN = (binding.MLA_ERR_INVALID_ARG, binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_BUFFER,
                                      binding.MLA_ERR_PLAN)


def call(name, good, change):
    args = dict(good, **change)
    return getattr(binding.load(), name)(*args.values())


APPEND = dict(rows=P, total_rows=100, cu_new=P, seq_lens=P, batch=4, max_new=40, kv_cache=P, kv_scales=P, block_tokens=16,
              page_table=P, page_table_stride=8, num_pages=50, status_dev=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=None), INVALID), (dict(cu_new=None), INVALID), (dict(seq_lens=None), INVALID), (dict(kv_cache=None), INVALID),
    (dict(kv_scales=None), INVALID), (dict(page_table=None), INVALID), (dict(rows=P + 8), INVALID),
    (dict(kv_cache=P + 8), INVALID), (dict(cu_new=P + 2), INVALID), (dict(status_dev=P + 1), INVALID),
    (dict(batch=0), INVALID), (dict(batch=65536), INVALID), (dict(total_rows=-1), INVALID), (dict(max_new=-1), INVALID),
    (dict(max_new=101), INVALID), (dict(num_pages=0), INVALID), (dict(page_table_stride=0), INVALID),
    (dict(block_tokens=0), UNSUPPORTED), (dict(block_tokens=3), UNSUPPORTED), (dict(block_tokens=128), UNSUPPORTED),
    (dict(block_tokens=-16), UNSUPPORTED)])
def test_append_refusals(change, code):
    assert call("mla_cache_append", APPEND, change) == code
    assert binding.last_error()


def test_append_of_nothing_is_no_call():
    assert call("mla_cache_append", APPEND, dict(max_new=0, rows=None)) == binding.MLA_OK


EVICT = dict(weights=P, weights_stride=1000, seq_lens=P, batch=3, max_seq=900, budget=100, n_first=4, n_last=16,
             kv_dtype=binding.MLA_KV_FP8_E4M3, kv_cache=P, kv_scales=P, block_tokens=64, page_table=P, page_table_stride=15,
             num_pages=60, kv_cache_dst=P, kv_scales_dst=P, page_table_dst=P, page_table_dst_stride=2, num_pages_dst=10,
             kept=P, seq_lens_dst=P, weights_dst=P, weights_dst_stride=100, workspace=None, workspace_bytes=0, status_dev=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(weights=None), INVALID), (dict(seq_lens=None), INVALID), (dict(kv_cache=None), INVALID),
    (dict(page_table=None), INVALID), (dict(kv_cache_dst=None), INVALID), (dict(page_table_dst=None), INVALID),
    (dict(kept=None), INVALID), (dict(seq_lens_dst=None), INVALID), (dict(kv_scales=None), INVALID),
    (dict(kv_scales_dst=None), INVALID), (dict(kv_cache=P + 4), INVALID), (dict(kept=P + 2), INVALID),
    (dict(batch=0), INVALID), (dict(batch=70000), INVALID), (dict(max_seq=-1), INVALID), (dict(budget=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_last=-1), INVALID), (dict(n_first=85), INVALID),
    (dict(n_first=2**31 - 1, n_last=2**31 - 1), INVALID), (dict(kv_dtype=2), INVALID),
    (dict(kv_dtype=binding.MLA_KV_BF16), INVALID), (dict(weights_stride=899), INVALID), (dict(weights_dst_stride=99), INVALID),
    (dict(page_table_stride=14), INVALID), (dict(page_table_dst_stride=1), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages_dst=0), INVALID), (dict(block_tokens=48), UNSUPPORTED),
    (dict(max_seq=2**21 + 1, weights_stride=2**22, page_table_stride=2**16), UNSUPPORTED),
    (dict(batch=1, max_seq=2**20, weights_stride=2**20, page_table_stride=2**14), BUFFER),
    (dict(batch=1, max_seq=2**20, weights_stride=2**20, page_table_stride=2**14, workspace=P + 16, workspace_bytes=1 << 20), INVALID)])
def test_evict_refusals(change, code):
    assert call("mla_cache_evict", EVICT, change) == code
    assert binding.last_error()


def test_evict_workspace():
    assert binding.cache_evict_workspace(32, 32768) == 0
    assert binding.cache_evict_workspace(1, 1 << 20) > 0
    assert binding.load().mla_cache_evict_workspace(0, 10, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert binding.load().mla_cache_evict_workspace(1, 10, None) == INVALID


def plan(kv, seq=(900, 64), q=(4, 1)):
    buf, _ = binding.plan(seq, q, 12, kv, 152)
    return buf


def weights_args(buf):
    return dict(plan_dev=P, plan_host=buf.ctypes.data, plan_bytes=buf.nbytes, q=P, kv_cache=P, kv_scales=P, block_tokens=16,
                page_table=P, page_table_stride=15, num_pages=60, lse=P, counted=None, sm_scale=0.07, kv_scale=1.0,
                decay=1.0, weights=P, weights_stride=900, workspace=P,
                workspace_bytes=binding.key_weights_workspace(buf), status_dev=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(plan_dev=None), INVALID), (dict(q=None), INVALID), (dict(kv_cache=None), INVALID), (dict(page_table=None), INVALID),
    (dict(lse=None), INVALID), (dict(weights=None), INVALID), (dict(plan_host=None), INVALID), (dict(plan_bytes=10), PLAN),
    (dict(q=P + 8), INVALID), (dict(lse=P + 2), INVALID), (dict(counted=P + 1), INVALID), (dict(block_tokens=5), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(page_table_stride=14), INVALID), (dict(sm_scale=0.0), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(kv_scale=-1.0), INVALID), (dict(decay=float("inf")), INVALID),
    (dict(decay=float("nan")), INVALID), (dict(weights_stride=899), INVALID), (dict(workspace=None), BUFFER),
    (dict(workspace_bytes=1000), BUFFER), (dict(workspace=P + 16), INVALID)])
def test_key_weights_refusals(change, code):
    assert call("mla_key_weights", weights_args(plan(binding.MLA_KV_FP8_E4M3)), change) == code
    assert binding.last_error()


def test_key_weights_of_a_bf16_plan():
    """No scratch, and no block scales."""
    buf = plan(binding.MLA_KV_BF16)
    assert binding.key_weights_workspace(buf) == 0
    assert call("mla_key_weights", weights_args(buf), {}) == INVALID  # it names kv_scales


def test_key_weights_workspace():
    rows = 5 * 12
    assert rows * (1152 + 4) <= binding.key_weights_workspace(plan(binding.MLA_KV_FP8_E4M3)) <= rows * (1152 + 4) + 512
    lib = binding.load()
    n = ctypes.c_size_t()
    assert lib.mla_key_weights_workspace(None, 0, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("change,code", [(dict(kv_scales=None), INVALID), (dict(kv_scales=P + 2), INVALID),
                                         (dict(block_tokens=0), UNSUPPORTED), (dict(block_tokens=65), UNSUPPORTED),
                                         (dict(q=None), INVALID), (dict(sm_scale=-1.0), INVALID)])
def test_decode_scaled_refusals(change, code):
    buf = plan(binding.MLA_KV_FP8_E4M3)
    good = dict(plan_dev=P, plan_host=buf.ctypes.data, plan_bytes=buf.nbytes, q=P, kv_cache=P, kv_scales=P, block_tokens=16,
                page_table=P, page_table_stride=15, num_pages=60, seq_lens=P, q_lens=P, sm_scale=0.07, out=P, lse=P,
                workspace=P, workspace_bytes=1 << 30, status_dev=None, stream=None)
    assert call("mla_decode_run_scaled", good, change) == code
    bf16 = plan(binding.MLA_KV_BF16)
    assert call("mla_decode_run_scaled", good, dict(plan_host=bf16.ctypes.data, plan_bytes=bf16.nbytes)) == INVALID


def test_tensors_have_to_be_on_a_gpu():
    t = torch.zeros
    with pytest.raises(ValueError):
        cache.append(t((4, 576), dtype=torch.bfloat16), t((1, 64, 576), dtype=torch.uint8), t((1, 4)),
                     t((1, 1), dtype=torch.int32), t(1, dtype=torch.int32), t(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        i = torch.int32
        cache.evict(t((1, 64)), t(1, dtype=i), 8, 0, 0, t((1, 64, 576), dtype=torch.bfloat16), t((1, 1), dtype=i),
                    t((1, 64, 576), dtype=torch.bfloat16), t((1, 1), dtype=i), t((1, 8), dtype=i), t(1, dtype=i))
    d = VerifyDecoder([64], [1], 12, "bf16", device="cpu", num_sms=152)
    with pytest.raises(ValueError):
        d.key_weights(t((1, 12, 576), dtype=torch.bfloat16), t((1, 64, 576), dtype=torch.bfloat16),
                      t((1, 1), dtype=torch.int32), t((1, 12)), t((1, 64)))


# ---------------------------------------------------------------- the plain forms themselves
def test_reference_rounding():
    """Every bf16 value against torch's e4m3 cast, and the block scales at their borders."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    assert np.array_equal(ref.to_e4m3(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    assert [ref.block_scale(a) for a in (0.0, 448.0, 448.001, 896.0, 1.0, 1e30)] == [2.0**-60, 1.0, 2.0, 2.0, 2.0**-8, 2.0**60]


def test_reference_keep():
    w = np.array([5, 1, 1, 3, np.nan, 1, -np.inf, 9], np.float32)
    assert ref.keep(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert ref.keep(w, 8, 4, 1, 1).tolist() == [0, 1, 3, 7]
    assert ref.keep(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]


def test_reference_attend_and_weights():
    """The plain decode against the float64 oracle (one scale), and weights that sum to the rows."""
    import oracle

    b = ref.Batch(6, [130, 70], [2, 3], "e4m3", 0, seed=5)
    out, _, lse, _ = ref.attend(b)
    o, l = oracle.decode(b.q.view(torch.int16).numpy().view(np.uint16), b.kv.view(-1, 576).numpy(), oracle.KV_FP8_E4M3,
                         b.kv_scale, b.table, 64, b.seq_lens, b.q_lens, 6, 1.0 / np.sqrt(192.0))
    assert np.abs(out - o).max() < 1e-5 and np.abs(lse - l).max() < 1e-5  # (the oracle's kv_scale is an fp32)
    w, _ = ref.weights(b, lse, 0.0, np.zeros((2, 130)))
    assert np.allclose(w.sum(1), [12, 18])
