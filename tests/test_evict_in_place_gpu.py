"""Evictions that write the new lengths over the old ones."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq,budget", [([3, 400, 64, 0, 200], 64), ([60000, 5, 40000], 3000), ([60000, 9000], 9000),
                                        ([150000, 70000, 12], 7000), ([150000, 7000], 7000)])
def test_lengths_in_place(seq, budget):
    """One CTA, a cluster, and the whole GPU to a request; lengths that stay, lengths that shrink
    (a reader that came late would see them at the budget and keep the first keys), an empty one.
    Against lengths of their own, and against the definition."""
    g = np.random.default_rng(len(seq))
    n = np.asarray(seq, np.int32)
    per = -(-n // 64)
    table = np.zeros((len(seq), int(per.max())), np.int32)
    for b, k in enumerate(per):
        table[b, :k] = per[:b].sum() + np.arange(k)
    per_dst = -(-np.minimum(n, budget) // 64)
    table_dst = np.zeros((len(seq), int(per_dst.max())), np.int32)
    for b, k in enumerate(per_dst):
        table_dst[b, :k] = per.sum() + per_dst[:b].sum() + np.arange(k)
    pages = int(per.sum() + per_dst.sum())
    gen = torch.Generator(device="cuda").manual_seed(budget)
    kv = torch.randint(0, 120, (pages, 64, 576), generator=gen, device="cuda", dtype=torch.uint8)
    weights = g.random((len(seq), int(n.max()))).astype(np.float32)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    w, t, td = dev(weights), dev(table), dev(table_dst)
    want = [ref.keep(weights[b], int(k), budget, 2, 5) for b, k in enumerate(n)]
    for again in range(8):
        lens, kept = dev(n.copy()), torch.empty((len(seq), budget), dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache.evict(w, lens, budget, 2, 5, kv, t, kv, td, kept, lens, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert lens.tolist() == [len(k) for k in want]
        for b, k in enumerate(want):
            assert kept[b].cpu().tolist() == k.tolist() + [-1] * (budget - len(k)), (again, b)
            if len(k) and again == 0:
                src = torch.from_numpy(table[b, k // 64].astype(np.int64) * 64 + k % 64).cuda()
                r = np.arange(len(k))
                dst = torch.from_numpy(table_dst[b, r // 64].astype(np.int64) * 64 + r % 64).cuda()
                rows = kv.view(-1, 576)
                assert torch.equal(rows[src], rows[dst]), b


def test_lengths_out_of_range_in_place():
    """A length that does not fit is reported and becomes 0, in place too."""
    kv = torch.zeros((4, 64, 576), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    lens, kept = torch.tensor([65, 20], dtype=torch.int32, device="cuda"), torch.empty((2, 8), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.evict(torch.rand((2, 64), device="cuda"), lens, 8, 0, 0, kv, table, kv, table + 2, kept, lens, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH
    assert lens.tolist() == [0, 8] and (kept[0] == -1).all() and (kept[1] >= 0).all()


def test_overlaps_are_refused():
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    kv, w = z(4, 64, 576, t=torch.uint8), z(2, 64, t=torch.float32)
    good = dict(weights=w, seq_lens=z(2), budget=8, n_first=0, n_last=0, kv=kv, page_table=z(2, 1), kv_dst=kv,
                page_table_dst=z(2, 1), kept=z(2, 8), seq_lens_dst=z(2))
    lens = z(3)
    for change in (dict(weights_dst=w), dict(seq_lens=lens[:2], seq_lens_dst=lens[1:]), dict(page_table_dst=good["page_table"])):
        with pytest.raises(binding.MlaError):
            cache.evict(**dict(good, **change))
