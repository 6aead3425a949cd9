"""What the documentation says of a server's steps beyond a single call: rejected drafts, places that
new tokens take, requests that are short already."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import cache
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("block", [1, 16, 64])
def test_a_rejected_draft(block):
    """A prompt, a draft whose first row is accepted and whose others are larger, the next draft over those."""
    g = torch.Generator().manual_seed(block)
    prompt, draft, second = (torch.randn((n, 576), generator=g).to(torch.bfloat16) for n in (70, 4, 4))
    draft[1:] *= 64  # (the first one is accepted)
    table = np.array([[1, 0]], np.int32)
    values, want_s = np.zeros((2, 64, 576)), np.ones((2, 64 // block))
    codes, scales = torch.zeros((2, 64, 576), dtype=torch.uint8, device="cuda"), torch.ones((2, 64 // block), device="cuda")
    for rows, end in ((prompt, 70), (draft, 74), (second, 75)):
        n = rows.shape[0]
        ref.append(rows, values, want_s, table, [end], [0, n], block)
        cache.append(rows.cuda(), codes, scales, dev(table), dev(np.array([end], np.int32)),
                     dev(np.array([0, n], np.int32)), n)
    assert np.array_equal(codes.cpu().view(F8).double().numpy(), values)
    assert np.array_equal(scales.cpu().double().numpy(), want_s)
    if block > 1:  # the scale that the rejected rows asked for stays with the older tokens
        assert want_s[0, 6 // block] >= 16 * want_s[1, 0]


def test_an_append_of_nothing():
    """max_new = 0 does nothing, whatever the lengths say; so do requests without new rows."""
    rows = torch.randn((8, 576), device="cuda").to(torch.bfloat16)
    codes, scales = torch.full((2, 64, 576), 7, dtype=torch.uint8, device="cuda"), torch.full((2, 4), 3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.append(rows, codes, scales, i32([[0], [1]]), i32([8, 0]), i32([0, 8, 8]), 0, status)
    cache.append(rows, codes, scales, i32([[0], [1]]), i32([8, 0]), i32([3, 3, 3]), 8, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (codes == 7).all() and (scales == 3.0).all()


def test_places_of_new_tokens():
    """A sum starts from what is in its place: zeroed there, it is the sum of a fresh row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randn((2, 64, 576), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    q = torch.randn((2, 12, 576), generator=g, device="cuda").to(torch.bfloat16)
    d = VerifyDecoder([100], [2], 12, "bf16")
    out, lse = torch.empty((2, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 12), device="cuda")
    d.run(q, kv, table, out, lse)
    fresh, used = torch.zeros((1, 128), device="cuda"), torch.zeros((1, 128), device="cuda")
    used[:, 98:] = 5.0
    d.key_weights(q, kv, table, lse, fresh, decay=0.5)
    stale = used.clone()
    d.key_weights(q, kv, table, lse, stale, decay=0.5)
    used[:, 98:100] = 0.0
    d.key_weights(q, kv, table, lse, used, decay=0.5)
    torch.cuda.synchronize()
    assert torch.equal(used[:, :100], fresh[:, :100]) and (used[:, 100:] == 5.0).all()
    assert torch.allclose(stale[:, 98:100], fresh[:, 98:100] + 2.5)


def test_short_requests_move_too():
    g = torch.Generator(device="cuda").manual_seed(4)
    kv = torch.randn((4, 64, 576), generator=g, device="cuda").to(torch.bfloat16)
    before = kv.clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, kept, status = i32([70]), torch.empty((1, 80), dtype=torch.int32, device="cuda"), i32([0])
    w_dst = torch.full((1, 80), -1.0, device="cuda")
    w = torch.rand((1, 128), generator=g, device="cuda")
    cache.evict(w, lens, 80, 1, 1, kv, i32([[0, 1]]), kv, i32([[3, 2]]), kept, lens, w_dst, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lens.item() == 70
    assert torch.equal(kv[3], before[0]) and torch.equal(kv[2, :6], before[1, :6]) and torch.equal(kv[2, 6:], before[2, 6:])
    assert torch.equal(w_dst[0, :70], w[0, :70]) and (w_dst[0, 70:] == -1.0).all()
