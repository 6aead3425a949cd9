"""How near the key weights come to 64 bits: bounds on the norm of the whole error, and cases in
which one of the kernel's roundings would stand alone."""
import math

import pytest
import torch

from mla_speculative_verify_gb300 import inputs
from mla_speculative_verify_gb300.decoder import VerifyDecoder

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
D = 576
F32_SCALE = torch.tensor(inputs.SM_SCALE).item()  # what the kernel is given


def cache(kind, n, gen, magnitude=0.5):
    """kv [pages, 64, 576], scales or None, kv_scale, and the keys [n, 576] in 64 bits."""
    pages = -(-n // 64)
    x = torch.randn((pages * 64, D), generator=gen, device="cuda")
    x *= torch.exp(magnitude * torch.randn((pages * 64, 1), generator=gen, device="cuda"))
    if kind == "bf16":
        kv = x.to(torch.bfloat16)
        return kv.view(pages, 64, D), None, 1.0, kv[:n].double()
    if kind == "e4m3":
        codes = (x * 32).clamp(-448, 448).to(F8)
        return codes.view(pages, 64, D), None, 1 / 32, codes[:n].double() / 32
    scales = torch.exp2(torch.randint(-6, -3, (pages, 4), generator=gen, device="cuda").float())
    per_key = scales.repeat_interleave(16, 1).view(-1, 1)
    codes = (x / per_key).clamp(-448, 448).to(F8)
    return codes.view(pages, 64, D), scales, 1.0, (codes.double() * per_key.double())[:n]


def weights(kv, scales, kv_scale, q, lse, n, sm_scale=inputs.SM_SCALE):
    d = VerifyDecoder([n], [q.shape[0]], q.shape[1], "bf16" if kv.dtype == torch.bfloat16 else "fp8")
    w, status = torch.zeros((1, n), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.arange(kv.shape[0], dtype=torch.int32, device="cuda").view(1, -1)
    d.key_weights(q, kv, table, lse, w, sm_scale=sm_scale, kv_scale=kv_scale, kv_scales=scales, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return w[0].double()


def exact_and_error(kind, q, k, n):
    """lse as fp32, the weights [n] in 64 bits for that lse, and the 2-norm of their expected error.

    A score is summed in parts (bf16: nine of four steps of 16 columns; e4m3: three of six steps of
    32, each for both parts of q), and a step cuts what is below the last bit of its sum: anything up
    to a unit, always towards zero, so half a unit on average. What is rounded instead (the parts'
    sum, score - lse, its value to base 2, the rows' sum) is off by half a unit at most in
    either direction: 1/sqrt(12) of a unit in the mean square, and independent. exp2 is off by 2^-22."""
    step, parts, per_step = (16, 9, 1) if kind == "bf16" else (32, 3, 2)
    tokens, heads = q.shape[:2]
    lse = torch.empty((tokens, heads), device="cuda")
    want, err = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    unit = lambda x: torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -100))) - 23)  # noqa: E731
    for i in range(tokens):
        seen = n - tokens + i + 1
        for h in range(heads):
            row = q[i, h].double()
            c = (k[:seen] * row).view(seen, parts, D // parts // step, step).sum(-1)
            cut = unit(c.cumsum(-1)).flatten(1)
            add = unit(c.sum(-1).cumsum(-1)[:, 1:])
            score = torch.sqrt((per_step * cut.sum(1) / 2) ** 2 + (per_step * (cut ** 2).sum(1) + (add ** 2).sum(1)) / 12)
            s = F32_SCALE * c.sum((-1, -2))
            lse[i, h] = torch.logsumexp(s, 0)
            v = s - lse[i, h].double()
            p = torch.exp(v)
            want[:seen] += p
            err[:seen] += p * (F32_SCALE * score + 2 * unit(v) / math.sqrt(12) + 2.0 ** -22)
    return lse, want, (err + math.sqrt(tokens * heads / 12) * 2.0 ** -23 * want).norm()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("n,q,heads", [(4096, 2, 12), (300001, 1, 4), (30000, 4, 96)])
def test_norm_of_the_error(n, q, heads, kind):
    gen = torch.Generator(device="cuda").manual_seed(n)
    kv, scales, kv_scale, k = cache(kind, n, gen)
    queries = torch.randn((q, heads, D), generator=gen, device="cuda").to(torch.bfloat16)
    lse, want, error = exact_and_error(kind, queries, k, n)
    off = (weights(kv, scales, kv_scale, queries, lse, n) - want).norm()
    print(f"{kind} n={n} q={q} heads={heads}: {(off / want.norm()).item():.2e}, expected below {(error / want.norm()).item():.2e}")
    assert error < 2e-5 * want.norm()  # (one sum over all 576 columns would be off by 1.6e-5 to 3e-5)
    assert off <= error


@pytest.mark.parametrize("kind", ["e4m3", "scaled"])
def test_small_entries_of_the_queries(kind):
    """Queries whose largest entry (at a column where the keys are zero) is 512 and whose others are
    0.125 and more, 2^-12 of it: the e4m3 part and the remainder in e5m2 hold all of their bits."""
    n = 4096
    gen = torch.Generator(device="cuda").manual_seed(5)
    kv, scales, kv_scale, k = cache(kind, n, gen)
    kv.view(-1, D).view(torch.uint8)[:, 100] = 0
    k[:, 100] = 0
    x = torch.randn((2, 12, D), generator=gen, device="cuda")
    queries = (x + 0.125 * x.sign()).to(torch.bfloat16)
    queries[..., 100] = 512.0
    lse, want, error = exact_and_error(kind, queries, k, n)
    off = (weights(kv, scales, kv_scale, queries, lse, n) - want).norm()
    print(f"{kind}: {(off / want.norm()).item():.2e}, expected below {(error / want.norm()).item():.2e}")
    assert off <= error


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
def test_large_scores_and_lse(kind):
    """Scores of about 256, all of whose products and sums are whole numbers: what is left is the
    rounding of score - lse at its own size, not at that of the score."""
    n = 5000
    gen = torch.Generator(device="cuda").manual_seed(6)
    pages = -(-n // 64)
    x = torch.randint(-4, 5, (pages * 64, D), generator=gen, device="cuda").float()
    x[:, :256] = 4.0
    q = torch.randint(-2, 3, (1, 1, D), generator=gen, device="cuda").float()
    q[..., :256] = 2.0
    k = x[:n].double()
    scales = None
    if kind == "bf16":
        kv = x.to(torch.bfloat16)
    else:
        kv = x.to(F8)
        if kind == "scaled":
            scales = torch.exp2(torch.randint(0, 2, (pages, 1), generator=gen, device="cuda").float())
            k = k * scales.double().repeat_interleave(64, 0)[:n]
            q = q / 2  # so that the larger scale's scores are those of the other kinds
    s = (k @ q[0, 0].double()) / 8
    lse = torch.logsumexp(s, 0).float()
    assert lse > 200
    v = s - lse.double()
    want = torch.exp(v)
    got = weights(kv.view(pages, 64, D), scales, 1.0, q.to(torch.bfloat16), lse.view(1, 1), n, sm_scale=0.125)
    # score - lse and its value to base 2 round by 2^-24 of themselves, the base's constant by 2^-25; exp2 by 2^-22
    bound = want * (2.5 * 2.0 ** -24 * v.abs() + 2.0 ** -22) + 2.0 ** -126
    assert ((got - want).abs() <= bound).all()
