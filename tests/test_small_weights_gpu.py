"""The decodes over an e4m3 cache where small softmax weights count: one strong key before a long,
flat rest that is together as heavy as it, in one unit (one CTA goes through all the keys)."""
import pytest
import torch

from mla_speculative_verify_gb300 import binding, inputs
from mla_speculative_verify_gb300.decoder import VerifyDecoder

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
D, DV = 576, 512


def strong_and_flat(n, rest, kind, seed):
    """Codes [pages, 64, 576], per-key scales (fp64), the scale argument, queries [2, 6, 576]: key 0
    gets a weight between 0.2 and 0.8 that goes by the row, every other key about the same small one
    (rest "equal": exactly the same; "spread": times exp(0.5 N(0, 1))). Only the last 64 columns,
    which hold no values, make the scores."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-n // 64)
    x = torch.randn((pages * 64, D), generator=g, device="cuda")
    x[:, :DV] += 0.7 * torch.randn(DV, generator=g, device="cuda")  # values with something in common
    if rest == "equal":
        x[:, DV:] = 0.0
    x[0, DV:] = 0.0
    if kind == "one":
        arg, scales = 2.0 ** -7, None
        per_key = torch.full((pages * 64,), arg, device="cuda")
    else:
        arg = 1.0
        scales = torch.exp2(torch.randint(-7, -4, (pages, 4), generator=g, device="cuda").float())
        per_key = scales.repeat_interleave(16, 1).view(-1)
    if rest == "spread":
        x[:, DV] = 0.0  # key 0's alone; the other 63 columns spread the rest
    x[0, DV] = 2.0
    codes = (x / per_key[:, None]).clamp(-448, 448).to(F8)
    strong = torch.linspace(0.2, 0.8, 12, device="cuda").view(2, 6)
    want = torch.log(n * strong / (1 - strong)) + (0.125 if rest == "spread" else 0.0)  # key 0's score
    q = 0.0625 * torch.randn((2, 6, D), generator=g, device="cuda") / inputs.SM_SCALE
    q[..., :DV] = 0.0
    q[..., DV] = want / (inputs.SM_SCALE * 2.0)
    return codes.view(pages, 64, D), per_key.double(), arg, scales, q.to(torch.bfloat16)


def exact(codes, per_key, q, n):
    """out [2, 6, 512] in 64 bits and a bound of the norm of each row's error."""
    k = codes.view(-1, D)[:n].double() * per_key[:n, None]
    out = torch.empty((2, 6, DV), dtype=torch.float64, device="cuda")
    bound = torch.empty((2, 6), dtype=torch.float64, device="cuda")
    for i in range(2):
        seen = n - 1 + i
        rows = q[i].double()
        p = torch.softmax(inputs.SM_SCALE * (rows @ k[:seen].T), 1)
        v = k[:seen, :DV]
        out[i] = p @ v
        # P is held to 2^-8 of itself and the output rounds to 2^-8. A small P rounds up or down, with
        # the odds that make it right on average, by less than a step of 2^-2 of itself: such an
        # error's standard deviation is at most half a step. Six of the sum's.
        term = p * per_key[:seen]
        small = p * (term < 2.0 ** -10 * term.amax(1, keepdim=True))
        noise = 6 * 2.0 ** -3 * ((small ** 2) @ (v ** 2).sum(1)).sqrt()
        # scores: 576 fp32 sums that may cut, 2^-23 of the magnitudes each; q in two e4m3 parts, 2^-17
        # of the row's largest. Both ends of the softmax see them.
        ds = 2 * inputs.SM_SCALE * (576 * 2.0 ** -23 * (rows.abs() @ k[:seen].abs().T).amax(1)
                                    + 2.0 ** -17 * rows.abs().amax(1) * k[:seen, DV:].abs().sum(1).max())
        bound[i] = 2.0 ** -8 * out[i].norm(dim=1) + (2.0 ** -8 + ds) * (p @ v.abs()).norm(dim=1) + noise
    return out, bound


@pytest.mark.parametrize("kind", ["one", "scaled"])
@pytest.mark.parametrize("rest", ["equal", "spread"])
@pytest.mark.parametrize("n", [4000, 16384, 65536, 500001])
def test_a_strong_key_before_a_flat_rest(n, rest, kind):
    codes, per_key, arg, scales, q = strong_and_flat(n, rest, kind, n)
    want, bound = exact(codes, per_key, q, n)
    d = VerifyDecoder([n], [2], 6, "fp8", options=binding.PlanOptions(force_splits=1))
    pages = codes.shape[0]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    out = torch.empty((2, 6, DV), dtype=torch.bfloat16, device="cuda")
    lse, status = torch.empty((2, 6), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    d.run(q, codes.view(torch.uint8), table, out, lse, kv_scale=arg, kv_scales=scales, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    off = (out.double() - want).norm(dim=2)
    size = want.norm(dim=2)
    print(f"n={n} {rest} {kind}: error {(off / size).max().item():.2e}, bound {(bound / size).max().item():.2e}")
    assert (bound < 0.1 * size).all()  # the bound means something
    assert (off <= bound).all()
