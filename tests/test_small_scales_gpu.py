"""Block scales at the ends of their range: below 2^-60 the decode's scores and the key weights' are
the same, those of the scales as they are; scales far apart leave every key its weight."""
import math

import pytest
import torch

from mla_speculative_verify_gb300 import binding, inputs
from mla_speculative_verify_gb300.decoder import VerifyDecoder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mixed", [False, True])
def test_scores_of_small_scales(mixed):
    """Queries of 2^70 against keys whose codes are scaled by 2^-72 to 2^-70 (and, mixed, by 2^-59
    with codes that much smaller, and by 0)."""
    n, q, H = 500, 2, 12
    g = torch.Generator(device="cuda").manual_seed(61)
    codes = (torch.randn((8, 64, 576), generator=g, device="cuda")).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-72, -69, (8, 4), generator=g, device="cuda").float())
    if mixed:
        scales[2], scales[5] = 0.0, 2.0 ** -59
        codes[5] = (codes[5].float() * 2.0 ** -9).to(torch.float8_e4m3fn)
    queries = (torch.randn((q, H, 576), generator=g, device="cuda") * 2.0 ** 70).to(torch.bfloat16)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, -1)
    d = VerifyDecoder([n], [q], H, "fp8")
    out, lse = torch.empty((q, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((q, H), device="cuda")
    w, status = torch.zeros((1, n), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    d.run(queries, codes.view(torch.uint8), table, out, lse, kv_scales=scales, status=status)
    d.key_weights(queries, codes, table, lse, w, kv_scales=scales, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    k = (codes.double() * scales.double().repeat_interleave(16, 1)[:, :, None]).view(-1, 576)[:n]
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(q):
        rows = queries[i].double()
        s = inputs.SM_SCALE * (rows @ k[:n - q + i + 1].T)
        # 576 fp32 sums, 2^-23 of the magnitudes each; q in two parts, 2^-17 of its largest entry
        ds = inputs.SM_SCALE * (576 * 2.0 ** -23 * (rows.abs() @ k[:n - q + i + 1].abs().T)
                                + 2.0 ** -17 * rows.abs().amax(1, keepdim=True) * k[:n - q + i + 1].abs().sum(1)).amax(1)
        exact = torch.logsumexp(s, 1)
        assert ((lse[i].double() - exact).abs() <= ds + 1e-5 * (1 + exact.abs())).all()
        want[:n - q + i + 1] += torch.exp(s - exact[:, None]).sum(0)
    assert ((w[0].double() - want).abs() <= 0.02 * want + 1e-12).all()  # ds and lse's: below 1 % of a weight
    assert torch.isfinite(out).all() and out.float().abs().max() < 2.0 ** -51


@pytest.mark.parametrize("octaves", [0, 52, 90])
def test_scales_far_apart(octaves):
    """A key with half of the weight in a block whose scale is 2^octaves of all others', whose keys
    share the other half (52: a block of zeros, which an append gives 2^-60, beside rows of size 1)."""
    n, H = 20000, 2
    pages = -(-n // 64)
    g = torch.Generator(device="cuda").manual_seed(62)
    codes = (torch.randn((pages, 64, 576), generator=g, device="cuda") * 60).clamp(-448, 448)
    codes[..., 512:] = 0.0
    codes[0, 1:] = 0.0
    codes[0, 0, 512] = 64.0
    scales = torch.full((pages, 1), 2.0 ** -(octaves // 2), device="cuda")
    scales[0] = 2.0 ** (octaves - octaves // 2)
    queries = torch.zeros((1, H, 576), device="cuda")
    queries[..., 512] = torch.tensor([1.0, 1.1], device="cuda") * math.log(n) / (inputs.SM_SCALE * 64.0 * scales[0, 0].item())
    queries = queries.to(torch.bfloat16)
    codes = codes.to(torch.float8_e4m3fn)
    d = VerifyDecoder([n], [1], H, "fp8", options=binding.PlanOptions(force_splits=1))
    out, lse = torch.empty((1, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((1, H), device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    d.run(queries, codes, table, out, lse, kv_scales=scales)
    torch.cuda.synchronize()
    k = (codes.double() * scales.double()[:, :, None]).view(-1, 576)[:n]
    s = inputs.SM_SCALE * (queries[0].double() @ k.T)
    want = torch.softmax(s, 1) @ k[:, :512]
    assert ((lse[0].double() - torch.logsumexp(s, 1)).abs() <= 1e-4).all()
    # the strong key's weight to 2^-8, the output's rounding 2^-8, the others' 2^-3 of theirs, independent: 6 deviations
    noise = 6 * 2.0 ** -3 / n * k[1:, :512].norm()
    assert ((out[0].double() - want).norm(dim=1) <= 2.0 ** -7 * want.norm(dim=1) + noise).all()
