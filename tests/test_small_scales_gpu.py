"""Block scales below 2^-60: the decode's scores and the key weights' are the same, those of the
scales as they are."""
import pytest
import torch

from mla_speculative_verify_gb300 import inputs
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
