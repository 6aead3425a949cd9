"""A build of the key weights' kernel with fewer registers than its warpgroups share out: the call
is refused with that reason, and every other entry point works."""
import shutil

import pytest
import torch

from mla_speculative_verify_gb300 import binding, build
from mla_speculative_verify_gb300.decoder import VerifyDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture
def other_build(tmp_path, monkeypatch):
    """The library from the same sources but for the number of registers that the kernel asks for,
    which no build can give: in the place of a compiler that gives fewer. Nothing of it is
    launched that waits for registers, since the host compares the numbers first."""
    src = tmp_path / "csrc"
    shutil.copytree(build.CSRC, src)
    f = src / "weights_sm103.cu"
    text = f.read_text()
    assert text.count("kRegsLaunch = 168") == 1
    f.write_text(text.replace("kRegsLaunch = 168", "kRegsLaunch = 256"))
    with monkeypatch.context() as m:
        m.setattr(build, "CSRC", str(src))
        m.setattr(build, "OUT_DIR", str(tmp_path / "lib"))
        m.setattr(build, "LIB_PATH", str(tmp_path / "lib" / build.LIB_NAME))
        path = build.build(force=True)
    lib = binding.load(path)
    monkeypatch.setattr(binding, "_lib", lib)
    return lib


def test_only_the_key_weights_are_refused(other_build):
    q = torch.randn((2, 12, 576), device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 64, 576), device="cuda").to(torch.bfloat16)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    out, lse = torch.empty((2, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 12), device="cuda")
    d = VerifyDecoder([100], [2], 12, "bf16")
    d.run(q, kv, table, out, lse)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    for _ in range(2):
        with pytest.raises(binding.MlaError, match="registers"):
            d.key_weights(q, kv, table, lse, torch.zeros((1, 100), device="cuda"))
    d.run(q, kv, table, out, lse)
    torch.cuda.synchronize()
