"""Outputs that overlap operands which the tensor forms copy onto 16-byte boundaries first:
refused as those of other operands are, before anything is launched.  (Stand-ins for the
library and the device, no GPU; and both forms on the GPU.)"""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
from test_block128_streams import fake  # noqa: E402,F401

BF16 = torch.bfloat16


def overlapping(device):
    """Calls whose output lies on an operand, by name; all operands have odd rows."""
    def room(n):
        return torch.zeros(n, dtype=BF16, device=device)
    x, w = room(20 * 255).view(20, 255), room(64 * 255).view(64, 255)
    q, s = torch.zeros(64, 128, dtype=torch.uint8, device=device), torch.ones(64, 2, dtype=BF16, device=device)
    return {
        "X": lambda: gnt.gated_linear(x, w, out=x[:, :32]),
        "X's end": lambda: gnt.gated_linear(x, w, out=x.flatten()[-32 * 20:].view(20, 32)),
        "W13": lambda: gnt.gated_linear(x, w, out=w.flatten()[:20 * 32].view(20, 32)),
        "W13, one token": lambda: gnt.gated_linear(x[:1], w, out=w[5:6, 3:35]),
        "X, 4 bits": lambda: gnt.linear_w4(x, q, s, out=x[:, :64]),
        "X, gated in 4 bits": lambda: gnt.gated_linear_w4(x, q, s, out=x[:, 7:39]),
    }


NAMES = ["X", "X's end", "W13", "W13, one token", "X, 4 bits", "X, gated in 4 bits"]


@pytest.mark.parametrize("name", NAMES)
def test_refused_before_anything_runs(fake, name, monkeypatch):  # noqa: F811
    monkeypatch.setattr(gnt, "error_string", lambda status: "overlap")
    with pytest.raises(gnt.GemmError) as e:
        overlapping("cpu")[name]()
    assert e.value.status == gnt.Status.OVERLAP
    assert not fake[1].launched


def test_neighbours_are_not_refused(fake):  # noqa: F811
    """An output that ends where an operand begins or begins where it ends, and empty ones."""
    store = torch.zeros(20 * 32 + 20 * 255 + 20 * 32, dtype=BF16)
    before, x, after = store[:640].view(20, 32), store[640:640 + 5100].view(20, 255), store[5740:].view(20, 32)
    w = torch.zeros(64, 255, dtype=BF16)
    for out in (before, after):
        assert gnt.gated_linear(x, w, out=out) is out
    assert gnt.gated_linear(x[:, :0], w[:, :0], out=x[:, :32]).shape == (20, 32)
    assert gnt.gated_linear(x[:0], w, out=w[:0, :32]).shape == (0, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_both_forms_refuse(name, monkeypatch):
    gnt.quantize_w4(torch.zeros(1, 32, device="cuda"))  # (binds the extension)
    call, extension = overlapping("cuda")[name], gnt._calls
    for calls in (extension, None):
        monkeypatch.setattr(gnt, "_calls", calls)
        with pytest.raises(gnt.GemmError) as e:
            call()
        assert e.value.status == gnt.Status.OVERLAP
