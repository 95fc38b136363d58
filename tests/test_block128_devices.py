"""The tensor forms of the 8-bit layers and the expert layer refuse tensors that are
not all on the current CUDA device, before anything is allocated or called."""
import types

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


def operands(device):
    """A call's tensors, by name, and the call."""
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device=device)

    def codes(*shape):
        return z(*shape, dtype=torch.uint8).view(F8)

    def scales(*shape):
        return z(*shape, dtype=torch.float32)
    return {
        "product": (dict(A=codes(8, 256), SA=scales(8, 2), B=codes(16, 256), SB=scales(16, 2), out=scales(8, 16)),
                    lambda A, SA, B, SB, out: gnt.gemm_nt_block128_tensors(A, SA, B, SB, out=out)),
        "quantise": (dict(X=z(8, 256)), gnt.quantize_block128),
        "forward": (dict(X=z(8, 256), W=codes(16, 256), SW=scales(1, 2)), gnt.linear_block128),
        "backward": (dict(dY=z(8, 16), qt=codes(256, 8), st=scales(256, 1), WT=codes(256, 16), SWT=scales(2, 1)),
                     lambda dY, qt, st, WT, SWT: gnt.linear_block128_backward(dY, (qt, st), WT, SWT)),
        "experts": (dict(X=z(2, 64), logits=scales(2, 4), W13=codes(4, 32, 64), W2=codes(4, 64, 16),
                         S13=scales(4, 1, 1), S2=scales(4, 1, 1), out=z(2, 64), workspace=z(1024, dtype=torch.uint8)),
                    lambda X, logits, W13, W2, S13, S2, out, workspace: gnt.moe_few_tokens(
                        X, logits, W13, W2, 1, S13=S13, S2=S2, out=out, workspace=workspace)),
    }


@pytest.fixture
def no_calls(monkeypatch):
    """Fails the test if the library is called."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(gnt, "_lib", Library())


@pytest.mark.parametrize("name", ["product", "quantise", "forward", "backward", "experts"])
def test_host_tensors_are_refused(name, no_calls):
    tensors, call = operands("cpu")[name]
    with pytest.raises(ValueError, match="CUDA device"):
        call(**tensors)


def test_mixed_and_other_devices_are_refused(monkeypatch):
    gnt._init_torch()
    monkeypatch.setattr(gnt, "_torch", types.SimpleNamespace(_C=types.SimpleNamespace(_cuda_getDevice=lambda: 0)))
    on = lambda i: types.SimpleNamespace(get_device=lambda: i, device="device %d" % i)  # noqa: E731
    assert gnt._same_device(on(0), on(0), None, on(0)) == 0
    for tensors in ([on(0), on(1)], [on(0), None, on(-1)], [on(-1), on(0)], [on(1), on(1)]):
        with pytest.raises(ValueError):
            gnt._same_device(*tensors)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["product", "forward", "backward", "experts"])
def test_one_operand_on_the_host_is_refused(name, no_calls):
    tensors, call = operands("cuda")[name]
    for one in tensors:
        with pytest.raises(ValueError):
            call(**{k: v.cpu() if k == one else v for k, v in tensors.items()})


@pytest.mark.gpu
def test_workspace_of_any_type_counts_its_bytes():
    tensors, call = operands("cuda")["experts"]
    del tensors["workspace"]
    need = gnt.gemm_nt_moe_workspace_bytes(2, 1, 16)
    call(workspace=torch.empty(need // 4, device="cuda"), **tensors)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    with pytest.raises(gnt.GemmError) as e:
        call(workspace=torch.empty(need // 4 - 4, device="cuda"), **tensors)
    assert e.value.status == gnt.Status.SCRATCH_TOO_SMALL
    with pytest.raises(ValueError):
        call(workspace=torch.empty(4 * need, dtype=torch.uint8, device="cuda")[::2], **tensors)
