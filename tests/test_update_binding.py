"""The binding of the 8-bit operators and the updates on hosts without a GPU, and beside other versions of torch."""
from __future__ import annotations

import pytest

import dense_gemm_optimisation_f32_amd as dg

torch = pytest.importorskip("torch")


def cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape).to(dtype)


E4M3 = torch.float8_e4m3fn
CALLS = {
    "quant_e4m3_f32": lambda: dg.quant_e4m3_f32(0, 1, 4, 128, cpu(4, 128), 128, 512, cpu(4, 128, dtype=E4M3), 128, 512, cpu(1, 4), 4, 4, stream=0),
    "quant_e4m3_f16": lambda: dg.quant_e4m3_f16(0, 1, 4, 128, cpu(4, 128, dtype=torch.float16), 128, 512, cpu(4, 128, dtype=E4M3), 128, 512,
                                                cpu(1, 4), 4, 4, stream=0),
    "quant_e4m3_bf16": lambda: dg.quant_e4m3_bf16(0, 1, 4, 128, cpu(4, 128, dtype=torch.bfloat16), 128, 512, cpu(4, 128, dtype=E4M3), 128, 512,
                                                  cpu(1, 4), 4, 4, stream=0),
    "gemm_e4m3_f32acc": lambda: dg.gemm_e4m3_f32acc(1, 4, 4, 128, 1.0, cpu(4, 128, dtype=E4M3), 128, cpu(1, 4), 4, cpu(4, 128, dtype=E4M3), 128,
                                                    cpu(1, 4), 4, 0.0, cpu(4, 4), 4, stream=0),
    "gemm_grouped_e4m3_f32acc": lambda: dg.gemm_grouped_e4m3_f32acc(
        1, 1, 4, 4, 128, 1.0, cpu(4, 128, dtype=E4M3), 4, 128, cpu(1, 4), 4, None, cpu(4, 128, dtype=E4M3), 128, 512, cpu(1, 4), 4, 4,
        torch.tensor([0, 4], dtype=torch.int32), 0.0, cpu(4, 4), 4, stream=0),
    "orthogonalise_f32": lambda: dg.orthogonalise_f32(4, 4, [(1.0, 0.0, 0.0)], 1.0, cpu(4, 4), 4, 16, cpu(4, 4, dtype=torch.bfloat16), 4, 16, stream=0),
}


class _Never:
    def __init__(self, name):
        self.__name__ = name

    def __call__(self, *args):
        pytest.fail(f"{self.__name__} called with host memory")


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [None, 0])
def test_host_tensors_are_refused(monkeypatch, name, device):
    """Tensors of the right types and sizes, but in host memory: without a device (torch raises, a host tensor's index is -1) and
    with device 0 the current one.  None of them reaches the library."""
    def current():
        if device is None:
            raise RuntimeError("no device")
        return device

    dg._load_torch()
    monkeypatch.setattr(dg, "_device", current)
    monkeypatch.setattr(dg, "_function", _Never)
    with pytest.raises(ValueError, match="CUDA"):
        CALLS[name]()


def test_torch_without_8_bit_floats(monkeypatch):
    """A torch that has no float8_e4m3fn: the operators of other types work as before, the 8-bit ones take raw addresses."""
    monkeypatch.delattr(torch, "float8_e4m3fn")
    for name in ("_torch", "_Tensor", "_device", "_raw_stream"):
        monkeypatch.setattr(dg, name, None)
    monkeypatch.setattr(dg, "_DTYPES", {})
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="CUDA"):        # (a host tensor; nothing about torch)
        dg.moe_combine_f32(4, 1, 4, x, 4, 4, None, None, 0.0, x, 4, stream=0)
    assert dg._DTYPES["float32"] is torch.float32
    monkeypatch.setattr(dg, "_device", lambda: 0)
    with pytest.raises(ValueError, match="CUDA|dtype"):
        dg.quant_e4m3_f32(0, 1, 4, 4, 0x10000, 4, 16, x, 4, 16, 0x10000, 4, 4, stream=0)
    with pytest.raises(dg.GemmError):                    # (block 7: the library's own refusal)
        dg.quant_e4m3_f32(0, 7, 4, 4, 0x10000, 4, 16, 0x10000, 4, 16, 0x10000, 4, 4, stream=0)
