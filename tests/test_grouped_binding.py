"""The expert layer's binding, without a GPU: on which device and in which stream's memory a
call runs, with torch.cuda's contexts replaced by recorders."""
import contextlib

import pytest
import torch

import fp8_block_scaled_08_b200 as fq


class OnDevice(torch.Tensor):
    """A host tensor that says that it lies on device 1."""

    def get_device(self):
        return 1


def recorder(log, kind):
    @contextlib.contextmanager
    def context(x):
        log.append((kind, x))
        yield
        log.append((kind, None))
    return context


def test_weights_are_quantized_on_their_own_device(monkeypatch):
    """The weight quantizer launches on the current device: it has to be the weights'."""
    log = []
    monkeypatch.setattr(torch.cuda, "device", recorder(log, "device"))
    E, N, K = 2, 128, 256

    def quantize(w, want_t, stream):
        log.append(("call", tuple(w.shape)))
        return (torch.zeros(E * N, K, dtype=torch.uint8), torch.zeros(E, K // 128),
                torch.zeros(K, E * N, dtype=torch.uint8))

    monkeypatch.setattr(fq, "quant_weight_alloc", quantize)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16).as_subclass(OnDevice)
    qw, sw, qwT = fq.grouped_quant_weight_alloc(w)
    assert log == [("device", 1), ("call", (E * N, K)), ("device", None)]
    assert qw.shape == (E, N, K) and sw.shape == (E, 1, 2) and qwT.shape == (K, E, N)


def test_weights_on_the_host_are_refused():
    with pytest.raises(ValueError, match="CUDA tensors"):
        fq.grouped_quant_weight_alloc(torch.zeros(2, 128, 256, dtype=torch.bfloat16))
