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


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


OFF = torch.zeros(3, dtype=torch.int32)
M, N, K = 128, 128, 256
ALLOC = {
    "add_rmsnorm_quant": (bf16(M, N), bf16(M, N), bf16(N), 1e-5),
    "grouped_transpose_quant_bf16": (bf16(M, N), OFF),
    "grouped_transpose_quant_fp8": (u8(M, N), torch.zeros(1, M), OFF),
    "quant_act_1x128": (bf16(M, N),),
    "quant_weight": (bf16(M, N),),
    "rmsnorm_quant": (bf16(M, N), bf16(N), 1e-5),
    "rmsnorm_quant_dual": (bf16(M, N), bf16(N), 1e-5),
    "rmsnorm_bwd_quant_dual": (bf16(M, N), bf16(N), bf16(M, N), None, 1e-5),
    "swiglu_quant": (bf16(M, 2 * N),),
    "swiglu_quant_dual": (bf16(M, 2 * N),),
    "swiglu_bwd_quant_dual": (bf16(M, 2 * N), bf16(M, N)),
    "transpose_quant_bf16": (bf16(M, N),),
    "transpose_quant_fp8": (u8(M, N), torch.zeros(1, M)),
    "linear_fwd": (u8(M, K), torch.zeros(2, M), u8(N, K), torch.zeros(1, 2)),
    "linear_dgrad": (u8(M, N), torch.zeros(1, M), u8(K, N), torch.zeros(1, 2)),
    "linear_wgrad": (u8(N, M), torch.zeros(1, N), u8(K, M), torch.zeros(1, K)),
}


def test_every_allocating_form_is_listed():
    forms = {n[:-len("_alloc")] for n in dir(fq) if n.endswith("_alloc") and not n.startswith("_")}
    # the stacked weights are quantize_weight's outputs; split-K allocates in the library
    assert forms - set(ALLOC) <= {"grouped_quant_weight", "linear_fwd_splitk_no"}


class Stream:
    cuda_stream = 0


@pytest.mark.parametrize("name", list(ALLOC))
def test_outputs_belong_to_the_stream_of_the_call(monkeypatch, name):
    """Outputs (and a workspace) of a call on another stream are allocated in that stream."""
    log, side = [], Stream()
    empty = torch.empty

    def alloc(*a, **k):
        log.append("empty")
        return empty(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", recorder(log, "stream"))
    monkeypatch.setattr(torch, "empty", alloc)
    with pytest.raises(ValueError, match="CUDA tensors"):
        getattr(fq, name + "_alloc")(*ALLOC[name], stream=side)
    assert log and len(log) % 3 == 0
    for i in range(0, len(log), 3):
        assert log[i:i + 3] == [("stream", side), "empty", ("stream", None)], log
    log.clear()
    with pytest.raises(ValueError, match="CUDA tensors"):
        getattr(fq, name + "_alloc")(*ALLOC[name])
    assert log and set(log) == {"empty"}
