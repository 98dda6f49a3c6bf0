"""The tensor marshalling of the 8-bit and training helpers on a machine without a GPU: every refusal
that needs no device memory, and that the module's functions take their arguments and nothing else."""

import pytest

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402

BF = torch.zeros(4, 8, dtype=torch.bfloat16)
Q = torch.zeros(4, 8, dtype=torch.int8)
S = torch.zeros(4)


@pytest.mark.parametrize("call", [
    lambda: g.i8_quantize(Q), lambda: g.i8_quantize(3), lambda: g.i8_quantize(None),
    lambda: g.i8_matmul(BF, S, Q, S), lambda: g.i8_swiglu_matmul("x", S, Q, S),
    lambda: g.i8_linear(Q, Q, S), lambda: g.i8_swiglu_linear(BF.float(), Q, S),
    lambda: g.matmul_backward(BF, BF.half(), BF), lambda: g.swiglu_forward(BF.double(), BF),
    lambda: g.swiglu_backward(BF, BF, Q, BF)])
def test_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [
    lambda: g.i8_quantize(BF), lambda: g.i8_quantize(BF[0]), lambda: g.i8_matmul(Q, S, Q, S),
    lambda: g.i8_linear(BF, Q, S), lambda: g.matmul_backward(BF, BF, BF), lambda: g.swiglu_forward(BF, BF),
    lambda: g.swiglu_backward(BF, BF, BF, BF)])
def test_host_tensors_and_vectors(call):
    with pytest.raises(ValueError):
        call()


def test_argument_counts():
    m = g._load_ops()
    for name, n in (("quantize", 2), ("i8", 7), ("i8_dynamic", 7), ("bwd", 6), ("train", 3), ("swiglu_bwd", 8),
                    ("bind", 9)):
        with pytest.raises(TypeError):
            getattr(m, name)(*[None] * (n - 1))
        with pytest.raises(TypeError):
            getattr(m, name)(*[None] * (n + 1))
