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


def grad(t):
    return t.clone().requires_grad_()


@pytest.mark.parametrize("call,name", [
    (lambda: g.swiglu_forward(grad(BF), BF.t()), "A"), (lambda: g.i8_linear(grad(BF), Q, S), "A"),
    (lambda: g.i8_swiglu_linear(grad(BF), Q, S), "A"), (lambda: g.matmul_backward(BF, grad(BF), BF), "A"),
    (lambda: g.swiglu_backward(BF, BF, grad(BF), BF), "A")])
def test_a_graph_is_not_lost_without_a_word(call, name):
    with pytest.raises(RuntimeError, match=f"{name} requires grad"):
        call()
    with torch.no_grad(), pytest.raises(ValueError):     # as for any host tensor
        call()


def test_codes_have_no_gradient():
    with pytest.raises(ValueError):                      # refused as a host tensor only
        g.i8_quantize(grad(BF))
