"""The cases on which the 8-bit and the training operators of the library are measured.

The operators are those of a gated MLP that the bf16 inference products leave open:

  i8       C = (Aq Wq^T) * sa * sw: 8-bit integer codes with a scale for each token and each
           output channel (gemm_i8)
  i8_lin   the same product from bf16 activations, whose codes and scales are made in the call
           (gemm_i8_bf16)
  i8_glu   silu(g) * u of an 8-bit gate/up product, from bf16 activations (gemm_i8_swiglu_bf16)
  ffn_fwd  the training forward of the gated block: silu(g) * u, and g and u for the backward
           pass (gemm_bf16_swiglu_train)
  ffn_bwd  its backward pass: the gradients of g and u, of the activations and of the gate/up
           weight (gemm_bf16_swiglu_bwd)
  lin_bwd  the backward pass of a plain product, as the down projection needs it
           (gemm_bf16_bwd)

M is the number of tokens, K the input width and N the output width (of the gate and of the up
half each, for the gated forms). bf16 weights are K x N (K x 2N) row-major, 8-bit weights N x K
(2N x K), each row with a scale.
"""

import torch

own = False

_gemm = None


def _lib():
    """The framework's binding, initialised on the current device once."""
    global _gemm
    if _gemm is None:
        import gemv_layers_amd

        gemv_layers_amd.gemm_init(torch.cuda.current_device())
        _gemm = gemv_layers_amd
    return _gemm


def listed():
    return [
        # one token through the up projection of a 4096-wide model with an 11008-wide MLP: a
        # stream of weight codes
        {"name": "i8_dec_M1", "op": "i8", "M": 1, "N": 11008, "K": 4096},
        # a mid-length prompt against a weight whose widths are odd (rows padded to 16 codes)
        {"name": "i8_ragged", "op": "i8", "M": 509, "N": 2501, "K": 1003},
        # the down projection over 4096 prompt tokens
        {"name": "i8_prefill", "op": "i8", "M": 4096, "N": 4096, "K": 11008},
        # a decode batch of 64 sequences through the down projection, codes made in the call
        {"name": "i8lin_dec_M64", "op": "i8_lin", "M": 64, "N": 4096, "K": 11008},
        # a small decode batch through the gate/up projections
        {"name": "i8glu_dec_M16", "op": "i8_glu", "M": 16, "N": 11008, "K": 4096},
        # the gate/up projections over 4096 prompt tokens
        {"name": "i8glu_prefill", "op": "i8_glu", "M": 4096, "N": 11008, "K": 4096},
        # a training step of a toy block, where launches count
        {"name": "ffn_fwd_small", "op": "ffn_fwd", "M": 300, "N": 520, "K": 328},
        # a training step's 4096 tokens through the gate/up projections
        {"name": "ffn_fwd", "op": "ffn_fwd", "M": 4096, "N": 11008, "K": 4096},
        # the backward pass of a small block over an odd number of tokens
        {"name": "ffn_bwd_small", "op": "ffn_bwd", "M": 509, "N": 1376, "K": 512},
        # the backward pass of the full gate/up block, the largest case
        {"name": "ffn_bwd", "op": "ffn_bwd", "M": 4096, "N": 11008, "K": 4096},
        # the backward pass of a square layer of a small model
        {"name": "lin_bwd_512", "op": "lin_bwd", "M": 512, "N": 512, "K": 512},
        # the backward pass of the full down projection
        {"name": "lin_bwd", "op": "lin_bwd", "M": 4096, "N": 4096, "K": 11008},
    ]


def _size(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of `step`."""
    v = lo * (hi / lo) ** rng.random()
    v = max(lo, min(hi, int(v / step + 0.5) * step))
    return v + step if v == 3 << 10 else v


def draw(rng):
    op = rng.choice(["i8", "i8_lin", "i8_glu", "ffn_fwd", "ffn_bwd", "lin_bwd"])
    if op in ("i8", "i8_lin", "i8_glu"):
        # from single tokens to prompts; widths of any residue
        m, n, k = _size(rng, 1, 4096), _size(rng, 64, 11008), _size(rng, 64, 11008)
    else:
        # training batches of any length; widths of eight
        m, n, k = _size(rng, 64, 4096), _size(rng, 64, 11008, 8), _size(rng, 64, 11008, 8)
    while m * n * k > 4096 * 11008 * 4096:
        k = max(64, k // 16 * 8)
    return {"op": op, "M": m, "N": n, "K": k}


def _codes(x, pad):
    """8-bit codes of each row of x (values in [-127, 127] times the row's scale) in rows padded
    to 16 bytes, the padding holding arbitrary codes, and the scales."""
    scale = x.abs().amax(1) / 127
    q = torch.round(x / scale[:, None]).to(torch.int8)
    rows, k = q.shape
    ld = -(-k // 16) * 16
    if ld != k:
        pad = torch.randint(-127, 128, (rows, ld - k), generator=pad, device=x.device).to(torch.int8)
        q = torch.cat([q, pad], 1)[:, :k]
    return q, scale


def prepare(case, seed):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"op": op, "N": N}
    # activations of unit size, a hundredth of the channels sixteen times as large
    x = randn(M, K) * (1 + 15 * (torch.rand(K, generator=gen, device="cuda") < 0.01))
    if op in ("i8", "i8_lin", "i8_glu"):
        s["W"], s["sw"] = _codes(0.02 * randn(2 * N if op == "i8_glu" else N, K), gen)
        if op == "i8":
            s["A"], s["sa"] = _codes(x, gen)
        else:
            s["A"] = x.bfloat16()
        return s
    s["A"] = x.bfloat16()
    s["B"] = (randn(K, N if op == "lin_bwd" else 2 * N) * K**-0.5).bfloat16()
    if op != "ffn_fwd":
        # gradients as a mean loss leaves them; a tenth of the tokens is masked out of the loss
        live = torch.rand(M, 1, generator=gen, device="cuda") < 0.9
        s["dC"] = (randn(M, N) * live / M).bfloat16()
    if op == "ffn_bwd":
        s["GU"] = (s["A"].float() @ s["B"].float()).bfloat16()
    return s


def _plain_codes(a):
    a = a.float()
    sa = a.abs().amax(1, keepdim=True) / 127
    return torch.round(a / sa), sa


def _plain(s):
    op, N = s["op"], s["N"]
    if op == "i8":
        return (s["A"].float() @ s["W"].float().t() * s["sa"][:, None] * s["sw"]).bfloat16()
    if op in ("i8_lin", "i8_glu"):
        q, sa = _plain_codes(s["A"])
        y = q @ s["W"].float().t() * sa * s["sw"]
        if op == "i8_glu":
            y = y[:, :N] / (1 + torch.exp(-y[:, :N])) * y[:, N:]
        return y.bfloat16()
    a, b = s["A"].float(), s["B"].float()
    if op == "ffn_fwd":
        gu = a @ b
        g, u = gu[:, :N], gu[:, N:]
        return (g / (1 + torch.exp(-g)) * u).bfloat16(), gu.bfloat16()
    d = s["dC"].float()
    if op == "ffn_bwd":
        g, u = s["GU"][:, :N].float(), s["GU"][:, N:].float()
        sig = 1 / (1 + torch.exp(-g))
        d = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1)
        return (d @ b.t()).bfloat16(), (a.t() @ d).bfloat16(), d.bfloat16()
    return (d @ b.t()).bfloat16(), (a.t() @ d).bfloat16()


def run(state):
    if not own:
        return _plain(state)
    g, s = _lib(), state
    op = s["op"]
    if op == "i8":
        return g.i8_matmul(s["A"], s["sa"], s["W"], s["sw"])
    if op == "i8_lin":
        return g.i8_linear(s["A"], s["W"], s["sw"])
    if op == "i8_glu":
        return g.i8_swiglu_linear(s["A"], s["W"], s["sw"])
    if op == "ffn_fwd":
        return g.swiglu_forward(s["A"], s["B"])
    if op == "ffn_bwd":
        return g.swiglu_backward(s["dC"], s["GU"], s["A"], s["B"])
    return g.matmul_backward(s["dC"], s["A"], s["B"])


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    mk, nk, mn = M * K, N * K, M * N
    if op == "i8":
        return {"bytes": mk + nk + 4 * (M + N) + 2 * mn, "flops": 2 * mn * K}
    if op == "i8_lin":
        return {"bytes": 2 * mk + nk + 4 * N + 2 * mn, "flops": 2 * mn * K}
    if op == "i8_glu":
        return {"bytes": 2 * mk + 2 * nk + 8 * N + 2 * mn, "flops": 4 * mn * K}
    if op == "ffn_fwd":
        return {"bytes": 2 * (mk + 2 * nk + 3 * mn), "flops": 4 * mn * K}
    if op == "ffn_bwd":
        return {"bytes": 2 * (2 * mk + 4 * nk + 5 * mn), "flops": 8 * mn * K}
    return {"bytes": 2 * (2 * mk + 2 * nk + mn), "flops": 4 * mn * K}


def exact(case, seed):
    s = prepare(case, seed)
    op, N = case["op"], case["N"]
    A = s["A"].double()
    if op in ("i8", "i8_lin", "i8_glu"):
        if op == "i8":
            sa = s["sa"].double()
        else:
            sa = A.abs().max(dim=1).values.div(127)
            A = torch.div(A, sa.unsqueeze(1)).round()
        y = torch.mm(A * sa.unsqueeze(1), (s["W"].double() * s["sw"].double().unsqueeze(1)).T)
        if op == "i8_glu":
            gate, up = y.split(N, dim=1)
            y = gate * torch.sigmoid(gate) * up
        return y
    B = s["B"].double()
    if op == "ffn_fwd":
        gate, up = torch.mm(A, B[:, :N]), torch.mm(A, B[:, N:])
        return gate * torch.sigmoid(gate) * up, torch.cat([gate, up], dim=1)
    if op == "ffn_bwd":
        gu = s["GU"].double().requires_grad_()
        gate, up = gu.split(N, dim=1)
        (dY,) = torch.autograd.grad(gate * torch.sigmoid(gate) * up, gu, s["dC"].double())
        return torch.mm(dY, B.T), torch.mm(A.T, dY), dY
    dY = s["dC"].double()
    return torch.mm(dY, B.T), torch.mm(A.T, dY)
