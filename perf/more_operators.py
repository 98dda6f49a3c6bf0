"""The cases on which the 8-bit floating-point products and the products grouped by expert are
measured.

  f8       C = sum over blocks of 128 inputs of (Aq Wq^T) * sa * sw: e4m3 codes, a scale for each
           token and block, and for each 128 x 128 block of the weight (gemm_f8)
  f8_lin   the same product from bf16 activations, whose codes and scales are made in the call
           (gemm_f8_bf16)
  grp      the product of a mixture of experts: every expert's rows of A times its own weight
           (gemm_bf16_grouped)
  grp_bwd  its backward pass: the gradients of the activations and of every expert's weight
           (gemm_bf16_grouped_bwd)
  f8_grp   the experts' products with 8-bit floating-point weights, from bf16 activations
           (gemm_f8_grouped_bf16)

M is the number of rows (tokens, or token and expert pairs sorted by expert), K the input width and
N the output width. bf16 expert weights are E x K x N, 8-bit weights N x K or E x N x K. Of the E
experts `hit` have rows, in sizes that a router leaves uneven, and the last `pad` of the M rows
belong to none: their outputs are zeros.
"""

import random

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
        {"name": "f8_dec_M1", "op": "f8", "M": 1, "N": 11008, "K": 4096},
        # a mid-length prompt against a weight whose widths are odd and whose last blocks are short
        {"name": "f8_ragged", "op": "f8", "M": 509, "N": 2501, "K": 1003},
        # the down projection over 4096 prompt tokens
        {"name": "f8_prefill", "op": "f8", "M": 4096, "N": 4096, "K": 11008},
        # a decode batch of 16 sequences through the down projection, codes made in the call
        {"name": "f8lin_dec_M16", "op": "f8_lin", "M": 16, "N": 4096, "K": 11008},
        # the up projection over 4096 prompt tokens from bf16 activations
        {"name": "f8lin_prefill", "op": "f8_lin", "M": 4096, "N": 11008, "K": 4096},
        # a decode step of 8 sequences, two experts each: small groups, some experts without rows
        {"name": "grp_dec", "op": "grp", "M": 16, "E": 8, "hit": 7, "pad": 0, "N": 1376, "K": 4096},
        # a training step of a toy layer, padded batch, where launches count
        {"name": "grp_small", "op": "grp", "M": 600, "E": 8, "hit": 7, "pad": 23, "N": 520, "K": 328},
        # 4096 prompt tokens, two of 8 full-size experts each
        {"name": "grp_prefill", "op": "grp", "M": 8192, "E": 8, "hit": 8, "pad": 0, "N": 11008, "K": 4096},
        # the backward pass of a small layer over an odd number of tokens, padded
        {"name": "grpbwd_small", "op": "grp_bwd", "M": 1018, "E": 8, "hit": 8, "pad": 37, "N": 1376, "K": 512},
        # the backward pass of the full layer, the largest case
        {"name": "grpbwd", "op": "grp_bwd", "M": 8192, "E": 8, "hit": 8, "pad": 0, "N": 11008, "K": 4096},
        # a decode step of 16 sequences, four of 64 small experts each
        {"name": "f8grp_dec", "op": "f8_grp", "M": 64, "E": 64, "hit": 41, "pad": 0, "N": 1376, "K": 4096},
        # 2048 prompt tokens, four of 64 small experts each, one of them without rows
        {"name": "f8grp_prefill", "op": "f8_grp", "M": 8192, "E": 64, "hit": 63, "pad": 0, "N": 1376, "K": 4096},
    ]


def _size(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of `step`."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["f8", "f8_lin", "grp", "grp_bwd", "f8_grp"])
    if op in ("f8", "f8_lin"):
        # from single tokens to prompts; widths of any residue
        m, n, k = _size(rng, 1, 4096), _size(rng, 64, 11008), _size(rng, 64, 11008)
        while m * n * k > 4096 * 11008 * 4096:
            k = max(64, k // 2)
        return {"op": op, "M": m, "N": n, "K": k}
    # from a few rows to prompts over few or many experts; bf16 widths of eight
    step = 1 if op == "f8_grp" else 8
    m, e, n, k = _size(rng, 2, 8192), _size(rng, 2, 64), _size(rng, 64, 11008, step), _size(rng, 64, 11008, step)
    while m * n * k > 8192 * 11008 * 4096 or e * n * k > 8 * 11008 * 4096:
        k = max(64, k // 16 * 8)
        if k == 64:
            n = max(64, n // 16 * 8)
    pad = rng.choice([0, 0, rng.randint(0, m // 8)])
    return {"op": op, "M": m, "E": e, "hit": rng.randint(1, min(e, m - pad)), "pad": pad, "N": n, "K": k}


def _group_sizes(case, seed):
    """Rows of each expert: at least one for `hit` of them, the others as an uneven router leaves them."""
    rng = random.Random(seed)
    sizes = [0] * case["E"]
    hit = rng.sample(range(case["E"]), case["hit"])
    likes = [rng.lognormvariate(0.0, 0.7) for _ in hit]
    for e in hit + rng.choices(hit, likes, k=case["M"] - case["pad"] - case["hit"]):
        sizes[e] += 1
    return sizes


def _rows_padded(q, gen):
    """The codes of a matrix in rows padded to 16 bytes, the padding holding arbitrary bytes."""
    rows, k = q.shape
    ld = -(-k // 16) * 16
    if ld == k:
        return q
    pad = torch.randint(0, 256, (rows, ld - k), generator=gen, device=q.device, dtype=torch.uint8)
    return torch.cat([q.view(torch.uint8), pad], 1).view(torch.float8_e4m3fn)[:, :k]


def _blocks(x):
    """x (rows x K) as rows x blocks x 128, the last block filled with zeros."""
    rows, k = x.shape
    return torch.nn.functional.pad(x, (0, -k % 128)).view(rows, -1, 128)


def _token_codes(x):
    """e4m3 codes (as x) and scales (blocks x rows) of each block of 128 values of each row."""
    b = _blocks(x.float())
    most = b.abs().amax(2)
    q = (b * 448 / torch.where(most > 0, most, 1.0)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(x.shape[0], -1)[:, : x.shape[1]], (most / 448).t().contiguous()


def _weight_codes(w):
    """e4m3 codes (as w) and scales of each 128 x 128 block of a weight (N x K)."""
    n, k = w.shape
    b = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    b = b.view(b.shape[0] // 128, 128, -1, 128)
    most = b.abs().amax((1, 3))
    q = (b * 448 / torch.where(most > 0, most, 1.0)[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(q.shape[0] * 128, -1)[:n, :k], most / 448


def prepare(case, seed):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"op": op, "K": K}
    # activations of unit size, a hundredth of the channels sixteen times as large
    x = randn(M, K) * (1 + 15 * (torch.rand(K, generator=gen, device="cuda") < 0.01))
    s["A"] = x.bfloat16()
    if op in ("f8", "f8_lin"):
        q, s["sw"] = _weight_codes(0.02 * randn(N, K))
        s["W"] = _rows_padded(q, gen)
        if op == "f8":
            q, s["sa"] = _token_codes(x)
            s["A"] = _rows_padded(q, gen)
        return s
    s["sizes"] = _group_sizes(case, seed)
    ends = torch.tensor([0] + s["sizes"]).cumsum(0)
    s["offsets"] = ends.to(device="cuda", dtype=torch.int32)
    E = case["E"]
    if op == "f8_grp":
        ld = -(-K // 16) * 16
        codes = torch.empty(E, N, ld, dtype=torch.float8_e4m3fn, device="cuda")
        s["sw"] = torch.empty(E, -(-N // 128), -(-K // 128), device="cuda")
        for e in range(E):
            q, s["sw"][e] = _weight_codes(0.02 * randn(N, K))
            codes[e, :, :K] = q
            if ld != K:
                codes[e] = torch.as_strided(_rows_padded(codes[e, :, :K].contiguous(), gen), (N, ld), (ld, 1))
        s["W"] = codes[:, :, :K]
        return s
    s["B"] = torch.empty(E, K, N, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        s["B"][e] = randn(K, N) * K**-0.5
    if op == "grp_bwd":
        # gradients as a mean loss leaves them, a tenth of the tokens masked out of the loss
        live = torch.rand(M, 1, generator=gen, device="cuda") < 0.9
        s["dC"] = (randn(M, N) * live / M).bfloat16()
    return s


def _plain_f8(q, sa, w, sw):
    """Codes (rows x K), scales (blocks x rows) and an 8-bit weight: the product in float32."""
    n, k = w.shape
    a = q.float() * sa.t().repeat_interleave(128, 1)[:, :k]
    b = w.float() * sw.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return a @ b.t()


def _plain(s):
    op = s["op"]
    if op == "f8":
        return _plain_f8(s["A"], s["sa"], s["W"], s["sw"]).bfloat16()
    if op == "f8_lin":
        q, sa = _token_codes(s["A"])
        return _plain_f8(q, sa, s["W"], s["sw"]).bfloat16()
    M, first = s["A"].shape[0], 0
    if op == "f8_grp":
        q, sa = _token_codes(s["A"])
        C = torch.zeros(M, s["W"].shape[1], dtype=torch.bfloat16, device=q.device)
        for e, rows in enumerate(s["sizes"]):
            at = slice(first, first + rows)
            if rows:
                C[at] = _plain_f8(q[at], sa[:, at], s["W"][e], s["sw"][e]).bfloat16()
            first += rows
        return C
    B = s["B"]
    if op == "grp":
        C = torch.zeros(M, B.shape[2], dtype=torch.bfloat16, device=B.device)
        for e, rows in enumerate(s["sizes"]):
            at = slice(first, first + rows)
            if rows:
                C[at] = (s["A"][at].float() @ B[e].float()).bfloat16()
            first += rows
        return C
    dA, dB = torch.zeros_like(s["A"]), torch.zeros_like(B)
    for e, rows in enumerate(s["sizes"]):
        at = slice(first, first + rows)
        if rows:
            d = s["dC"][at].float()
            dA[at] = (d @ B[e].float().t()).bfloat16()
            dB[e] = (s["A"][at].float().t() @ d).bfloat16()
        first += rows
    return dA, dB


def run(state):
    if not own:
        return _plain(state)
    g, s = _lib(), state
    op = s["op"]
    if op == "f8":
        return g.f8_matmul(s["A"], s["sa"], s["W"], s["sw"])
    if op == "f8_lin":
        return g.f8_linear(s["A"], s["W"], s["sw"])
    if op == "grp":
        return g.grouped_matmul(s["A"], s["B"], s["offsets"])
    if op == "grp_bwd":
        return g.grouped_matmul_backward(s["dC"], s["A"], s["B"], s["offsets"])
    return g.f8_grouped_linear(s["A"], s["W"], s["sw"], s["offsets"])


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    blocks_n, blocks_k = -(-N // 128), -(-K // 128)
    if op in ("f8", "f8_lin"):
        a = M * K + 4 * M * blocks_k if op == "f8" else 2 * M * K
        return {"bytes": a + N * K + 4 * blocks_n * blocks_k + 2 * M * N, "flops": 2 * M * N * K}
    # rows of no expert are neither read nor multiplied, and their outputs written
    rows, hit = M - case["pad"], case["hit"]
    if op == "grp":
        return {"bytes": 2 * (rows * K + hit * K * N + M * N), "flops": 2 * rows * N * K}
    if op == "grp_bwd":
        return {"bytes": 2 * (rows * (N + K) + hit * K * N + M * K + case["E"] * K * N), "flops": 4 * rows * N * K}
    return {"bytes": 2 * rows * K + hit * (N * K + 4 * blocks_n * blocks_k) + 2 * M * N, "flops": 2 * rows * N * K}


def _exact_round(v):
    """The e4m3 value nearest to each of v (magnitudes up to 448), ties to even, in 64 bits."""
    _, exponent = torch.frexp(v)
    step = torch.exp2(torch.clamp(exponent.double() - 4, min=-9.0))
    return torch.round(v / step) * step


def _exact_activations(A):
    """A with every block of 128 values of each row rounded to its codes, in 64 bits."""
    cut = [b.double() for b in A.split(128, dim=1)]
    for i, b in enumerate(cut):
        most = b.abs().max(dim=1, keepdim=True).values
        most = torch.where(most == 0, torch.ones_like(most), most)
        cut[i] = _exact_round(b.mul(448).div(most)) * most / 448
    return torch.cat(cut, dim=1)


def _exact_weight(w, sw):
    out = w.double()
    for i in range(sw.shape[0]):
        for j in range(sw.shape[1]):
            out[128 * i : 128 * i + 128, 128 * j : 128 * j + 128] *= sw[i, j].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("f8", "f8_lin"):
        if op == "f8_lin":
            A = _exact_activations(s["A"])
        else:
            A = torch.cat([b.double() * f.double().unsqueeze(1) for b, f in zip(s["A"].split(128, dim=1), s["sa"])], dim=1)
        return torch.mm(A, _exact_weight(s["W"], s["sw"]).T)
    ends = s["offsets"].tolist()
    spans = [(e, a, b) for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a]
    double = {"dtype": torch.float64, "device": s["A"].device}
    if op == "f8_grp":
        A, out = _exact_activations(s["A"]), torch.zeros(case["M"], case["N"], **double)
        for e, a, b in spans:
            torch.mm(A[a:b], _exact_weight(s["W"][e], s["sw"][e]).T, out=out[a:b])
        return out
    if op == "grp":
        out = torch.zeros(case["M"], case["N"], **double)
        for e, a, b in spans:
            torch.mm(s["A"][a:b].double(), s["B"][e].double(), out=out[a:b])
        return out
    dA, dB = torch.zeros(case["M"], case["K"], **double), torch.zeros(case["E"], case["K"], case["N"], **double)
    for e, a, b in spans:
        dY = s["dC"][a:b].double()
        torch.mm(dY, s["B"][e].double().T, out=dA[a:b])
        torch.mm(s["A"][a:b].double().T, dY, out=dB[e])
    return dA, dB
