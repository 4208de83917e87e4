"""Operators of a transformer block around its products: the norm before them, products grouped by expert, and the
4-bit block-scaled form of an operand.

Cases, inputs, plain forms and exact values of the operators

    rmsnorm           forward   h = x + residual, y = h * rstd * w, y in x's type or in 8 bits with block scales
                      backward  the gradients of h (the residual stream's own added) and of w
    gemm_grouped      rows sorted by expert, offsets in GPU memory, one weight matrix per expert:
                      forward   D[rows of g] = round(act(A[rows of g] @ W[g]^T + bias[g]))
                      input     dX[rows of g] = dY[rows of g] @ W[g]
                      weight    dW[g] = dY[rows of g]^T @ X[rows of g] + beta * C[g]
    gemm_grouped_mx   the forward direction from 8-bit activations and 8- or 4-bit weights, both block-scaled
    mx4_quantize      rows to 4-bit floating point (E2M1) with one power-of-two scale per 32

Formats.  8-bit elements: rows padded to a multiple of 32 with zeros; 4-bit elements: two per byte, the lower
index in the low nibble, rows of ceil(K / 32) * 16 bytes.  Scale words of both (ceil(K / 128) x rows, int32): byte
q of word t is the exponent e (value 2^(e - 127)) of block 4t + q; 127 for blocks past K.  Offsets: int32, one more
than experts; rows behind the last offset belong to no expert and stay as they were.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1, "fp4": 0.5}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# exponent of the largest element and the fp32 fraction bits of its significand
_TOP = {"e4m3": (8, 0x600000), "e5m2": (15, 0x600000), "fp4": (2, 0x400000)}
_LARGEST = {"e4m3": 448.0, "e5m2": 57344.0, "fp4": 6.0}


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # one sequence answers token by token: a row of the residual stream before a projection, latency counts
        dict(name="norm_token", op="rmsnorm", way="forward", M=1, N=4096, type="bf16", w="bf16", out="same", residual=True),
        # a training step or a long prompt: the normed rows leave in 8 bits for the block-scaled product
        dict(name="norm_to_8_bits", op="rmsnorm", way="forward", M=8192, N=8192, type="bf16", w="bf16", out="e4m3",
             residual=True),
        # its backward pass, the gradient of the residual stream added
        dict(name="norm_backward", op="rmsnorm", way="backward", M=8192, N=8192, type="bf16", w="fp32", residual=True),
        # one token through two of sixteen experts: the weights of two are read
        dict(name="experts_token", op="gemm_grouped", way="forward", M=2, G=16, active=2, tail=0, N=4096, K=4096,
             type="bf16", out="same", bias=True, relu=False),
        # a batch of prompts, two experts a token, through the experts' first product
        dict(name="experts_prompt", op="gemm_grouped", way="forward", M=8192, G=16, active=16, tail=0, N=4096, K=4096,
             type="bf16", out="same", bias=False, relu=True),
        # the gradient of its input; some experts without rows, rows behind the last expert
        dict(name="experts_input_gradient", op="gemm_grouped", way="input", M=8190, G=16, active=14, tail=22, N=2048,
             K=4096, type="fp16", out="same", bias=False, relu=False),
        # the gradient of the experts' weights, added to that of the steps before
        dict(name="experts_weight_gradient", op="gemm_grouped", way="weight", M=8192, G=8, active=8, tail=0, N=4096,
             K=2048, type="bf16", out="fp32", beta=1.0),
        # the same for a small layer: few rows, odd sizes, two experts without rows
        dict(name="experts_weight_gradient_ragged", op="gemm_grouped", way="weight", M=1000, G=7, active=5, tail=3,
             N=1001, K=520, type="fp16", out="same", beta=0.0),
        # a small batch answers token by token from 4-bit experts: as many experts as rows are read
        dict(name="experts_4_bit_tokens", op="gemm_grouped_mx", M=16, G=64, active=16, tail=0, N=4096, K=4096,
             type="e4m3", weights="fp4", out="bf16", bias=False, relu=False),
        # a prompt through 4-bit experts
        dict(name="experts_4_bit_prompt", op="gemm_grouped_mx", M=4096, G=16, active=16, tail=0, N=4096, K=8192,
             type="e4m3", weights="fp4", out="bf16", bias=True, relu=False),
        # the experts' weights brought to 4 bits, as loaded; and activations of odd sizes
        dict(name="weights_to_4_bits", op="mx4_quantize", M=16384, K=8192, type="bf16"),
        dict(name="rows_to_4_bits_ragged", op="mx4_quantize", M=777, K=1000, type="fp32"),
    ]


def _size(rng, lo, hi):
    """A whole number in lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm", "gemm_grouped", "gemm_grouped", "gemm_grouped", "gemm_grouped_mx",
                     "gemm_grouped_mx", "mx4_quantize"])
    if op == "mx4_quantize":
        return dict(op=op, M=_size(rng, 1, 16384), K=_size(rng, 32, 8192), type=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "rmsnorm":
        case = dict(op=op, way=rng.choice(["forward", "backward"]), M=_size(rng, 1, 8192), N=_size(rng, 64, 8192),
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), w=rng.choice(["same", "fp32"]),
                    residual=rng.random() < 0.7)
        if case["type"] == "fp32":
            case["M"] = min(case["M"], 4096)
        if case["way"] == "forward":
            case["out"] = rng.choice(["same", "e4m3", "e4m3", "e5m2"])
        return case
    G = _size(rng, 2, 64)
    N, K = _size(rng, 256, 8192), _size(rng, 256, 8192)
    M = _size(rng, 1, 8192)
    most = 16 * 4096 * 4096                      # elements of all weights
    G = max(2, min(G, most // (N * K)))
    M = max(1, min(M, 8192 * 4096 * 4096 // (N * K)))
    case = dict(op=op, M=M, G=G, active=max(1, min(G, M, int(G * rng.uniform(0.5, 1.2)))), N=N, K=K)
    case["tail"] = min(M - case["active"], rng.choice([0, 0, 5]))
    if op == "gemm_grouped_mx":
        return dict(case, K=32 * max(8, min(K // 32, 256)), M=min(M, 4096), active=min(case["active"], 4096),
                    tail=min(case["tail"], max(0, min(M, 4096) - case["active"])),
                    type=rng.choice(["e4m3", "e4m3", "e5m2"]), weights=rng.choice(["fp4", "fp4", "e4m3"]),
                    out=rng.choice(["bf16", "fp16", "fp32"]), bias=rng.random() < 0.5, relu=rng.random() < 0.3)
    way = rng.choice(["forward", "input", "weight"])
    case.update(way=way, type=rng.choice(["bf16", "bf16", "fp16"]), out=rng.choice(["same", "same", "fp32"]))
    if way == "weight":
        return dict(case, beta=rng.choice([0.0, 1.0]))
    return dict(case, bias=way == "forward" and rng.random() < 0.5, relu=way == "forward" and rng.random() < 0.3)


def work(case):
    op = case["op"]
    t = _SIZES[case["type"]]
    if op == "mx4_quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * (K * t + -(-K // 32) * 16 + -(-K // 128) * 4), "flops": 2 * M * K}
    if op == "rmsnorm":
        M, N = case["M"], case["N"]
        w = N * _SIZES[_w(case)]
        if case["way"] == "backward":
            return {"bytes": M * N * t * (4 if case["residual"] else 3) + 4 * M + w + 4 * N, "flops": 10 * M * N}
        y = N * t if case["out"] == "same" else -(-N // 32) * 32 + -(-N // 128) * 4
        return {"bytes": M * (N * t * (3 if case["residual"] else 1) + y + 4) + w, "flops": 5 * M * N}
    M, G, N, K, rows = case["M"], case["G"], case["N"], case["K"], case["M"] - case["tail"]
    o = _SIZES[_out(case)]
    if op == "gemm_grouped_mx":
        words = -(-K // 128) * 4
        weights = case["active"] * N * (K * _SIZES[case["weights"]] + words)
        extra = case["active"] * N * 4 if case["bias"] else 0
        return {"bytes": weights + rows * (K + words) + rows * N * o + extra + 4 * (G + 1), "flops": 2 * rows * N * K}
    if case["way"] == "weight":
        return {"bytes": rows * (N + K) * t + G * N * K * o * (2 if case["beta"] else 1) + 4 * (G + 1),
                "flops": 2 * rows * N * K}
    extra = case["active"] * N * 4 if case["bias"] else 0
    return {"bytes": case["active"] * N * K * t + rows * (K * t + N * o if case["way"] == "forward" else N * t + K * o) +
            extra + 4 * (G + 1), "flops": 2 * rows * N * K}


def _w(case):
    return case["type"] if case["w"] == "same" else case["w"]


def _out(case):
    return case["type"] if case["out"] == "same" else case["out"]


# ---- formats, in plain torch -------------------------------------------------------------------

def _padded(x, multiple):
    pad = -x.shape[-1] % multiple
    return torch.nn.functional.pad(x, (0, pad)) if pad else x


def _blocks(x, kind):
    """Rows (fp32) -> elements (M x blocks x 32, scaled, not yet rounded) and exponents (M x blocks)."""
    M = x.shape[0]
    x = _padded(x, 32).view(M, -1, 32)
    top, fraction = _TOP[kind]
    bits = x.abs().amax(-1).view(torch.int32)
    e = ((bits + (0x7fffff - fraction)) >> 23) - top
    e = torch.where(bits == 0, torch.full_like(e, 127), e.clamp(1, 254))
    return x * ((254 - e) << 23).view(torch.float32).unsqueeze(-1), e


def _words(e):
    b = torch.nn.functional.pad(e, (0, -e.shape[1] % 4), value=127).view(e.shape[0], -1, 4)
    return (b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24)).t().contiguous()


def _quantize8(x, kind):
    y, e = _blocks(x, kind)
    return y.to(_TYPES[kind]).view(x.shape[0], -1), _words(e)


def _quantize4(x):
    """The nearest E2M1 value, ties to the even code: steps of 1/2 below 2, of 1 below 4, of 2 above."""
    y, e = _blocks(x, "fp4")
    a = y.abs()
    n = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    n = (n.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).view(x.shape[0], -1)
    return n[:, 0::2] | (n[:, 1::2] << 4), _words(e)


def _scales(words, rows, blocks, dtype):
    """Scale words (... x strips x rows) -> the blocks' scales (... x rows x blocks)."""
    w = words.transpose(-1, -2)
    e = torch.stack((w & 255, (w >> 8) & 255, (w >> 16) & 255, (w >> 24) & 255), -1).flatten(-2)[..., :blocks]
    return (e << 23).view(torch.float32).to(dtype)


def _values(q, words, kind, dtype):
    """The matrix that elements and scale words stand for (... x rows x K)."""
    if kind == "fp4":
        n = torch.stack((q & 15, q >> 4), -1).flatten(-2).int()
        v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=dtype, device=q.device)[n]
    else:
        v = q.to(torch.float32).to(dtype)
    s = _scales(words, v.shape[-2], v.shape[-1] // 32, dtype)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


# ---- inputs ------------------------------------------------------------------------------------

def _pitched(x):
    """The same values in rows whose pitch is a multiple of 16 bytes."""
    per = 16 // x.element_size()
    if x.shape[-1] % per == 0:
        return x.contiguous()
    buf = torch.zeros(*x.shape[:-1], -(-x.shape[-1] // per) * per, dtype=x.dtype, device=x.device)
    buf[..., :x.shape[-1]] = x
    return buf[..., :x.shape[-1]]


def _activations(M, K, gen, device):
    """Hidden states: unit scale, a few columns that are much larger."""
    x = torch.randn(M, K, generator=gen, device=device)
    loud = torch.rand(K, generator=gen, device=device) < 0.01
    return torch.where(loud, x * 20, x)


def _routing(case, gen, device):
    """Offsets of rows sorted by expert: `active` experts have rows, some of them many times others'; also which
    ones, and the largest number of rows of one, which a router's program keeps on the host."""
    G, active, rows = case["G"], case["active"], case["M"] - case["tail"]
    who = torch.randperm(G, generator=gen, device=device)[:active].sort().values
    liked = torch.exp(0.5 * torch.randn(active, generator=gen, device=device))
    more = torch.multinomial(liked, max(1, rows - active), replacement=True, generator=gen)[:rows - active]
    counts = torch.zeros(G, dtype=torch.int64, device=device)
    counts[who] = torch.bincount(more, minlength=active) + 1
    offsets = torch.zeros(G + 1, dtype=torch.int32, device=device)
    offsets[1:] = counts.cumsum(0)
    return offsets, who, int(counts.max())


def prepare(case, seed):
    device = torch.device("cuda", 0)
    gen = torch.Generator(device=device).manual_seed(seed)
    t, op = _TYPES[case["type"]], case["op"]
    state = {"case": case}

    def empty(*shape, dtype):
        return _pitched(torch.zeros(*shape, dtype=dtype, device=device))

    if op == "mx4_quantize":
        M, K = case["M"], case["K"]
        state["X"] = _pitched((torch.randn(M, K, generator=gen, device=device) / math.sqrt(K)).to(t))
        state["Xq"] = torch.empty(M, -(-K // 32) * 16, dtype=torch.uint8, device=device)
        state["SX"] = torch.empty(-(-K // 128), M, dtype=torch.int32, device=device)
        return state
    if op == "rmsnorm":
        M, N = case["M"], case["N"]
        state["w"] = (1 + 0.1 * torch.randn(N, generator=gen, device=device)).to(_TYPES[_w(case)])
        if case["way"] == "backward":
            H = _activations(M, N, gen, device).to(t)
            state["H"] = _pitched(H)
            state["rstd"] = torch.rsqrt(H.double().square().mean(-1) + 1e-5).float()
            state["dY"] = _pitched((torch.randn(M, N, generator=gen, device=device) / 64).to(t))
            state["dH"] = _pitched((torch.randn(M, N, generator=gen, device=device) / 64).to(t)) if case["residual"] else None
            state["dX"] = empty(M, N, dtype=t)
            state["dW"] = torch.empty(N, dtype=torch.float32, device=device)
            return state
        state["X"] = _pitched(_activations(M, N, gen, device).to(t))
        state["R"] = _pitched(_activations(M, N, gen, device).to(t)) if case["residual"] else None
        state["H"] = empty(M, N, dtype=t) if case["residual"] else None
        state["rstd"] = torch.empty(M, dtype=torch.float32, device=device)
        if case["out"] == "same":
            state["Y"] = empty(M, N, dtype=t)
        else:
            state["Y"] = torch.empty(M, -(-N // 32) * 32, dtype=_TYPES[case["out"]], device=device)
            state["SY"] = torch.empty(-(-N // 128), M, dtype=torch.int32, device=device)
        return state
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    state["offsets"], state["active"], state["most"] = _routing(case, gen, device)
    o = _TYPES[_out(case)]
    if case.get("bias"):
        state["bias"] = torch.randn(G, N, generator=gen, device=device)
    if op == "gemm_grouped_mx":
        state["A"], state["SA"] = _quantize8(_activations(M, K, gen, device), case["type"])
        wide = K // 2 if case["weights"] == "fp4" else K
        state["B"] = torch.empty(G, N, wide, dtype=torch.uint8 if case["weights"] == "fp4" else _TYPES["e4m3"], device=device)
        state["SB"] = torch.empty(G, -(-K // 128), N, dtype=torch.int32, device=device)
        for g in range(G):
            W = torch.randn(N, K, generator=gen, device=device) / math.sqrt(K)
            state["B"][g], state["SB"][g] = _quantize4(W) if case["weights"] == "fp4" else _quantize8(W, case["weights"])
        state["D"] = torch.zeros(M, N, dtype=o, device=device)
        return state
    if case["way"] == "weight":
        state["dY"] = _pitched((torch.randn(M, N, generator=gen, device=device) / 64).to(t))
        state["X"] = _pitched(_activations(M, K, gen, device).to(t))
        state["C"] = torch.randn(G, N, K, generator=gen, device=device).to(o) if case["beta"] else None
        state["D"] = torch.empty(G, N, K, dtype=o, device=device)
        return state
    state["W"] = torch.empty(G, N, -(-K // 8) * 8, dtype=t, device=device)[..., :K]
    for g in range(G):
        state["W"][g] = torch.randn(N, K, generator=gen, device=device) / math.sqrt(K)
    if case["way"] == "forward":
        state["A"] = _pitched(_activations(M, K, gen, device).to(t))
        state["D"] = torch.zeros(M, N, dtype=o, device=device)
    else:
        state["A"] = _pitched((torch.randn(M, N, generator=gen, device=device) / 64).to(t))
        state["D"] = torch.zeros(M, K, dtype=o, device=device)
    return state


# ---- one pass ----------------------------------------------------------------------------------

def _own(state):
    import sparse_matrix_multiply_amd as mm

    case, op = state["case"], state["case"]["op"]
    if op == "mx4_quantize":
        return mm.mx4_quantize(state["X"], state["Xq"], state["SX"])
    if op == "rmsnorm":
        if case["way"] == "backward":
            if "workspace" not in state:         # kept with the layer, as a program does
                state["workspace"] = mm.rmsnorm_grad_workspace(case["M"], case["N"], device=state["dY"].device)
            mm.rmsnorm_grad(state["dY"], state["H"], state["w"], state["rstd"], state["dX"], dW=state["dW"],
                            dH=state["dH"], workspace=state["workspace"])
            return state["dX"], state["dW"]
        mm.rmsnorm(state["X"], state["w"], state["Y"], eps=1e-5, residual=state["R"], H=state["H"], rstd=state["rstd"],
                   SY=state.get("SY"))
        if case["out"] == "same":
            return state["H"], state["Y"], state["rstd"]
        return state["H"], state["Y"], state["SY"].view(torch.float8_e8m0fnu), state["rstd"]
    act = mm.ACT_RELU if case.get("relu") else mm.ACT_NONE
    if op == "gemm_grouped_mx":
        return mm.gemm_grouped_mx(state["A"], state["SA"], state["offsets"], state["B"], state["SB"], state["D"],
                                  b_type=mm.FP4_E2M1 if case["weights"] == "fp4" else None, bias=state.get("bias"), act=act)
    if case["way"] == "weight":
        return mm.gemm_grouped_wgrad(state["dY"], state["X"], state["offsets"], state["D"], beta=case["beta"],
                                     C=state["C"])
    return mm.gemm_grouped(state["A"], state["offsets"], state["W"], state["D"], trans_b=case["way"] == "input",
                           bias=state.get("bias"), act=act)


def _by_expert(state):
    """For each expert with rows, its rows' numbers (experts x most rows of one) and which of them it has."""
    first, end = state["offsets"][state["active"]], state["offsets"][state["active"] + 1]
    row = first.unsqueeze(1) + torch.arange(state["most"], device=first.device)
    return row.long(), row < end.unsqueeze(1)


def _rows_by_expert(x, row, has):
    """The rows of x as batches of equal size, zeros where an expert has fewer."""
    return torch.where(has.unsqueeze(-1), x[row.clamp(max=x.shape[0] - 1)].float(), 0.0)


def run(state):
    if own:
        return _own(state)
    case, op = state["case"], state["case"]["op"]
    if op == "mx4_quantize":
        return _quantize4(state["X"].float())
    if op == "rmsnorm":
        w = state["w"].float()
        if case["way"] == "backward":
            dy, xhat = state["dY"].float(), state["H"].float() * state["rstd"].unsqueeze(1)
            v = dy * w
            dx = state["rstd"].unsqueeze(1) * (v - xhat * (v * xhat).mean(-1, keepdim=True))
            if state["dH"] is not None:
                dx = dx + state["dH"].float()
            return dx.to(state["dX"].dtype), (dy * xhat).sum(0)
        h, kept = state["X"], None
        if state["R"] is not None:
            h = kept = (h.float() + state["R"].float()).to(h.dtype)
        h = h.float()
        rstd = torch.rsqrt(h.square().mean(-1) + 1e-5)
        y = h * rstd.unsqueeze(1) * w
        if case["out"] == "same":
            return kept, y.to(state["X"].dtype), rstd
        q, words = _quantize8(y, case["out"])
        return kept, q, words.view(torch.float8_e8m0fnu), rstd
    row, has = _by_expert(state)
    active = state["active"]
    if op == "gemm_grouped" and case["way"] == "weight":
        y, x = _rows_by_expert(state["dY"], row, has), _rows_by_expert(state["X"], row, has)
        d = torch.zeros(state["D"].shape, dtype=torch.float32, device=y.device)
        d[active] = torch.bmm(y.transpose(1, 2).contiguous(), x)
        if state["C"] is not None:
            d = d + case["beta"] * state["C"].float()
        return d.to(state["D"].dtype)
    if op == "gemm_grouped_mx":
        a = _values(state["A"], state["SA"], case["type"], torch.float32)
        W = _values(state["B"][active], state["SB"][active], case["weights"], torch.float32).transpose(1, 2).contiguous()
    else:
        a = state["A"]
        W = state["W"][active].float()
        if case["way"] == "forward":
            W = W.transpose(1, 2).contiguous()
    d = torch.bmm(_rows_by_expert(a, row, has), W)
    if "bias" in state:
        d = d + state["bias"][active].unsqueeze(1)
    if case["relu"]:
        d = d.clamp(min=0)
    out = torch.zeros(state["D"].shape, dtype=state["D"].dtype, device=d.device)
    out[row[has]] = d[has].to(out.dtype)
    return out


# ---- the definition in 64 bits -----------------------------------------------------------------

def _exponents(x, largest):
    """The smallest powers of two (not below 2^-126) that bring the blocks' largest to `largest` or below; 0 for zeros."""
    top = x.abs().amax(-1)
    mantissa, exponent = torch.frexp(top / largest)
    power = torch.where(mantissa == 0.5, exponent - 1, exponent).clamp(min=-126)
    return torch.where(top == 0, torch.zeros_like(power), power)


def _exact_words(power):
    b = torch.nn.functional.pad(power, (0, -power.shape[1] % 4)).view(power.shape[0], -1, 4).long() + 127
    b = (b * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], device=b.device)).sum(-1)
    return torch.where(b >= 1 << 31, b - (1 << 32), b).int().t().contiguous()


def _matrix(q, words, kind):
    """One matrix in 64 bits from its elements and scale words."""
    if kind == "fp4":
        n = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
        n[:, 0::2], n[:, 1::2] = (q % 16).double(), (q // 16).double()
        m = n % 8
        v = torch.where(n >= 8, -1.0, 1.0) * torch.where(m < 2, m / 2, (1 + (m % 2) / 2) * torch.pow(2.0, torch.floor(m / 2) - 1))
    else:
        v = q.float().double()
    block = torch.arange(v.shape[1], device=q.device) // 32
    bits = words.to(torch.int64) & 0xffffffff
    e = (bits[block // 4] >> (8 * (block % 4)).unsqueeze(1)) & 255
    return torch.ldexp(v, (e.t() - 127).double())


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "mx4_quantize":
        x = _padded(state["X"].double(), 32)
        x = x.view(x.shape[0], -1, 32)
        power = _exponents(x, 6.0)
        y = torch.ldexp(x, -power.unsqueeze(-1)).flatten(1)
        n = torch.zeros(y.shape, dtype=torch.int64, device=y.device)
        for i in range(7):                       # up past the middle of two values, and on it where the next code is even
            middle = (_E2M1[i] + _E2M1[i + 1]) / 2
            n += (y.abs() > middle) | ((y.abs() == middle) & bool(i % 2))
        n += 8 * torch.signbit(y)
        return (n[:, 0::2] + 16 * n[:, 1::2]).to(torch.uint8), _exact_words(power)
    if op == "rmsnorm" and case["way"] == "backward":
        dy, h, w, N = state["dY"].double(), state["H"].double(), state["w"].double(), case["N"]
        r = state["rstd"].double().unsqueeze(1)
        dot = (dy * w * h).sum(-1, keepdim=True)
        dx = dy * w * r - h * (r ** 3) * dot / N
        return (dx + state["dH"].double() if state["dH"] is not None else dx), (dy * h * r).sum(0)
    if op == "rmsnorm":
        h, kept = state["X"].double(), None
        if state["R"] is not None:               # the norm is that of the sum as it is kept
            kept = h + state["R"].double()
            h = kept.float().to(state["X"].dtype).double()
        r = 1 / torch.sqrt((h * h).sum(-1) / case["N"] + 1e-5)
        y = h * state["w"].double() * r.unsqueeze(1)
        if case["out"] == "same":
            return kept, y, r
        x = _padded(y, 32).view(y.shape[0], -1, 32)
        power = _exponents(x, _LARGEST[case["out"]])
        q = torch.ldexp(x, -power.unsqueeze(-1)).flatten(1).to(_TYPES[case["out"]])
        scales = torch.ldexp(torch.ones_like(power, dtype=torch.float64), power.double())
        scales = torch.nn.functional.pad(scales, (0, -scales.shape[1] % 4), value=1.0).view(y.shape[0], -1, 4)
        return kept, q.float(), scales.transpose(0, 1).reshape(scales.shape[1], -1), r
    offsets = state["offsets"].tolist()
    out = torch.zeros(state["D"].shape, dtype=torch.float64, device=state["D"].device)
    if op == "gemm_grouped" and case["way"] == "weight":
        for g in range(case["G"]):
            rows = slice(offsets[g], offsets[g + 1])
            out[g] = state["dY"][rows].double().t() @ state["X"][rows].double()
            if state["C"] is not None:
                out[g] += case["beta"] * state["C"][g].double()
        return out
    a = _matrix(state["A"], state["SA"], case["type"]) if op == "gemm_grouped_mx" else state["A"].double()
    for g in range(case["G"]):
        rows = slice(offsets[g], offsets[g + 1])
        if op == "gemm_grouped_mx":
            W = _matrix(state["B"][g], state["SB"][g], case["weights"]).t()
        else:
            W = state["W"][g].double() if case["way"] == "input" else state["W"][g].double().t()
        d = a[rows] @ W
        if case.get("bias"):
            d = d + state["bias"][g].double()
        out[rows] = d.clamp(min=0) if case["relu"] else d
    return out
