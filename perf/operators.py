"""Low-bit operands of a linear layer: 4-bit weights with group scales and 8-bit activation
checkpoints with a scale per block, each with the call that makes it and the products that read it.

Cases, inputs, plain forms and exact values of the operators

    w4_quantize     weights (N x K) -> 4-bit codes and one scale word per group of a row
    gemm_w4         D = round(act(alpha * A @ W^T + beta * C + bias)), W the matrix the codes stand for
    mx8_quantize    activations (M x K) -> 8-bit elements and one power-of-two scale per 32 of a row
    mx8_dequantize  the activations that they stand for
    gemm_mx8_wgrad  D = alpha * dY^T @ X + beta * C, the weight's gradient, X read in its 8 bits

Formats.  Codes: two per byte, the lower k in the low nibble, rows of ceil(K / 32) * 16 bytes.  Scale
words (groups x N, int32): the top 24 bits are those of an fp32 scale with 16 significant bits, the low
byte is the zero point.  A group is `group` consecutive k of a row, or the whole row (0).  U4: (n - z) * s;
FP4: the E2M1 value of n times s.  8-bit elements: rows padded to a multiple of 32 with zeros; scale words
(ceil(K / 128) x M, int32): byte q of word t is the exponent e (value 2^(e - 127)) of block 4t + q.
"""
import math

import torch

own = False

U4, FP4 = 9, 6                                   # code types, as the package numbers them
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# exponent of the largest element and the fp32 fraction bits of its significand
_TOP = {"e4m3": (8, 0x600000), "e5m2": (15, 0x600000), "int8": (6, 0x7e0000)}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # one sequence answers token by token: one square projection, where latency counts
        dict(name="w4_one_token", op="gemm_w4", M=1, N=4096, K=4096, group=128, codes="u4", symmetric=True, type="bf16",
             out="bf16", bias=False, relu=False, beta=0.0),
        # a small batch of sequences, sizes that end inside every tile, group and line
        dict(name="w4_ragged_batch", op="gemm_w4", M=13, N=10250, K=4100, group=64, codes="u4", symmetric=False,
             type="fp16", out="fp16", bias=True, relu=False, beta=0.0),
        # the scores over a large vocabulary for a few sequences: 134 MB of codes, small groups
        dict(name="w4_scores", op="gemm_w4", M=4, N=32768, K=8192, group=32, codes="fp4", symmetric=True, type="bf16",
             out="fp32", bias=False, relu=False, beta=0.0),
        # a prompt goes through the same weights: compute counts
        dict(name="w4_prompt", op="gemm_w4", M=2048, N=8192, K=8192, group=128, codes="u4", symmetric=False, type="bf16",
             out="bf16", bias=True, relu=True, beta=0.0),
        # weights of one projection brought to 4 bits, as loaded; and one scale per row at odd sizes
        dict(name="w4_from_bf16", op="w4_quantize", N=8192, K=8192, group=128, codes="u4", symmetric=False, type="bf16"),
        dict(name="w4_whole_rows", op="w4_quantize", N=1000, K=2057, group=0, codes="u4", symmetric=True, type="fp16"),
        # a training step keeps a layer's input for the backward pass in 8 bits
        dict(name="mx8_save", op="mx8_quantize", M=8192, K=8192, type="bf16", codes="e4m3"),
        dict(name="mx8_save_ragged", op="mx8_quantize", M=777, K=1000, type="fp16", codes="int8"),
        # the backward pass of an activation function needs that input itself
        dict(name="mx8_restore", op="mx8_dequantize", M=8192, K=8192, type="bf16", codes="e4m3"),
        dict(name="mx8_restore_ragged", op="mx8_dequantize", M=777, K=1000, type="fp32", codes="int8"),
        # the gradient of a low-rank adapter's first factor (few rows, long sum), and of a full weight, added to
        # the gradient of the steps before
        dict(name="wgrad_adapter", op="gemm_mx8_wgrad", M=8192, N=32, K=8192, type="bf16", codes="e4m3", out="fp32",
             beta=0.0),
        dict(name="wgrad_full", op="gemm_mx8_wgrad", M=8190, N=4096, K=4096, type="bf16", codes="e4m3", out="fp32",
             beta=1.0),
    ]


def _size(rng, lo, hi):
    """A whole number in lo .. hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm_w4", "gemm_w4", "w4_quantize", "mx8_quantize", "mx8_dequantize", "gemm_mx8_wgrad"])
    if op in ("gemm_w4", "w4_quantize"):
        codes = rng.choice(["u4", "u4", "fp4"])
        case = dict(op=op, N=_size(rng, 512, 32768), K=_size(rng, 512, 8192), group=rng.choice([0, 32, 64, 128]),
                    codes=codes, symmetric=codes == "fp4" or rng.random() < 0.5)
        if op == "w4_quantize":
            return dict(case, N=min(case["N"], 8192), type=rng.choice(["bf16", "fp16", "fp32"]))
        rows = _size(rng, 1, 2048)
        rows = max(1, min(rows, (2048 * 8192 * 8192) // (case["N"] * case["K"])))
        return dict(case, M=rows, type=rng.choice(["bf16", "fp16"]), out=rng.choice(["same", "fp32"]),
                    bias=rng.random() < 0.5, relu=rng.random() < 0.3, beta=rng.choice([0.0, 0.0, 1.0]))
    codes = rng.choice(["e4m3", "e4m3", "e5m2", "int8"])
    if op == "gemm_mx8_wgrad":
        return dict(op=op, M=_size(rng, 64, 8192), N=_size(rng, 8, 4096), K=_size(rng, 512, 4096),
                    type=rng.choice(["bf16", "bf16", "fp16"]), codes=codes, out=rng.choice(["fp32", "fp32", "same"]),
                    beta=rng.choice([0.0, 1.0]))
    return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, 512, 8192), type=rng.choice(["bf16", "fp16", "fp32"]), codes=codes)


def _groups(case):
    return 1 if case["group"] == 0 else -(-case["K"] // case["group"])


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    K, op = case["K"], case["op"]
    t = size[case["type"]]
    if op in ("gemm_w4", "w4_quantize"):
        N = case["N"]
        weight = N * K / 2 + 4 * N * _groups(case)
        if op == "w4_quantize":
            return {"bytes": N * K * t + weight, "flops": 4 * N * K}
        M = case["M"]
        o = t if case["out"] in ("same", case["type"]) else 4
        extra = (4 * N if case["bias"] else 0) + (M * N * o if case["beta"] else 0)
        return {"bytes": weight + M * K * t + M * N * o + extra, "flops": 2 * M * N * K}
    M = case["M"]
    kept = M * K + 4 * M * -(-K // 128)
    if op == "gemm_mx8_wgrad":
        N = case["N"]
        o = t if case["out"] == "same" else 4
        return {"bytes": kept + M * N * t + N * K * o * (2 if case["beta"] else 1), "flops": 2 * M * N * K}
    return {"bytes": kept + M * K * t, "flops": 2 * M * K}


# ---- formats, in plain torch -------------------------------------------------------------------

def _round16(s):
    """fp32 scales rounded to 16 significant bits, ties to even."""
    u = s.view(torch.int32)
    return ((u + 0x7f + ((u >> 8) & 1)) & ~0xff).view(torch.float32)


def _padded(x, multiple):
    pad = -x.shape[-1] % multiple
    return torch.nn.functional.pad(x, (0, pad)) if pad else x


def _by_group(x, group):
    """N x K -> N x groups x group, zeros past K."""
    group = group or x.shape[1]
    x = _padded(x, group)
    return x.view(x.shape[0], -1, group)


def _pack(n, K):
    """Codes (N x K) -> N x 16 ceil(K / 32) bytes, zero codes past K."""
    n = _padded(n[:, :K].to(torch.uint8), 32)
    return (n[:, 0::2] | (n[:, 1::2] << 4)).contiguous()


def _quantize4(W, case):
    """The operator's definition: codes and scale words, with every quotient in 64 bits."""
    x = _by_group(W.float(), case["group"])
    if case["codes"] == "fp4":
        top, steps = x.abs().amax(-1), 6.0
    elif case["symmetric"]:
        top, steps = x.abs().amax(-1), 7.0
    else:
        top, steps = x.amax(-1).clamp(min=0) - x.amin(-1).clamp(max=0), 15.0
    s = (top.double() / torch.full_like(top, steps, dtype=torch.float64)).float()
    s = _round16(torch.where(s < 2.0 ** -126, torch.zeros_like(s), s))
    nil = s == 0
    ratio = x.double() / torch.where(nil, torch.ones_like(s), s).double().unsqueeze(-1)
    ratio = torch.where(nil.unsqueeze(-1), torch.zeros_like(ratio), ratio)
    if case["codes"] == "fp4":
        z = torch.zeros_like(s)
        # the nearest E2M1 value, ties to the even code: steps of 1/2 below 2, of 1 below 4, of 2 above
        a = ratio.abs()
        n = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4)).clamp(max=7)
        n = n + 8 * (ratio < 0)
    else:
        if case["symmetric"]:
            z = torch.full_like(s, 8.0)
        else:
            lo = x.amin(-1).clamp(max=0).double()
            z = torch.round(-lo / torch.where(nil, torch.ones_like(s), s).double()).clamp(0, 15)
            z = torch.where(nil, torch.zeros_like(z), z)
        n = (torch.round(ratio) + z.unsqueeze(-1)).clamp(0, 15)
    words = (s.view(torch.int32) | z.to(torch.int32)).t().contiguous()
    return _pack(n.flatten(1), W.shape[1]), words


def _weights4(Wq, words, case, dtype):
    """The matrix (N x K) that the codes stand for."""
    N, K = Wq.shape[0], case["K"]
    n = torch.stack((Wq & 15, Wq >> 4), -1).view(N, -1)[:, :K]
    w = words[:, :N].t()
    s, z = (w & ~0xff).view(torch.float32).to(dtype), (w & 0xff).to(dtype)
    if case["codes"] == "fp4":
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=Wq.device)
        v = table[n.long()]
    else:
        v = n.to(dtype)
    v = _by_group(v, case["group"])
    if case["codes"] != "fp4":
        v = v - z.unsqueeze(-1)
    return (v * s.unsqueeze(-1)).flatten(1)[:, :K]


def _quantize8(X, codes):
    M, K = X.shape
    x = _padded(X.float(), 32).view(M, -1, 32)
    top, fraction = _TOP[codes]
    bits = x.abs().amax(-1).view(torch.int32)
    e = ((bits + (0x7fffff - fraction)) >> 23) - top
    e = torch.where(bits == 0, torch.full_like(e, 127), e.clamp(1, 254))
    y = x * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)
    q = (torch.round(y).to(torch.int8) if codes == "int8" else y.to(_TYPES[codes])).view(M, -1)
    pad = -e.shape[1] % 4
    b = torch.nn.functional.pad(e, (0, pad), value=127).view(M, -1, 4)
    words = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24)
    return q, words.t().contiguous()


def _values8(Xq, words, K, dtype):
    """The matrix (M x K) that the 8-bit elements stand for."""
    M = Xq.shape[0]
    w = words[:, :M].t()
    e = torch.stack((w & 255, (w >> 8) & 255, (w >> 16) & 255, (w >> 24) & 255), -1).view(M, -1)[:, :Xq.shape[1] // 32]
    s = (e << 23).view(torch.float32).to(dtype)
    return (Xq.to(torch.float32).to(dtype).view(M, -1, 32) * s.unsqueeze(-1)).view(M, -1)[:, :K]


# ---- inputs ------------------------------------------------------------------------------------

def _pitched(x):
    """The same values in rows whose pitch is a multiple of 16 bytes."""
    per = 16 // x.element_size()
    if x.shape[1] % per == 0:
        return x.contiguous()
    buf = torch.zeros(x.shape[0], -(-x.shape[1] // per) * per, dtype=x.dtype, device=x.device)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def _activations(M, K, gen, device):
    """Hidden states: unit scale, a few columns that are much larger."""
    x = torch.randn(M, K, generator=gen, device=device)
    loud = torch.rand(K, generator=gen, device=device) < 0.01
    return torch.where(loud, x * 20, x)


def prepare(case, seed):
    device = torch.device("cuda", 0)
    gen = torch.Generator(device=device).manual_seed(seed)
    t = _TYPES[case["type"]]
    K, op = case["K"], case["op"]
    state = {"case": case}
    if op in ("gemm_w4", "w4_quantize"):
        N = case["N"]
        W = torch.randn(N, K, generator=gen, device=device) / math.sqrt(K)
        rows = -(-K // 32) * 16
        if op == "w4_quantize":
            state["W"] = _pitched(W.to(t))
            state["Wq"] = torch.empty(N, rows, dtype=torch.uint8, device=device)
            state["SW"] = torch.empty(_groups(case), N, dtype=torch.int32, device=device)
            return state
        state["Wq"], state["SW"] = _quantize4(W, case)
        del W
        M = case["M"]
        o = t if case["out"] in ("same", case["type"]) else torch.float32
        state["A"] = _pitched(_activations(M, K, gen, device).to(t))
        state["bias"] = torch.randn(N, generator=gen, device=device) if case["bias"] else None
        state["C"] = torch.randn(M, N, generator=gen, device=device).to(o) if case["beta"] else None
        state["D"] = torch.empty(M, N, dtype=o, device=device)
        return state
    M = case["M"]
    X = _activations(M, K, gen, device)
    wide = -(-K // 32) * 32
    if op == "mx8_quantize":
        state["X"] = _pitched(X.to(t))
        state["Xq"] = torch.empty(M, wide, dtype=_TYPES[case["codes"]], device=device)
        state["SX"] = torch.empty(-(-K // 128), M, dtype=torch.int32, device=device)
        return state
    state["Xq"], state["SX"] = _quantize8(X, case["codes"])
    del X
    if op == "mx8_dequantize":
        state["X"] = _pitched(torch.empty(M, K, dtype=t, device=device))
        return state
    N = case["N"]
    o = t if case["out"] == "same" else torch.float32
    state["dY"] = _pitched((torch.randn(M, N, generator=gen, device=device) / 64).to(t))
    state["C"] = torch.randn(N, K, generator=gen, device=device).to(o) if case["beta"] else None
    state["D"] = torch.empty(N, K, dtype=o, device=device)
    return state


# ---- one pass ----------------------------------------------------------------------------------

def _own(state):
    import sparse_matrix_multiply_amd as mm

    case, op = state["case"], state["case"]["op"]
    q4 = mm.FP4_E2M1 if case["codes"] == "fp4" else mm.U4
    if op == "gemm_w4":
        if "workspace" not in state:             # kept with the weights, as a program does
            state["workspace"] = mm.w4_workspace(case["M"], case["N"], case["K"], device=state["A"].device)
        return mm.gemm_w4(state["A"], state["Wq"], state["SW"], state["D"], group=case["group"], q_type=q4,
                          beta=case["beta"], C=state["C"], bias=state["bias"],
                          act=mm.ACT_RELU if case["relu"] else mm.ACT_NONE, workspace=state["workspace"])
    if op == "w4_quantize":
        return mm.w4_quantize(state["W"], state["Wq"], state["SW"], group=case["group"], q_type=q4,
                              symmetric=case["symmetric"])
    if op == "mx8_quantize":
        return mm.mx8_quantize(state["X"], state["Xq"], state["SX"])
    if op == "mx8_dequantize":
        return mm.mx8_dequantize(state["Xq"], state["SX"], state["X"])
    if "workspace" not in state:
        state["workspace"] = mm.mx8_wgrad_workspace(case["M"], case["N"], case["K"], device=state["dY"].device)
    return mm.gemm_mx8_wgrad(state["dY"], state["Xq"], state["SX"], state["D"], beta=case["beta"], C=state["C"],
                             workspace=state["workspace"])


def run(state):
    if own:
        return _own(state)
    case, op = state["case"], state["case"]["op"]
    if op == "gemm_w4":
        d = state["A"].float() @ _weights4(state["Wq"], state["SW"], case, torch.float32).t()
        if state["C"] is not None:
            d = d + case["beta"] * state["C"].float()
        if state["bias"] is not None:
            d = d + state["bias"]
        if case["relu"]:
            d = d.clamp(min=0)
        return d.to(state["D"].dtype)
    if op == "w4_quantize":
        return _quantize4(state["W"], case)
    if op == "mx8_quantize":
        return _quantize8(state["X"], case["codes"])
    if op == "mx8_dequantize":
        return _values8(state["Xq"], state["SX"], case["K"], torch.float32).to(state["X"].dtype)
    d = state["dY"].float().t() @ _values8(state["Xq"], state["SX"], case["K"], torch.float32)
    if state["C"] is not None:
        d = d + case["beta"] * state["C"].float()
    return d.to(state["D"].dtype)


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "w4_quantize":
        W = state["W"].double()
        N, K = W.shape
        group = case["group"] or K
        x = _padded(W, group).view(N, -1, group)
        high, low = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
        if case["codes"] == "fp4" or case["symmetric"]:
            high, low = torch.maximum(high, -low), torch.zeros_like(low)
        steps = 6.0 if case["codes"] == "fp4" else 7.0 if case["symmetric"] else 15.0
        mantissa, exponent = torch.frexp(((high - low).float().double() / steps).float().double())
        s = torch.ldexp(torch.round(mantissa * 65536), exponent - 16)        # 16 significant bits
        s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
        r = torch.where(s.unsqueeze(-1) > 0, x / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1), torch.zeros_like(x))
        if case["codes"] == "fp4":
            z = torch.zeros_like(s)
            n = torch.zeros_like(r)
            for i in range(7):                   # up past the middle of two values, and on it where the next code is even
                middle = (_E2M1[i] + _E2M1[i + 1]) / 2
                n += (r.abs() > middle) | ((r.abs() == middle) & bool(i % 2))
            n += 8 * (r < 0)
        else:
            z = torch.where(s > 0, torch.round(-low / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15), torch.zeros_like(s))
            z = torch.full_like(s, 8) if case["symmetric"] else z
            n = (torch.round(r) + z.unsqueeze(-1)).clamp(0, 15)
        n = torch.nn.functional.pad(n.flatten(1)[:, :K], (0, -K % 32)).long()
        return (n[:, 0::2] + 16 * n[:, 1::2]).to(torch.uint8), (s.float().view(torch.int32) + z.int()).t().contiguous()
    if op == "mx8_quantize":
        x = _padded(state["X"].double(), 32)
        x = x.view(x.shape[0], -1, 32)
        top = x.abs().amax(-1)
        largest = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}[case["codes"]]
        # the smallest power of two (not below 2^-126) that brings the block's largest to the type's largest or below
        mantissa, exponent = torch.frexp(top / largest)
        power = torch.where(mantissa == 0.5, exponent - 1, exponent).clamp(min=-126)
        power = torch.where(top == 0, torch.zeros_like(power), power)
        y = torch.ldexp(x, -power.unsqueeze(-1)).flatten(1)
        words = torch.nn.functional.pad(power, (0, -power.shape[1] % 4)).view(x.shape[0], -1, 4).long() + 127
        words = (words * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], device=words.device)).sum(-1)
        words = torch.where(words >= 1 << 31, words - (1 << 32), words).int().t().contiguous()
        return torch.round(y).to(torch.int8) if case["codes"] == "int8" else y, words
    if op == "gemm_w4":
        N, K = case["N"], case["K"]
        packed = state["Wq"].to(torch.int16)
        n = torch.empty(N, 2 * packed.shape[1], dtype=torch.float64, device=packed.device)
        n[:, 0::2], n[:, 1::2] = (packed % 16).double(), (packed // 16).double()
        n = n[:, :K]
        group = torch.arange(K, device=n.device) // (case["group"] or K)
        bits = state["SW"].to(torch.int64) & 0xffffffff
        s = torch.ldexp(((bits >> 8 & 0x7fff) + 0x8000).double(), ((bits >> 23) - 142).double())
        s = torch.where(bits >> 23 == 0, torch.zeros_like(s), s)
        z = (bits & 0xff).double()
        if case["codes"] == "fp4":
            sign = torch.where(n >= 8, -1.0, 1.0)
            m = n % 8
            n = sign * torch.where(m < 2, m / 2, (1 + (m % 2) / 2) * torch.pow(2.0, torch.floor(m / 2) - 1))
        else:
            n = n - z[group].t()
        d = state["A"].double() @ (n * s[group].t()).t()
        if state["C"] is not None:
            d = d + case["beta"] * state["C"].double()
        if state["bias"] is not None:
            d = d + state["bias"].double()
        return d.clamp(min=0) if case["relu"] else d
    M, K = case["M"], case["K"]
    block = torch.arange(K, device=state["Xq"].device) // 32
    bits = state["SX"].to(torch.int64) & 0xffffffff
    e = (bits[block // 4] >> (8 * (block % 4)).unsqueeze(1)) & 255          # K x M
    x = torch.ldexp(state["Xq"][:, :K].float().double(), (e.t() - 127).double())
    if op == "mx8_dequantize":
        return x
    d = state["dY"].double().t() @ x
    return d + case["beta"] * state["C"].double() if state["C"] is not None else d
