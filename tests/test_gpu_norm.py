"""GPU tests of the RMS norm (forward, gradients) and of the 4-bit quantizer against the formulas in 64 bits.

Bounds, with u = 2^-24.  A row's sum of squares has positive terms only: each thread adds at most n = 32 (long rows:
8 * ceil(N / 8192)) of them in turn and 6 + 16 partial sums follow, so it is within (n + 22) u of its value, r within half
of that and 4 u for the mean, eps, root and quotient, y within 2 u more: (n / 2 + 17) u < 64 u up to N = 200 000 (n <= 200 would
need 117: long rows use 128 u).  An output of fewer bits adds half a step.  8-bit outputs: each element is within half a step
of the scaled y, and the exponent is the smallest that holds the block, for a y within that bound.  Gradients: the mean of v * x
has terms of either sign, so its error counts against the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import lowbit_ref as R
import sparse_matrix_multiply_amd as mm
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LOW = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}   # smallest subnormal


def rng(*key):
    return np.random.default_rng([int.from_bytes(str(k).encode(), "little") % (1 << 32) for k in key])


def pitched(x, t, pad=0):
    """Host float64 matrix -> device tensor of type t whose row pitch is a multiple of 16 bytes; the padding is NaN."""
    x = torch.from_numpy(np.ascontiguousarray(x))
    rows, cols = x.shape
    per = 16 // torch.empty((), dtype=t).element_size()
    buf = torch.full((rows, -(-cols // per) * per + pad * per), float("nan"), dtype=t, device=dev())
    buf[:, :cols] = x.to(dev()).to(t)
    return buf[:, :cols]


def guarded(rows, cols, t, fill, per=None):
    """(buffer, view): one guard row above and below and guard columns after each row."""
    per = per or 16 // torch.empty((), dtype=t).element_size()
    buf = torch.full((rows + 2, -(-cols // per) * per + per), fill, device=dev()).to(t)
    return buf, buf[1:rows + 1, :cols]


def check_guards(buf, rows, cols):
    host = buf.float().cpu()
    fill = host[0, 0]
    assert (host[0] == fill).all() and (host[rows + 1] == fill).all() and (host[1:rows + 1, cols:] == fill).all(), "guard cells"


def f64(t):
    return t.double().cpu().numpy()


def half_step(x, t):
    return torch.finfo(t).eps / 2 * np.abs(x) + TINY[t] / 2


def rel(N):
    return (64 if N <= 32768 else 128) * U


def forward(x, r, w, eps, t):
    """h as kept (rounded to t, exact sum of two values of t rounded once to fp32 first only for fp32), r and y in 64 bits."""
    h = x if r is None else torch.from_numpy(x + r).float().to(t).double().numpy()
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


SIZES = [(1, 1), (3, 7), (5, 8), (2, 33), (7, 255), (4, 512), (9, 513), (3, 1000), (2, 1025), (5, 2049), (3, 4104), (2, 8190), (1, 16383), (2, 16400),
         (1, 32768), (2, 40001)]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N", SIZES)
def test_forward(t, residual, M, N):
    t = TYPES[t]
    g = rng(M, N, residual)
    X = pitched(g.standard_normal((M, N)) * 3, t, pad=1)
    Rs = pitched(g.standard_normal((M, N)), t, pad=2) if residual else None
    wt = [torch.float32, t][(M + N) % 2]
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(N)).to(dev()).to(wt)
    ybuf, Y = guarded(M, N, t, 5.0)
    hbuf, H = guarded(M, N, t, 5.0)
    rstd = torch.full((M,), -1.0, device=dev())
    mm.rmsnorm(X, w, Y, eps=1e-5, residual=Rs, H=H, rstd=rstd)
    torch.cuda.synchronize()
    check_guards(ybuf, M, N)
    check_guards(hbuf, M, N)
    h, r, y = forward(f64(X), f64(Rs) if residual else None, f64(w), np.float32(1e-5), t)
    assert np.array_equal(f64(H), h)
    assert (np.abs(f64(rstd) - r) <= rel(N) * r).all()
    assert (np.abs(f64(Y) - y) <= rel(N) * np.abs(y) + (0 if t is torch.float32 else half_step(y * (1 + rel(N)), t)) + TINY[t]).all()


def check_low(Y, SY, y, kind, N, slack):
    """8-bit elements and scale words against y (64 bits), whose fp32 form is within slack * |y| of it."""
    M = y.shape[0]
    kp, nb = -(-N // 32) * 32, -(-N // 32)
    words = SY.cpu().numpy().view(np.uint32)
    e = np.stack([(words >> (8 * q)) & 255 for q in range(4)], 2).transpose(1, 0, 2).reshape(M, -1).astype(np.int64)
    assert (e[:, nb:] == 127).all(), "exponents past the row"
    e = e[:, :nb]
    q = Y.float().double().cpu().numpy()
    assert (q[:, N:] == 0).all(), "elements past the row"
    x = np.zeros((M, kp))
    x[:, :N] = y
    x = x.reshape(M, nb, 32)
    top, T = np.abs(x).max(2), R.TOP[kind]
    s = np.ldexp(1.0, e - 127)
    zero = top == 0
    assert (e[zero] == 127).all()
    assert (top * (1 - slack) <= T * s)[~zero].all(), "a block that its scale does not hold"
    assert ((top * (1 + slack) > T * s / 2) | (e == 1))[~zero].all(), "a scale larger than needed"
    eps, low = (2.0 ** -4, 2.0 ** -10) if kind == "e4m3" else (2.0 ** -3, 2.0 ** -17)
    v = q.reshape(M, nb, 32) * s[:, :, None]
    assert (np.abs(v - x) <= np.maximum(eps * np.abs(x), low * s[:, :, None]) * (1 + slack) + slack * np.abs(x)).all()


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("kind", list(LOW))
@pytest.mark.parametrize("M,N", SIZES)
def test_forward_to_8_bits(t, kind, M, N):
    t = TYPES[t]
    g = rng(M, N, kind)
    x = g.standard_normal((M, N)) * np.exp(2 * g.standard_normal((M, N)))
    x[:, : N // 3 // 32 * 32] *= 2.0 ** -12
    x[-1, 32:64] = 0.0
    X, Rs = pitched(x, t, pad=1), pitched(g.standard_normal((M, N)), t) if M % 2 else None
    if Rs is not None:
        Rs[-1, 32:64] = 0.0
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(N)).float().to(dev())
    kp = -(-N // 32) * 32
    ybuf, Y = guarded(M, kp, torch.uint8, 77, 16)
    sbuf = torch.full((-(-N // 128) + 2, M + 3), -7, dtype=torch.int32, device=dev())
    mm.rmsnorm(X, w, Y.view(LOW[kind]), eps=1e-5, residual=Rs, SY=sbuf[1:-1, :M])
    torch.cuda.synchronize()
    check_guards(ybuf, M, kp)
    s = sbuf.cpu()
    assert (s[0] == -7).all() and (s[-1] == -7).all() and (s[:, M:] == -7).all(), "guard cells"
    _, _, y = forward(f64(X), f64(Rs) if Rs is not None else None, f64(w), np.float32(1e-5), t)
    check_low(Y.view(LOW[kind]), sbuf[1:-1, :M], y, kind, N, rel(N))


@pytest.mark.parametrize("kind", list(LOW))
@pytest.mark.parametrize("N", [96, 777, 4100, 33000])
def test_8_bits_are_the_quantizers(kind, N):
    """Elements of magnitude 1 have r = 1 exactly (eps 0), so y = +-w is exact and the outputs are mx8_quantize's, bit for bit."""
    M = 37
    g = rng(N, kind)
    X = pitched(g.choice([-1.0, 1.0], (M, N)), torch.bfloat16)
    w = torch.from_numpy(g.standard_normal(N) * np.exp(3 * g.standard_normal(N))).float().to(dev())
    y = pitched(f64(X) * f64(w), torch.float32)
    kp = -(-N // 32) * 32
    got = torch.empty(M, kp, dtype=LOW[kind], device=dev()), torch.empty(-(-N // 128), M, dtype=torch.int32, device=dev())
    want = torch.empty_like(got[0]), torch.empty_like(got[1])
    mm.rmsnorm(X, w, got[0], eps=0.0, SY=got[1])
    mm.mx8_quantize(y, *want)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("N", [64, 3001, 40000])
def test_in_place(N):
    """H in the place of X or of the residual, Y in the place of X: the bits of separate buffers."""
    M, t = 11, torch.bfloat16
    g = rng(N)
    X, Rs = pitched(g.standard_normal((M, N)), t), pitched(g.standard_normal((M, N)), t)
    w = torch.from_numpy(g.standard_normal(N)).to(dev()).to(t)
    H, Y = pitched(np.zeros((M, N)), t), pitched(np.zeros((M, N)), t)
    mm.rmsnorm(X, w, Y, residual=Rs, H=H)

    def again(x):
        return pitched(f64(x), t)

    x, r = again(X), again(Rs)
    y = pitched(np.zeros((M, N)), t)
    mm.rmsnorm(x, w, y, residual=r, H=r)
    assert torch.equal(r, H) and torch.equal(y, Y) and torch.equal(x, X)
    x, r = again(X), again(Rs)
    mm.rmsnorm(x, w, y, residual=r, H=x)
    assert torch.equal(x, H) and torch.equal(y, Y)
    x, r = again(X), again(Rs)
    mm.rmsnorm(x, w, x, residual=r, H=r)
    assert torch.equal(x, Y) and torch.equal(r, H)


@pytest.mark.parametrize("N", [200, 5000, 33000])
def test_rows_apart(N):
    """A row with a NaN or an infinity, one of zeros and one whose squares pass fp32 leave the others as they are."""
    M, t = 9, torch.bfloat16
    g = rng(N)
    x = g.standard_normal((M, N))
    clean = pitched(x, t)
    x[1, 5], x[3, N - 1], x[4, 0] = np.nan, np.inf, -np.inf
    x[6] = 0.0
    x[7] = 1e30
    X = pitched(x, t)
    w = torch.ones(N, device=dev())
    out, want = pitched(np.full((M, N), 3.0), t), pitched(np.full((M, N), 3.0), t)
    mm.rmsnorm(X, w, out)
    mm.rmsnorm(clean, w, want)
    for i in (0, 2, 5, 8):
        assert torch.equal(out[i], want[i])
    assert torch.isnan(out[1]).all() and torch.isnan(out[3, N - 1]) and torch.isnan(out[4, 0])
    assert (out[3, : N - 1] == 0).all() and (out[6] == 0).all() and (out[7] == 0).all()
    kp = -(-N // 32) * 32
    q, s = torch.empty(M, kp, dtype=torch.float8_e4m3fn, device=dev()), torch.empty(-(-N // 128), M, dtype=torch.int32, device=dev())
    mm.rmsnorm(X, w, q, SY=s)
    v = q.float()
    assert torch.isnan(v[1, :N]).all() and (v[:, N:] == 0).all() and torch.isnan(v[3, N - 1]) and (v[3, : N - 1] == 0).all() and (v[6] == 0).all()


GRADS = [(1, 1), (2, 7), (5, 64), (13, 257), (700, 512), (33, 1000), (2100, 1024), (6, 2048), (600, 2050), (7, 4099), (3, 8192), (5, 16001),
         (3, 16390), (530, 17000)]


def gradients(dy, h, r, w, dh):
    x, v = h * r[:, None], dy * w
    m = (v * x).mean(1, keepdims=True)
    dx = r[:, None] * (v - x * m)
    mags = r[:, None] * (np.abs(v) + np.abs(x) * (np.abs(v * x)).mean(1, keepdims=True))
    if dh is not None:
        dx, mags = dx + dh, mags + np.abs(dh)
    return dx, mags, (dy * x).sum(0), np.abs(dy * x).sum(0)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,N", GRADS)
def test_gradients(t, M, N):
    t = TYPES[t]
    g = rng(M, N, "grad")
    H, dY = pitched(2 * g.standard_normal((M, N)), t, pad=1), pitched(g.standard_normal((M, N)), t)
    dH = pitched(g.standard_normal((M, N)), t, pad=1) if (M + N) % 3 else None
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(N)).to(dev()).to([torch.float32, t][N % 2])
    rstd = torch.from_numpy(1 / np.sqrt((f64(H) ** 2).mean(1) + 1e-5)).float().to(dev())
    xbuf, dX = guarded(M, N, t, 5.0)
    wbuf = torch.full((N + 8,), 5.0, device=dev())
    ws = mm.rmsnorm_grad_workspace(M, N, dev())
    ws.fill_(255)                                        # need not be cleared, and its first KiB is left alone
    mm.rmsnorm_grad(dY, H, w, rstd, dX, dW=wbuf[:N], dH=dH, workspace=ws)
    torch.cuda.synchronize()
    check_guards(xbuf, M, N)
    assert (wbuf[N:] == 5.0).all() and (ws[:1024] == 255).all()
    dx, mags, dw, dwmags = gradients(f64(dY), f64(H), f64(rstd), f64(w), f64(dH) if dH is not None else None)
    tol = (128 if N <= 32768 else 256) * U * mags
    assert (np.abs(f64(dX) - dx) <= tol + (0 if t is torch.float32 else half_step(np.abs(dx) + tol, t)) + TINY[t]).all()
    # sums over at most ceil(M / parts) rows in turn, 4 waves, ceil(parts / 16) and 16 partial sums; 3 roundings a term
    assert (np.abs(f64(wbuf[:N]) - dw) <= (-(-M // 128) + 60) * U * dwmags + 1e-45).all()
    plain = pitched(np.zeros((M, N)), t)
    mm.rmsnorm_grad(dY, H, w, rstd, plain, dH=dH)        # without dW, without a workspace
    assert torch.equal(plain, dX)
    place = pitched(f64(dY), t)
    mm.rmsnorm_grad(place, H, w, rstd, place, dH=dH)
    assert torch.equal(place, dX)
    if dH is not None:
        place = pitched(f64(dH), t)
        mm.rmsnorm_grad(dY, H, w, rstd, place, dH=place)
        assert torch.equal(place, dX)


def test_gradient_without_rows():
    dW = torch.full((40,), 5.0, device=dev())
    z = torch.empty(0, 40, device=dev())
    mm.rmsnorm_grad(z, z, torch.ones(40, device=dev()), torch.empty(0, device=dev()), z, dW=dW, workspace=mm.rmsnorm_grad_workspace(0, 40, dev()))
    assert (dW == 0).all()


@pytest.mark.parametrize("N", [40, 1500, 9000, 16384, 16388, 40000])
def test_gradient_without_rows_reads_no_workspace(N):
    """dW is zero whatever the workspace holds, in every kernel's range of N; and so without the pointers that no row needs."""
    ws = torch.full_like(mm.rmsnorm_grad_workspace(0, N, dev()), 255)
    z, w, r = torch.empty(0, N, device=dev()), torch.ones(N, device=dev()), torch.empty(0, device=dev())
    dW = torch.full((N + 4,), 5.0, device=dev())
    mm.rmsnorm_grad(z, z, w, r, z, dW=dW[:N], workspace=ws)
    assert (dW[:N] == 0).all() and (dW[N:] == 5).all()


@pytest.mark.parametrize("t", list(TYPES))
def test_without_elements(t):
    """New tensors without rows or columns, whose pitches are no multiple of 16 bytes: nothing to do but a dW of zeros."""
    t = TYPES[t]
    for M, N in ((0, 33), (4, 0), (0, 0)):
        x, w, r = (torch.empty(M, N, dtype=t, device=dev()) for _ in range(5)), torch.ones(N, device=dev()), torch.empty(M, device=dev())
        x, y, h, q, d = x
        mm.rmsnorm(x, w, y, residual=q, H=h, rstd=r)
        dW = torch.full((N,), 5.0, device=dev())
        mm.rmsnorm_grad(y, h, w, r, d, dW=dW, dH=q, workspace=mm.rmsnorm_grad_workspace(M, max(N, 1), dev()))
        assert (dW == 0).all()
        codes = torch.empty(M, -(-N // 32) * 16, dtype=torch.uint8, device=dev())
        mm.mx4_quantize(x, codes, torch.empty(-(-N // 128), M, dtype=torch.int32, device=dev()))


@pytest.mark.parametrize("N", [40, 1500, 9000, 16384, 16388, 40000])
def test_gradient_without_rows_or_pointers(N):
    ws = torch.full_like(mm.rmsnorm_grad_workspace(0, N, dev()), 255)
    dW = torch.full((N,), 5.0, device=dev())
    ld = -(-N // 8) * 8
    assert mm.raw_call("mmac_rmsnorm_grad", mm.BF16, mm.F32, 0, N, None, ld, None, ld, None, None, None, 0, None, ld, dW.data_ptr(),
                       ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == mm.OK
    torch.cuda.synchronize()
    assert (dW == 0).all() and (ws == 255).all()


@pytest.mark.parametrize("N", [40, 1500])
def test_gradients_by_differences(N):
    """The forward pass's central differences along random directions (in 64 bits) against the kernels' gradients: the formula's
    own third-order term, at steps of 1e-4, is far below the bound."""
    M = 6
    g = rng(N, "differences")
    x, w, c = g.standard_normal((M, N)), 1 + 0.2 * g.standard_normal(N), g.standard_normal((M, N))
    x, w, c = (v.astype(np.float32).astype(np.float64) for v in (x, w, c))

    def loss(x, w):
        return (c * x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-5) * w).sum()

    X, W, Y = pitched(x, torch.float32), torch.from_numpy(w).float().to(dev()), pitched(x, torch.float32)
    rstd, dX, dW = torch.empty(M, device=dev()), pitched(x, torch.float32), torch.empty(N, device=dev())
    mm.rmsnorm(X, W, Y, eps=1e-5, rstd=rstd)
    mm.rmsnorm_grad(pitched(c, torch.float32), X, W, rstd, dX, dW=dW, workspace=mm.rmsnorm_grad_workspace(M, N, dev()))
    for _ in range(4):
        d, s = g.standard_normal((M, N)), 1e-4
        want = (loss(x + s * d, w) - loss(x - s * d, w)) / (2 * s)
        assert abs((f64(dX) * d).sum() - want) <= 1e-4 * np.abs(f64(dX) * d).sum()
        d = g.standard_normal(N)
        want = (loss(x, w + s * d) - loss(x, w - s * d)) / (2 * s)
        assert abs((f64(dW) * d).sum() - want) <= 1e-4 * np.abs(f64(dW) * d).sum()


def test_many_rows():
    """More rows than workgroups, and 16-bit rows whose matrix passes 2^31 bytes: the last rows are right."""
    M, N, t = 300_000, 4096, torch.bfloat16
    X = torch.ones(M, N, dtype=t, device=dev())
    X[-2:] = torch.from_numpy(rng(1).standard_normal((2, N))).to(dev()).to(t)
    w = torch.ones(N, device=dev())
    Y, rstd = torch.empty_like(X), torch.empty(M, device=dev())
    mm.rmsnorm(X, w, Y, eps=0.0, rstd=rstd)
    assert (rstd[:-2] == 1).all() and (Y[:-2] == 1).all()
    _, r, y = forward(f64(X[-2:]), None, np.ones(N), 0.0, t)
    assert (np.abs(f64(Y[-2:]) - y) <= rel(N) * np.abs(y) + half_step(y * 1.0001, t)).all()
    dX = torch.empty_like(X)
    dW = torch.empty(N, device=dev())
    mm.rmsnorm_grad(Y, X, w, rstd, dX, dW=dW, workspace=mm.rmsnorm_grad_workspace(M, N, dev()))
    assert (dX[:-2] == 0).all()
    want = (M - 2) + (f64(Y[-2:]) * f64(X[-2:]) * f64(rstd[-2:])[:, None]).sum(0)
    assert (np.abs(f64(dW) - want) <= (M / 128 + 60) * U * (M + 100)).all()


# ---- rows to 4 bits -----------------------------------------------------------------------------

def mx4_reference(x):
    """x float64 (M x K) -> packed codes and exponents."""
    M, K = x.shape
    b = np.zeros((M, -(-K // 32) * 32))
    b[:, :K] = x
    b = b.reshape(M, -1, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(2)
    e = np.full(top.shape, 127, np.int64)
    for i, v in np.ndenumerate(top):                     # the smallest exponent whose power of two holds the block
        if v > 0:
            k = int(np.floor(np.log2(v / 6))) - 1
            while 6 * 2.0 ** k < v:
                k += 1
            e[i] = max(k + 127, 1)
    y = np.ldexp(b, (127 - e)[:, :, None])
    c = R.rne_codes(np.abs(y), R.E2M1) + 8 * np.signbit(y)
    c[bad] = 0
    e[bad] = 255
    return R.pack_codes(c.reshape(M, -1)[:, :K]), e


def run_mx4(X):
    M, K = X.shape
    rb = -(-K // 32) * 16
    qbuf, Xq = guarded(M, rb, torch.uint8, 77, 16)
    sbuf = torch.full((-(-K // 128) + 2, M + 3), -7, dtype=torch.int32, device=dev())
    mm.mx4_quantize(X, Xq, sbuf[1:-1, :M])
    torch.cuda.synchronize()
    check_guards(qbuf, M, rb)
    s = sbuf.cpu()
    assert (s[0] == -7).all() and (s[-1] == -7).all() and (s[:, M:] == -7).all(), "guard cells"
    return Xq, sbuf[1:-1, :M]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 31), (33, 127), (65, 300), (31, 512), (37, 2305)])
def test_mx4_bits(t, M, K):
    g = rng(M, K, "mx4")
    X = pitched(g.standard_normal((M, K)) * np.exp(2 * g.standard_normal((M, 1))), TYPES[t], pad=1)
    Xq, SX = run_mx4(X)
    q, e = mx4_reference(f64(X))
    assert np.array_equal(SX.cpu().numpy(), R.sx_words(e))
    assert np.array_equal(Xq.cpu().numpy(), q)


def test_mx4_special_blocks():
    """Zeros of either sign, ties on every middle, the largest at and next to 6 * 2^k, tiny and huge blocks, NaN and infinities."""
    g = rng("special")
    K = 256
    x = g.standard_normal((16, K)).astype(np.float32).astype(np.float64)
    x[0], x[1] = 0.0, -0.0
    x[2] = g.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], K) * g.choice([-1, 1], K)
    x[2, ::32] = 6.0
    x[3] = x[2] * np.float64(np.float32(1 + 2.0 ** -23))
    x[4] = np.float64(np.nextafter(np.float32(6), np.float32(7)))
    x[5] = np.float64(np.nextafter(np.float32(6), np.float32(5)))
    x[6] *= 2.0 ** -126
    x[7] = 2.0 ** -149
    x[8] = g.choice([-3.4e38, 3.4e38], K)
    x[9, 40], x[10, 200], x[11, 0] = np.nan, np.inf, -np.inf
    x[12] = 1e-30
    x[12, 5::32] = 1.0
    x[13] = -5.0
    X = pitched(x, torch.float32)
    Xq, SX = run_mx4(X)
    q, e = mx4_reference(f64(X))
    assert np.array_equal(SX.cpu().numpy(), R.sx_words(e))
    assert np.array_equal(Xq.cpu().numpy(), q)


def test_mx4_feeds_the_product():
    """gemm_mx from two quantized operands, against the values that they stand for (small integers times powers of two: exact)."""
    M, N, K = 65, 48, 256
    g = rng("product")
    a, b = g.choice([0, 1, -2, 3, 4, -6.0], (M, K)), g.choice([0, -1, 1, 2, 6.0], (N, K))
    a[:, ::32], b[:, ::32] = 6.0, 6.0
    A, SA = run_mx4(pitched(a, torch.bfloat16))
    SA = torch.nn.functional.pad(SA, (0, -M % 4)).contiguous()
    B, SB = run_mx4(pitched(b, torch.bfloat16))
    SB = SB.contiguous()
    D = torch.empty(M, N, device=dev())
    mm.gemm_mx(A.contiguous(), SA, B.contiguous(), SB, D, a_type=mm.FP4_E2M1, b_type=mm.FP4_E2M1)
    assert np.array_equal(f64(D), a @ b.T)
