"""GPU tests of the products grouped by expert against the formulas in 64 bits.

With S the sum of the magnitudes of a sum's terms and u = 2^-24, fp32 sums of n terms are within 2 (n + 32) u S element by element
(each addition rounds once, doubled for an accumulator that truncates; 32 covers the epilogue and the joins of partial sums).  The block-scaled matrix
instructions add an error of their own, 2^-13 S (outputs of 16 bits or fewer; fp32 outputs are formed without them), and an output
of fewer bits half a step.  Small integers with power-of-two scales make every sum exact: those must match bit for bit.
"""
import numpy as np
import pytest
import torch

import lowbit_ref as R
import sparse_matrix_multiply_amd as mm
from gpu_helpers import dev
from test_gpu_norm import check_guards, f64, guarded, half_step, pitched, rng

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
OUT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}

# sizes of the groups, rows before the first and behind the last
ROWS = {
    "one": ([1], 0, 0),
    "single": ([0, 0, 1, 0], 0, 0),
    "few": ([2, 0, 5, 1], 0, 3),
    "none": ([0, 0, 0], 2, 4),
    "uneven": ([0, 33, 1, 0, 130, 64, 15], 3, 5),
    "edges": ([16, 17, 32, 31, 64, 65, 127, 128, 129], 0, 0),
    "all_in_one": ([0, 300, 0], 0, 0),
    "long": ([257, 0, 513], 1, 2),
    "many": ([0, 1, 3, 0, 2] * 27, 0, 1),
    "many_long": ([0, 70, 3, 0, 140] * 27, 2, 0),
    "crowd": ([1, 0, 2] * 90 + [150, 0, 20] * 3, 1, 0),
}


def offsets(sizes, before, behind):
    o = np.concatenate([[before], before + np.cumsum(sizes)]).astype(np.int32)
    return o, int(o[-1]) + behind


def matrices(x, t, pad=0):
    """Host float64 (groups x rows x cols) -> device tensor whose row pitch is a multiple of 16 bytes; padding NaN, a gap between groups."""
    G, rows, cols = x.shape
    per = 16 // torch.empty((), dtype=t).element_size()
    ld = -(-cols // per) * per + pad * per
    buf = torch.full((G, rows + pad, ld), float("nan"), dtype=t, device=dev())
    buf[:, :rows, :cols] = torch.from_numpy(x).to(dev()).to(t)
    return buf[:, :rows, :cols]


def check_sums(got, want, mags, n, t, extra=0.0):
    tol = (2 * (n + 32) * U + extra) * mags
    if t is not torch.float32:
        want = np.clip(want, -torch.finfo(t).max, torch.finfo(t).max)          # finite outputs saturate
        tol = tol + half_step(np.abs(want) + tol, t) if t.itemsize == 2 else tol + np.maximum(torch.finfo(t).eps / 2 * (np.abs(want) + tol), torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(got - want) / tol):.3g} of the bound"


def forward_case(sizes, before, behind, N, K, t, trans, integers, key, bias, beta):
    g = rng(len(sizes), N, K, str(t), trans, integers, key)
    o, M = offsets(sizes, before, behind)
    G = len(sizes)
    a = g.integers(-3, 4, (M, K)) if integers else g.standard_normal((M, K))
    b = g.integers(-3, 4, (G, N, K)) if integers else g.standard_normal((G, N, K)) / np.sqrt(max(K, 1))
    A = pitched(a.astype(np.float64), t, pad=1)
    A[:before], A[M - behind:] = float("nan"), float("nan")      # rows of no group are not read
    B = matrices((np.swapaxes(b, 1, 2) if trans else b).astype(np.float64), t, pad=1)
    vec = g.integers(-3, 4, (G, N)).astype(np.float64) if bias else None
    c = (g.integers(-3, 4, (M, N)) if integers else g.standard_normal((M, N))) if beta else None
    return o, M, A, B, vec, c


def run_forward(rows, N, K, t, trans=False, out=torch.float32, integers=False, bias=False, relu=False, alpha=1.0, beta=0.0, key=0):
    sizes, before, behind = rows
    o, M, A, B, vec, c = forward_case(sizes, before, behind, N, K, t, trans, integers, key, bias, beta)
    C = pitched(c.astype(np.float64), out, pad=1) if c is not None else None
    dbuf, D = guarded(M, N, out, 5.0)
    mm.gemm_grouped(A, torch.from_numpy(o).to(dev()), B, D, trans_b=trans, alpha=alpha, beta=beta, C=C,
                    bias=torch.from_numpy(vec).float().to(dev()) if bias else None, act=mm.ACT_RELU if relu else mm.ACT_NONE)
    torch.cuda.synchronize()
    check_guards(dbuf, M, N)
    got, a, b = f64(D), f64(A), f64(B)
    assert (got[:o[0]] == 5).all() and (got[o[-1]:] == 5).all(), "rows of no group"
    cc = f64(C) if C is not None else None
    for i in range(len(sizes)):
        r = slice(o[i], o[i + 1])
        w = b[i] if trans else b[i].T
        want, mags = alpha * (a[r] @ w), abs(alpha) * (np.abs(a[r]) @ np.abs(w))
        if cc is not None:
            want, mags = want + beta * cc[r], mags + abs(beta) * np.abs(cc[r])
        if bias:
            want, mags = want + vec[i], mags + np.abs(vec[i])
        if relu:
            want = np.maximum(want, 0)
        if integers:
            assert np.array_equal(got[r], torch.from_numpy(want).to(out).double().numpy()), f"group {i}"
        elif want.size:
            check_sums(got[r], want, mags, K, out)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", [(1, 1), (37, 71), (130, 520), (200, 128)])
def test_forward(t, trans, rows, N, K):
    run_forward(ROWS[rows], N, K, TYPES[t], trans=trans)


@pytest.mark.parametrize("tile", [16, 32, 64, 128, 1282, 256])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K", [1, 64, 200, 704])
def test_every_tile_exact(tile, trans, K, monkeypatch):
    """Each tile shape on groups of every size, all epilogue terms, bit for bit on small integers."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    for k, rows in enumerate(("uneven", "edges", "long", "many", "none", "many_long", "crowd")):
        run_forward(ROWS[rows], 270 if k % 2 else 263, K, torch.bfloat16, trans=trans, integers=True, bias=k % 2 == 0, relu=k == 1,
                    alpha=[1.0, 2.0, -1.0][k % 3], beta=[0.0, 1.0, 2.0][k % 3])


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("tile", [16, 64, 256])
def test_epilogue(out, tile, monkeypatch):
    monkeypatch.setenv("MMAC_TILE", str(tile))
    run_forward(ROWS["uneven"], 72, 96, torch.float16, out=OUT[out], bias=True, relu=True, alpha=0.5, beta=-0.25)
    run_forward(ROWS["few"], 71, 96, torch.float16, out=OUT[out], beta=1.0)
    run_forward(ROWS["few"], 64, 0, torch.float16, out=OUT[out], bias=True, beta=2.0)


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("tile", [16, 64, 128, 256])
def test_outputs_of_any_alignment(out, tile, monkeypatch):
    """C and D of odd pitches that start at odd elements: the wide accesses at any address, and nothing beside the matrix written."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    sizes, before, behind = ROWS["uneven"]
    g = rng("odd", out, tile)
    o, M = offsets(sizes, before, behind)
    t = OUT[out]
    for N in (135, 270):
        a, b, c = g.integers(-2, 3, (M, 64)), g.integers(-2, 3, (len(sizes), N, 64)), g.integers(-2, 3, (M, N))
        buf = torch.full((M + 2, N + 4), 5.0, device=dev()).to(t)
        if buf.shape[1] % 2 == 0:
            buf = torch.full((M + 2, N + 5), 5.0, device=dev()).to(t)
        D = buf[1:M + 1, 1:N + 1]
        C = torch.zeros(M, N + 3 + N % 2, device=dev()).to(t)[:, 1:N + 1]
        C.copy_(torch.from_numpy(c.astype(np.float64)).to(dev()).to(t))
        mm.gemm_grouped(pitched(a.astype(np.float64), torch.bfloat16), torch.from_numpy(o).to(dev()), matrices(b.astype(np.float64), torch.bfloat16), D,
                        alpha=0.5, beta=2.0, C=C)
        torch.cuda.synchronize()
        host, got = buf.float().cpu(), f64(D.float())
        assert (host[0] == 5).all() and (host[-1] == 5).all() and (host[:, 0] == 5).all() and (host[:, N + 1:] == 5).all(), "guard cells"
        for i in range(len(sizes)):
            r = slice(o[i], o[i + 1])
            want = torch.from_numpy(0.5 * (a[r] @ b[i].T) + 2.0 * c[r]).to(t).double().numpy()
            assert np.array_equal(got[r], want), f"group {i}"


def test_the_skinny_products_bits():
    """A group of at most 16 rows has gemm_dense's bits for those rows (the same kernel, the same order)."""
    g = rng("skinny")
    a, b = pitched(g.standard_normal((16, 1000)), torch.bfloat16), matrices(g.standard_normal((3, 130, 1000)), torch.bfloat16)
    o = torch.tensor([0, 5, 5, 16], dtype=torch.int32, device=dev())
    D, E = torch.empty(16, 130, device=dev()), torch.empty(16, 130, device=dev())
    mm.gemm_grouped(a, o, b, D)
    mm.gemm_dense(a[:5], b[0], E[:5])
    mm.gemm_dense(a[5:], b[2], E[5:])
    assert torch.equal(D, E)


def test_other_groups_do_not_leak():
    """NaN in one group's rows, weights or bias stays there."""
    g = rng("leak")
    o = np.array([0, 20, 45, 70], np.int32)
    for tile in (None, 256):
        a, b = g.standard_normal((70, 256)), g.standard_normal((3, 96, 256))
        a[20:45], b[1] = np.nan, np.nan
        bias = torch.zeros(3, 96, device=dev())
        bias[1] = float("nan")
        A, B, D = pitched(a, torch.bfloat16), matrices(b, torch.bfloat16), torch.empty(70, 96, device=dev())
        mm.gemm_grouped(A, torch.from_numpy(o).to(dev()), B, D, bias=bias)
        assert torch.isnan(D[20:45]).all() and torch.isfinite(D[:20]).all() and torch.isfinite(D[45:]).all()
        W = torch.empty(3, 96, 256, device=dev())
        mm.gemm_grouped_wgrad(pitched(g.standard_normal((70, 96)), torch.bfloat16), A, torch.from_numpy(o).to(dev()), W)
        assert torch.isnan(W[1]).all() and torch.isfinite(W[0]).all() and torch.isfinite(W[2]).all()


@pytest.mark.parametrize("tile", [None, 16, 32, 64, 128, 1282, 256])
@pytest.mark.parametrize("trans", [False, True])
def test_other_groups_do_not_leak_in_any_tile(tile, trans, monkeypatch):
    """NaN in one group's rows, weights or bias stays there: whole and half tiles of 150 and 300 rows beside the group's own, K in the
    middle of a k-tile."""
    if tile is not None:
        monkeypatch.setenv("MMAC_TILE", str(tile))
    g = rng("leak", trans)
    K, N, o = 200, 280, np.cumsum([0, 150, 20, 300, 45, 130]).astype(np.int32)
    a, b = g.standard_normal((o[-1], K)), g.standard_normal((5, N, K))
    rows = np.zeros(o[-1], bool)
    for i in (1, 3):
        rows[o[i]:o[i + 1]] = True
        b[i] = np.nan
    a[rows] = np.nan
    bias = torch.zeros(5, N, device=dev())
    bias[1] = float("nan")
    A, off = pitched(a, torch.bfloat16), torch.from_numpy(o).to(dev())
    B = matrices(np.swapaxes(b, 1, 2) if trans else b, torch.bfloat16)
    for t in (torch.float32, torch.bfloat16):
        D = torch.empty(int(o[-1]), N, dtype=t, device=dev())
        mm.gemm_grouped(A, off, B, D, trans_b=trans, bias=bias)
        bad = torch.isnan(D).cpu().numpy()
        assert bad[rows].all() and not bad[~rows].any()
        W = torch.empty(5, N, K, dtype=t, device=dev())
        mm.gemm_grouped_wgrad(pitched(g.standard_normal((o[-1], N)), torch.bfloat16), A, off, W)
        assert torch.isnan(W[[1, 3]]).all() and torch.isfinite(W[[0, 2, 4]]).all()


@pytest.mark.parametrize("bad", [[0, 40, 20, 64], [-5, 10, 30, 64], [0, 10, 1000, 2000], [70, 80, 90, 100], [2 ** 31 - 1, -(2 ** 31), 5, 2 ** 31 - 1]])
def test_bad_offsets_stay_inside(bad):
    """Offsets that decrease or leave the arrays: nothing outside them is touched."""
    M, N, K = 64, 48, 64
    A, B = pitched(np.ones((M, K)), torch.bfloat16), matrices(np.ones((3, N, K)), torch.bfloat16)
    o = torch.tensor(bad, dtype=torch.int32, device=dev())
    dbuf, D = guarded(M, N, torch.float32, 5.0)
    mm.gemm_grouped(A, o, B, D)
    W = torch.full((5, N, K), 5.0, device=dev())
    mm.gemm_grouped_wgrad(pitched(np.ones((M, N)), torch.bfloat16), A, o, W[1:4])
    torch.cuda.synchronize()
    check_guards(dbuf, M, N)
    assert (W[0] == 5).all() and (W[4] == 5).all()
    assert ((D == 5) | (D == K)).all()


@pytest.mark.parametrize("G,N,K", [(80_000, 2048, 16), (34_000, 16384, 8)])
def test_forward_of_many_tiles(G, N, K):
    """A row a group and more workgroups than 2^21 (the second: than small tiles can be launched): every row meets its group's weights."""
    gen = torch.Generator(device=dev()).manual_seed(G)
    A = torch.randint(-2, 3, (G, K), device=dev(), generator=gen, dtype=torch.int8).to(torch.bfloat16)
    B = torch.randint(-2, 3, (G, N, K), device=dev(), generator=gen, dtype=torch.int8).to(torch.bfloat16)    # 5.2 and 8.9 GB
    o = torch.arange(G + 1, dtype=torch.int32, device=dev())
    D = torch.full((G, N), 99.0, dtype=torch.bfloat16, device=dev())
    mm.gemm_grouped(A, o, B, D)
    for i in range(0, G, 5_000):
        want = torch.zeros(min(5_000, G - i), N, device=dev())
        for k in range(K):
            want += A[i:i + 5_000, k:k + 1].float() * B[i:i + 5_000, :, k].float()
        assert torch.equal(D[i:i + 5_000].float(), want), i                     # sums of at most 64: exact in bf16


# ---- weight gradient ----------------------------------------------------------------------------

def run_wgrad(rows, N, K, t, out=torch.float32, integers=False, alpha=1.0, beta=0.0, same=False, key=0):
    sizes, before, behind = rows
    g = rng(len(sizes), N, K, str(t), integers, key)
    o, M = offsets(sizes, before, behind)
    G = len(sizes)
    dy = g.integers(-3, 4, (M, N)).astype(np.float64) if integers else g.standard_normal((M, N))
    x = g.integers(-3, 4, (M, K)).astype(np.float64) if integers else g.standard_normal((M, K))
    dY, X = pitched(dy, t, pad=1), pitched(x, t)
    for v in (dY, X):
        v[:before], v[M - behind:] = float("nan"), float("nan")
    buf = torch.full((G + 2, N + 1, K + 3), 5.0, device=dev()).to(out)
    D = buf[1:G + 1, :N, :K]
    C = None
    if beta:
        c = torch.from_numpy(g.integers(-3, 4, (G, N, K)).astype(np.float64)).to(dev()).to(out)
        C = D if same else c
        if same:
            D.copy_(c)
        cc = f64(c)
    mm.gemm_grouped_wgrad(dY, X, torch.from_numpy(o).to(dev()), D, alpha=alpha, beta=beta, C=C)
    torch.cuda.synchronize()
    host = buf.float().cpu()
    assert (host[0] == 5).all() and (host[-1] == 5).all() and (host[:, N] == 5).all() and (host[:, :, K:] == 5).all(), "guard cells"
    got, dy, x = f64(D), f64(dY), f64(X)
    for i in range(G):
        r = slice(o[i], o[i + 1])
        want, mags = alpha * (dy[r].T @ x[r]), abs(alpha) * (np.abs(dy[r]).T @ np.abs(x[r]))
        if beta:
            want, mags = want + beta * cc[i], mags + abs(beta) * np.abs(cc[i])
        if integers:
            assert np.array_equal(got[i], torch.from_numpy(want).to(out).double().numpy()), f"group {i}"
        else:
            check_sums(got[i], want, mags, sizes[i], out)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("N,K", [(1, 1), (37, 71), (96, 130)])
def test_wgrad(t, rows, N, K):
    run_wgrad(ROWS[rows], N, K, TYPES[t])


@pytest.mark.parametrize("tile", [64, 128, 1282, 256])
@pytest.mark.parametrize("beta,same", [(0.0, False), (1.0, True), (2.0, False)])
def test_wgrad_every_tile_exact(tile, beta, same, monkeypatch):
    monkeypatch.setenv("MMAC_TILE", str(tile))
    for rows in ("uneven", "long", "none", "single"):
        run_wgrad(ROWS[rows], 263, 270, torch.bfloat16, integers=True, alpha=[1.0, 2.0][beta == 2.0], beta=beta, same=same)


@pytest.mark.parametrize("out", list(OUT))
def test_wgrad_outputs(out):
    run_wgrad(ROWS["uneven"], 40, 64, torch.float16, out=OUT[out], alpha=0.5, beta=-0.25)
    run_wgrad(ROWS["few"], 33, 65, torch.float16, out=OUT[out], beta=1.0, same=True)


@pytest.mark.parametrize("G,N,K", [(256, 1100, 7168), (300_000, 65, 80), (4200, 4100, 66)])
def test_wgrad_of_many_tiles(G, N, K):
    """More workgroups than 2^18 of them: every group's matrix is written, those without rows with zeros."""
    g = rng("many tiles", G)
    sizes = np.zeros(G, int)
    sizes[g.integers(0, G, 40)], sizes[0], sizes[-1] = 3, 2, 5
    o, M = offsets(sizes, 0, 0)
    dy, x = g.integers(-2, 3, (M, N)).astype(np.float64), g.integers(-2, 3, (M, K)).astype(np.float64)
    D = torch.full((G, N, K), 5.0, dtype=torch.bfloat16, device=dev())            # 4.0, 3.1 and 2.3 GB
    mm.gemm_grouped_wgrad(pitched(dy, torch.bfloat16), pitched(x, torch.bfloat16), torch.from_numpy(o).to(dev()), D)
    some = sizes > 0
    for i in np.flatnonzero(some):
        assert np.array_equal(f64(D[i]), dy[o[i]:o[i + 1]].T @ x[o[i]:o[i + 1]]), f"group {i}"
    written = (D.view(G, -1) == 0).all(1).cpu().numpy()
    assert written[~some].all()


def test_wgrad_rows_past_one_descriptor():
    """A pitch so wide that one buffer descriptor covers 255 rows (192 are walked at a time): the parts add up, exactly."""
    M, N, K, ld = 700, 40, 72, 1 << 22
    g = rng("wide")
    dy, x = g.integers(-2, 3, (M, N)), g.integers(-2, 3, (M, K))
    wide = torch.empty((M - 1) * ld + K, dtype=torch.bfloat16, device=dev())      # 5.9 GB
    X = torch.as_strided(wide, (M, K), (ld, 1))
    X.copy_(torch.from_numpy(x).to(dev()))
    dY = pitched(dy.astype(np.float64), torch.bfloat16)
    o = np.array([0, 3, 650, 700], np.int32)
    D = torch.empty(3, N, K, device=dev())
    C = torch.ones(3, N, K, device=dev())
    mm.gemm_grouped_wgrad(dY, X, torch.from_numpy(o).to(dev()), D, beta=1.0, C=C)
    for i in range(3):
        assert np.array_equal(f64(D[i]), 1 + dy[o[i]:o[i + 1]].T @ x[o[i]:o[i + 1]])


def test_rows_past_32_bits():
    """Rows that start more than 2^32 bytes into A and D, and weights that far into B."""
    M, N, K, G = 600_000, 40, 4096, 3
    A = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())                     # 4.9 GB
    g = rng("far")
    a = g.integers(-2, 3, (50, K))
    A[-50:] = torch.from_numpy(a).to(dev())
    B = torch.empty(G, (1 << 31) // 16 * 9, dtype=torch.bfloat16, device=dev())   # groups 2.4 GB apart
    b = g.integers(-2, 3, (G, N, K))
    W = torch.as_strided(B, (G, N, K), (B.stride(0), K, 1))
    W.copy_(torch.from_numpy(b).to(dev()))
    o = torch.tensor([0, M - 50, M - 20, M], dtype=torch.int32, device=dev())
    D = torch.full((M, N), 5.0, device=dev())
    mm.gemm_grouped(A, o, W, D)
    assert (D[:-50] == 0).all()
    assert np.array_equal(f64(D[-50:-20]), a[:30] @ b[1].T) and np.array_equal(f64(D[-20:]), a[30:] @ b[2].T)


# ---- block-scaled operands ----------------------------------------------------------------------

KINDS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def mx8_operand(g, shape, kind, integers):
    """Codes (uint8) and exponents of a block-scaled operand, and its values."""
    pos = R.E4M3_POS if kind == "e4m3" else R.E5M2_POS
    if kind == "fp4":
        pos = R.E2M1
    small = [i for i, v in enumerate(pos) if v in (0, 1, 2, 3, 4)]
    sign = 8 if kind == "fp4" else 128
    rows, K = shape
    if integers:
        c = g.choice(small, (rows, K))
        e = 127 + g.integers(-1, 2, (rows, K // 32))
    else:
        v = np.abs(g.standard_normal((rows, K))) * (2 if kind == "fp4" else 20)
        c = R.rne_codes(np.minimum(v, pos[-1]), pos)
        e = 127 + g.integers(-6, 4, (rows, K // 32))
    c = c + sign * g.integers(0, 2, (rows, K))
    values = np.where(c >= sign, -1.0, 1.0) * pos[c % sign] * np.repeat(np.ldexp(1.0, e - 127), 32, 1)
    return c.astype(np.uint8), e, values


def run_mx(rows, N, K, ka, kb, out=torch.bfloat16, integers=False, bias=False, beta=0.0, pad=1):
    sizes, before, behind = rows
    g = rng(len(sizes), N, K, ka, kb, integers)
    o, M = offsets(sizes, before, behind)
    G = len(sizes)
    ca, ea, a = mx8_operand(g, (M, K), ka, integers)
    cb, eb, b = mx8_operand(g, (G * N, K), kb, integers)
    ea[:before], ea[M - behind:] = 255, 255                    # rows of no group: NaN
    fill = 255                                                 # blocks past K: NaN scales, ignored
    abuf = torch.full((M, K + 16 * pad), 0x7f, dtype=torch.uint8, device=dev())
    abuf[:, :K] = torch.from_numpy(ca).to(dev())
    A = abuf.view(KINDS[ka])[:, :K]
    sabuf = torch.from_numpy(R.sx_words(ea, fill)).to(dev())
    SA = torch.nn.functional.pad(sabuf, (0, pad), value=-1)[:, :M + pad]
    packed = (cb[:, 0::2] | (cb[:, 1::2] << 4)) if kb == "fp4" else cb
    width = packed.shape[1]
    bbuf = torch.full((G, N + pad, width + 16 * pad), 0x7f, dtype=torch.uint8, device=dev())
    bbuf[:, :N, :width] = torch.from_numpy(packed.reshape(G, N, width)).to(dev())
    B = bbuf[:, :N, :width] if kb == "fp4" else bbuf.view(KINDS[kb])[:, :N, :width]
    words = np.stack([R.sx_words(eb[i * N:(i + 1) * N], fill) for i in range(G)])
    SB = torch.nn.functional.pad(torch.from_numpy(words).to(dev()), (0, 2 * pad, 0, pad), value=-1)[:, :words.shape[1], :N + pad]
    c = g.integers(-3, 4, (M, N)).astype(np.float64)
    C = pitched(c, out) if beta else None
    vec = g.integers(-3, 4, (G, N)).astype(np.float64)
    dbuf, D = guarded(M, N, out, 5.0)
    mm.gemm_grouped_mx(A, SA, torch.from_numpy(o).to(dev()), B, SB, D, b_type=mm.FP4_E2M1 if kb == "fp4" else None, beta=beta, C=C,
                       bias=torch.from_numpy(vec).float().to(dev()) if bias else None)
    torch.cuda.synchronize()
    check_guards(dbuf, M, N)
    got = f64(D.float())
    assert (got[:o[0]] == 5).all() and (got[o[-1]:] == 5).all(), "rows of no group"
    b = b.reshape(G, N, K)
    for i in range(G):
        r = slice(o[i], o[i + 1])
        want, mags = a[r] @ b[i].T, np.abs(a[r]) @ np.abs(b[i].T)
        if beta:
            want, mags = want + beta * c[r], mags + abs(beta) * np.abs(c[r])
        if bias:
            want, mags = want + vec[i], mags + np.abs(vec[i])
        if integers:
            assert np.array_equal(got[r], torch.from_numpy(want).to(out).double().numpy()), f"group {i}"
        elif want.size:
            check_sums(got[r], want, mags, K, out, 0.0 if out is torch.float32 else 2.0 ** -13)


@pytest.mark.parametrize("ka", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kb", ["e4m3", "e5m2", "fp4"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,N,K", [("single", 1, 32), ("few", 37, 96), ("uneven", 130, 544), ("all_in_one", 70, 256), ("none", 8, 64)])
def test_mx(ka, kb, out, rows, N, K):
    run_mx(ROWS[rows], N, K, ka, kb, OUT[out], bias=K == 96, beta=1.0 if K == 544 else 0.0)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("kb", ["e4m3", "fp4"])
@pytest.mark.parametrize("out", ["fp32", "fp16"])
@pytest.mark.parametrize("K", [32, 160, 704, 1024])
def test_mx_every_tile_exact(tile, kb, out, K, monkeypatch):
    """Elements and scales that differ by block and keep every partial sum exact: bit for bit, so each element meets its partner and
    each block its scale."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    for k, rows in enumerate(("edges", "uneven", "many")):
        run_mx(ROWS[rows], 70 if k == 2 else 263, K, ["e4m3", "e5m2"][k % 2], kb, OUT[out] if out == "fp32" or K < 500 else torch.float32,
               integers=True, bias=k == 1, pad=k % 2)


@pytest.mark.parametrize("out", list(OUT))
def test_mx_outputs(out):
    run_mx(ROWS["uneven"], 64, 128, "e4m3", "fp4", OUT[out], bias=True, beta=0.5)


@pytest.mark.parametrize("tile", [16, 128])
def test_mx_fp32_outputs_are_exact_to_fp32(tile, monkeypatch):
    """Blocks of very different scales: the sums stay within fp32's bound."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    run_mx(ROWS["edges"], 64, 4096, "e4m3", "e4m3", torch.float32)
    run_mx(ROWS["edges"], 64, 4096, "e5m2", "fp4", torch.float32)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("kb", ["e4m3", "e5m2", "fp4"])
@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [704, 1024])
def test_mx_every_tile_exact_in_16_bits(tile, kb, out, K, monkeypatch):
    """The block-scaled instructions over many k-tiles: every sum is a multiple of 1/4 below 2^17, exact in any order, and the output
    its nearest value, bit for bit."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    for k, rows in enumerate(("edges", "uneven", "long")):
        run_mx(ROWS[rows], 70 if k == 2 else 263, K, ["e4m3", "e5m2"][k % 2], kb, OUT[out], integers=True, bias=k == 1, pad=k % 2)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("ka", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kb", ["e4m3", "e5m2", "fp4"])
@pytest.mark.parametrize("K", [512, 1120, 4096])
def test_mx_16_bit_outputs_in_every_tile(tile, ka, kb, K, monkeypatch):
    monkeypatch.setenv("MMAC_TILE", str(tile))
    run_mx(ROWS["edges"], 130, K, ka, kb, torch.bfloat16)
    run_mx(ROWS["long"], 70, K, ka, kb, torch.float16, beta=1.0)


def scaled(c, e, kind):
    """Values of codes (rows x K) with a scale per 32."""
    pos, sign = (R.E2M1, 8) if kind == "fp4" else (R.E4M3_POS, 128)
    return np.where(c >= sign, -1.0, 1.0) * pos[c % sign] * np.repeat(np.ldexp(1.0, e.astype(np.int64) - 127), 32, 1)


def run_mx_codes(ca, ea, cb, eb, kb, out):
    """One group's product of given codes (A E4M3): its values, the sums in 64 bits and those of the magnitudes."""
    A = torch.from_numpy(ca.astype(np.uint8)).to(dev()).view(torch.float8_e4m3fn)
    packed = (cb[:, 0::2] | (cb[:, 1::2] << 4)) if kb == "fp4" else cb
    B = torch.from_numpy(packed.astype(np.uint8)).to(dev()).unsqueeze(0)
    B = B if kb == "fp4" else B.view(torch.float8_e4m3fn)
    SA, SB = (torch.from_numpy(R.sx_words(e, 127)).to(dev()) for e in (ea, eb))
    D = torch.empty(len(ca), len(cb), dtype=out, device=dev())
    mm.gemm_grouped_mx(A, SA, torch.tensor([0, len(ca)], dtype=torch.int32, device=dev()), B, SB.unsqueeze(0), D,
                       b_type=mm.FP4_E2M1 if kb == "fp4" else None)
    a, b = scaled(ca, ea, "e4m3"), scaled(cb, eb, kb)
    return f64(D), a @ b.T, np.abs(a) @ np.abs(b.T)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("kb", ["e4m3", "fp4"])
@pytest.mark.parametrize("out", list(OUT))
def test_mx_sums_that_cancel(tile, kb, out, monkeypatch):
    """The second half of K takes back the first but for one block, so a result is some thousandths of the magnitudes: within 2^-13
    of those (outputs of 16 bits or fewer; fp32 ones without that) and the output's half step."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    g = rng("cancel", kb)
    K, M, N = 2048, 70, 96
    ca, cb = g.integers(0, 0x60, (M, K)) + 128 * g.integers(0, 2, (M, K)), g.integers(0, 8 if kb == "fp4" else 0x60, (N, K))
    ea, eb = 127 + g.integers(-3, 4, (M, K // 32)), 127 + g.integers(-3, 4, (N, K // 32))
    h, q = K // 2, K // 64
    ca[:, h:], cb[:, h:], ea[:, q:], eb[:, q:] = ca[:, :h] ^ 128, cb[:, :h], ea[:, :q], eb[:, :q]
    ea[:, -1] -= 4
    got, want, mags = run_mx_codes(ca, ea, cb, eb, kb, OUT[out])
    assert np.median(np.abs(want) / mags) < 2.0 ** -6
    check_sums(got, want, mags, K, OUT[out], 0.0 if out == "fp32" else 2.0 ** -13)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("kb", ["e4m3", "fp4"])
@pytest.mark.parametrize("out", ["bf16", "fp16"])
def test_mx_exponents_far_apart(tile, kb, out, monkeypatch):
    """Scales near the ends of their range that meet their opposites: the products, of the size of one, count in 16-bit outputs."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    g = rng("far apart", kb)
    K, M, N = 512, 70, 96
    ca, cb = g.integers(0, 0x60, (M, K)) + 128 * g.integers(0, 2, (M, K)), g.integers(0, 8 if kb == "fp4" else 0x60, (N, K))
    low = g.integers(0, 2, K // 32).astype(bool)
    ea, eb = g.integers(1, 4, (M, K // 32)), g.integers(250, 253, (N, K // 32))
    ea, eb = np.where(low, ea, 254 - ea), np.where(low, eb, 254 - eb)
    got, want, mags = run_mx_codes(ca, ea, cb, eb, kb, OUT[out])
    check_sums(got, want, mags, K, OUT[out], 2.0 ** -13)


@pytest.mark.parametrize("tile", [16, 64, 128, 1282])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_mx_scale_words_at_the_end_of_their_arrays(tile, out, monkeypatch):
    """Scale words as columns of a wider array, whose last row ends with the last word that is used."""
    monkeypatch.setenv("MMAC_TILE", str(tile))
    g = rng("words", tile, out)
    sizes, N, K = [50, 3, 0, 87], 101, 416
    o, M = offsets(sizes, 0, 0)
    G = len(sizes)
    ca, ea, a = mx8_operand(g, (M, K), "e4m3", True)
    cb, eb, b = mx8_operand(g, (G * N, K), "fp4", True)
    A = torch.from_numpy(ca).to(dev()).view(torch.float8_e4m3fn)
    B = torch.from_numpy((cb[:, 0::2] | (cb[:, 1::2] << 4)).reshape(G, N, K // 2)).to(dev())
    words = np.stack([R.sx_words(eb[i * N:(i + 1) * N], 255) for i in range(G)])
    SA = torch.nn.functional.pad(torch.from_numpy(R.sx_words(ea, 255)).to(dev()), (37, 0), value=-1)[:, 37:]
    SB = torch.nn.functional.pad(torch.from_numpy(words).to(dev()), (29, 0), value=-1)[:, :, 29:]
    D = torch.empty(M, N, dtype=OUT[out], device=dev())
    mm.gemm_grouped_mx(A, SA, torch.from_numpy(o).to(dev()), B, SB, D, b_type=mm.FP4_E2M1)
    for i in range(G):
        r = slice(o[i], o[i + 1])
        assert np.array_equal(f64(D[r]), torch.from_numpy(a[r] @ b[i * N:(i + 1) * N].T).to(OUT[out]).double().numpy()), f"group {i}"


def test_matrices_without_elements():
    """New tensors without rows or columns, whose pitches are no multiple of 16 bytes."""
    def e(*shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device=dev())

    o = torch.tensor([0, 1, 3], dtype=torch.int32, device=dev())
    none = torch.zeros(3, dtype=torch.int32, device=dev())
    mm.gemm_grouped(e(3, 16), o, e(2, 16, 0), e(3, 0), trans_b=True)
    mm.gemm_grouped(e(0, 33), none, e(2, 8, 40)[:, :, :33], e(0, 8))
    D = torch.full((3, 8), 5.0, device=dev())
    mm.gemm_grouped(e(3, 0), o, e(2, 8, 0), D)
    assert (D == 0).all()
    mm.gemm_grouped_wgrad(e(3, 0), e(3, 16), o, torch.empty(2, 0, 16, device=dev()))
    mm.gemm_grouped_wgrad(e(3, 16), e(3, 0), o, torch.empty(2, 16, 0, device=dev()))
    D, C = torch.full((2, 33, 5), 5.0, device=dev()), torch.ones(2, 33, 5, device=dev())
    mm.gemm_grouped_wgrad(e(0, 33), e(0, 5), none, D, beta=2.0, C=C)
    assert (D == 2).all()


def test_mx_of_zero_length():
    D = torch.full((4, 8), 5.0, device=dev())
    e = torch.empty(4, 0, dtype=torch.float8_e4m3fn, device=dev())
    s = torch.empty(0, 4, dtype=torch.int32, device=dev())
    mm.gemm_grouped_mx(e, s, torch.tensor([0, 1, 3], dtype=torch.int32, device=dev()), torch.empty(2, 8, 0, dtype=torch.float8_e4m3fn, device=dev()),
                       torch.empty(2, 0, 8, dtype=torch.int32, device=dev()), D, bias=torch.ones(2, 8, device=dev()))
    assert (D[:3] == 1).all() and (D[3] == 5).all()


# ---- together -----------------------------------------------------------------------------------

def block(T, H, F, G, seed):
    """A feed-forward block of G experts, one expert a token: what a training step has in hand."""
    g = rng(T, H, F, G, seed)
    t = torch.bfloat16

    def normal(*shape, scale=1.0):
        return torch.from_numpy(g.standard_normal(shape) * scale).to(dev()).to(t)

    return dict(x=normal(T, H), res=normal(T, H), w=torch.ones(H, device=dev()) + 0.1 * normal(H).float(), W1=normal(G, F, H, scale=H ** -0.5),
                W2=normal(G, H, F, scale=F ** -0.5), dout=normal(T, H), offsets=torch.from_numpy(offsets(np.bincount(g.integers(0, G, T), minlength=G), 0, 0)[0]).to(dev()))


def step(p):
    """Norm, two grouped products with a ReLU between, and all gradients, by this library's calls alone; tokens are sorted by expert."""
    T, H = p["x"].shape
    G, F = p["W1"].shape[:2]
    t = torch.bfloat16
    o = p["offsets"]
    h, y, rstd = torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty(T, device=dev())
    mm.rmsnorm(p["x"], p["w"], y, eps=1e-5, residual=p["res"], H=h, rstd=rstd)
    a = torch.empty(T, F, dtype=t, device=dev())
    mm.gemm_grouped(y, o, p["W1"], a, act=mm.ACT_RELU)
    out = torch.empty(T, H, dtype=t, device=dev())
    mm.gemm_grouped(a, o, p["W2"], out, beta=1.0, C=h)                            # added to the residual stream
    da = torch.empty(T, F, dtype=t, device=dev())
    mm.gemm_grouped(p["dout"], o, p["W2"], da, trans_b=True)
    da = torch.where(a > 0, da, torch.zeros_like(da))
    dW2, dW1 = torch.empty(G, H, F, device=dev()), torch.empty(G, F, H, device=dev())
    mm.gemm_grouped_wgrad(p["dout"], a, o, dW2)
    mm.gemm_grouped_wgrad(da, y, o, dW1)
    dy, dx, dw = torch.empty(T, H, dtype=t, device=dev()), torch.empty(T, H, dtype=t, device=dev()), torch.empty(H, device=dev())
    mm.gemm_grouped(da, o, p["W1"], dy, trans_b=True)
    p.setdefault("ws", mm.rmsnorm_grad_workspace(T, H, dev()))
    mm.rmsnorm_grad(dy, h, p["w"], rstd, dx, dW=dw, dH=p["dout"], workspace=p["ws"])
    return dict(out=out, dx=dx, dw=dw, dW1=dW1, dW2=dW2, a=a)


def reference_step(p, on):
    """The same in 64 bits by autograd on the CPU, from the same 16-bit inputs; `on`: where the ReLU let values pass (its gradient jumps where
    a rounding moves a value across zero)."""
    q = {k: v.double().cpu().requires_grad_(k in ("x", "w", "W1", "W2")) for k, v in p.items() if k not in ("offsets", "ws")}
    o = p["offsets"].tolist()
    h = q["x"] + q["res"]
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-5) * q["w"]
    outs = [(y[o[g]:o[g + 1]] @ q["W1"][g].t() * on[o[g]:o[g + 1]]) @ q["W2"][g].t() for g in range(len(o) - 1)]
    out = torch.cat(outs) + h
    out.backward(q["dout"])
    return dict(out=out.detach(), dx=q["x"].grad, dw=q["w"].grad, dW1=q["W1"].grad, dW2=q["W2"].grad)


def test_block_forward_and_backward():
    """Every 16-bit rounding on the way (h, y, a, da, dy and the outputs: at most six in turn, each 2^-9 relative, norms) leaves a
    result within 6 * 2^-9 times the growth of a relative error through two products and the norm, which are contractions of
    independent roundings here: 8 * 2^-8 covers it normwise."""
    p = block(300, 96, 160, 5, 1)
    got = step(p)
    want = reference_step(p, (got["a"] > 0).double().cpu())
    for k, v in want.items():
        d = (got[k].double().cpu() - v).norm() / v.norm()
        assert d <= 8 * 2.0 ** -8, f"{k}: {d:.3g}"


def test_block_from_8_bits():
    """The serving form: the norm's 8-bit output through 4-bit experts, against the values the stored operands stand for."""
    T, H, F, G = 100, 256, 192, 4
    p = block(T, H, F, G, 2)
    yq, sy = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev()), torch.empty(2, T, dtype=torch.int32, device=dev())
    mm.rmsnorm(p["x"], p["w"], yq, residual=p["res"], SY=sy)
    q, s = torch.empty(G, F, H // 2, dtype=torch.uint8, device=dev()), torch.empty(G, 2, F, dtype=torch.int32, device=dev())
    for g in range(G):
        mm.mx4_quantize(p["W1"][g], q[g], s[g])
    D = torch.empty(T, F, device=dev())
    mm.gemm_grouped_mx(yq, sy, p["offsets"], q, s, D, b_type=mm.FP4_E2M1)
    y = torch.empty(T, H, device=dev())
    mm.mx8_dequantize(yq, sy, y)
    y, o = f64(y), p["offsets"].tolist()
    for g in range(G):
        e = np.stack([(s[g].cpu().numpy().view(np.uint32) >> (8 * i)) & 255 for i in range(4)], 2).transpose(1, 0, 2).reshape(F, -1)[:, : H // 32]
        c = R.unpack_codes(q[g].cpu().numpy(), H)
        w = np.where(c >= 8, -1.0, 1.0) * R.E2M1[c & 7] * np.repeat(np.ldexp(1.0, e.astype(np.int64) - 127), 32, 1)
        r = slice(o[g], o[g + 1])
        check_sums(f64(D[r]), y[r] @ w.T, np.abs(y[r]) @ np.abs(w.T), H, torch.float32)


def test_two_streams():
    """Two blocks at once on streams of their own give the bits of one after the other."""
    p, q = block(500, 128, 256, 6, 3), block(333, 256, 96, 3, 4)
    want = step(p), step(q)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, v in enumerate((p, q)):
            s[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s[i]):
                got[i] = step(v)
    torch.cuda.synchronize()
    for i in range(2):
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), k


def test_captured_and_replayed():
    """A captured step follows new offsets and inputs: every replay has the eager bits, with eager work between the replays."""
    p = block(260, 128, 192, 4, 5)
    step(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(p)
    for k, sizes in enumerate(([260, 0, 0, 0], [1, 2, 250, 7], [0, 0, 0, 260], [65, 65, 65, 65])):
        p["offsets"].copy_(torch.from_numpy(offsets(sizes, 0, 0)[0]))
        p["x"].copy_(block(260, 128, 192, 4, 6 + k)["x"])
        graph.replay()
        torch.cuda.synchronize()
        first = {n: v.clone() for n, v in got.items()}
        eager = step(p)
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(first[n], eager[n]), (k, n)
