"""The norm, the ragged grouped products and clipping on the GPU, against
plain 64-bit formulas.

Tolerances, derived from the arithmetic.  A stored value is off by at most
half a step of its type, u(t) = eps(t) / 2 of its size.  An fp32 sum of K
products accumulated in any order is off by at most K steps of 2^-23 (a step
for an addition, rounded or truncated) of the sum of the products' sizes:
e = (K + 8) 2^-23 sum |a b|.  Elementwise fp32 work adds a few steps of 2^-23.
"""
import math

import pytest
import torch

from block_sparse_gemm_amd import bsg

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
STEP = 2.0 ** -23


def u(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def padded(t, extra, fill=float("nan")):
    """The same values in a tensor whose rows are `extra` longer, the rest filled."""
    big = torch.full((t.shape[0], t.shape[1] + extra), fill, device=t.device).to(t.dtype)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def close(name, got, want, tol):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
        f"{got[bad][0].item()} for {want[bad][0].item()}")


# ------------------------------------------------------------------- norm

EPS = 1e-5


def norm_exact(x, residual, weight):
    dt = x.dtype
    # the sum of two values of a type rounded once (fp64 holds it exactly, or
    # to far below half a step)
    h = x if residual is None else (x.double() + residual.double()).to(dt)
    hd = h.double()
    rstd = 1.0 / torch.sqrt(hd.square().mean(1) + EPS)
    return h, rstd, hd * rstd[:, None] * weight.double()


WIDTHS = [8, 64, 512, 520, 1000, 1024, 2048, 2056, 4096, 4104, 8192, 16384]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T, res", [(1, True), (3, False), (131, True)])
def test_rms_norm(dtype, d, T, res):
    if d * dtype.itemsize > 32768:
        d //= 2
    g = gen(d + T)
    x, r = randn(g, T, d, dtype=dtype), randn(g, T, d, dtype=dtype, std=2.0) if res else None
    w = randn(g, d, dtype=dtype)
    if T > 2:
        x[1] = 0
        if res:
            r[1] = 0
    h0, rstd0, y0 = norm_exact(x, r, w)
    # longer rows in memory, NaN behind each row; rows behind T poisoned
    xs = padded(x, 8)
    h = torch.full((T + 1, d), 7.0, device="cuda", dtype=dtype)
    y = torch.full((T + 1, d + 16), 7.0, device="cuda", dtype=dtype)
    rstd = torch.full((T + 1,), 7.0, device="cuda")
    bsg.rms_norm(xs, w, EPS, y[:T, :d], h=h[:T] if res else None, residual=r, rstd=rstd[:T])
    if res:  # fp32 sums of fp32 are rounded as the fp64 sum is
        assert torch.equal(h[:T], h0)
    # relative: d additions of squares, then half of that by the root, and some ten operations
    rel = (d + 8) * STEP / 2 + 10 * STEP
    close("rstd", rstd[:T], rstd0, rel * rstd0)
    close("y", y[:T, :d], y0, (u(dtype) + rel) * y0.abs() + 1e-38)
    assert bool((h[T] == 7).all()) and bool((y[T] == 7).all()) and float(rstd[T]) == 7
    assert bool((y[:, d:] == 7).all()) and (res or bool((h == 7).all()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, d, res", [(1, 4096, True), (37, 1000, True), (5, 8, False),
                                       (64, 2056, False), (9, 8192, True)])
def test_rms_norm_e4m3(dtype, T, d, res):
    g = gen(d)
    x, r = randn(g, T, d, dtype=dtype), randn(g, T, d, dtype=dtype) if res else None
    w = randn(g, d, dtype=dtype)
    if T > 2:
        x[1] = 0
        if res:
            r[1] = 0
    _, _, y0 = norm_exact(x, r, w)
    y = torch.empty(T, d, device="cuda", dtype=E4M3)
    scale = torch.empty(T, device="cuda")
    bsg.rms_norm(x, w, EPS, y, residual=r, y_scale=scale)
    rel = (d + 8) * STEP / 2 + 16 * STEP
    most = y0.abs().amax(1)
    want = torch.where(most == 0, torch.ones_like(most), most / 448)
    close("scale", scale, want, rel * want)
    # half a step of e4m3: 2^-4 of the value, and 2^-10 below its smallest normal 2^-6
    got = y.double() * scale.double()[:, None]
    close("y", got, y0, (u(E4M3) + rel) * y0.abs() + 2.0 ** -10 * want[:, None] * (1 + rel))
    assert bool((y.float().abs().amax(1)[most > 0] == 448).all())


def test_rms_norm_nan_and_infinity():
    d = 264
    x = torch.ones(4, d, device="cuda", dtype=BF16)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    w = torch.ones(d, device="cuda", dtype=BF16)
    y = torch.empty_like(x)
    bsg.rms_norm(x, w, EPS, y)
    assert bool(y[0].isfinite().all()) and bool(y[3].isfinite().all())
    assert bool(y[1].isnan().all()) and bool(y[2, 7].isnan())
    q, s = torch.empty(4, d, device="cuda", dtype=E4M3), torch.empty(4, device="cuda")
    bsg.rms_norm(x, w, EPS, q, y_scale=s)
    assert s.isfinite().tolist() == [True, False, False, True]
    assert torch.equal(q[0].float(), torch.full((d,), 448.0, device="cuda"))


def test_rms_norm_in_place_and_empty():
    g = gen(1)
    x, r, w = (randn(g, *s, dtype=BF16) for s in ((33, 1024), (33, 1024), (1024,)))
    y, h = torch.empty_like(x), torch.empty_like(x)
    bsg.rms_norm(x, w, EPS, y, h=h, residual=r)
    x2, r2 = x.clone(), r.clone()
    bsg.rms_norm(x2, w, EPS, x2, h=r2, residual=r2)   # y over x, h over the residual
    assert torch.equal(x2, y) and torch.equal(r2, h)
    bsg.rms_norm(x[:0], w, EPS, y[:0])
    dw = torch.full((1024,), 3.0, device="cuda")
    ws = torch.empty(bsg.rms_norm_backward_workspace_bytes(0, 1024), device="cuda", dtype=torch.uint8)
    bsg.rms_norm_backward(x[:0], h[:0], w, torch.empty(0, device="cuda"), y[:0], dw, ws)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, d, res", [(1, 8, True), (3, 520, False), (700, 1024, True),
                                       (9000, 136, True), (65, 2048, False), (65, 4096, True),
                                       (19, 8192, True), (5, 16384, False)])
def test_rms_norm_backward(dtype, T, d, res):
    if d * dtype.itemsize > 32768:
        d //= 2
    g = gen(T + d)
    h, dy, w = (randn(g, *s, dtype=dtype) for s in ((T, d), (T, d), (d,)))
    dh = randn(g, T, d, dtype=dtype) if res else None
    rstd = torch.empty(T, device="cuda")
    y = torch.empty_like(h)
    bsg.rms_norm(h, w, EPS, y, rstd=rstd)
    dx = torch.full((T + 1, d + 8), 5.0, device="cuda", dtype=dtype)
    dw = torch.full((d,), 5.0, device="cuda")
    ws = torch.full((bsg.rms_norm_backward_workspace_bytes(T, d) // 4,), float("nan"), device="cuda")
    bsg.rms_norm_backward(padded(dy, 16), padded(h, 8), w, rstd, dx[:T, :d], dw, ws, dh=dh)
    hd, dyd, wd, r = h.double(), dy.double(), w.double(), rstd.double()[:, None]
    n = hd * r
    dot = (wd * dyd * n).mean(1, keepdim=True)
    want = r * (wd * dyd - n * dot)
    if res:
        want = want + dh.double()
    # the mean's sum of d terms, and some ten operations on the terms' sizes
    e_dot = (d + 8) * STEP * (wd * dyd * n).abs().mean(1, keepdim=True)
    size = r * ((wd * dyd).abs() + n.abs() * dot.abs()) + (dh.double().abs() if res else 0)
    close("dx", dx[:T, :d], want, u(dtype) * want.abs() + 10 * STEP * size + r * n.abs() * e_dot)
    close("dw", dw, (dyd * n).sum(0), (T + 8) * STEP * (dyd * n).abs().sum(0) + 1e-38)
    assert bool((dx[T] == 5).all()) and bool((dx[:, d:] == 5).all())


def test_rms_norm_backward_against_differences():
    g = gen(4)
    T, d = 3, 24
    h, w, dy = randn(g, T, d), randn(g, d), randn(g, T, d)
    rstd, dx, dw = torch.empty(T, device="cuda"), torch.empty_like(h), torch.empty(d, device="cuda")
    bsg.rms_norm(h, w, EPS, torch.empty_like(h), rstd=rstd)
    ws = torch.empty(bsg.rms_norm_backward_workspace_bytes(T, d) // 4, device="cuda")
    bsg.rms_norm_backward(dy, h, w, rstd, dx, dw, ws)

    def loss(hh, ww):
        return (dy.double() * norm_exact(hh, None, ww)[2]).sum()

    hd, wd, step = h.double(), w.double(), 1e-5
    for i in range(d):
        e = torch.zeros_like(hd)
        e[1, i] = step
        num = (loss(hd + e, wd) - loss(hd - e, wd)) / (2 * step)
        # central differences: third derivatives of order 10 times step^2, and fp32 dx
        assert abs(float(num) - float(dx[1, i])) <= 1e-4 * max(1.0, abs(float(num)))
        num = (loss(hd, wd + e[1]) - loss(hd, wd - e[1])) / (2 * step)
        assert abs(float(num) - float(dw[i])) <= 1e-4 * max(1.0, abs(float(num)))


# ------------------------------------------------------- grouped products

def offsets(sizes, start=0):
    off = [start]
    for s in sizes:
        off.append(off[-1] + s)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def products_exact(a, b, off, trans):
    """fp64 products and the sums of their terms' sizes, by expert."""
    E = b.shape[0]
    N = b.shape[1] if trans else b.shape[2]
    p = torch.zeros(a.shape[0], N, dtype=torch.float64, device="cuda")
    s = torch.zeros_like(p)
    o = off.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            w = b[e].double()
            w = w.t().contiguous() if trans else w
            r = a[o[e]:o[e + 1]].double()
            p[o[e]:o[e + 1]] = r @ w
            s[o[e]:o[e + 1]] = r.abs() @ w.abs()
    return p, s


def weights(g, E, K, N, dtype, trans, layout):
    """Experts' matrices: one after the other with longer rows (NaN behind
    each row and each matrix), or side by side as the layer's W1."""
    rows, cols = (N, K) if trans else (K, N)
    vals = torch.randn(E, rows, cols, generator=g, device="cuda").mul_(0.5).to(dtype)
    if layout == "side":
        big = torch.empty(rows, E * cols, device="cuda", dtype=dtype)
        v = big.view(rows, E, cols).permute(1, 0, 2)
    else:
        big = torch.full((E, rows + 1, cols + 16), float("nan"), device="cuda").to(dtype)
        v = big[:, :rows, :cols]
    v.copy_(vals)
    return v


def e_sum(K, s, dtype=F32):
    """Error of a sum of K products with sum of sizes s.  The 8-bit matrix
    instruction adds the products of 8 neighbouring k at once, cut 13 bits
    below the leading bit of the largest: each of the 7 others loses less than
    2^-13 of the largest, in all less than 7 * 2^-13 of the group's sizes."""
    return ((K + 8) * STEP + (7 * 2.0 ** -13 if dtype == E4M3 else 0)) * s


SIZES = {
    "one": [1],
    "tile edges": [127, 128, 129, 0, 255, 256, 257, 1],
    "few": [3, 0, 0, 17, 1, 16, 33, 0, 64, 65],
    "many": [(i * 7) % 11 for i in range(200)],
    "long": [0, 1500, 2],
}
SHAPES = [(64, 256), (8, 8), (24, 136), (72, 264), (520, 1000), (2048, 128)]


OPERANDS = [(BF16, False), (BF16, True), (F32, False), (F32, True), (E4M3, True)]


@pytest.mark.parametrize("dtype, trans", OPERANDS)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K, N", SHAPES)
def test_grouped_gemm(dtype, sizes, K, N, trans):
    if dtype == E4M3:
        K = -(-K // 16) * 16
    sizes = SIZES[sizes]
    g = gen(K * N + len(sizes))
    E, before, after = len(sizes), 3, 5
    M = before + sum(sizes) + after
    off = offsets(sizes, before)
    a = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    a0 = a.clone()
    # rows of no group hold NaN, and so does what lies behind each row
    a.view(torch.uint8)[:before] = 0x7f if dtype == E4M3 else 0xff
    a.view(torch.uint8)[M - after:] = 0x7f if dtype == E4M3 else 0xff
    b = weights(g, E, K, N, dtype, trans, "side" if K % 3 else "apart")
    cdt = BF16 if dtype == E4M3 else dtype
    sa = sb = None
    p, s = products_exact(a0.float(), b.float(), off, trans)
    if dtype == E4M3:
        sa = torch.rand(M, generator=g, device="cuda") + 0.5
        sb = torch.rand(E, N, generator=g, device="cuda") + 0.5
        of = torch.repeat_interleave(torch.arange(E, device="cuda"),
                                     torch.tensor(sizes, device="cuda"))
        f = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        f[before:M - after] = sa[before:M - after].double()[:, None] * sb.double()[of]
        p, s = p * f, s * f
    as_ = padded(a, 16)
    c = torch.full((M, N + 16), 9.0, device="cuda", dtype=cdt)
    ws = None
    n = bsg.grouped_gemm_workspace_bytes(M, K, N, E)
    if n:
        ws = torch.full((n // 4,), float("nan"), device="cuda")
    bsg.grouped_gemm(as_, off, b, c[:, :N], trans_b=trans, a_scale=sa, b_scale=sb, workspace=ws)
    live = slice(before, M - after)
    close("c", c[live, :N], p[live], u(cdt) * p[live].abs() + e_sum(K, s[live], dtype) + 1e-38)
    assert bool((c[:before] == 9).all()) and bool((c[M - after:] == 9).all())
    assert bool((c[:, N:] == 9).all())
    if dtype == E4M3:
        return
    # without the workspace, and with an fp32 output
    c2 = torch.full((M, N), 9.0, device="cuda")
    bsg.grouped_gemm(as_, off, b, c2, trans_b=trans)
    close("c fp32", c2[live], p[live], 4 * STEP * p[live].abs() + e_sum(K, s[live]) + 1e-38)
    assert bool((c2[:before] == 9).all()) and bool((c2[M - after:] == 9).all())


def acts_exact(epi, p, q, aux):
    """(outputs, saved), and for each a bound on its change per unit of error in p and in q."""
    one = torch.ones_like(p)
    if epi == "gelu":
        cdf = torch.special.ndtr(p)
        pdf = torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        # |gelu'| <= 1.13, |gelu''| <= 0.8
        return [p * cdf, cdf + p * pdf], [(1.13 * one, 0), (0.8 * one, 0)]
    if epi == "silu_mul":
        sg = torch.sigmoid(p)
        silu, dsilu = p * sg, sg * (1 + p * (1 - sg))
        # |silu'| <= 1.1, |silu''| <= 0.5
        return ([silu * q, silu, q * dsilu],
                [(1.1 * q.abs(), silu.abs()), (1.1 * one, 0), (0.5 * q.abs(), dsilu.abs())])
    if epi == "gelu_bwd":
        return [p * aux], [(aux.abs(), 0)]
    return [p * aux[1], p * aux[0]], [(aux[1].abs(), 0), (aux[0].abs(), 0)]


# e4m3 has forward products only, and the backward ones save nothing
EPILOGUES = [(dt, tr, epi, save) for dt, tr in OPERANDS
             for epi in ("gelu", "silu_mul", "gelu_bwd", "silu_mul_bwd") for save in (False, True)
             if not (save and epi.endswith("bwd")) and
             not (dt == E4M3 and (save or epi.endswith("bwd")))]


@pytest.mark.parametrize("dtype, trans, epi, save", EPILOGUES)
@pytest.mark.parametrize("sizes", ["tile edges", "few"])
@pytest.mark.parametrize("K, N", [(64, 264), (200, 136), (1032, 512)])
def test_grouped_gemm_epilogues(dtype, sizes, K, N, trans, epi, save):
    bwd = epi.endswith("bwd")
    if dtype == E4M3:
        K = -(-K // 16) * 16
    sizes = SIZES[sizes]
    E, M = len(sizes), sum(sizes)
    g = gen(K + N)
    off = offsets(sizes)
    a = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    scale = 1.5 / math.sqrt(K)
    b = [weights(g, E, K, N, dtype, trans, "side") for _ in range(2 if epi == "silu_mul" else 1)]
    cdt = BF16 if dtype == E4M3 else dtype
    sa = sb = f = None
    if dtype == E4M3:
        sa = torch.rand(M, generator=g, device="cuda") + 0.5
        sb = (torch.rand(len(b), E, N, generator=g, device="cuda") + 0.5) * scale
        of = torch.repeat_interleave(torch.arange(E, device="cuda"),
                                     torch.tensor(sizes, device="cuda"))
        f = sa.double()[:, None] * sb.double()[:, of]
    else:
        for w in b:
            w.mul_(scale)
    ps = [products_exact(a.float(), w.float(), off, trans) for w in b]
    if f is not None:
        ps = [(p * f[i], s * f[i]) for i, (p, s) in enumerate(ps)]
    two = epi == "silu_mul_bwd"
    aux = randn(g, *((2,) if two else ()), M, N, dtype=cdt) if bwd else None
    c = torch.full((2 if two else 1, M, N), 9.0, device="cuda", dtype=cdt)
    saved = None
    if save:
        saved = torch.full((2 if epi == "silu_mul" else 1, M, N), 9.0, device="cuda", dtype=cdt)
    n = bsg.grouped_gemm_workspace_bytes(M, K, N, E, epi)
    ws = torch.full((n // 4,), float("nan"), device="cuda") if n else None
    bsg.grouped_gemm(a, off, b[0], c if two else c[0], epilogue=epi, trans_b=trans,
                     b2=b[1] if len(b) > 1 else None, a_scale=sa, b_scale=sb, aux_in=aux,
                     aux_out=None if saved is None else saved if epi == "silu_mul" else saved[0],
                     workspace=ws)
    q, qs = ps[1] if len(ps) > 1 else (None, None)
    want, slopes = acts_exact(epi, ps[0][0], q, None if aux is None else aux.double())
    got = list(c) + (list(saved) if save else [])
    e0, e1 = e_sum(K, ps[0][1], dtype), 0 if qs is None else e_sum(K, qs, dtype)
    for i, t in enumerate(got):
        w, (k0, k1) = want[i], slopes[i]
        # the activations' own error: 1.5e-7 in erf (scaled by h in gelu), hardware exp2 and
        # reciprocal, a few steps of the result's and the factors' sizes
        own = 8 * STEP * (w.abs() + (0 if q is None else (ps[0][0] * q).abs()) + ps[0][0].abs() + 1)
        if q is not None:
            own = own + 8 * STEP * q.abs()
        close(f"{epi} output {i}", t, w, u(cdt) * w.abs() + k0 * e0 + k1 * e1 + own)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K, N", [(64, 256), (40, 72), (520, 136), (1024, 384)])
def test_grouped_gemm_two_sets(dtype, trans, K, N):
    sizes = [5, 0, 300, 130, 16]
    E, M = len(sizes), sum(sizes)
    g = gen(K + N)
    off = offsets(sizes)
    a = [randn(g, M, K, dtype=dtype) for _ in range(2)]
    b = [weights(g, E, K, N, dtype, trans, "apart") for _ in range(2)]
    p, s = (sum(x) for x in zip(*[products_exact(a[i], b[i], off, trans) for i in range(2)]))
    c = torch.full((M, N), 9.0, device="cuda", dtype=dtype)
    n = bsg.grouped_gemm_workspace_bytes(M, K, N, E)
    ws = torch.full((n // 4,), float("nan"), device="cuda") if n else None
    bsg.grouped_gemm(a[0], off, b[0], c, trans_b=trans, a2=a[1], b2=b[1], workspace=ws)
    close("c", c, p, u(dtype) * p.abs() + e_sum(2 * K, s))


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("epi", ["none", "gelu", "silu_mul"])
def test_grouped_gemm_split_along_k(dtype, epi):
    """Few rows, a long sum: workspaces that hold every number of segments,
    the same bits on every run, nothing behind the workspace's end touched."""
    sizes, K, N = [1, 0, 5, 2], 4112, 136
    E, M = len(sizes), sum(sizes)
    g = gen(8)
    trans, cdt = dtype == E4M3, BF16 if dtype == E4M3 else dtype
    off = offsets(sizes)
    a = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    two = epi == "silu_mul"
    b = [weights(g, E, K, N, dtype, trans, "apart") for _ in range(2 if two else 1)]
    sa = sb = None
    scale = 1.0 / math.sqrt(K)
    if dtype == E4M3:
        sa = torch.ones(M, device="cuda")
        sb = torch.full((len(b), E, N), scale, device="cuda")
    else:
        for w in b:
            w.mul_(scale)
            scale = 1.0
    share = M * N * len(b)
    most = bsg.grouped_gemm_workspace_bytes(M, K, N, E, epi) // 4
    assert most >= 4 * share
    ps = [products_exact(a.float(), w.float(), off, trans) for w in b]
    f = 1.0 / math.sqrt(K) if dtype == E4M3 else 1.0
    ps = [(p * f, s * f) for p, s in ps]
    if epi == "none":
        want, slope = ps[0][0], [torch.ones_like(ps[0][0])]
    else:
        out, k = acts_exact(epi, ps[0][0], ps[1][0] if two else None, None)
        want, slope = out[0], list(k[0])
    for floats in (0, share, 2 * share, 3 * share + 1, most):
        ws = torch.full((floats + 64,), 7.0, device="cuda")
        got = []
        for _ in range(2):
            c = torch.full((M, N), 9.0, device="cuda", dtype=cdt)
            bsg.grouped_gemm(a, off, b[0], c, epilogue=epi, trans_b=trans, b2=b[1] if two else None,
                             a_scale=sa, b_scale=sb, workspace=ws[:floats] if floats else None)
            got.append(c)
        assert torch.equal(got[0], got[1]) and bool((ws[floats:] == 7).all())
        err = slope[0] * e_sum(K, ps[0][1], dtype)
        if two:
            err = err + slope[1] * e_sum(K, ps[1][1], dtype)
        own = 8 * STEP * (want.abs() + ps[0][0].abs() * (1 + (ps[1][0].abs() if two else 0)) + 1)
        close(f"{floats} floats", got[0], want, u(cdt) * want.abs() + err + own)


def test_grouped_gemm_single_row_and_expert_strides():
    """One row, and one expert: strides that no address depends on may be odd."""
    g = gen(2)
    a, b = randn(g, 1, 64, dtype=BF16), randn(g, 1, 64, 72, dtype=BF16)
    off = offsets([1])
    want = torch.empty(1, 72, device="cuda", dtype=BF16)
    bsg.grouped_gemm(a, off, b, want)
    odd = torch.as_strided(a, (1, 64), (67, 1))
    oddb = torch.as_strided(b, (1, 64, 72), (4611, 72, 1))
    got = torch.empty_like(want)
    bsg.grouped_gemm(odd, off, oddb, torch.as_strided(got, (1, 72), (75, 1)))
    assert torch.equal(got, want)
    y, y2, w = torch.empty_like(a), torch.empty_like(a), a[0].clone()
    bsg.rms_norm(a, w, EPS, y)
    bsg.rms_norm(odd, w, EPS, torch.as_strided(y2, (1, 64), (71, 1)))
    assert torch.equal(y, y2)


def test_grouped_gemm_groups_do_not_mix():
    """NaN and infinity in one expert's rows and weights stay with that expert."""
    sizes = [40, 70, 300, 10]
    E, M, K, N = len(sizes), sum(sizes), 72, 136
    for dtype in (BF16, F32):
        g = gen(3)
        off = offsets(sizes)
        a, b = randn(g, M, K, dtype=dtype), randn(g, E, K, N, dtype=dtype)
        bad = slice(40, 110)
        clean = torch.empty(M, N, device="cuda", dtype=dtype)
        bsg.grouped_gemm(a, off, b, clean)
        a[bad] = float("nan")
        b[1] = float("inf")
        c = torch.empty_like(clean)
        bsg.grouped_gemm(a, off, b, c)
        assert bool(c[bad].isnan().all())
        assert torch.equal(c[:40], clean[:40]) and torch.equal(c[110:], clean[110:])
        dw = torch.empty(E, K, N, device="cuda", dtype=dtype)
        bsg.grouped_wgrad(a, clean, off, dw)
        assert bool(dw[1].isnan().all()) and bool(dw[[0, 2, 3]].isfinite().all())


def test_grouped_gemm_bad_offsets_write_no_row_behind_m():
    """Offsets that leave [0, M], or fall, are cut to it."""
    M, K, N = 96, 64, 64
    g = gen(5)
    a, b = randn(g, M, K, dtype=BF16), randn(g, 3, K, N, dtype=BF16)
    big = torch.full((M + 64, N), 9.0, device="cuda", dtype=BF16)
    off = torch.tensor([-5, 40, 20, 5000], dtype=torch.int32, device="cuda")
    bsg.grouped_gemm(a, off, b, big[:M])
    torch.cuda.synchronize()
    assert bool((big[M:] == 9).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K, N", [(64, 256), (8, 8), (24, 136), (264, 72), (520, 384)])
@pytest.mark.parametrize("side", [False, True])
def test_grouped_wgrad(dtype, sizes, K, N, side):
    sizes = SIZES[sizes]
    g = gen(K * N)
    E, before, after = len(sizes), 2, 4
    M = before + sum(sizes) + after
    off = offsets(sizes, before)
    a, d = randn(g, M, K, dtype=dtype), randn(g, M, N, dtype=dtype)
    for t in (a, d):
        t[:before] = float("nan")
        t[M - after:] = float("nan")
    big = torch.full((K, E * N) if side else (E, K + 1, N + 8), 9.0, device="cuda", dtype=dtype)
    c = big.view(K, E, N).permute(1, 0, 2) if side else big[:, :K, :N]
    f = torch.full((E, K, N), 9.0, device="cuda")
    bsg.grouped_wgrad(padded(a, 8), padded(d, 24), off, c)
    bsg.grouped_wgrad(a, d, off, f)
    o = off.tolist()
    for e in range(E):
        r = slice(o[e], o[e + 1])
        ad, dd = a[r].double().t().contiguous(), d[r].double()
        want, s = ad @ dd, ad.abs() @ dd.abs()
        n = sizes[e]
        close(f"expert {e}", c[e], want, u(dtype) * want.abs() + e_sum(n, s))
        close(f"expert {e} fp32", f[e], want, 4 * STEP * want.abs() + e_sum(n, s))
    if not side:
        assert bool((big[:, K:] == 9).all()) and bool((big[:, :, N:] == 9).all())
    f.fill_(9.0)
    bsg.grouped_wgrad(a[:0], d[:0], torch.zeros_like(off), f)
    assert bool((f == 0).all())


@pytest.mark.parametrize("dtype, out", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("sizes, K, N", [([5000], 136, 72), ([0, 2100, 3, 1300], 64, 264),
                                         ([1500, 1600], 256, 128)])
def test_grouped_wgrad_split_along_rows(dtype, out, sizes, K, N):
    """Few small matrices over long groups: every number of segments."""
    g = gen(6)
    E, M = len(sizes), sum(sizes)
    off = offsets(sizes)
    a, d = randn(g, M, K, dtype=dtype), randn(g, M, N, dtype=dtype)
    share = E * K * N
    most = bsg.grouped_wgrad_workspace_bytes(M, K, N, E) // 4
    assert most >= 2 * share
    o = off.tolist()
    for floats in (0, share, 2 * share, most):
        ws = torch.full((floats + 64,), 7.0, device="cuda")
        got = []
        for _ in range(2):
            big = torch.full((K, E * N + 8), 9.0, device="cuda", dtype=out)
            c = big[:, :E * N].unflatten(1, (E, N)).permute(1, 0, 2)
            bsg.grouped_wgrad(a, d, off, c, workspace=ws[:floats] if floats else None)
            got.append(big)
        assert torch.equal(got[0], got[1]) and bool((ws[floats:] == 7).all())
        assert bool((big[:, E * N:] == 9).all())
        for e in range(E):
            r = slice(o[e], o[e + 1])
            ad, dd = a[r].double().t().contiguous(), d[r].double()
            want, s = ad @ dd, ad.abs() @ dd.abs()
            close(f"expert {e}, {floats} floats", c[e], want,
                  u(out) * want.abs() + e_sum(sizes[e], s))


# --------------------------------------------------------------- clipping

def grads_of(g, sizes, std=1.0):
    """Gradients of both types, some not at a 16-byte boundary."""
    out = []
    for i, n in enumerate(sizes):
        dt = (BF16, F32)[i % 2]
        shift = (0, 1, 3, 8)[i % 4]
        out.append((torch.randn(n + shift, generator=g, device="cuda") * std).to(dt)[shift:])
    return out


def workspace():
    return torch.full((bsg.grad_norm_workspace_bytes() // 8,), float("nan"), device="cuda",
                      dtype=torch.float64)


CLIP = {
    "one value": [1],
    "none": [],
    "empty ones": [0, 5, 0, 0, 7, 0],
    "odd": [1, 2, 3, 7, 8, 9, 15, 16, 17, 4095, 4096, 4097, 16384, 16385, 131071],
    "many": [(i * 37) % 301 for i in range(250)],
    "exact lists": [5] * 192,
    "large": [3_000_001, 10, 7_000_003],
}


@pytest.mark.parametrize("sizes", list(CLIP))
@pytest.mark.parametrize("most", [1e30, 0.5, 0.0])
def test_grad_norm_and_clip(sizes, most):
    g = gen(len(sizes))
    grads = grads_of(g, CLIP[sizes])
    norm = torch.full((), float("nan"), device="cuda")
    bsg.grad_norm(grads, norm, workspace())
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    # fp64 sums; the root rounded to fp32
    assert abs(float(norm) - want) <= 2.0 ** -24 * want + 1e-9 * want
    out = [torch.empty(t.numel() + 3, device="cuda", dtype=t.dtype)[i % 4:][:t.numel()]
           for i, t in enumerate(grads)]
    bsg.grad_clip(grads, norm, most, out=out)
    nm = float(norm)
    s = torch.tensor(1.0 if nm <= most else most / nm, device="cuda", dtype=torch.float64)
    same = [t.clone() for t in grads]
    bsg.grad_clip(same, norm, most)
    for i, (t, o, p) in enumerate(zip(grads, out, same)):
        # the quotient and the product in fp32, then the type's rounding (subnormal: an absolute one)
        w = t.double() * s
        close(f"tensor {i}", o, w, (u(t.dtype) + 3 * STEP) * w.abs() + 1e-40)
        assert torch.equal(o, p)
        if nm <= most:
            assert torch.equal(p, t)


def test_grad_norm_of_large_and_unusual_values():
    ws, norm = workspace(), torch.empty((), device="cuda")
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((9,), 1e30, device="cuda", dtype=BF16)]
    bsg.grad_norm(big, norm, ws)           # squares of 1e60
    want = math.sqrt(sum(float(t.double().square().sum()) for t in big))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    bsg.grad_clip(big, norm, 1.0)
    bsg.grad_norm(big, norm, ws)
    assert abs(float(norm) - 1.0) <= 2.0 ** -8
    small = [torch.full((1000,), 1e-30, device="cuda")]
    bsg.grad_norm(small, norm, ws)
    assert abs(float(norm) - math.sqrt(1000) * 1e-30) <= 1e-6 * 3.2e-29
    for bad in (float("nan"), float("inf")):
        t = [torch.ones(100, device="cuda", dtype=BF16), torch.ones(33, device="cuda")]
        t[0][17] = bad
        bsg.grad_norm(t, norm, ws)
        assert (math.isnan if math.isnan(bad) else math.isinf)(float(norm))
        bsg.grad_clip(t, norm, 1.0)
        if math.isnan(bad):
            assert all(bool(x.isnan().all()) for x in t)
        else:
            assert bool(t[0][17].isnan()) and float(t[0][3]) == 0 and bool((t[1] == 0).all())


def test_same_bits_on_every_run():
    g = gen(9)
    grads = grads_of(g, [100_003, 5_000_001, 77])
    ws = workspace()
    norms = [torch.empty((), device="cuda") for _ in range(3)]
    for n in norms:
        bsg.grad_norm(grads, n, ws)
    assert torch.equal(norms[0], norms[1]) and torch.equal(norms[0], norms[2])
    h, dy, w = randn(g, 3000, 512, dtype=BF16), randn(g, 3000, 512, dtype=BF16), randn(g, 512, dtype=BF16)
    rstd = torch.rsqrt(h.float().square().mean(1))
    ws = torch.empty(bsg.rms_norm_backward_workspace_bytes(3000, 512), device="cuda", dtype=torch.uint8)
    dws = [torch.empty(512, device="cuda") for _ in range(3)]
    for dw in dws:
        bsg.rms_norm_backward(dy, h, w, rstd, torch.empty_like(h), dw, ws)
    assert torch.equal(dws[0], dws[1]) and torch.equal(dws[0], dws[2])


# ------------------------------------------- many tiles, offsets past 32 bits

@pytest.mark.parametrize("dtype, trans", OPERANDS)
@pytest.mark.parametrize("K, most", [(96, 2), (1040, 1)])
def test_grouped_gemm_over_many_tiles(dtype, trans, K, most):
    """Several hundred tiles of uneven groups.  Small integers: every sum is
    below 2^24 and so exact in any order (8-bit: no product below 2^-13 of
    another but 0), and the result is its one rounding."""
    E, N = 37, 1304
    sizes = [(i * 61) % 401 for i in range(E)]
    M = sum(sizes) + 50
    g = gen(K)
    a = torch.randint(-most, most + 1, (M, K), generator=g, device="cuda").float().to(dtype)
    b = torch.randint(-most, most + 1, (E, N, K) if trans else (E, K, N), generator=g,
                      device="cuda").float().to(dtype)
    off = offsets(sizes)
    out = F32 if dtype == F32 else BF16
    c = torch.full((M, N), 9.0, device="cuda", dtype=out)
    scales = dict(a_scale=torch.ones(M, device="cuda"),
                  b_scale=torch.ones(E, N, device="cuda")) if dtype == E4M3 else {}
    bsg.grouped_gemm(a, off, b, c, trans_b=trans, **scales)
    want = products_exact(a, b, off, trans)[0]
    assert torch.equal(c[:-50], want[:-50].to(out)) and bool((c[-50:] == 9).all())


def test_rows_past_4_gib():
    """Rows so far apart that their byte offsets pass 2^32: the same bits as
    from rows side by side."""
    M, K, N, ld = 33000, 64, 72, 65544
    g = gen(7)
    a, d, r = randn(g, M, K, dtype=BF16), randn(g, M, N, dtype=BF16), randn(g, M, K, dtype=BF16)
    b = randn(g, 4, K, N, dtype=BF16)
    off = offsets([20000, 0, 12990, 10])

    def apart(t):
        v = torch.empty(M, ld, device="cuda", dtype=t.dtype)[:, :t.shape[1]]
        v.copy_(t)
        return v

    A, D, R = apart(a), apart(d), apart(r)
    c, C = torch.empty(M, N, device="cuda", dtype=BF16), apart(d)
    bsg.grouped_gemm(a, off, b, c)
    bsg.grouped_gemm(A, off, b, C)
    assert torch.equal(c, C)
    w, W = (torch.empty(4, K, N, device="cuda", dtype=BF16) for _ in range(2))
    bsg.grouped_wgrad(a, d, off, w)
    bsg.grouped_wgrad(A, D, off, W)
    assert torch.equal(w, W)
    wn = randn(g, K, dtype=BF16)
    y, h, s = torch.empty_like(a), torch.empty_like(a), torch.empty(M, device="cuda")
    bsg.rms_norm(a, wn, 1e-5, y, h=h, residual=r, rstd=s)
    bsg.rms_norm(A, wn, 1e-5, A, h=R, residual=R)
    assert torch.equal(y, A) and torch.equal(h, R)
    ws = torch.empty(bsg.rms_norm_backward_workspace_bytes(M, K), device="cuda", dtype=torch.uint8)
    dx, dw, dW = torch.empty_like(a), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    bsg.rms_norm_backward(a, h, wn, s, dx, dw, ws)
    A.copy_(a)
    bsg.rms_norm_backward(A, R, wn, s, A, dW, ws)
    assert torch.equal(dx, A) and torch.equal(dw, dW)


def test_clipping_a_tensor_of_more_than_2_31_values():
    n = (1 << 31) + 5
    t = torch.full((n,), 2.0 ** -10, device="cuda", dtype=BF16)
    t[-1] = 2.0 ** 10
    ws = workspace()
    norm = torch.zeros((), device="cuda")
    bsg.grad_norm([t], norm, ws)
    # squares and their sum are exact in fp64 (below 2^53 steps of 2^-20); one root, one rounding
    want = float(torch.tensor((2.0 ** -20 * (n - 1) + 2.0 ** 20) ** 0.5, dtype=torch.float64).float())
    assert float(norm) == want
    norm.fill_(4.0)
    bsg.grad_clip([t], norm, 2.0)
    assert float(t[-1]) == 512.0 and bool((t[:-1] == 2.0 ** -11).all())
