"""Refusals of the norm, the ragged grouped products and clipping, without a
GPU: bad arguments are reported before any HIP call (pointers here are never
dereferenced), and the binding refuses tensors that do not agree."""
import ctypes as C

import pytest
import torch

from block_sparse_gemm_amd import bsg

P = C.c_void_p(0x10000)
MIS = C.c_void_p(0x10004)     # 4-byte but not 16-byte aligned
ODD = C.c_void_p(0x10002)
NAN = float("nan")
INF = float("inf")


@pytest.fixture(scope="module")
def L():
    return bsg.lib()


def caller(fn, names, ok):
    def call(**over):
        a = list(ok)
        for key, v in over.items():
            a[names.index(key)] = v
        return fn(*a)
    return call


NORM = ("x ldx r ldr w eps T d dt h ldh y ldy ydt scale rstd s".split(),
        [P, 64, P, 64, P, 1e-5, 3, 64, bsg.BF16, P, 64, P, 64, bsg.BF16, None, P, None])


@pytest.mark.parametrize("over, want", [
    (dict(x=None), bsg.EINVAL), (dict(x=MIS), bsg.EINVAL), (dict(w=None), bsg.EINVAL),
    (dict(y=None), bsg.EINVAL), (dict(y=MIS), bsg.EINVAL), (dict(r=MIS), bsg.EINVAL),
    (dict(h=MIS), bsg.EINVAL), (dict(rstd=ODD), bsg.EINVAL), (dict(ldx=63), bsg.EINVAL),
    (dict(ldx=68), bsg.EINVAL), (dict(ldr=8), bsg.EINVAL), (dict(ldh=0), bsg.EINVAL),
    (dict(ldy=-64), bsg.EINVAL), (dict(T=-1), bsg.EINVAL), (dict(T=1 << 31), bsg.EINVAL),
    (dict(d=0), bsg.EINVAL), (dict(d=60), bsg.EINVAL), (dict(d=-8), bsg.EINVAL),
    (dict(d=1 << 25), bsg.EINVAL), (dict(dt=7), bsg.EINVAL), (dict(dt=bsg.E4M3), bsg.EINVAL),
    (dict(ydt=bsg.F32), bsg.EINVAL), (dict(eps=-1.0), bsg.EINVAL), (dict(eps=NAN), bsg.EINVAL),
    (dict(eps=INF), bsg.EINVAL), (dict(r=None), bsg.EINVAL),     # h without a residual
    (dict(scale=P), bsg.EINVAL), (dict(ydt=bsg.E4M3), bsg.EINVAL),   # scale and e4m3 go together
    (dict(ydt=bsg.E4M3, scale=P, ldy=68), bsg.EINVAL),
    (dict(ydt=bsg.E4M3, scale=P, y=MIS), bsg.EINVAL),
    (dict(d=16392, ldx=16392, ldr=16392, ldh=16392, ldy=16392), bsg.EUNSUPPORTED),
    (dict(T=0, x=None, y=None, w=None), bsg.OK),
])
def test_rms_norm_refusals(L, over, want):
    assert caller(L.bsg_rms_norm, *NORM)(**over) == want
    assert bool(L.bsg_last_error()) == (want != bsg.OK)


def test_rms_norm_backward_refusals(L):
    need = bsg.rms_norm_backward_workspace_bytes(1000, 64)
    assert need == 512 * 64 * 4
    assert bsg.rms_norm_backward_workspace_bytes(3, 64) == 3 * 64 * 4
    assert bsg.rms_norm_backward_workspace_bytes(-1, 64) == 0
    assert bsg.rms_norm_backward_workspace_bytes(3, 0) == 0
    call = caller(L.bsg_rms_norm_backward,
                  "dy lddy dh lddh h ldh w rstd T d dt dx lddx dw ws wsb s".split(),
                  [P, 64, P, 64, P, 64, P, P, 1000, 64, bsg.BF16, P, 64, P, P, need, None])
    for over in (dict(dy=None), dict(dh=MIS), dict(h=None), dict(w=MIS), dict(rstd=None),
                 dict(dx=None), dict(dw=None), dict(ws=None), dict(ws=MIS), dict(wsb=need - 1),
                 dict(lddy=8), dict(lddh=60), dict(ldh=0), dict(lddx=63), dict(d=63), dict(T=-1),
                 dict(dt=bsg.E4M3)):
        assert call(**over) == bsg.EINVAL, over


GEMM_NAMES = ("a a2 lda asc b b2 ldb sb bsc trans off E M K N epi auxi c ldc cdt auxo dt ws wsb "
              "s").split()
GEMM = [P, None, 64, None, P, None, 128, 8192, None, 0, P, 4, 100, 64, 128, bsg.EPI_NONE, None, P,
        128, bsg.BF16, None, bsg.BF16, None, 0, None]
F8 = dict(dt=bsg.E4M3, trans=1, ldb=64, asc=P, bsc=P)


@pytest.mark.parametrize("over, want", [
    (dict(a=None), bsg.EINVAL), (dict(a=MIS), bsg.EINVAL), (dict(b=None), bsg.EINVAL),
    (dict(c=None), bsg.EINVAL), (dict(off=None), bsg.EINVAL), (dict(off=ODD), bsg.EINVAL),
    (dict(E=0), bsg.EINVAL), (dict(E=1025), bsg.EINVAL), (dict(M=-1), bsg.EINVAL),
    (dict(M=1 << 31), bsg.EINVAL), (dict(K=0), bsg.EINVAL), (dict(K=60), bsg.EINVAL),
    (dict(N=0), bsg.EINVAL), (dict(N=124), bsg.EINVAL), (dict(K=72), bsg.EINVAL),  # lda < K
    (dict(lda=68), bsg.EINVAL), (dict(ldb=64), bsg.EINVAL), (dict(ldb=132), bsg.EINVAL),
    (dict(sb=-8), bsg.EINVAL), (dict(sb=4), bsg.EINVAL), (dict(ldc=64), bsg.EINVAL),
    (dict(ldc=132), bsg.EINVAL), (dict(trans=2), bsg.EINVAL), (dict(epi=9), bsg.EINVAL),
    (dict(dt=5), bsg.EINVAL), (dict(cdt=bsg.E4M3), bsg.EINVAL),
    (dict(lda=1 << 25), bsg.EUNSUPPORTED), (dict(ldb=1 << 27), bsg.EUNSUPPORTED),
    (dict(cdt=bsg.F32, epi=bsg.EPI_GELU), bsg.EUNSUPPORTED),
    (dict(dt=bsg.F32), bsg.EUNSUPPORTED),                          # fp32 operands, bf16 output
    (dict(a2=P), bsg.EINVAL), (dict(b2=P), bsg.EINVAL), (dict(a2=MIS, b2=P), bsg.EINVAL),
    (dict(epi=bsg.EPI_SILU_MUL), bsg.EINVAL), (dict(epi=bsg.EPI_SILU_MUL, b2=P, a2=P), bsg.EINVAL),
    (dict(epi=bsg.EPI_GELU, b2=P), bsg.EINVAL), (dict(epi=bsg.EPI_GELU_BWD), bsg.EINVAL),
    (dict(epi=bsg.EPI_GELU, auxi=P), bsg.EINVAL), (dict(auxo=P), bsg.EINVAL),
    (dict(epi=bsg.EPI_GELU, auxo=MIS), bsg.EINVAL), (dict(asc=P), bsg.EINVAL),
    (dict(bsc=P), bsg.EINVAL), (dict(ws=MIS, wsb=64), bsg.EINVAL),
    (dict(F8, trans=0, ldb=128), bsg.EUNSUPPORTED), (dict(F8, asc=None), bsg.EINVAL),
    (dict(F8, bsc=MIS), bsg.EINVAL), (dict(F8, K=56), bsg.EINVAL),
    (dict(F8, epi=bsg.EPI_GELU, auxo=P), bsg.EUNSUPPORTED),
    (dict(F8, epi=bsg.EPI_GELU_BWD, auxi=P), bsg.EUNSUPPORTED),
    (dict(F8, a2=P, b2=P), bsg.EUNSUPPORTED), (dict(F8, cdt=bsg.F32), bsg.EUNSUPPORTED),
    (dict(E=1024, M=(1 << 31) - 1, N=1 << 24, ldb=1 << 24, ldc=1 << 24), bsg.EUNSUPPORTED),
    (dict(M=0, a=None, c=None), bsg.OK),
])
def test_grouped_gemm_refusals(L, over, want):
    assert caller(L.bsg_grouped_gemm, GEMM_NAMES, GEMM)(**over) == want


def test_grouped_wgrad_refusals(L):
    call = caller(L.bsg_grouped_wgrad, "a lda d ldd off E M K N c ldc sc cdt dt ws wsb s".split(),
                  [P, 64, P, 128, P, 4, 100, 64, 128, P, 128, 8192, bsg.BF16, bsg.BF16, None, 0,
                   None])
    for over in (dict(a=None), dict(d=MIS), dict(off=None), dict(c=None), dict(E=0), dict(E=1025),
                 dict(M=-1), dict(K=4), dict(N=4), dict(K=72), dict(N=136), dict(lda=68),
                 dict(ldd=132), dict(ldc=64), dict(ldc=132), dict(sc=0), dict(sc=4),
                 dict(dt=bsg.E4M3), dict(cdt=3), dict(ws=MIS, wsb=64)):
        assert call(**over) == bsg.EINVAL, over
    assert call(dt=bsg.F32) == bsg.EUNSUPPORTED
    assert call(lda=1 << 27) == bsg.EUNSUPPORTED
    assert call(E=1024, K=1 << 24, N=1 << 24, lda=1 << 24, ldd=1 << 24,
                ldc=1 << 24) == bsg.EUNSUPPORTED


def _list(ptrs, counts, dtypes):
    n = len(ptrs)
    return (C.c_void_p * n)(*ptrs), (C.c_int64 * n)(*counts), (C.c_int * n)(*dtypes), n


def test_grad_norm_refusals(L):
    wsb = bsg.grad_norm_workspace_bytes()

    def call(ptrs=(0x1000, 0x2000), counts=(5, 7), dtypes=(bsg.F32, bsg.BF16), norm=P, ws=P,
             wsb=wsb):
        a, b, c, n = _list(ptrs, counts, dtypes)
        return L.bsg_grad_norm(a, b, c, n, norm, ws, wsb, None)

    assert call(ptrs=(0x1000, None)) == bsg.EINVAL
    assert call(ptrs=(0x1002, 0x2000)) == bsg.EINVAL      # fp32 at a 2-byte boundary
    assert call(ptrs=(0x1000, 0x2001)) == bsg.EINVAL
    assert call(counts=(5, -1)) == bsg.EINVAL
    assert call(counts=(5, 1 << 50)) == bsg.EINVAL
    assert call(dtypes=(bsg.F32, bsg.E4M3)) == bsg.EINVAL
    assert call(norm=None) == bsg.EINVAL
    assert call(ws=None) == bsg.EINVAL
    assert call(ws=MIS) == bsg.EINVAL
    assert call(wsb=wsb - 1) == bsg.EINVAL
    assert L.bsg_grad_norm(None, None, None, 1, P, P, wsb, None) == bsg.EINVAL
    assert L.bsg_grad_norm(None, None, None, -1, P, P, wsb, None) == bsg.EINVAL


def test_grad_clip_refusals(L):
    def call(ptrs=(0x1000, 0x2000), out=None, counts=(5, 7), dtypes=(bsg.F32, bsg.F32), norm=P,
             most=1.0):
        a, b, c, n = _list(ptrs, counts, dtypes)
        o = (C.c_void_p * n)(*out) if out else None
        return L.bsg_grad_clip(a, o, b, c, n, norm, most, None)

    assert call(norm=None) == bsg.EINVAL
    assert call(most=-1.0) == bsg.EINVAL
    assert call(most=NAN) == bsg.EINVAL
    assert call(out=(0x3000, None)) == bsg.EINVAL
    assert call(out=(0x3000, 0x4002)) == bsg.EINVAL
    # the same tensor twice in place; overlapping ends; an output on another's input
    assert call(ptrs=(0x1000, 0x1000)) == bsg.EINVAL
    assert call(ptrs=(0x1000, 0x1010)) == bsg.EINVAL
    assert call(ptrs=(0x1010, 0x1000)) == bsg.EINVAL
    assert call(out=(0x2000, 0x3000)) == bsg.EINVAL
    assert call(out=(0x1004, 0x3000)) == bsg.EINVAL
    assert call(out=(0x3000, 0x3000)) == bsg.EINVAL


@pytest.mark.parametrize("T, k, E", [(1, 1, 1), (7, 2, 5), (4096, 4, 64)])
def test_bins_without_padding(T, k, E):
    assert bsg.max_padded_rows(T, k, E, 1) == T * k


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current GPU"):
        bsg.rms_norm(x, x[0], 1e-5, x)
    with pytest.raises(ValueError, match="current GPU"):
        bsg.grouped_gemm(x, torch.zeros(2, dtype=torch.int32), x.view(1, 64, 4), x)
    with pytest.raises(ValueError, match="current GPU"):
        bsg.grad_norm([x], torch.zeros(1), x)


def test_grad_clip_refuses_a_norm_that_it_would_write(L):
    a, b, c, n = _list((0x1000, 0x2000), (5, 7), (bsg.F32, bsg.F32))
    o = (C.c_void_p * n)(0x3000, 0x4000)
    for out, norm in ((None, 0x1000), (None, 0x1010), (None, 0x2018), (o, 0x3000), (o, 0x4008)):
        assert L.bsg_grad_clip(a, out, b, c, n, norm, 1.0, None) == bsg.EINVAL


def test_binding_refuses_sizes_beyond_the_c_types():
    def empty(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="meta")

    wide = empty(2, (1 << 32) + 64)
    with pytest.raises(ValueError):
        bsg._rows("rms_norm", "x", wide, wide.shape, wide.dtype)
    for shape in ((1, 8, (1 << 32) + 64), (1, (1 << 32) + 64, 8), ((1 << 32) + 1, 1, 8)):
        b = empty(*shape)
        with pytest.raises(ValueError):
            bsg._matrices("grouped_gemm", "b", b, b.shape, b.dtype)
