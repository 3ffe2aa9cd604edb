"""The norm, the ragged products and clipping as a user runs them: routing
without padding, the ragged layer forward and backward, a training step and a
serving step end to end, captured and replayed, and on other streams."""
import math

import numpy as np
import pytest
import torch

from block_sparse_gemm_amd import bsg, layer

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# ----------------------------------------------------- routing, no padding

@pytest.mark.parametrize("T, E, k", [(1, 8, 2), (5, 64, 1), (777, 40, 3), (5000, 8, 2),
                                     (66000, 3, 1)])
def test_route_without_padding(T, E, k):
    g = gen(T)
    logits = randn(g, T, E)
    i32 = dict(dtype=torch.int32, device="cuda")
    A, d = T * k, 64
    x = randn(g, T, d, dtype=BF16)
    outs = []
    for how in range(3):
        o = [torch.full((n,), -7, **i32) for n in (A, A, E, E + 1)]
        gate = torch.full((A,), float("nan"), device="cuda")
        idx, dest, counts, off = o
        ws = torch.zeros(bsg.route_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda")
        xp = torch.full((A + 8, d), 5.0, device="cuda", dtype=BF16)
        src = torch.full((A,), -7, **i32)
        if how == 0:
            bsg.route(logits, k, True, idx, gate, dest, counts, off, ws, bin_rows=1)
            bsg.permute_pad(x, k, dest, None, counts, off, E, A, src, xp, bin_rows=1)
        elif how == 1:
            bsg.route_noalloc(logits, k, True, idx, gate, dest, counts, off, bin_rows=1)
            bsg.permute_pad(x, k, dest, None, counts, off, E, A, src, xp, bin_rows=1)
        else:
            bsg.route_permute_topology(logits, k, True, idx, gate, dest, counts, off, ws, x, A,
                                       src, xp, bin_rows=1)
        outs.append([t.cpu().numpy() for t in (idx, dest, counts, off, src)] + [xp])
    idx, dest, counts, off, src, xp = outs[0]
    want = np.argsort(-logits.cpu().numpy(), axis=1, kind="stable")[:, :k].reshape(-1)
    assert np.array_equal(idx, want)
    assert np.array_equal(counts, np.bincount(want, minlength=E))
    assert np.array_equal(off, np.concatenate([[0], np.cumsum(counts)]))
    # ascending assignments inside each group, every row taken once
    place = np.empty(A, np.int64)
    place[np.argsort(want, kind="stable")] = np.arange(A)
    assert np.array_equal(dest, place)
    assert np.array_equal(src[dest], np.arange(A))
    assert torch.equal(xp[torch.from_numpy(dest).long().cuda()], x.repeat_interleave(k, 0))
    assert bool((xp[A:] == 5).all())
    for o in outs[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(o[:5], outs[0][:5]))
        assert torch.equal(o[5], xp)


# --------------------------------------------------------- the ragged layer

def layer_exact(x, logits, W1, W2, W3, k, renorm, E, picks):
    """The layer in fp64 on the CPU by autograd's rules; picks fixed."""
    d, f = W1.shape[0], W1.shape[1] // E
    p = torch.softmax(logits, 1)
    gate = torch.gather(p, 1, picks)
    if renorm:
        gate = gate / gate.sum(1, keepdim=True)
    y = 0
    for j in range(k):
        e = picks[:, j]
        parts = torch.zeros(x.shape[0], d, dtype=x.dtype)
        for ex in range(E):
            r = (e == ex).nonzero()[:, 0]
            if len(r) == 0:
                continue
            h = x[r] @ W1[:, ex * f:(ex + 1) * f]
            if W3 is None:
                a = 0.5 * h * (1 + torch.erf(h / math.sqrt(2)))
            else:
                a = torch.nn.functional.silu(h) * (x[r] @ W3[:, ex * f:(ex + 1) * f])
            parts = parts.index_put((r,), a @ W2[ex * f:(ex + 1) * f])
        y = y + gate[:, j:j + 1] * parts
    return y


LAYERS = [  # T, d, E, f, k, act, dtype, renorm
    (1, 64, 8, 72, 2, "swiglu", "f32", True),
    (3, 128, 64, 128, 1, "gelu", "f32", False),
    (300, 72, 5, 200, 2, "gelu", "f32", True),
    (257, 128, 7, 136, 3, "swiglu", "f32", False),
    (600, 128, 4, 256, 1, "gelu", "bf16", False),
    (333, 64, 6, 264, 2, "swiglu", "bf16", True),
]


def make_layer(T, d, E, f, k, act, dtype, renorm, seed=3):
    dt = BF16 if dtype == "bf16" else F32
    g = gen(seed)
    s = layer.Shape(T, d, E, f, k, act, dtype, yp_dtype=dtype, renorm=renorm, backward=True,
                    bin_rows=1)
    std = 1 / math.sqrt(d)
    t = dict(x=randn(g, T, d, dtype=dt), logits=randn(g, T, E), dy=randn(g, T, d, dtype=dt),
             W1=randn(g, d, E * f, dtype=dt, std=std),
             W2=randn(g, E * f, d, dtype=dt, std=1 / math.sqrt(f)),
             W3=randn(g, d, E * f, dtype=dt, std=std) if act == "swiglu" else None)
    return s, t


def leaf(t):
    return None if t is None else t.detach().double().cpu().requires_grad_()


@pytest.mark.parametrize("shape", LAYERS)
def test_ragged_layer_forward_and_backward(shape):
    s, t = make_layer(*shape)
    L = layer.Layer(s)
    L.forward(t["x"], t["logits"], t["W1"], t["W2"], t["W3"])
    L.backward(t["dy"], t["W1"], t["W2"], t["W3"])
    torch.cuda.synchronize()
    v = {n: leaf(t[n]) for n in ("x", "logits", "W1", "W2", "W3")}
    picks = torch.topk(t["logits"].cpu(), s.k, dim=1).indices
    assert torch.equal(L.expert_idx.cpu().view(-1, s.k).long(), picks)
    y = layer_exact(*(v[n] for n in ("x", "logits", "W1", "W2", "W3")), s.k, s.renorm, s.E, picks)
    y.backward(t["dy"].double().cpu())
    got = dict(y=(L.y, y.detach()), dx=(L.dx, v["x"].grad), dW1=(L.dW1, v["W1"].grad),
               dW2=(L.dW2, v["W2"].grad), dlogits=(L.dlogits, v["logits"].grad))
    if s.act == "swiglu":
        got["dW3"] = (L.dW3, v["W3"].grad)
    # each value passes at most four products; the sums of sizes are within a
    # few times the tensors' largest value, so a bound relative to that covers
    # them: fp32 sums of at most 600 terms, 4 * 600 * 2^-23 < 3e-4; bf16 storage of
    # each of the at most six tensors on the way, 6 * 2^-8 of it
    tol = 3e-4 if s.dtype == "f32" else 6 * 2.0 ** -8
    for name, (a, b) in got.items():
        d = (a.double().cpu() - b).abs().max().item()
        assert d <= tol * b.abs().max().item(), (name, d, b.abs().max().item())


@pytest.mark.parametrize("yp", ["bf16", "f32"])
def test_ragged_layer_agrees_with_the_padded_one(yp):
    shape = (700, 128, 6, 256, 2, "swiglu", "bf16", True)
    s, t = make_layer(*shape)
    s.yp_dtype = yp
    outs = []
    for rows in (1, 128):
        s.bin_rows = rows
        L = layer.Layer(s)
        L.forward(t["x"], t["logits"], t["W1"], t["W2"], t["W3"])
        outs.append([L.y] + list(L.backward(t["dy"], t["W1"], t["W2"], t["W3"])) + [L.dlogits])
    for a, b in zip(*outs):  # the same roundings; sums in another order move a few of them
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()


# ------------------------------------------------------- a step end to end

class Block:
    """norm(x + residual) -> router -> ragged experts, trained with clipping."""

    def __init__(self, T, d, E, f, k, act):
        self.s = layer.Shape(T, d, E, f, k, act, "f32", yp_dtype="f32", renorm=True, backward=True,
                             bin_rows=1)
        g = gen(7)
        std = 1 / math.sqrt(d)
        self.W1, self.W3 = (randn(g, d, E * f, std=std) for _ in range(2))
        self.W2 = randn(g, E * f, d, std=1 / math.sqrt(f))
        self.Wr = randn(g, 1, d, E, std=std)
        if act == "gelu":
            self.W3 = None
        self.wn = 1 + 0.1 * randn(g, d)
        self.norm = layer.Norm(T, d, self.wn, backward=True)
        self.L = layer.Layer(self.s)
        self.off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        self.logits = torch.empty(T, E, device="cuda")
        self.dn, self.dWr = torch.empty(T, d, device="cuda"), torch.empty_like(self.Wr)

    def step(self, x, r, dy, dh):
        n = self.norm.forward(x, r)
        bsg.grouped_gemm(n, self.off, self.Wr, self.logits)
        self.L.forward(n, self.logits, self.W1, self.W2, self.W3)
        dx = self.L.backward(dy, self.W1, self.W2, self.W3)[0]
        # the router's gradients; n is reached from the experts and the router
        bsg.grouped_wgrad(n, self.L.dlogits, self.off, self.dWr)
        bsg.grouped_gemm(self.L.dlogits, self.off, self.Wr, self.dn, trans_b=True)
        self.dn.add_(dx)
        self.norm.backward(self.dn, dh)
        self.L.clip_grads(0.5, more=[self.dWr, self.norm.dweight])

    def outputs(self):
        L = self.L
        w = [L.dW1, L.dW2] + ([L.dW3] if L.s.act == "swiglu" else [])
        return [self.norm.h, L.y, self.norm.dx, L.grad_norm, self.dWr, self.norm.dweight] + w


def block_inputs(B, seed):
    g = gen(seed)
    return [randn(g, B.s.T, B.s.d) for _ in range(4)]


def test_training_step_against_autograd():
    B = Block(120, 64, 8, 72, 2, "swiglu")
    x, r, dy, dh = block_inputs(B, 1)
    B.step(x, r, dy, dh)
    torch.cuda.synchronize()
    v = [leaf(t) for t in (x, r, B.wn, B.Wr[0], B.W1, B.W2, B.W3)]
    h = v[0] + v[1]
    n = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * v[2]
    logits = n @ v[3]
    picks = B.L.expert_idx.cpu().view(-1, B.s.k).long()
    assert torch.equal(picks, torch.topk(logits, B.s.k, dim=1).indices)
    y = layer_exact(n, logits, v[4], v[5], v[6], B.s.k, True, B.s.E, picks)
    ((y * dy.double().cpu()).sum() + (h * dh.double().cpu()).sum()).backward()
    grads = [v[4].grad, v[5].grad, v[6].grad, v[3].grad, v[2].grad]
    norm = math.sqrt(sum(float(t.square().sum()) for t in grads))
    assert norm > 0.5
    c = 0.5 / norm
    want = [h.detach(), y.detach(), v[0].grad, torch.tensor(norm), (v[3].grad * c)[None],
            v[2].grad * c, v[4].grad * c, v[5].grad * c, v[6].grad * c]
    for i, (a, b) in enumerate(zip(B.outputs(), want)):
        d = (a.double().cpu() - b).abs().max().item()
        # fp32 throughout, sums of at most 240 terms over at most seven products in a row:
        # 7 * 240 * 2^-23 = 2e-4 of the sums of sizes, which are a few times the largest value
        assert d <= 1e-3 * b.abs().max().item(), (i, d, b.abs().max().item())


def test_training_step_captured_and_replayed():
    B = Block(200, 64, 8, 128, 2, "gelu")
    x, r, dy, dh = block_inputs(B, 2)
    B.step(x, r, dy, dh)  # buffers exist
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.step(x, r, dy, dh)
    for seed in (11, 12, 13, 12):
        for to, of in zip((x, r, dy, dh), block_inputs(B, seed)):
            to.copy_(of)
        for t in B.outputs():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in B.outputs()]
        B.step(x, r, dy, dh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, B.outputs()))


@pytest.mark.parametrize("T", [1, 7, 64])
def test_serving_step_in_8_bits(T):
    d, E, f, k = 256, 8, 272, 2
    g = gen(T)
    x, r, wn = randn(g, T, d, dtype=BF16), randn(g, T, d, dtype=BF16), randn(g, d, dtype=BF16)
    q8, n16 = layer.Norm(T, d, wn, e4m3=True), layer.Norm(T, d, wn)
    q8.forward(x, r)
    n16.forward(x, r)
    logits = randn(g, T, E)
    W1, W3 = (randn(g, E, f, d).to(E4M3) for _ in range(2))
    ws = torch.rand(2, E, f, generator=g, device="cuda") * 0.1
    W2 = randn(g, E, f, d, dtype=BF16, std=0.1)
    i32 = dict(dtype=torch.int32, device="cuda")
    A = T * k
    idx, dest, src = (torch.empty(A, **i32) for _ in range(3))
    counts, off, gate = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(A, device="cuda")
    rows = torch.empty(A, d, device="cuda", dtype=E4M3)
    # 8-bit rows move as rows of d / 4 fp32 values
    bsg.route_noalloc(logits, k, True, idx, gate, dest, counts, off, bin_rows=1)
    bsg.permute_pad(q8.y.view(torch.float32), k, dest, None, counts, off, E, A, src,
                    rows.view(torch.float32), bin_rows=1)
    scale = q8.y_scale[src.long() // k]
    a, yp = torch.empty(A, f, device="cuda", dtype=BF16), torch.empty(A, d, device="cuda", dtype=BF16)
    y = torch.empty(T, d, device="cuda", dtype=BF16)
    w = torch.empty(max(bsg.grouped_gemm_workspace_bytes(A, d, f, E, "silu_mul"),
                        bsg.grouped_gemm_workspace_bytes(A, f, d, E), 16), device="cuda",
                    dtype=torch.uint8)
    bsg.grouped_gemm(rows, off, W1, a, "silu_mul", trans_b=True, b2=W3, a_scale=scale, b_scale=ws,
                     workspace=w)
    bsg.grouped_gemm(a, off, W2, yp, workspace=w)
    bsg.unpermute_combine(yp, dest, gate, T, k, d, y)
    # the same with the stored 8-bit values, in fp64
    n = q8.y.double() * q8.y_scale.double()[:, None]
    p = torch.softmax(logits.double(), 1)
    top = torch.topk(logits, k, dim=1).indices
    gates = torch.gather(p, 1, top)
    gates = gates / gates.sum(1, keepdim=True)
    want, size = torch.zeros(T, d, dtype=torch.float64, device="cuda"), 0
    for t in range(T):
        for j in range(k):
            e = int(top[t, j])
            h = (W1[e].double() * ws[0, e].double()[:, None]) @ n[t]
            u = (W3[e].double() * ws[1, e].double()[:, None]) @ n[t]
            act = torch.nn.functional.silu(h) * u
            want[t] += gates[t, j] * (act @ W2[e].double())
            size = max(size, float((act.abs() @ W2[e].double().abs()).max()))
    # per value: two 8-bit sums (7 * 2^-13 of sums of sizes a few times the values), bf16
    # storage of the activation, of the expert's row and of the result
    assert (y.double() - want).abs().max() <= 4 * 2.0 ** -8 * size
    # 8 bits against 16: half a step of e4m3 a value
    assert (n - n16.y.double()).abs().max() <= (2.0 ** -4 + 2.0 ** -8) * n.abs().max()


def test_two_streams_at_once():
    """The same calls on two streams, each with its own buffers, as on one."""
    Bs = [Block(300, 64, 8, 72, 2, "swiglu") for _ in range(2)]
    ins = [block_inputs(B, 20 + i) for i, B in enumerate(Bs)]
    want = []
    for B, i in zip(Bs, ins):
        B.step(*i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in B.outputs()])
    streams = [torch.cuda.Stream() for _ in Bs]
    for _ in range(3):
        for B in Bs:
            for t in B.outputs():
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for st, B, i in zip(streams, Bs, ins):
            with torch.cuda.stream(st):
                B.step(*i)
        torch.cuda.synchronize()
        for B, w in zip(Bs, want):
            assert all(torch.equal(a, b) for a, b in zip(B.outputs(), w))


def test_refusals_of_tensors_that_do_not_agree():
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    w, s4 = x[0].clone(), torch.zeros(4, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    b = torch.zeros(1, 64, 128, device="cuda", dtype=BF16)
    c = torch.zeros(4, 128, device="cuda", dtype=BF16)
    for bad in (lambda: bsg.rms_norm(x, w[:32], 1e-5, x), lambda: bsg.rms_norm(x, w.float(), 1e-5, x),
                lambda: bsg.rms_norm(x, w, 1e-5, x[:3]), lambda: bsg.rms_norm(x, w, 1e-5, x.float()),
                lambda: bsg.rms_norm(x, w, 1e-5, x, rstd=s4[:3]),
                lambda: bsg.rms_norm(x.t(), w, 1e-5, x.t()),
                lambda: bsg.rms_norm(x.cpu(), w, 1e-5, x),
                lambda: bsg.grouped_gemm(x, off, b[:, :32], c),
                lambda: bsg.grouped_gemm(x, off.long(), b, c),
                lambda: bsg.grouped_gemm(x, off[:1], b, c),
                lambda: bsg.grouped_gemm(x, off, b, c[:3]),
                lambda: bsg.grouped_gemm(x, off, b, c[:, :64]),
                lambda: bsg.grouped_gemm(x, off, b.float(), c),
                lambda: bsg.grouped_gemm(x, off, b, c, "gelu", aux_out=c[:, :120]),
                lambda: bsg.grouped_gemm(x, off, b, c, "silu_mul", b2=b.transpose(1, 2)),
                lambda: bsg.grouped_gemm(x, off, b, c, "silu_mul_bwd", aux_in=c),
                lambda: bsg.grouped_wgrad(x, c, off, b[:, :, :64]),
                lambda: bsg.grouped_wgrad(x, c[:3], off, b),
                lambda: bsg.grad_clip([s4], s4[0], 1.0, out=[s4[:2]]),
                lambda: bsg.grad_clip([x.t()], s4[0], 1.0),
                lambda: bsg.grad_norm([s4], s4, torch.zeros(4096, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bsg.grad_norm([off], s4[0], torch.zeros(4096, device="cuda"))
    with pytest.raises(bsg.BsgError) as e:  # the norm's tensors twice in place
        bsg.grad_clip([s4, s4], torch.zeros((), device="cuda"), 1.0)
    assert e.value.status == bsg.EINVAL


def test_norm_with_and_without_a_residual():
    g = gen(5)
    x, r, dy = (randn(g, 9, 72) for _ in range(3))
    w = randn(g, 72)
    both, plain = layer.Norm(9, 72, w, backward=True), layer.Norm(9, 72, w, residual=False,
                                                                  backward=True)
    both.forward(r, x)
    assert torch.equal(both.forward(x), plain.forward(x))
    assert all(torch.equal(a, b) for a, b in zip(both.backward(dy), plain.backward(dy)))
    with pytest.raises(ValueError):  # nowhere to keep the sum that the backward needs
        plain.forward(x, r)


def test_ragged_layer_rows_and_clipping_buffers():
    s = layer.Shape(T=16, d=64, E=4, f=72, k=2, dtype="f32", bin_rows=1, backward=True)
    m = layer.Layer(s)
    m.act.normal_()
    rows = torch.tensor([3, 0, 31], device="cuda", dtype=torch.int32)
    assert torch.equal(m.sparse_rows(m.act, rows), m.act[[3, 0, 31]])
    assert m.grad_norm.numel() == 1 and m.clip_ws.numel() == bsg.grad_norm_workspace_bytes()
