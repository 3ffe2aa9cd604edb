"""The operators around the expert layer, as they are measured: the cases, their inputs and their plain forms.

Five calls.  ``rms_norm`` adds the residual stream to a block's input and normalises the sum (in storage type, or in
e4m3 with one scale a row); ``rms_norm_backward`` is its gradient; ``grouped_gemm`` multiplies the rows of each expert
by that expert's weights, the rows of a group as many as the routing left there, with the expert layer's epilogues;
``grouped_wgrad`` is the gradient of those weights; ``grad_norm`` and ``grad_clip`` take the 2-norm over a list of
gradients and scale them down to a limit.

``own`` False: plain torch in 32 bits (sums over whole gradients in 64).  ``own`` True: the library's calls.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving, four sequences one token each: the add and the norm before the experts, rows handed on in 8 bits
        dict(name="norm_tokens_8bit", op="norm", T=4, d=4096, dtype="bf16", out="e4m3", residual=True),
        # the same norm over a prompt of 8192 tokens, or over a training batch, kept in bf16 with what backward needs
        dict(name="norm_prompt", op="norm", T=8192, d=4096, dtype="bf16", out="bf16", residual=True),
        # its gradient over the 65536 tokens of the skewed training layer, joined with the residual stream's
        dict(name="norm_backward", op="norm_backward", T=65536, d=1024, dtype="bf16", residual=True),
        # one token through two of eight SwiGLU experts: two rows against 235 MB of weights each for W1 and W3
        dict(name="experts_one_token", op="up", T=1, k=2, E=8, d=4096, f=14336, act="swiglu", dtype="bf16", save=False,
             skew=False),
        # a serving batch of 48 tokens, the experts' second product with weights and rows in 8 bits
        dict(name="experts_batch_8bit", op="down", T=48, k=2, E=8, d=4096, f=14336, act="swiglu", dtype="e4m3",
             save=False, skew=False),
        # a training batch of the small layer's first product, GeLU, its derivative kept: about 256 rows an expert
        dict(name="experts_up", op="up", T=16384, k=1, E=64, d=512, f=2048, act="gelu", dtype="bf16", save=True,
             skew=False),
        # a prompt through SwiGLU experts in 8 bits
        dict(name="experts_prompt_8bit", op="up", T=8192, k=2, E=8, d=4096, f=14336, act="swiglu", dtype="e4m3",
             save=False, skew=False),
        # the gradient of the skewed layer's input: 131072 rows, ten hot experts with most of them
        dict(name="experts_input_grad", op="input_grad", T=65536, k=2, E=64, d=1024, f=4096, act="gelu", dtype="bf16",
             save=False, skew=True),
        # weight gradients: the small layer's W1 (64 experts of about 256 rows), and the large one's (8 of about 2048)
        dict(name="weight_grad_small", op="weight_grad", T=16384, k=1, E=64, d=512, f=2048, dtype="bf16", skew=False),
        dict(name="weight_grad_large", op="weight_grad", T=8192, k=2, E=8, d=4096, f=14336, dtype="bf16", skew=False),
        # clipping: the 40 gradients of a small model, odd sizes among them, and a whole skewed layer's two
        dict(name="clip_many_small", op="clip", tensors=40, most=200003, dtype="mixed"),
        dict(name="clip_layer", op="clip", tensors=2, most=268435456, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, dtype):
    step = 16 if dtype == "e4m3" else 8
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "up", "up", "down", "up_grad", "input_grad", "weight_grad", "clip"])
    if op == "norm":
        c = dict(op=op, T=_log(rng, 1, 16384), d=_width(rng, 64, 8192, "bf16"), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 residual=rng.random() < 0.7)
        c["out"] = rng.choice([c["dtype"], "e4m3"])
        return c
    if op == "norm_backward":
        return dict(op=op, T=_log(rng, 1, 32768), d=_width(rng, 64, 4096, "bf16"), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7)
    if op == "clip":
        n = rng.randint(1, 60)
        return dict(op=op, tensors=n, most=_log(rng, 10, 200_000_000 // n), dtype=rng.choice(["bf16", "f32", "mixed"]))
    kinds = {"up": ["bf16", "bf16", "e4m3", "f32"], "down": ["bf16", "bf16", "e4m3", "f32"]}.get(op, ["bf16", "bf16", "f32"])
    dtype = rng.choice(kinds)
    E = _log(rng, 1, 64)
    c = dict(op=op, T=_log(rng, 1, 16384), k=rng.randint(1, min(E, 4)), E=E, d=_width(rng, 128, 4096, dtype),
             f=_width(rng, 128, 8192, dtype), dtype=dtype, skew=rng.random() < 0.3)
    if op != "weight_grad":
        c["act"] = rng.choice(["gelu", "swiglu"])
        c["save"] = op == "up" and dtype != "e4m3" and rng.random() < 0.5
    # no costlier than the largest listed: at most 2 TFLOP, and the weights within a few GB
    while 4.0 * c["T"] * c["k"] * c["d"] * c["f"] > 2e12:
        c["T"] = max(1, c["T"] // 2)
    while c["E"] * c["d"] * c["f"] > 500_000_000:
        c["f"] = max(128, c["f"] // 2 // 16 * 16)
    return c


# ----------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device=g.device, dtype=torch.float32 if dtype == E4M3 else dtype)
    return t.mul_(std).to(dtype)


def _counts(case, g):
    """Rows of each expert: a top-k routing of the case's tokens, with a few hot and starved experts where it is skewed."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn((T, E), generator=g, device=g.device)
    if case["skew"]:
        bias = torch.zeros(E, device=g.device)
        bias[:max(1, E * 10 // 64)] = 1.33
        bias[E - E * 6 // 64:] = -1.0
        logits += bias[torch.randperm(E, generator=g, device=g.device)]
    picks = torch.topk(logits, k, dim=1).indices.reshape(-1)
    return torch.bincount(picks, minlength=E)


def _clip_sizes(case):
    """Sizes from one value to `most`, odd ones among them, the last of them `most` itself (every one, where there are two)."""
    n, most = case["tensors"], case["most"]
    if n <= 2:
        return [most] * n
    return [max(1, int(most ** ((i % 10) / 9.0)) - (i // 10) % 3) if i % 10 else 1 + i for i in range(n - 1)] + [most]


def prepare(case, seed):
    device = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = _gen(seed, device)
    op, dtype = case["op"], TYPES.get(case["dtype"])
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        s["x"] = _randn(g, (T, d), dtype)
        s["residual"] = _randn(g, (T, d), dtype, 3.0) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=device)).to(dtype)
        if op == "norm":
            out = TYPES[case["out"]]
            s["h"] = torch.empty((T, d), dtype=dtype, device=device) if case["residual"] else None
            s["y"] = torch.empty((T, d), dtype=out, device=device)
            s["scale"] = torch.empty(T, dtype=torch.float32, device=device) if out == E4M3 else None
            s["rstd"] = torch.empty(T, dtype=torch.float32, device=device)
        else:  # h, 1/rms of its rows and two gradients are what the forward and the blocks above leave
            s["h"] = _randn(g, (T, d), dtype, 2.0)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = s.pop("x")
            s["dh"] = s.pop("residual")
            s["dx"] = torch.empty((T, d), dtype=dtype, device=device)
            s["dweight"] = torch.empty(d, dtype=torch.float32, device=device)
    elif op == "clip":
        kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32, torch.bfloat16]}
        kinds = kinds[case["dtype"]]
        s["grads"] = [_randn(g, (n,), kinds[i % len(kinds)], 0.01) for i, n in enumerate(_clip_sizes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty((), dtype=torch.float32, device=device)
        s["max_norm"] = 1.0
    else:
        counts = _counts(case, g)
        E, d, f, M = case["E"], case["d"], case["f"], case["T"] * case["k"]
        s["row_offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=device)
        s["row_offsets"][1:] = torch.cumsum(counts, 0)
        # what the plain form's padded batch goes by: the experts that have rows, and each row's place in the batch
        sizes = counts.tolist()
        s["most"] = max(sizes)
        s["active"] = torch.tensor([e for e in range(E) if sizes[e]], device=device)
        rank = torch.cumsum((counts > 0).long(), 0) - 1
        of = torch.repeat_interleave(torch.arange(E, device=device), counts)
        s["place"] = rank[of] * s["most"] + torch.arange(M, device=device) - s["row_offsets"][of].long()
        two = case.get("act") == "swiglu"
        f8 = dtype == E4M3
        cdt = torch.bfloat16 if f8 else dtype
        if op == "weight_grad":
            s["a"], s["b"] = _randn(g, (M, d), dtype), _randn(g, (M, f), dtype, 0.1)
            s["c"] = torch.empty((d, E * f), dtype=dtype, device=device).view(d, E, f).permute(1, 0, 2)
            return s
        K, N = {"up": (d, f), "down": (f, d), "up_grad": (d, f), "input_grad": (f, d)}[op]
        n_b = 2 if two and op in ("up", "input_grad") else 1
        n_a = 2 if two and op == "input_grad" else 1
        s["a"] = [_randn(g, (M, K), dtype, 1.0 if op == "up" else 0.5) for _ in range(n_a)]
        if f8:  # weights laid out once with K contiguous, a scale for each output column, a scale for each row
            s["b"] = [_randn(g, (E, N, K), dtype) for _ in range(n_b)]
            s["trans_b"] = True
            s["a_scale"] = 0.5 + torch.rand(M, generator=g, device=device)
            s["b_scale"] = 0.02 * (0.5 + torch.rand((n_b, E, N), generator=g, device=device))
        else:  # W1, W3 [d, E f] and W2 [E f, d] as the expert layer holds them, seen expert by expert
            s["trans_b"] = op in ("up_grad", "input_grad")
            if op in ("up", "input_grad"):
                s["b"] = [_randn(g, (d, E * f), dtype, 0.02).view(d, E, f).permute(1, 0, 2) for _ in range(n_b)]
            else:
                s["b"] = [_randn(g, (E * f, d), dtype, 0.02).view(E, f, d) for _ in range(n_b)]
            s["a_scale"] = s["b_scale"] = None
        planes = (2,) if two else ()
        s["aux_in"] = _randn(g, planes + (M, N), cdt) if op == "up_grad" else None
        s["aux_out"] = torch.empty(planes + (M, N), dtype=cdt, device=device) if case["save"] else None
        s["c"] = torch.empty((planes if op == "up_grad" else ()) + (M, N), dtype=cdt, device=device)
    return s


# -------------------------------------------------------------------- run

def _workspace(s, nbytes, *args):
    """The state's workspace, made on its first pass and kept, as a program that calls again and again keeps it."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(nbytes(*args), 256), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    from block_sparse_gemm_amd import bsg
    case = s["case"]
    op = case["op"]
    if op == "norm":
        bsg.rms_norm(s["x"], s["weight"], EPS, s["y"], h=s["h"], residual=s["residual"], y_scale=s["scale"], rstd=s["rstd"])
        return s["h"], s["y"], s["scale"], s["rstd"]
    if op == "norm_backward":
        ws = _workspace(s, bsg.rms_norm_backward_workspace_bytes, case["T"], case["d"])
        bsg.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], ws, dh=s["dh"])
        return s["dx"], s["dweight"]
    if op == "clip":
        ws = _workspace(s, bsg.grad_norm_workspace_bytes)
        bsg.grad_norm(s["grads"], s["norm"], ws)
        bsg.grad_clip(s["grads"], s["norm"], s["max_norm"], out=s["out"])
        return [s["norm"]] + s["out"]
    if op == "weight_grad":
        bsg.grouped_wgrad(s["a"], s["b"], s["row_offsets"], s["c"])
        return s["c"]
    two = case["act"] == "swiglu"
    epilogue = "none"
    if op == "up":
        epilogue = "silu_mul" if two else "gelu"
    elif op == "up_grad":
        epilogue = "silu_mul_bwd" if two else "gelu_bwd"
    (M, K), N = s["a"][0].shape, s["c"].shape[-1]
    ws = _workspace(s, bsg.grouped_gemm_workspace_bytes, M, K, N, case["E"], epilogue)
    bsg.grouped_gemm(s["a"][0], s["row_offsets"], s["b"][0], s["c"], epilogue=epilogue, trans_b=s["trans_b"],
                     a2=s["a"][1] if len(s["a"]) > 1 else None, b2=s["b"][1] if len(s["b"]) > 1 else None,
                     a_scale=s["a_scale"], b_scale=s["b_scale"], aux_in=s["aux_in"], aux_out=s["aux_out"], workspace=ws)
    return s["c"], s["aux_out"]


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------ plain forms

def _plain(s):
    return {"norm": _norm, "norm_backward": _norm_backward, "clip": _clip, "weight_grad": _weight_grad}.get(
        s["case"]["op"], _products)(s)


def _norm(s):
    x = s["x"].float()
    h = None
    if s["residual"] is not None:
        h = (x + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
    rstd = torch.rsqrt((x * x).mean(1) + EPS)
    y = x * rstd[:, None] * s["weight"].float()
    scale = None
    if s["y"].dtype == E4M3:
        most = y.abs().amax(1)
        scale = torch.where(most == 0, torch.ones_like(most), most / E4M3_MAX)
        y = y / scale[:, None]
    return h, y.to(s["y"].dtype), scale, rstd


def _norm_backward(s):
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    dn = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (dn - n * (dn * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), (dy * n).sum(0)


def _clip(s):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    scale = torch.where(norm <= s["max_norm"], torch.ones_like(norm), s["max_norm"] / norm)
    return [norm] + [(g.float() * scale).to(g.dtype) for g in s["grads"]]


def _batch(s, rows):
    """[M, K] rows as a zero-padded [experts with rows, most rows of one, K] batch, in 32 bits."""
    n = s["active"].numel()
    out = torch.zeros((n * s["most"], rows.shape[1]), dtype=torch.float32, device=rows.device)
    out[s["place"]] = rows.float()
    return out.view(n, s["most"], -1)


def _weight_grad(s):
    c = torch.zeros((s["case"]["d"], s["case"]["E"], s["case"]["f"]), dtype=s["a"].dtype, device=s["a"].device)
    c = c.permute(1, 0, 2)
    c[s["active"]] = torch.bmm(_batch(s, s["a"]).transpose(1, 2).contiguous(), _batch(s, s["b"])).to(c.dtype)
    return c


def _product(s, rows, weights, which):
    w = weights[s["active"]].float()
    if s["trans_b"]:
        w = w.transpose(1, 2).contiguous()
    p = torch.bmm(_batch(s, rows), w)
    p = p.view(-1, p.shape[2])[s["place"]]
    if s["a_scale"] is not None:
        of = s["active"][s["place"] // s["most"]]
        p = p * s["a_scale"][:, None] * s["b_scale"][which][of]
    return p


def _products(s):
    op, two = s["case"]["op"], s["case"]["act"] == "swiglu"
    cdt = s["c"].dtype
    p = _product(s, s["a"][0], s["b"][0], 0)
    saved = None
    if op == "up" and two:
        u = _product(s, s["a"][0], s["b"][1], 1)
        sig = 1.0 / (1.0 + torch.exp(-p))
        silu = p * sig
        saved = torch.stack([silu, u * (sig * (1.0 + p * (1.0 - sig)))])
        p = silu * u
    elif op == "up":
        cdf = 0.5 * (1.0 + torch.erf(p * math.sqrt(0.5)))
        saved = cdf + p * torch.exp(-0.5 * p * p) * (1.0 / math.sqrt(2.0 * math.pi))
        p = p * cdf
    elif op == "up_grad" and two:
        aux = s["aux_in"].float()
        p = torch.stack([p * aux[1], p * aux[0]])
    elif op == "up_grad":
        p = p * s["aux_in"].float()
    elif op == "input_grad" and two:
        p = p + _product(s, s["a"][1], s["b"][1], 1)
    return p.to(cdt), saved.to(cdt) if s["case"]["save"] else None


# ------------------------------------------------------------------- work

_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, d, b = case["T"], case["d"], _BYTES[case["dtype"]]
        r = case["residual"]
        if op == "norm":
            out = _BYTES[case["out"]]
            bytes_ = T * d * (b * (3 if r else 1) + out) + d * b + 4 * T * (2 if case["out"] == "e4m3" else 1)
            return dict(bytes=bytes_, flops=T * d * (5 if r else 4))
        return dict(bytes=T * d * b * (4 if r else 3) + d * (b + 4) + 4 * T, flops=T * d * 10)
    if op == "clip":
        kinds = {"bf16": [2], "f32": [4], "mixed": [2, 4, 2]}[case["dtype"]]
        sizes = _clip_sizes(case)
        each = sum(n * kinds[i % len(kinds)] for i, n in enumerate(sizes))
        return dict(bytes=2 * each + 4, flops=3 * sum(sizes))
    T, k, E, d, f, b = case["T"], case["k"], case["E"], case["d"], case["f"], _BYTES[case["dtype"]]
    M = T * k
    active = E * (1.0 - (1.0 - k / E) ** T)  # experts that are expected to have rows
    if op == "weight_grad":
        return dict(bytes=b * (M * (d + f) + E * d * f) + 4 * (E + 1), flops=2.0 * M * d * f)
    two = case["act"] == "swiglu"
    K, N = {"up": (d, f), "down": (f, d), "up_grad": (d, f), "input_grad": (f, d)}[op]
    n_b = 2 if two and op in ("up", "input_grad") else 1
    n_a = 2 if two and op == "input_grad" else 1
    cb = 2 if b == 1 else b
    outs = (2 if two and op == "up_grad" else 1) + ((2 if two else 1) if case["save"] else 0)
    ins = (2 if two else 1) if op == "up_grad" else 0
    bytes_ = b * (n_a * M * K + n_b * active * K * N) + cb * M * N * (outs + ins) + 4 * (E + 1)
    if b == 1:
        bytes_ += 4 * (M + n_b * active * N)
    return dict(bytes=bytes_, flops=2.0 * M * K * N * n_b)


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        stored = h.to(s["x"].dtype).double()  # the norm is of the sum as it is stored
        inv = 1.0 / torch.sqrt(stored.pow(2).sum(1) / case["d"] + EPS)
        y = torch.einsum("td,t,d->td", stored, inv, s["weight"].double())
        top = None
        if s["scale"] is not None:
            top = y.abs().max(1).values / E4M3_MAX
            top[top == 0] = 1.0
            y = y / top.unsqueeze(1)
        return (None if s["residual"] is None else h), y, top, inv
    if op == "norm_backward":
        h, w, dy = s["h"].double(), s["weight"].double(), s["dy"].double()
        r = s["rstd"].double().unsqueeze(1)
        along = (dy * w * h).sum(1, keepdim=True) / case["d"]
        dx = r * dy * w - r.pow(3) * along * h
        if s["dh"] is not None:
            dx += s["dh"].double()
        return dx, torch.einsum("td,td,t->d", dy, h, r.squeeze(1))
    if op == "clip":
        total = 0.0
        for g in s["grads"]:
            total += float(torch.linalg.vector_norm(g.double())) ** 2
        norm = math.sqrt(total)
        by = min(1.0, s["max_norm"] / norm) if norm else 1.0
        return [torch.tensor(norm, dtype=torch.float64)] + [g.double() * by for g in s["grads"]]
    at = s["row_offsets"].tolist()
    groups = [(e, slice(at[e], at[e + 1])) for e in range(case["E"]) if at[e + 1] > at[e]]
    if op == "weight_grad":
        c = torch.zeros((case["E"], case["d"], case["f"]), dtype=torch.float64, device=s["a"].device)
        for e, r in groups:
            c[e] = s["a"][r].double().t().contiguous() @ s["b"][r].double()
        return c
    M, N = s["c"].shape[-2:]

    def product(i, j):
        out = torch.empty((M, N), dtype=torch.float64, device=s["c"].device)
        for e, r in groups:
            w = s["b"][j][e].double()
            out[r] = s["a"][i][r].double() @ (w.t().contiguous() if s["trans_b"] else w)
            if s["a_scale"] is not None:
                out[r] *= s["a_scale"][r].double().unsqueeze(1)
                out[r] *= s["b_scale"][j, e].double()
        return out

    p = product(0, 0)
    two = case["act"] == "swiglu"
    kept = None
    if op == "up":
        if two:
            sig = torch.sigmoid(p)
            u = product(0, 1)
            kept = torch.stack([p * sig, u * sig * (1.0 + p - p * sig)]) if case["save"] else None
            p = p * sig * u
        else:
            phi = torch.special.ndtr(p)
            kept = phi + p * torch.exp(-p.pow(2) / 2) / math.sqrt(2 * math.pi) if case["save"] else None
            p = p * phi
    elif op == "up_grad":
        p = torch.stack([p * s["aux_in"][1].double(), p * s["aux_in"][0].double()]) if two else p * s["aux_in"].double()
    elif op == "input_grad" and two:
        p += product(1, 1)
    return p, kept
