"""The dense operators beside the MoE layer, measured: a matrix product with
bias, activation and residual in its epilogue, the gated feed-forward block,
and the clipping of a step's gradients by their global norm.

``run`` computes one pass of an operator: in elementary torch operations in
32 bits where ``own`` is false, through the package's entry points where it
is true.  ``exact`` evaluates the definitions in 64 bits.

    linear           z = x W^T + b,  y = act(z) + r
    linear_backward  dz = dy act'(z);  dx = dz W,  dW = dz^T x,  db = sum dz
    gated            a = x W1^T + b1, u = x W3^T + b3, h = act(a) u,
                     y = h W2^T + b2 + r
    gated_backward   dh = dy W2; dA = dh u act'(a), dU = dh act(a);
                     dx = dA W1 + dU W3, dW1 = dA^T x, dW3 = dU^T x,
                     dW2 = dy^T h, and the biases' column sums
    clip             n = sqrt(sum g^2),  c = min(1, max_norm / (n + 1e-6)),
                     g c for every gradient

The backward passes take what a forward pass leaves behind (z, or a and u, in
the layer's type) as inputs.
"""
import math

import torch

own = False

ACTS = ("identity", "relu", "silu", "gelu", "gelu_tanh")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP_EPS = 1e-6


# --------------------------------- the cases ---------------------------------

def listed():
    return [
        # one token through a Mixtral-shaped down-projection: serving, where
        # only the stream of the weights counts
        dict(name="linear_one_token", op="linear", dtype="bf16", M=1, K=14336, N=4096, act="identity",
             bias=False, residual=True, save=False, pad=0),
        # the first projection of the tiny fp32 layer: launch latency
        dict(name="linear_tiny_f32", op="linear", dtype="f32", M=256, K=64, N=128, act="relu",
             bias=True, residual=False, save=True, pad=0),
        # odd everything: rows of a wider buffer, no side a multiple of 8
        dict(name="linear_odd", op="linear", dtype="bf16", M=1001, K=1411, N=2049, act="gelu",
             bias=True, residual=True, save=True, pad=3),
        # the first projection of an ungated dense FFN on a long batch
        dict(name="linear_long", op="linear", dtype="bf16", M=16384, K=4096, N=16384, act="gelu_tanh",
             bias=True, residual=False, save=False, pad=0),
        # training a GShard-shaped dense FFN's first projection
        dict(name="linear_backward", op="linear_backward", dtype="bf16", M=4096, K=1024, N=4096,
             act="gelu", bias=True, pad=0),
        # four sequences decoding through a Mixtral-shaped dense FFN
        dict(name="gated_decode", op="gated", dtype="bf16", T=4, d=4096, f=14336, act="silu",
             bias=False, residual=True, save=False, pad=0),
        # the same block on a prompt batch
        dict(name="gated_prompt", op="gated", dtype="bf16", T=8192, d=4096, f=14336, act="silu",
             bias=False, residual=True, save=False, pad=0),
        # training forward of a ragged batch with biases, pre-activations kept
        dict(name="gated_ragged", op="gated", dtype="bf16", T=2047, d=2048, f=5632, act="gelu",
             bias=True, residual=True, save=True, pad=0),
        # the training backward at DeepSeekMoE's width and four times its expert size
        dict(name="gated_backward", op="gated_backward", dtype="bf16", T=8192, d=2048, f=5632,
             act="silu", bias=False, pad=0),
        # a small fp32 block, ragged, with biases: tests and small models
        dict(name="gated_backward_f32", op="gated_backward", dtype="f32", T=777, d=320, f=1000,
             act="gelu_tanh", bias=True, pad=0),
        # the gradients of the tiny fp32 layer (x, router, w1, w2), in place
        # and below the limit: what most steps of a run that has settled see
        dict(name="clip_tiny", op="clip", tensors="16384:f32,512:f32,65536:f32,65536:f32",
             clip=False, inplace=True),
        # a Mixtral-shaped layer's fp32 gradients and a dense block's bf16
        # ones, over the limit
        dict(name="clip_layer", op="clip",
             tensors="33554432:f32,32768:f32,469762048:f32,469762048:f32,469762048:f32,"
                     "58720256:bf16,58720256:bf16,58720256:bf16", clip=True, inplace=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer width: half of them multiples of 64, a quarter of 8, a quarter anything."""
    v, k = _log(rng, lo, hi), rng.random()
    g = 64 if k < 0.5 else 8 if k < 0.75 else 1
    return max(g, v // g * g)


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "gated", "gated", "gated_backward", "clip"))
    if op == "clip":
        n, parts, total = _log(rng, 1, 60), [], 0
        for _ in range(n):
            k = min(_log(rng, 1, 1 << 28), (1 << 29) - total)
            if k > 0:
                parts.append("%d:%s" % (k, rng.choice(("f32", "f32", "bf16"))))
                total += k
        clip = rng.random() < 0.7
        return dict(op=op, tensors=",".join(parts), clip=clip, inplace=not clip)
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    most = 1.0e12 if dtype == "bf16" else 1.2e11
    rows = _log(rng, 1, 16384)
    pad = rng.choice((0, 0, 8, 3))
    c = dict(op=op, dtype=dtype, act=rng.choice(ACTS), bias=rng.random() < 0.5, pad=pad)
    if op.startswith("linear"):
        c |= dict(M=rows, K=_width(rng, 16, 16384), N=_width(rng, 16, 16384))
        while work(c | dict(save=False, residual=False))["flops"] > most:
            c["M"] = max(1, c["M"] // 2)
    else:
        c["act"] = rng.choice(ACTS[1:])
        c |= dict(T=rows, d=_width(rng, 16, 8192), f=_width(rng, 16, 16384))
        while work(c | dict(save=False, residual=False))["flops"] > most:
            c["T"] = max(1, c["T"] // 2)
    if not op.endswith("backward"):
        c |= dict(residual=rng.random() < 0.6, save=rng.random() < 0.4)
    return c


def work(case):
    op = case["op"]
    if op == "clip":
        t = _tensors(case)
        es = sum(n * (4 if d == "f32" else 2) for n, d in t)
        # below the limit nothing changes in place: the gradients are only read
        return {"bytes": es * (1 if case["inplace"] and not case["clip"] else 2) + 4,
                "flops": 3 * sum(n for n, _ in t)}
    es = 4 if case["dtype"] == "f32" else 2
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        b = M * K + N * K + N * case["bias"] + M * N * (1 + case["residual"] + case["save"])
        return {"bytes": es * b, "flops": 2 * M * N * K}
    if op == "linear_backward":
        M, K, N = case["M"], case["K"], case["N"]
        b = 2 * M * K + 2 * N * K + N * case["bias"] + M * N * (1 + (case["act"] != "identity"))
        return {"bytes": es * b, "flops": 4 * M * N * K}
    T, d, f = case["T"], case["d"], case["f"]
    if op == "gated":
        b = T * d * (2 + case["residual"]) + 3 * d * f + (2 * f + d) * case["bias"] + 2 * T * f * case["save"]
        return {"bytes": es * b, "flops": 6 * T * d * f}
    return {"bytes": es * (3 * T * d + 2 * T * f + 6 * d * f + (2 * f + d) * case["bias"]),
            "flops": 12 * T * d * f}


def _tensors(case):
    return [(int(n), d) for n, d in (p.split(":") for p in case["tensors"].split(","))]


# --------------------------------- the inputs --------------------------------

class _Maker:
    """Seeded tensors on the GPU, drawn in fp32 and rounded to the type."""

    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = dtype

    def normal(self, *shape, std=1.0, dtype=None):
        t = torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.float32)
        return t.mul_(std).to(dtype or self.dtype)

    def rows(self, n, width, pad, std=1.0):
        """[n, width] rows of a buffer `pad` columns wider."""
        return self.normal(n, width + pad, std=std)[:, :width]

    def room(self, n, width, pad):
        """The same for an output: nothing written yet."""
        return torch.empty(n, width + pad, dtype=self.dtype, device="cuda")[:, :width]


def prepare(case, seed):
    op = case["op"]
    if op == "clip":
        m = _Maker(seed, torch.float32)
        std = 1e-3
        grads = [m.normal(n, std=std, dtype=DTYPES[d]) for n, d in _tensors(case)]
        norm = std * math.sqrt(sum(t.numel() for t in grads))
        s = dict(case=case, grads=grads, max_norm=norm * (0.37 if case["clip"] else 3.0))
        if own:
            from mixture_experts_layer_63_b200 import api
            s["norm"] = torch.empty((), device="cuda")
            s["out"] = None if case["inplace"] else [torch.empty_like(t) for t in grads]
            s["ws"] = api.new_clip_workspace(grads)
        return s
    dt, pad = DTYPES[case["dtype"]], case["pad"]
    m = _Maker(seed, dt)
    s = dict(case=case)
    if op.startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        s |= dict(x=m.rows(M, K, pad), w=m.normal(N, K, std=K ** -0.5),
                  b=m.normal(N, std=0.3) if case["bias"] else None)
        if op == "linear":
            s["r"] = m.rows(M, N, pad) if case["residual"] else None
        else:
            s["dy"] = m.rows(M, N, pad)
            # the pre-activations that the forward pass left
            s["z"] = None
            if case["act"] != "identity":
                s["z"] = s["x"] @ s["w"].T if s["b"] is None else torch.addmm(s["b"], s["x"], s["w"].T)
        if own:
            from mixture_experts_layer_63_b200 import api
            s["cfg"] = api.linear_config(M, K, N, act=case["act"], dtype=dt, ld_x=K + pad, ld_y=N + pad,
                                         ld_r=N + pad)
            s["ws"] = api.new_linear_workspace(s["cfg"], backward=op != "linear")
            if op == "linear":
                s["y"] = m.room(M, N, pad)
                s["z"] = m.room(M, N, 0) if case["save"] else None
            else:
                s |= dict(dx=m.room(M, K, pad), dw=torch.empty_like(s["w"]),
                          db=torch.empty_like(s["b"]) if case["bias"] else None)
        return s
    T, d, f = case["T"], case["d"], case["f"]
    s |= dict(x=m.rows(T, d, pad), w1=m.normal(f, d, std=d ** -0.5), w3=m.normal(f, d, std=d ** -0.5),
              w2=m.normal(d, f, std=f ** -0.5), b1=None, b3=None, b2=None)
    if case["bias"]:
        s |= dict(b1=m.normal(f, std=0.3), b3=m.normal(f, std=0.3), b2=m.normal(d, std=0.3))
    if op == "gated":
        s["r"] = m.rows(T, d, pad) if case["residual"] else None
    else:
        s["dy"] = m.rows(T, d, pad)
        # the two pre-activations that the forward pass left
        for p, w, b in (("a", "w1", "b1"), ("u", "w3", "b3")):
            s[p] = s["x"] @ s[w].T if s[b] is None else torch.addmm(s[b], s["x"], s[w].T)
    if own:
        from mixture_experts_layer_63_b200 import api
        s["cfg"] = api.gated_ffn_config(T, d, f, act=case["act"], dtype=dt, ld_x=d + pad, ld_y=d + pad,
                                        ld_r=d + pad)
        s["ws"] = api.new_gated_ffn_workspace(s["cfg"], backward=op != "gated")
        if op == "gated":
            s["y"] = m.room(T, d, pad)
            for p in ("a", "u"):
                s[p] = m.room(T, f, 0) if case["save"] else None
        else:
            s["dx"] = m.room(T, d, pad)
            for p in ("w1", "w3", "w2", "b1", "b3", "b2"):
                s["d" + p] = torch.empty_like(s[p]) if s[p] is not None else None
    return s


# ------------------------------ the plain forms -------------------------------

def _act(z, name):
    if name == "identity":
        return z
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    c, t = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float().T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(t), "z": z.to(t) if c["save"] else None}


def _linear_backward(s):
    c, t = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if c["act"] != "identity":
        dz = dz * _act_grad(s["z"].float(), c["act"])
    return {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.T @ s["x"].float()).to(t),
            "db": dz.sum(0).to(t) if s["b"] is not None else None}


def _gated(s):
    c, t = s["case"], s["x"].dtype
    x = s["x"].float()
    a, u = x @ s["w1"].float().T, x @ s["w3"].float().T
    if s["b1"] is not None:
        a, u = a + s["b1"].float(), u + s["b3"].float()
    y = (_act(a, c["act"]) * u) @ s["w2"].float().T
    if s["b2"] is not None:
        y = y + s["b2"].float()
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(t), "a": a.to(t) if c["save"] else None, "u": u.to(t) if c["save"] else None}


def _gated_backward(s):
    c, t = s["case"], s["x"].dtype
    x, dy, a, u = s["x"].float(), s["dy"].float(), s["a"].float(), s["u"].float()
    g = _act(a, c["act"])
    dh = dy @ s["w2"].float()
    da, du = dh * u * _act_grad(a, c["act"]), dh * g
    dx = da @ s["w1"].float() + du @ s["w3"].float()
    out = {"dx": dx, "dw1": da.T @ x, "dw3": du.T @ x, "dw2": dy.T @ (g * u)}
    if s["b1"] is not None:
        out |= {"db1": da.sum(0), "db3": du.sum(0), "db2": dy.sum(0)}
    return {k: v.to(t) for k, v in out.items()}


def _clip(s):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp_max(1.0).float()
    if s["case"]["inplace"]:
        out = [g.copy_(g.float() * coef) for g in s["grads"]]
    else:
        out = [(g.float() * coef).to(g.dtype) for g in s["grads"]]
    return {"norm": norm.float(), "grads": out}


# ------------------------------ the calls of a user -----------------------------

def _run_own(s):
    from mixture_experts_layer_63_b200 import api
    op = s["case"]["op"]
    if op == "linear":
        api.moe_linear(s["cfg"], s["x"], s["w"], s["b"], s["r"], s["y"], s["z"], s["ws"])
        return {"y": s["y"], "z": s["z"]}
    if op == "linear_backward":
        api.moe_linear_backward(s["cfg"], s["x"], s["w"], s["z"], s["dy"], s["dx"], s["dw"], s["db"],
                                s["ws"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "gated":
        api.moe_gated_ffn(s["cfg"], s["x"], s["w1"], s["b1"], s["w3"], s["b3"], s["w2"], s["b2"], s["r"],
                          s["y"], s["a"], s["u"], s["ws"])
        return {"y": s["y"], "a": s["a"], "u": s["u"]}
    if op == "gated_backward":
        api.moe_gated_ffn_backward(s["cfg"], s["x"], s["w1"], s["w3"], s["w2"], s["a"], s["u"], s["dy"],
                                   s["dx"], s["dw1"], s["db1"], s["dw3"], s["db3"], s["dw2"], s["db2"],
                                   s["ws"])
        return {k: s[k] for k in ("dx", "dw1", "dw3", "dw2", "db1", "db3", "db2")}
    api.moe_clip_grads(s["grads"], s["max_norm"], s["norm"], s["ws"], out=s["out"])
    return {"norm": s["norm"], "grads": s["grads"] if s["out"] is None else s["out"]}


PLAIN = {"linear": _linear, "linear_backward": _linear_backward, "gated": _gated,
         "gated_backward": _gated_backward, "clip": _clip}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------ 64-bit evaluation -------------------------------

def _act64(z, name):
    """act(z) and its derivative at z (float64), by automatic differentiation
    of torch's own activations."""
    import torch.nn.functional as F
    fn = {"identity": lambda v: v * 1.0, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
          "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name]
    with torch.enable_grad():
        v = z.detach().requires_grad_(True)
        out = fn(v)
        grad, = torch.autograd.grad(out.sum(), v)
    return out.detach(), grad


def exact(case, seed):
    s = prepare(case, seed)
    q = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op == "clip":
        total = math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"])
        norm = math.sqrt(total)
        coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "grads": [g.double() * coef for g in s["grads"]]}
    if op == "linear":
        z = torch.einsum("mk,nk->mn", q["x"], q["w"])
        z = z if q["b"] is None else z + q["b"]
        y = _act64(z, case["act"])[0]
        return {"y": y if q["r"] is None else y + q["r"], "z": z if case["save"] else None}
    if op == "linear_backward":
        dz = q["dy"] if q["z"] is None else q["dy"] * _act64(q["z"], case["act"])[1]
        return {"dx": torch.einsum("mn,nk->mk", dz, q["w"]), "dw": torch.einsum("mn,mk->nk", dz, q["x"]),
                "db": None if q["b"] is None else torch.einsum("mn->n", dz)}
    if op == "gated":
        a = torch.einsum("td,fd->tf", q["x"], q["w1"])
        u = torch.einsum("td,fd->tf", q["x"], q["w3"])
        if q["b1"] is not None:
            a, u = a + q["b1"], u + q["b3"]
        y = torch.einsum("tf,df->td", _act64(a, case["act"])[0] * u, q["w2"])
        y = y if q["b2"] is None else y + q["b2"]
        return {"y": y if q["r"] is None else y + q["r"], "a": a if case["save"] else None,
                "u": u if case["save"] else None}
    act, grad = _act64(q["a"], case["act"])
    dh = torch.einsum("td,df->tf", q["dy"], q["w2"])
    da, du = dh * q["u"] * grad, dh * act
    out = {"dx": torch.einsum("tf,fd->td", da, q["w1"]) + torch.einsum("tf,fd->td", du, q["w3"]),
           "dw1": torch.einsum("tf,td->fd", da, q["x"]), "dw3": torch.einsum("tf,td->fd", du, q["x"]),
           "dw2": torch.einsum("td,tf->df", q["dy"], act * q["u"])}
    if q["b1"] is not None:
        out |= {"db1": da.sum(0), "db3": du.sum(0), "db2": q["dy"].sum(0)}
    return out
