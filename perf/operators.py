"""Timing cases of the unquantised-block operators: LayerNorm, the dense linear with its epilogue, 8-bit checkpoints.

A case is one call (or the few calls that belong together) of a training or inference step on random data of the
value distributions these operators meet: a residual stream with outlier channels and padding rows, weights of
std 0.02, unit gradients.  With `own` false the operators run as elementary torch operations in fp32 (fp64 where
a rounding border matters); with `own` true they run as the library's entry points.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 64          # columns that share one scale in an 8-bit checkpoint
TINY = 2.0 ** -118  # a block below this is stored as zeros


def listed():
    return [
        # one generated token through a LayerNorm: launch latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "d": 4096},
        # four sequences of 512 tokens at hidden size 4096
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 2048, "d": 4096},
        # an odd number of packed tokens at the hidden size of a small stack
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "rows": 333, "d": 576, "residual": True},
        # sixteen sequences of 512 tokens at hidden size 5120
        {"name": "ln_bwd_long", "op": "ln_bwd", "rows": 8192, "d": 5120, "residual": True},
        # a layer's checkpoint of a short sequence: saved, restored for the recompute, read by the norm's backward
        {"name": "ckpt_short", "op": "ckpt", "rows": 64, "d": 576},
        # the same for four sequences of 512 tokens
        {"name": "ckpt_batch", "op": "ckpt", "rows": 2048, "d": 4096},
        # and for sixteen sequences at hidden size 5120
        {"name": "ckpt_long", "op": "ckpt", "rows": 8192, "d": 5120},
        # one generated token through a linear of hidden size 4096: the weight's bytes decide
        {"name": "linear_fwd_token", "op": "linear_fwd", "rows": 1, "n": 4096, "k": 4096, "act": "gelu",
         "bias": True, "residual": False, "keep_z": False},
        # an odd number of tokens through the up projection of a small stack, training (the pre-activation is kept)
        {"name": "linear_fwd_ragged", "op": "linear_fwd", "rows": 333, "n": 1536, "k": 576, "act": "silu",
         "bias": True, "residual": True, "keep_z": True},
        # the up projection of hidden size 4096 over four sequences of 512 tokens, training
        {"name": "linear_fwd_up", "op": "linear_fwd", "rows": 2048, "n": 14336, "k": 4096, "act": "gelu_tanh",
         "bias": True, "residual": False, "keep_z": True},
        # backward of a small stack's linear over an odd number of tokens
        {"name": "linear_bwd_ragged", "op": "linear_bwd", "rows": 130, "n": 576, "k": 1536, "act": "gelu"},
        # backward of the up projection over four sequences of 512 tokens
        {"name": "linear_bwd_up", "op": "linear_bwd", "rows": 2048, "n": 14336, "k": 4096, "act": "gelu_tanh"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "ckpt", "linear_fwd", "linear_bwd"))
    if op in ("ln_fwd", "ln_bwd", "ckpt"):
        d = 8 * _log(rng, 8, 1536)
        rows = _log(rng, 1, min(16384, 8192 * 5120 // d))
        case = {"op": op, "rows": rows, "d": d}
        if op == "ln_bwd":
            case["residual"] = rng.random() < 0.5
        return case
    n, k = 8 * _log(rng, 8, 1792), 8 * _log(rng, 8, 1792)
    rows = _log(rng, 1, max(1, min(8192, 2048 * 14336 * 4096 // (n * k))))
    case = {"op": op, "rows": rows, "n": n, "k": k, "act": rng.choice(ACTS)}
    if op == "linear_fwd":
        case.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, keep_z=rng.random() < 0.5)
    return case


def work(case):
    rows = case["rows"]
    if case["op"] in ("ln_fwd", "ln_bwd", "ckpt"):
        d = case["d"]
        e = rows * d
        if case["op"] == "ln_fwd":      # x, g, b in; y, mean, rstd out
            return {"bytes": 4 * e + 4 * d + 8 * rows, "flops": 8 * e}
        if case["op"] == "ln_bwd":      # dy, x, (residual gradient), g, mean, rstd in; dx, dg, db out
            return {"bytes": (8 if case["residual"] else 6) * e + 10 * d + 8 * rows, "flops": 14 * e}
        c = e + 2 * rows * (-(-d // BLOCK))   # codes and block maxima
        save, restore, back = 4 * e + c, 4 * e + c, 6 * e + c
        return {"bytes": save + restore + back + 6 * d + 12 * rows, "flops": 24 * e}
    n, k = case["n"], case["k"]
    if case["op"] == "linear_fwd":
        outs = 1 + bool(case["residual"]) + bool(case["keep_z"])
        return {"bytes": 2 * (rows * k + n * k + outs * rows * n + (n if case["bias"] else 0)),
                "flops": 2 * rows * n * k}
    zs = 1 if case["act"] == "none" else 2
    return {"bytes": 2 * (zs * rows * n + 2 * rows * k + 2 * n * k) + 4 * n, "flops": 4 * rows * n * k}


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _stream(g, rows, d):
    """A residual stream: unit values, a few channels tens of times larger, every 61st row padding (zeros)."""
    x = torch.randn(rows, d, generator=g, device="cuda", dtype=torch.float32)
    gain = torch.ones(d, device="cuda")
    hot = torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")
    gain[hot] = 40.0
    x = x * gain + 0.25
    x[60::61] = 0.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = dict(case)
    rows = case["rows"]
    if case["op"] in ("ln_fwd", "ln_bwd", "ckpt"):
        d = case["d"]
        st["x"] = _stream(g, rows, d)
        st["g"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        st["eps"] = 1e-5
        if case["op"] == "ln_fwd":
            st["b"] = _normal(g, (d,), 0.1)
            return st
        st["dy"] = _normal(g, (rows, d))
        st["dy"][60::61] = 0.0          # no gradient reaches padding
        if case["op"] == "ckpt" or case["residual"]:
            st["dres"] = _normal(g, (rows, d))
        if case["op"] == "ln_bwd":      # the statistics that the forward pass left
            x = st["x"].double()
            st["mean"] = x.mean(1).float()
            st["rstd"] = (1.0 / torch.sqrt(x.var(1, unbiased=False) + st["eps"])).float()
        return st
    n, k = case["n"], case["k"]
    st["x"] = _normal(g, (rows, k))
    st["w"] = _normal(g, (n, k), 0.02)
    if case["op"] == "linear_fwd":
        st["b"] = _normal(g, (n,), 0.1) if case["bias"] else None
        st["res"] = _normal(g, (rows, n)) if case["residual"] else None
        return st
    st["dy"] = _normal(g, (rows, n))
    st["z"] = _normal(g, (rows, n)) if case["act"] != "none" else None   # the pre-activation the forward kept
    return st


# ---------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _round8(x):
    """bf16 [rows, d] -> the bf16 values its 8-bit checkpoint stands for."""
    rows, d = x.shape
    nb = -(-d // BLOCK)
    v = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :d] = x.double()
    v = v.view(rows, nb, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    safe = torch.where(top >= TINY, top, torch.ones_like(top))
    q = torch.sign(v) * torch.floor(v.abs() * 127.0 / safe + 0.5)
    out = torch.where(top >= TINY, q * safe / 127.0, torch.zeros_like(v))
    return out.view(rows, nb * BLOCK)[:, :d].to(torch.bfloat16)


def _rms(x, g, eps):
    v = x.float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + eps)
    return (v * rstd[:, None] * g.float()).to(torch.bfloat16), rstd


def _plain(st):
    op = st["op"]
    if op == "ln_fwd":
        v = st["x"].float()
        mean = v.mean(1)
        c = v - mean[:, None]
        rstd = 1.0 / torch.sqrt((c * c).mean(1) + st["eps"])
        y = c * rstd[:, None] * st["g"].float() + st["b"].float()
        return {"y": y.to(torch.bfloat16), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dy = st["dy"].float()
        xh = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        a = dy * st["g"].float()
        dx = st["rstd"][:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
        if st["residual"]:
            dx = dx + st["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dg": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "ckpt":
        y, _ = _rms(st["x"], st["g"], st["eps"])
        xr = _round8(st["x"])
        yr, rstd = _rms(xr, st["g"], st["eps"])
        a, v = st["dy"].float() * st["g"].float(), xr.float()
        dx = rstd[:, None] * a - v * (rstd ** 3)[:, None] * (a * v).mean(1, keepdim=True) + st["dres"].float()
        return {"y": y, "x_restored": xr, "y_restored": yr, "rstd": rstd, "dx": dx.to(torch.bfloat16)}
    if op == "linear_fwd":
        z = st["x"].float() @ st["w"].float().T
        if st["b"] is not None:
            z = z + st["b"].float()
        y = _act(z, st["act"])
        if st["res"] is not None:
            y = y + st["res"].float()
        out = {"y": y.to(torch.bfloat16)}
        if st["keep_z"]:
            out["z"] = z.to(torch.bfloat16)
        return out
    dz = st["dy"].float()
    if st["act"] != "none":
        dz = dz * _dact(st["z"].float(), st["act"])
    return {"dx": (dz @ st["w"].float()).to(torch.bfloat16), "dw": (dz.T @ st["x"].float()).to(torch.bfloat16),
            "db": dz.sum(0)}


# ---------------------------------------------------------------- the library's calls
def _buffers(st):
    """What a caller keeps between calls: the output tensors and the workspace, made at the first pass."""
    from nf4_layer_streamed_blockwise_b200 import lib as L
    rows = st["rows"]

    def bf(*shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")

    def f32(*shape):
        return torch.empty(*shape, dtype=torch.float32, device="cuda")

    def u8(size):
        return torch.empty(max(int(size), 1), dtype=torch.uint8, device="cuda")

    op = st["op"]
    st["lib"] = L
    if op == "ln_fwd":
        st["out"] = {"y": bf(rows, st["d"]), "mean": f32(rows), "rstd": f32(rows)}
    elif op == "ln_bwd":
        st["out"] = {"dx": bf(rows, st["d"]), "dg": f32(st["d"]), "db": f32(st["d"])}
        st["ws"] = u8(L.lsq_layernorm_bwd_workspace_size(rows, st["d"]))
    elif op == "ckpt":
        st["out"] = {"y": bf(rows, st["d"]), "x_restored": bf(rows, st["d"]), "y_restored": bf(rows, st["d"]),
                     "rstd": f32(rows), "dx": bf(rows, st["d"])}
        st["ckpt"] = u8(L.lsq_ckpt8_size(rows, st["d"]))
    elif op == "linear_fwd":
        st["out"] = {"y": bf(rows, st["n"])}
        if st["keep_z"]:
            st["out"]["z"] = bf(rows, st["n"])
    else:
        st["out"] = {"dx": bf(rows, st["k"]), "dw": bf(st["n"], st["k"]), "db": f32(st["n"])}
        st["ws"] = u8(L.lsq_linear_bwd_workspace_size(rows, st["n"], st["k"], ACTS.index(st["act"])))


def _library(st):
    if "out" not in st:
        _buffers(st)
    L, o, op, rows = st["lib"], st["out"], st["op"], st["rows"]
    if op == "ln_fwd":
        L.lsq_layernorm_fwd(st["x"], st["g"], st["b"], o["y"], o["mean"], o["rstd"], rows, st["d"], st["eps"])
    elif op == "ln_bwd":
        L.lsq_layernorm_bwd(st["dy"], st["x"], st["g"], st["mean"], st["rstd"], st.get("dres"), o["dx"], o["dg"],
                            o["db"], 0, rows, st["d"], st["ws"])
    elif op == "ckpt":
        L.lsq_rmsnorm_fwd_pack8(st["x"], st["g"], o["y"], None, st["ckpt"], rows, st["d"], st["eps"])
        L.lsq_rmsnorm_fwd_unpack8(st["ckpt"], st["g"], o["x_restored"], o["y_restored"], o["rstd"], rows, st["d"],
                                  st["eps"])
        L.lsq_rmsnorm_bwd_unpack8(st["dy"], st["ckpt"], st["g"], o["rstd"], st["dres"], o["dx"], rows, st["d"])
    elif op == "linear_fwd":
        L.lsq_linear_fwd(st["x"], st["w"], st["b"], ACTS.index(st["act"]), st["res"], o.get("z"), o["y"], rows,
                         st["n"], st["k"])
    else:
        L.lsq_linear_bwd(st["dy"], st["x"], st["w"], st["z"], ACTS.index(st["act"]), o["dx"], o["dw"], 0, o["db"], 0,
                         rows, st["n"], st["k"], st["ws"])
    return o


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_round8(x):
    """Each element's code from its block's largest magnitude, gathered by block index."""
    rows, d = x.shape
    v = x.double()
    block = (torch.arange(d, device=x.device) // BLOCK).expand(rows, d)
    top = torch.zeros(rows, -(-d // BLOCK), dtype=torch.float64, device=x.device)
    top = top.scatter_reduce(1, block, v.abs(), "amax")
    per = top.gather(1, block)
    code = torch.trunc((v.abs() * 254.0 + per) / (2.0 * per)) * torch.sign(v)
    back = code * per / 127.0
    return torch.where(per < TINY, torch.zeros_like(back), back).float().to(torch.bfloat16).double()


def _exact_rms_grad(v, g, dy, eps):
    """Gradient of g x / sqrt(mean x^2 + eps) by the product rule on the unit-norm form."""
    d = v.shape[1]
    s = ((v * v).sum(1, keepdim=True) / d + eps).sqrt()
    u = v / s
    w = dy * g
    return (w - u * ((w * u).sum(1, keepdim=True) / d)) / s


def exact(case, seed):
    st = prepare(case, seed)
    f = {name: t.double() for name, t in st.items() if isinstance(t, torch.Tensor)}
    op = case["op"]
    if op == "ln_fwd":
        var, mean = torch.var_mean(f["x"], dim=1, correction=0)
        sd = torch.sqrt(var + st["eps"])
        return {"y": (f["x"] - mean[:, None]) / sd[:, None] * f["g"] + f["b"], "mean": mean, "rstd": 1.0 / sd}
    if op == "ln_bwd":
        d = case["d"]
        xh = torch.addcmul(-(f["mean"] * f["rstd"])[:, None], f["x"], f["rstd"][:, None])
        w = f["dy"] * f["g"]
        proj = torch.einsum("ij,ij->i", w, xh)[:, None] / d
        dx = f["rstd"][:, None] * (w - w.sum(1, keepdim=True) / d - proj * xh)
        if case["residual"]:
            dx = dx + f["dres"]
        return {"dx": dx, "dg": torch.einsum("ij,ij->j", f["dy"], xh), "db": f["dy"].sum(0)}
    if op == "ckpt":
        d = case["d"]

        def unit(v):
            return v / ((v * v).sum(1, keepdim=True) / d + st["eps"]).sqrt()

        xr = _exact_round8(st["x"])
        return {"y": unit(f["x"]) * f["g"], "x_restored": xr, "y_restored": unit(xr) * f["g"],
                "rstd": ((xr * xr).sum(1) / d + st["eps"]) ** -0.5,
                "dx": _exact_rms_grad(xr, f["g"], f["dy"], st["eps"]) + f["dres"]}
    normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device="cuda"), 1.0)

    def phi(z, act):
        if act == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if act == "gelu":
            return z * normal.cdf(z)
        if act == "gelu_tanh":
            return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        if act == "silu":
            return z * torch.sigmoid(z)
        return z

    if op == "linear_fwd":
        z = torch.einsum("mk,nk->mn", f["x"], f["w"])
        if case["bias"]:
            z += f["b"]
        y = phi(z, case["act"])
        if case["residual"]:
            y = y + f["res"]
        return {"y": y, "z": z} if case["keep_z"] else {"y": y}
    dz = f["dy"]
    if case["act"] != "none":       # the derivative of phi, by differentiating it
        z = f["z"].requires_grad_(True)
        dz = torch.autograd.grad(phi(z, case["act"]), z, grad_outputs=dz)[0]
    return {"dx": torch.einsum("mn,nk->mk", dz, f["w"]), "dw": torch.einsum("mn,mk->nk", dz, f["x"]),
            "db": dz.sum(0)}
