"""Measured cases of the operators around the FP8 scaled matmul: the product
with activation and residual in its epilogue, its gradient forms, and layer
norm forward and backward.

``run`` computes an operator in plain 32-bit torch operations (``own`` false)
or through this package's entry points (``own`` true) on the same inputs;
``exact`` gives the definition's values in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token through an up-projection: a decode step, where latency counts
        dict(name="mm one token", op="mm", M=1, N=4096, K=4096, act="silu", bias=True, residual=False,
             preact=False, rowwise=True, a="e4m3", out="bf16"),
        # a short prompt through a down-projection of odd width: rows that are not 16-byte aligned
        dict(name="mm ragged", op="mm", M=300, N=4999, K=4112, act="gelu_tanh", bias=True, residual=True,
             preact=False, rowwise=False, a="e4m3", out="fp16"),
        # a training batch through the first product of an MLP; the value before the activation is kept
        dict(name="mm up train", op="mm", M=8192, N=16384, K=4096, act="gelu", bias=True, residual=False,
             preact=True, rowwise=True, a="e4m3", out="bf16"),
        # the second product of an MLP, added onto the residual stream: the largest case
        dict(name="mm down residual", op="mm", M=16384, N=4096, K=14336, act="none", bias=True, residual=True,
             preact=False, rowwise=True, a="e4m3", out="bf16"),
        # a small batch's gradient through the second product and the activation before it
        dict(name="mm grad small", op="mm_grad", M=512, N=4096, K=2048, act="silu", rowwise=True, a="e5m2",
             out="bf16"),
        # the same for a training batch
        dict(name="mm grad train", op="mm_grad", M=8192, N=14336, K=4096, act="gelu", rowwise=True, a="e5m2",
             out="bf16"),
        # activation and bias gradient of a small ragged batch
        dict(name="act grad ragged", op="act_grad", M=300, N=4999, act="gelu_tanh", dz=True, dbias=True, out="fp16"),
        # and of a training batch
        dict(name="act grad train", op="act_grad", M=16384, N=14336, act="gelu", dz=True, dbias=True, out="bf16"),
        # one token's normalisation, quantised for the product that follows
        dict(name="norm one token", op="norm", R=1, C=4096, x="bf16", y="bf16", q="e4m3"),
        # a training batch's, with the normalised rows and the statistics kept
        dict(name="norm train", op="norm", R=16384, C=8192, x="bf16", y="bf16", q="e4m3"),
        # backward of a small fp32 batch of odd width
        dict(name="norm grad ragged", op="norm_grad", R=300, C=4999, x="fp32", y="fp32", residual=False),
        # backward of a training batch, added onto the residual stream's gradient
        dict(name="norm grad train", op="norm_grad", R=16384, C=8192, x="bf16", y="bf16", residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 64, the others as they come."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["mm", "mm_grad", "act_grad", "norm", "norm_grad"])
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
    out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("mm", "mm_grad"):
        n = _width(rng, 64, 16384)
        k = 16 * _log_int(rng, 1, 896)
        m = min(_log_int(rng, 1, 16384), max(1, 16384 * 4096 * 8192 // (n * k)))
        c = dict(op=op, M=m, N=n, K=k, act=act, rowwise=rng.random() < 0.5, a=rng.choice(["e4m3", "e5m2"]), out=out)
        if op == "mm":
            c.update(act=rng.choice(["none", act]), bias=rng.random() < 0.75, residual=rng.random() < 0.5,
                     preact=rng.random() < 0.5)
        return c
    if op == "act_grad":
        n = _width(rng, 64, 16384)
        m = min(_log_int(rng, 1, 32768), 16384 * 14336 // (n * (2 if out == "fp32" else 1)))
        return dict(op=op, M=m, N=n, act=act, dz=True, dbias=rng.random() < 0.75, out=out)
    c = _width(rng, 64, 32768)
    x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    r = min(_log_int(rng, 1, 65536), 16384 * 8192 // (c * (2 if x == "fp32" else 1)))
    if op == "norm":
        return dict(op=op, R=r, C=c, x=x, y=rng.choice([x, "bf16"]), q=rng.choice(["", "e4m3", "e5m2"]))
    return dict(op=op, R=r, C=c, x=x, y=rng.choice([x, "bf16"]), residual=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op in ("mm", "mm_grad"):
        m, n, k, o = case["M"], case["N"], case["K"], BYTES[case["out"]]
        nbytes = m * k + n * k + m * n * o + 4 * ((m + n) if case["rowwise"] else 2)
        if op == "mm":
            nbytes += n * o * case["bias"] + m * n * o * (case["residual"] + case["preact"])
        else:
            nbytes += m * n * o
        return {"bytes": nbytes, "flops": 2.0 * m * n * k}
    if op == "act_grad":
        m, n, o = case["M"], case["N"], BYTES[case["out"]]
        return {"bytes": m * n * o * (2 + case["dz"]) + 4 * n * case["dbias"], "flops": 20.0 * m * n}
    r, c, x, y = case["R"], case["C"], BYTES[case["x"]], BYTES[case["y"]]
    if op == "norm":
        return {"bytes": r * c * (x + y + (1 if case["q"] else 0)) + 4 * r * (2 + bool(case["q"])) + 8 * c,
                "flops": 8.0 * r * c}
    return {"bytes": r * c * (y + 2 * x + x * case["residual"]) + 8 * r + 12 * c, "flops": 14.0 * r * c}


# ----------------------------------------------------------------- inputs ---

def _quantise(x, q, rowwise):
    """fp32 x [R, C] to fp8 codes and scales (amax / qmax), as the operands of a scaled product are made."""
    amax = x.abs().amax(dim=1, keepdim=True) if rowwise else x.abs().amax().reshape(1, 1)
    s = (amax / QMAX[q]).clamp_min(1e-30)
    return (x / s).clamp_(-QMAX[q], QMAX[q]).to(DTYPES[q]), s.reshape(-1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale)

    op = case["op"]
    s = dict(case)
    if op in ("mm", "mm_grad"):
        m, n, k, out = case["M"], case["N"], case["K"], DTYPES[case["out"]]
        s["A"], s["sa"] = _quantise(randn(m, k), case["a"], case["rowwise"])
        # weights of variance 2 / K: values before the activation spread over both of its ends
        bt, s["sb"] = _quantise(randn(n, k, scale=math.sqrt(2.0 / k)), "e4m3", case["rowwise"])
        s["B"] = bt.t()                     # [K, N], column-major
        if op == "mm":
            s["b"] = randn(n, scale=0.2).to(out) if case["bias"] else None
            s["r"] = randn(m, n, scale=1.5).to(out) if case["residual"] else None
        else:
            s["z"] = randn(m, n, scale=1.5).to(out)
    elif op == "act_grad":
        m, n, out = case["M"], case["N"], DTYPES[case["out"]]
        s["z"] = randn(m, n, scale=1.5).to(out)
        s["dy"] = randn(m, n, scale=0.5).to(out)
    else:
        r, c = case["R"], case["C"]
        # a residual stream: rows of different size, an offset, a few large channels
        x = randn(r, c)
        x.mul_(torch.exp(randn(r, 1, scale=0.3))).add_(randn(1, c, scale=0.3)).add_(0.1)
        s["x"] = x.to(DTYPES[case["x"]])
        s["gamma"] = randn(c, scale=0.2).add_(1.0)
        s["beta"] = randn(c, scale=0.1)
        if op == "norm_grad":
            xf = s["x"].float()
            mean = xf.mean(dim=1)
            s["mean"], s["rstd"] = mean, torch.rsqrt((xf - mean[:, None]).square_().mean(dim=1) + EPS)
            s["dy"] = randn(r, c, scale=0.5).to(DTYPES[case["y"]])
            s["res"] = randn(r, c, scale=0.5).to(s["x"].dtype) if case["residual"] else None
    return s


# ------------------------------------------------------------- plain form ---

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _product(s):
    z = s["A"].float() @ s["B"].float()
    if s["rowwise"]:
        return z * (s["sa"][:, None] * s["sb"][None, :])
    return z * (s["sa"] * s["sb"])


def _plain(s):
    op = s["op"]
    if op == "mm":
        out = DTYPES[s["out"]]
        z = _product(s)
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"out": y.to(out), "preact": z.to(out)} if s["preact"] else {"out": y.to(out)}
    if op == "mm_grad":
        return {"dz": (_product(s) * _act_grad(s["z"].float(), s["act"])).to(DTYPES[s["out"]])}
    if op == "act_grad":
        dz = s["dy"].float() * _act_grad(s["z"].float(), s["act"])
        r = {}
        if s["dbias"]:
            r["dbias"] = dz.sum(dim=0)
        if s["dz"]:
            r["dz"] = dz.to(DTYPES[s["out"]])
        return r
    x = s["x"].float()
    if op == "norm":
        mean = x.mean(dim=1)
        d = x - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(dim=1) + EPS)
        y = d * rstd[:, None] * s["gamma"] + s["beta"]
        r = {"y": y.to(DTYPES[s["y"]]), "mean": mean, "rstd": rstd}
        if s["q"]:
            scale = y.abs().amax(dim=1) / QMAX[s["q"]]
            r["q"] = (y / scale[:, None]).clamp(-QMAX[s["q"]], QMAX[s["q"]]).to(DTYPES[s["q"]])
            r["scale"] = scale
        return r
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    w = dy * s["gamma"]
    dx = s["rstd"][:, None] * (w - w.mean(dim=1, keepdim=True) - xhat * (w * xhat).mean(dim=1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(dim=0), "dbeta": dy.sum(dim=0)}


# -------------------------------------------------------- the entry points ---

def _own(s):
    import fp8_scaled_gemm_gb300 as fm
    act = {"none": fm.ACT_NONE, "relu": fm.ACT_RELU, "gelu": fm.ACT_GELU, "gelu_tanh": fm.ACT_GELU_TANH,
           "silu": fm.ACT_SILU}
    op = s["op"]
    if op in ("mm", "mm_grad"):
        mode = fm.SCALE_ROWWISE if s["rowwise"] else fm.SCALE_TENSOR
        out = DTYPES[s["out"]]
        if op == "mm_grad":
            return {"dz": fm.fp8_scaled_mm_act_grad(s["A"], s["B"], s["sa"], s["sb"], mode, s["z"], act[s["act"]],
                                                    out_dtype=out)}
        r = fm.fp8_scaled_mm_epilogue(s["A"], s["B"], s["sa"], s["sb"], mode, bias=s["b"], activation=act[s["act"]],
                                      residual=s["r"], out_dtype=out, return_preact=s["preact"])
        return {"out": r[0], "preact": r[1]} if s["preact"] else {"out": r}
    if op == "act_grad":
        dz, dbias = fm.fp8_act_grad(s["dy"], s["z"], act[s["act"]], return_dz=s["dz"], return_dbias=s["dbias"])
        return {k: v for k, v in (("dbias", dbias), ("dz", dz)) if v is not None}
    if op == "norm":
        r = fm.fp8_layer_norm(s["x"], s["gamma"], s["beta"], EPS, y_dtype=DTYPES[s["y"]],
                              q_dtype=DTYPES[s["q"]] if s["q"] else None)
        return dict(zip(("y", "mean", "rstd", "q", "scale"), r))
    dx, dgamma, dbeta = fm.fp8_layer_norm_grad(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                               residual_grad=s["res"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------- 64-bit values ---

def _phi64(z):
    """Normal distribution function."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _act64(z, act):
    """(value, slope) of an activation in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "gelu":
        return z * _phi64(z), _phi64(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        c = math.sqrt(8.0 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1.0 - p) * c * (1.0 + 0.134145 * z ** 2)
    p = torch.sigmoid(z)
    return z * p, p + z * p * (1.0 - p)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("mm", "mm_grad"):
            a = s["A"].double()
            b = s["B"].double()
            sa, sb = s["sa"].double(), s["sb"].double()
            if case["rowwise"]:
                acc = torch.mm(a * sa.unsqueeze(1), b * sb.unsqueeze(0))
            else:
                acc = torch.mm(a * sa, b * sb)
            del a, b
            if op == "mm_grad":
                return {"dz": acc.mul_(_act64(s["z"].double(), case["act"])[1])}
            if s["b"] is not None:
                acc += s["b"].double()
            value = _act64(acc, case["act"])[0]
            if s["r"] is not None:
                value = value + s["r"].double()
            return {"out": value, "preact": acc} if case["preact"] else {"out": value}
        if op == "act_grad":
            dz = s["dy"].double() * _act64(s["z"].double(), case["act"])[1]
            r = {"dbias": dz.sum(dim=0)} if case["dbias"] else {}
            if case["dz"]:
                r["dz"] = dz
            return r
        x = s["x"].double()
        gamma, beta = s["gamma"].double(), s["beta"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
            y = torch.addcmul(beta, (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), gamma)
            r = {"y": y, "mean": mean, "rstd": rstd}
            if case["q"]:
                scale = y.abs().max(dim=1).values / QMAX[case["q"]]
                r["q"], r["scale"] = y / scale.unsqueeze(1), scale
            return r
        rstd = s["rstd"].double().unsqueeze(1)
        h = (x - s["mean"].double().unsqueeze(1)) * rstd
        dy = s["dy"].double()
        n = x.shape[1]
        wsum = torch.mv(dy, gamma).unsqueeze(1)
        whsum = torch.mv(dy * h, gamma).unsqueeze(1)
        dx = (dy * gamma * n - wsum - h * whsum) * (rstd / n)
        if s["res"] is not None:
            dx = dx + s["res"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, h), "dbeta": dy.sum(dim=0)}
