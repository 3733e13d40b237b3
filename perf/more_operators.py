"""Measured cases of the end of a training step on FP8 products: softmax cross
entropy over a large vocabulary fused with the product that makes its logits,
its gradient, and the AdamW update of many tensors with states in 32 bits or
in 8.

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
IGNORE = -100
BLOCK = 256                     # elements of an 8-bit state that share a scale
TINIEST = 2.0 ** -9             # e4m3's smallest positive value
HYPER = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token scored against a vocabulary, as while sampling or ranking: latency counts
        dict(name="loss one token", op="loss", M=1, N=32000, K=4096, rowwise=True, a="e4m3", bias=False),
        # a short document of odd sizes, one scale per tensor, a bias that rules out the padding of the vocabulary
        dict(name="loss ragged", op="loss", M=300, N=50257, K=4112, rowwise=False, a="e4m3", bias=True),
        # a long batch of a narrow model: the sum over the vocabulary weighs more than the product
        dict(name="loss shallow", op="loss", M=16384, N=8192, K=512, rowwise=True, a="e4m3", bias=False),
        # a training batch against a large vocabulary: the largest case
        dict(name="loss train", op="loss", M=8192, N=131072, K=4096, rowwise=True, a="e4m3", bias=False),
        # the gradients of a small fine-tuning batch
        dict(name="loss grad small", op="loss_grad", M=128, N=32000, K=1024, rowwise=True, a="e4m3", bias=False,
             out="bf16"),
        # of a short document of odd sizes, with the bias's
        dict(name="loss grad ragged", op="loss_grad", M=300, N=50257, K=4112, rowwise=False, a="e4m3", bias=True,
             out="fp16"),
        # of a training batch
        dict(name="loss grad train", op="loss_grad", M=4096, N=131072, K=4096, rowwise=True, a="e4m3", bias=False,
             out="bf16"),
        # the parameters of one small MLP block, everything in 32 bits: latency counts
        dict(name="adamw one block", op="adamw", width=512, hidden=2048, layers=1, param="fp32", grad="fp32",
             master=False, bits=32, clip=False),
        # many small tensors of odd sizes, states in 8 bits
        dict(name="adamw ragged", op="adamw", width=333, hidden=1111, layers=8, param="bf16", grad="bf16",
             master=True, bits=8, clip=True),
        # a model's MLP blocks with states in 8 bits, bf16 weights beside their 32-bit originals
        dict(name="adamw train 8 bits", op="adamw", width=4096, hidden=14336, layers=4, param="bf16", grad="bf16",
             master=True, bits=8, clip=True),
        # and with states in 32 bits
        dict(name="adamw train 32 bits", op="adamw", width=4096, hidden=16384, layers=2, param="fp32", grad="fp32",
             master=False, bits=32, clip=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 64, the others as they come."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["loss", "loss_grad", "adamw"])
    if op == "adamw":
        width = _width(rng, 16, 6144)
        hidden = _width(rng, width, min(16384, 4 * width))
        layers = min(_log_int(rng, 1, 24), max(1, 4 * 4096 * 14336 // (width * hidden)))
        param = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, width=width, hidden=hidden, layers=layers, param=param, grad=rng.choice([param, "fp32"]),
                    master=param != "fp32" and rng.random() < 0.75, bits=rng.choice([8, 32]), clip=rng.random() < 0.5)
    n = _width(rng, 128, 131072)
    k = 16 * _log_int(rng, 2, 448)
    most = (8192 if op == "loss" else 4096) * 131072
    m = min(_log_int(rng, 1, 16384), most // n, max(1, most * 4096 // (n * k)))
    c = dict(op=op, M=m, N=n, K=k, rowwise=rng.random() < 0.5, a=rng.choice(["e4m3", "e4m3", "e5m2"]),
             bias=rng.random() < 0.5)
    if op == "loss_grad":
        c.update(out=rng.choice(["bf16", "bf16", "fp16"]))
    return c


def _shapes(case):
    """The parameters of `layers` MLP blocks: two weights, two biases, norm weight and bias."""
    w, h = case["width"], case["hidden"]
    return [(h, w), (h,), (w, h), (w,), (w,), (w,)] * case["layers"]


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        state = 4 * (4 if case["bits"] == 32 else 1 + 4 / BLOCK)                    # two states, read and written
        master = 8 if case["master"] else BYTES[case["param"]]                       # (and read what is updated)
        return {"bytes": n * (BYTES[case["grad"]] + BYTES[case["param"]] + master + state), "flops": 16.0 * n}
    m, n, k = case["M"], case["N"], case["K"]
    nbytes = m * k + n * k + 4 * ((m + n) if case["rowwise"] else 2) + 16 * m + 4 * n * case["bias"]
    if case["op"] == "loss":
        return {"bytes": nbytes, "flops": 2.0 * m * n * k}
    nbytes += (m + n) * k * BYTES[case["out"]] + 4 * n * case["bias"]
    return {"bytes": nbytes, "flops": 6.0 * m * n * k}


# ----------------------------------------------------------------- inputs ---

def _quantise(x, q, rowwise):
    """fp32 x [R, C] to fp8 codes and scales (amax / qmax), as the operands of a scaled product are made."""
    amax = x.abs().amax(dim=1, keepdim=True) if rowwise else x.abs().amax().reshape(1, 1)
    s = (amax / QMAX[q]).clamp_min(1e-30)
    return (x / s).clamp_(-QMAX[q], QMAX[q]).to(DTYPES[q]), s.reshape(-1).contiguous()


def _blocks(x):
    """x's elements in rows of BLOCK, the last one filled up with zeros."""
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).reshape(-1, BLOCK)


def _codes(x, scale, shape):
    """Rows of BLOCK as e4m3 codes of x / scale."""
    q = torch.where(scale[:, None] == 0, 0.0, (x / scale[:, None]).clamp(-448.0, 448.0))
    return q.reshape(-1)[:math.prod(shape)].reshape(shape).to(torch.float8_e4m3fn)


def _store(s, name, shapes, sizes, dtype, wanted, align=BLOCK):
    """s[name]: tensors of `shapes` in one buffer, each at a multiple of `align` elements; the buffer in s["all"]."""
    if not wanted:
        s[name] = []
        return
    room = [-(-n // align) * align for n in sizes]
    flat = torch.zeros(sum(room), dtype=dtype, device="cuda")
    s.setdefault("all", {})[name] = flat
    s[name] = [t[:n].view(shape) for t, n, shape in zip(flat.split(room), sizes, shapes)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale)

    s = dict(case)
    if case["op"] == "adamw":
        shapes, eight = _shapes(case), case["bits"] == 8
        sizes = [math.prod(x) for x in shapes]
        code = torch.float8_e4m3fn if eight else torch.float32
        for name, dtype, wanted in (("p", DTYPES[case["param"]], True), ("g", DTYPES[case["grad"]], True),
                                    ("master_w", torch.float32, case["master"]), ("m", code, True), ("v", code, True)):
            _store(s, name, shapes, sizes, dtype, wanted)
        for name in ("ms", "vs"):
            blocks = [-(-n // BLOCK) for n in sizes]
            _store(s, name, [(n,) for n in blocks], blocks, torch.float32, eight, align=1)
        for i, shape in enumerate(shapes):
            w = randn(*shape, scale=0.02)
            # gradients of rows of different size
            grad = randn(*shape).mul_(torch.exp(randn(shape[0], *([1] * (len(shape) - 1)))).mul_(1e-3))
            m = grad * 0.3 + randn(*shape, scale=3e-4)
            v = (grad.square() * 0.5).add_(randn(*shape, scale=7e-4).square_())
            s["p"][i].copy_(w)
            s["g"][i].copy_(grad)
            if case["master"]:
                s["master_w"][i].copy_(w)
            if not eight:
                s["m"][i].copy_(m)
                s["v"][i].copy_(v)
                continue
            for name, x in (("m", _blocks(m)), ("v", _blocks(v).sqrt())):
                s[name + "s"][i].copy_(x.abs().amax(dim=1) / 448.0)
                s[name][i].copy_(_codes(x, s[name + "s"][i], shape))
        s["step"] = 1000
        s["clip_by"] = torch.full((1,), 0.75, device="cuda") if case["clip"] else None
        return s
    m, n, k = case["M"], case["N"], case["K"]
    # a few rows are padding, which has no target
    target = torch.randint(0, n, (m,), generator=g, device="cuda")
    ignored = torch.rand(m, generator=g, device="cuda") < 0.05
    ignored[0] = False
    # logits of standard deviation 2; the hidden rows lean towards their target's weights
    w = randn(n, k, scale=2.0 / math.sqrt(k))
    h = randn(m, k).add_(w[target], alpha=1.5)
    s["A"], s["sa"] = _quantise(h, case["a"], case["rowwise"])
    wq, s["sb"] = _quantise(w, "e4m3", case["rowwise"])
    del w, h
    s["B"] = wq.t()                             # [K, N], column-major
    s["target"] = torch.where(ignored, IGNORE, target)
    s["b"] = None
    if case["bias"]:
        s["b"] = randn(n, scale=0.3)
        s["b"][torch.rand(n, generator=g, device="cuda") < 0.01] = float("-inf")
        s["b"][target] = 0.1                    # (no target is ruled out)
    if case["op"] == "loss_grad":
        z = _logits(s)
        s["lse"] = torch.logsumexp(z, dim=1)
        s["dloss"] = torch.rand(m, generator=g, device="cuda").add_(0.5).div_(m)
    return s


# ------------------------------------------------------------- plain form ---

def _logits(s):
    z = s["A"].float() @ s["B"].float()
    z = z * (s["sa"][:, None] * s["sb"][None, :]) if s["rowwise"] else z * (s["sa"] * s["sb"])
    return z if s["b"] is None else z + s["b"]


def _plain_loss(s):
    z = _logits(s)
    top = z.amax(dim=1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    live = s["target"] != IGNORE
    at = z.gather(1, torch.where(live, s["target"], 0)[:, None])[:, 0]
    return {"loss": torch.where(live, lse - at, 0.0), "lse": lse}


def _plain_grad(s):
    live = s["target"] != IGNORE
    dz = torch.exp(_logits(s) - s["lse"][:, None])
    dz[torch.arange(s["M"], device=dz.device), torch.where(live, s["target"], 0)] -= 1.0
    dz = dz * torch.where(live, s["dloss"], 0.0)[:, None]
    w = s["B"].t().float() * (s["sb"][:, None] if s["rowwise"] else s["sb"])
    h = s["A"].float() * (s["sa"][:, None] if s["rowwise"] else s["sa"])
    out = DTYPES[s["out"]]
    r = {"da": (dz @ w).to(out), "db": (dz.t() @ h).to(out)}
    if s["b"] is not None:
        r["dbias"] = dz.sum(dim=0)
    return r


def _plain_update(s, i):
    """One tensor's step, in place."""
    h = HYPER
    step_size = h["lr"] / (1.0 - h["beta1"] ** s["step"])
    root = 1.0 / math.sqrt(1.0 - h["beta2"] ** s["step"])
    p, shape = s["p"][i], s["p"][i].shape
    w = s["master_w"][i] if s["master"] else p.float()
    g = s["g"][i].float()
    if s["clip"]:
        g = g * s["clip_by"]
    if s["bits"] == 8:
        n = p.numel()
        m = (_blocks(s["m"][i].float()) * s["ms"][i][:, None]).reshape(-1)[:n].reshape(shape)
        v = (_blocks(s["v"][i].float()) * s["vs"][i][:, None]).reshape(-1)[:n].reshape(shape)
        v = v * v
    else:
        m, v = s["m"][i], s["v"][i]
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
    r = torch.sqrt(v)
    w = w * (1.0 - h["lr"] * h["weight_decay"]) - (m / (r * root + h["eps"])) * step_size
    p.copy_(w)
    if s["master"]:
        s["master_w"][i].copy_(w)
    if s["bits"] == 32:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
        return
    most = torch.full((1,), 448.0, device=p.device)
    m, r = _blocks(m), _blocks(r)
    s["ms"][i].copy_(m.abs().amax(dim=1) / most)
    s["vs"][i].copy_(r.amax(dim=1) / most)
    s["m"][i].copy_(_codes(m, s["ms"][i], shape))
    # the second moment's root is rounded up or down by chance, as far as it lies between two codes: a step changes it by
    # less than half of their distance, so that the nearest one would always be the one before. What is not zero does
    # not become zero: it divides
    q = (r / s["vs"][i][:, None]).clamp(max=448.0)
    q = torch.where(s["vs"][i][:, None] == 0, 0.0, q)
    u = _dither(p.numel(), s["step"], p.device)
    up = ((q.view(torch.int32) + u) & -(1 << 20)).view(torch.float32)
    low = torch.floor(q * 512.0 + u.float() * 2.0 ** -20) * TINIEST         # where codes are 2^-9 apart
    q = torch.where(q < 2.0 ** -6, torch.where(q > 0, low.clamp_min(TINIEST), q), torch.where(q == q, up, q))
    s["v"][i].copy_(q.reshape(-1)[:p.numel()].reshape(shape).to(torch.float8_e4m3fn))


def _dither(n, step, device):
    """20 bits for each of n elements (in rows of BLOCK), a hash of its place and of the step."""
    x = (torch.arange(-(-n // BLOCK) * BLOCK, device=device) * 0x9E3779B1 + step * 0x85EBCA77) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x2C1B3C6D) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0x297A2D39) & 0xFFFFFFFF
    return ((x ^ (x >> 16)) >> 12).to(torch.int32).reshape(-1, BLOCK)


def _plain(s):
    if s["op"] == "loss":
        return _plain_loss(s)
    if s["op"] == "loss_grad":
        return _plain_grad(s)
    [_plain_update(s, i) for i in range(len(s["p"]))]
    return _updated(s)


def _updated(s):
    """What a step writes, the buffers of each kind."""
    return {name: flat for name, flat in s["all"].items() if name != "g"}


# -------------------------------------------------------- the entry points ---

def _own(s):
    import fp8_scaled_gemm_gb300 as fm
    if s["op"] == "adamw":
        fm.fp8_adamw(s["p"], s["g"], s["m"], s["v"], s["step"], masters=s["master_w"] or None,
                     exp_avg_scales=s["ms"] or None, exp_avg_sq_scales=s["vs"] or None, grad_scale=s["clip_by"],
                     **HYPER)
        return _updated(s)
    mode = fm.SCALE_ROWWISE if s["rowwise"] else fm.SCALE_TENSOR
    if s["op"] == "loss":
        loss, lse = fm.fp8_cross_entropy(s["A"], s["B"], s["sa"], s["sb"], mode, s["target"], bias=s["b"],
                                         ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    da, db, dbias = fm.fp8_cross_entropy_grad(s["A"], s["B"], s["sa"], s["sb"], mode, s["target"], s["lse"],
                                              s["dloss"], bias=s["b"], ignore_index=IGNORE,
                                              out_dtype=DTYPES[s["out"]], return_dbias=s["b"] is not None)
    return {"da": da, "db": db} if dbias is None else {"da": da, "db": db, "dbias": dbias}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------- 64-bit values ---

def _exact_update(s):
    """The step on the whole buffers (what lies between the tensors is zero and stays so), in 64 bits."""
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], s["step"]
    buf = s["all"]
    w = (buf["master_w"] if s["master"] else buf["p"]).double()
    grad = buf["g"].double()
    if s["clip_by"] is not None:
        grad = grad * s["clip_by"].double()
    moments = {}
    for name in ("m", "v"):
        x = buf[name].double()
        if s["bits"] == 8:
            # every tensor starts at a block, so the buffer's blocks are the tensors'
            x = (x.reshape(-1, BLOCK) * buf[name + "s"].double().unsqueeze(1)).reshape(-1)
        moments[name] = x
    m = torch.lerp(grad, moments["m"], b1)
    old = moments["v"] ** 2 if s["bits"] == 8 else moments["v"]
    v = torch.lerp(grad ** 2, old, b2)
    mhat, vhat = m / (1.0 - b1 ** t), v / (1.0 - b2 ** t)
    w = w - HYPER["lr"] * (HYPER["weight_decay"] * w + mhat / (vhat ** 0.5 + HYPER["eps"]))
    r = {"p": w, "m": m, "v": v}
    if s["master"]:
        r["master_w"] = w
    if s["bits"] == 8:
        for name, x in (("m", m), ("v", v ** 0.5)):
            x = x.reshape(-1, BLOCK)
            scale = x.abs().max(dim=1).values / 448.0
            x = x / scale.unsqueeze(1)
            r[name] = (torch.where(x > 0, x.clamp_min(TINIEST), x) if name == "v" else x).nan_to_num(0.0).reshape(-1)
            r[name + "s"] = scale
    return r


def exact(case, seed):
    if case["op"] == "loss_grad" and 6.0 * case["M"] * case["N"] * case["K"] > 1.4e13:
        return None
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "adamw":
            return _exact_update(s)
        a = s["A"].double() * (s["sa"].double().unsqueeze(1) if case["rowwise"] else s["sa"].double())
        b = s["B"].double() * (s["sb"].double().unsqueeze(0) if case["rowwise"] else s["sb"].double())
        z = torch.mm(a, b)
        if s["b"] is not None:
            z += s["b"].double()
        index = s["target"].clamp_min(0).unsqueeze(1)
        live = (s["target"] >= 0).double()
        if case["op"] == "loss":
            lse = torch.logsumexp(z, dim=1)
            return {"loss": (lse - torch.take_along_dim(z, index, dim=1).squeeze(1)) * live, "lse": lse}
        dz = z.sub_(s["lse"].double().unsqueeze(1)).exp_()
        dz.scatter_add_(1, index, torch.full_like(index, -1.0, dtype=torch.float64))
        dz.mul_((s["dloss"].double() * live).unsqueeze(1))
        r = {"da": torch.mm(dz, b.t()), "db": torch.mm(dz.t(), a)}
        if s["b"] is not None:
            r["dbias"] = dz.sum(dim=0)
        return r
