"""Timed cases of the neural parameter decoder's operators: the root-mean-square norm with the
residual's addition (and an 8-bit output with scales), the linear map with bias, activation and
residual in its epilogue, and the gated feed-forward unit, forward and backward.

A case names an operator, a direction, sizes and types.  prepare() makes its inputs from a seed,
run() takes one pass through the operator: in elementary float32 torch operations where `own` is
false, through the package's entry points where it is true.  exact() evaluates the definition in
float64, with the gradients from differentiation instead of from the formulas.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one token between two blocks of a decoder that serves: latency alone
        dict(name="norm_token", op="norm", dir="fwd", rows=1, width=1024, dtype="bf16", quantize=False),
        # a batch of features before an 8-bit product: the sum goes on, the normed rows leave in 8 bits
        dict(name="norm_8bit", op="norm", dir="fwd", rows=16384, width=2048, dtype="bf16", quantize=True),
        # the gradient at 100K Gaussians with 256 features each, half precision
        dict(name="norm_bwd", op="norm", dir="bwd", rows=100_000, width=256, dtype="f16", quantize=False),
        # the down projection of a block for one token: every weight is read for one row
        dict(name="linear_token", op="linear", dir="fwd", rows=1, din=4096, dout=1024, dtype="bf16", y="bf16",
             act="none", bias=True, residual=True, channel_major=False),
        # 59 parameter rows (centre, scale, rotation, opacity, degree-3 colour) of 1M Gaussians from 64
        # features each, added to their base values, in the layout that the projection reads
        dict(name="linear_params", op="linear", dir="fwd", rows=1_000_000, din=64, dout=59, dtype="bf16", y="f32",
             act="none", bias=True, residual=True, channel_major=True),
        # its gradient from the projection's backward rows, at a count that no tile divides
        dict(name="linear_params_bwd", op="linear", dir="bwd", rows=300_001, din=64, dout=59, dtype="bf16", y="f32",
             act="none", bias=True, residual=False, channel_major=True),
        # the down projection of a block over a batch of 8192 rows, onto the residual stream
        dict(name="linear_wide", op="linear", dir="fwd", rows=8192, din=4096, dout=1024, dtype="bf16", y="bf16",
             act="none", bias=False, residual=True, channel_major=False),
        # a hidden layer's gradient through its activation, with sizes that no vector width divides
        dict(name="linear_odd_bwd", op="linear", dir="bwd", rows=4099, din=1000, dout=777, dtype="f16", y="f16",
             act="gelu", bias=True, residual=False, channel_major=False),
        # the gated unit of a block on 8-bit rows and weights with a scale each
        dict(name="gated_8bit", op="gated", dir="fwd", rows=8192, din=1024, hidden=4096, dtype="e4m3", act="silu",
             bias=False),
        # the gated unit for four tokens: the weights' bytes are the whole cost
        dict(name="gated_token", op="gated", dir="fwd", rows=4, din=1024, hidden=4096, dtype="bf16", act="silu",
             bias=False),
        # training a narrow decoder on 262144 Gaussians: long and thin, bound by memory
        dict(name="gated_narrow_bwd", op="gated", dir="bwd", rows=262_144, din=64, hidden=128, dtype="bf16",
             act="silu", bias=True),
        # training a wide block: the largest products
        dict(name="gated_wide_bwd", op="gated", dir="bwd", rows=8192, din=2048, hidden=8192, dtype="bf16",
             act="silu", bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: rows from a single token to a million Gaussians, widths from 16 to 8192, half of
    the sizes multiples of 16 and the others as they fall."""
    flops, most = (max(work(c)[k] for c in listed()) for k in ("flops", "bytes"))

    def size(lo, hi):
        n = _log(rng, lo, hi)
        return max(16, n // 16 * 16) if rng.random() < 0.5 else n

    while True:
        op = rng.choice(["norm", "linear", "linear", "gated", "gated"])
        d = rng.choice(["fwd", "bwd"])
        half = rng.choice(["bf16", "bf16", "f16"])
        if op == "norm":
            q = d == "fwd" and rng.random() < 0.4
            c = dict(op=op, dir=d, rows=_log(rng, 1, 300_000), width=size(16, 8192), dtype=half, quantize=q)
            if c["rows"] * c["width"] > 1 << 26:
                continue
            return c
        act = rng.choice(["none", "relu", "silu", "gelu"]) if op == "linear" else rng.choice(["silu", "gelu"])
        rows, din, dout = _log(rng, 1, 1_000_000), size(16, 8192), size(16, 8192)
        bias = rng.random() < 0.5
        if op == "linear":
            cm = rng.random() < 0.25
            dt = "e4m3" if d == "fwd" and not cm and rng.random() < 0.25 else half
            y = "f32" if cm else ("bf16" if dt == "e4m3" else dt)
            if cm:
                dout, act = rng.randint(3, 128), "none"
            c = dict(op=op, dir=d, rows=rows, din=din, dout=dout, dtype=dt, y=y, act=act, bias=bias,
                     residual=d == "fwd" and rng.random() < 0.5, channel_major=cm)
        else:
            dt = "e4m3" if d == "fwd" and rng.random() < 0.25 else half
            c = dict(op=op, dir=d, rows=rows, din=din, hidden=dout, dtype=dt, act=act, bias=bias)
        if d == "bwd" and act == "relu":
            c["bias"] = False  # a sum of steps jumps where rounding moves a value over zero
        w = work(c)
        if w["flops"] > flops or w["bytes"] > most or rows * max(din, 2 * dout) > 1 << 27:
            continue
        return c


def work(case):
    """Each input read once and each output written once; the backward of a map with an activation, and of
    the gated unit, computes its products again from the inputs."""
    es = {"bf16": 2, "f16": 2, "e4m3": 1, "f32": 4}
    m = case["rows"]
    if case["op"] == "norm":
        n, s = m * case["width"], es[case["dtype"]]
        w = case["width"] * 4
        if case["dir"] == "fwd":
            out = n * s + (n + 4 * m if case["quantize"] else n * s)
            return {"bytes": 2 * n * s + w + out, "flops": 6 * n}
        return {"bytes": 4 * n * s + 2 * w, "flops": 10 * n}
    k = case["din"]
    s = es[case["dtype"]]
    if case["op"] == "linear":
        n, t = case["dout"], es[case["y"]]
        scales = 4 * (m + n) if case["dtype"] == "e4m3" else 0
        if case["dir"] == "fwd":
            b = m * k * s + n * k * s + scales + m * n * t * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0)
            return {"bytes": b, "flops": 2 * m * n * k}
        b = 2 * m * k * s + 2 * n * k * s + m * n * t + (8 * n if case["bias"] else 0)
        return {"bytes": b, "flops": (4 if case["act"] == "none" else 6) * m * n * k}
    h = case["hidden"]
    n = 2 * h
    scales = 4 * (m + n) if case["dtype"] == "e4m3" else 0
    t = 2
    if case["dir"] == "fwd":
        return {"bytes": m * k * s + n * k * s + scales + m * h * t + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    return {"bytes": 2 * m * k * s + 2 * n * k * s + m * h * t + (8 * n if case["bias"] else 0), "flops": 6 * m * n * k}


def _rows8(x):
    """Rows in 8 bits with a scale each."""
    scale = x.abs().amax(1) / E4M3_MAX
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    m = case["rows"]
    if case["op"] == "norm":
        d = case["width"]
        t = {"weight": 1.0 + normal(d, std=0.2)}
        # the residual stream grows along a decoder: rows of different size, a few large features
        size = torch.exp(normal(m, 1, std=0.7)) * (1.0 + 4.0 * (torch.arange(d, device="cuda") % 61 == 7))
        if case["dir"] == "fwd":
            t["x"] = normal(m, d).to(dt)
            t["residual"] = (normal(m, d) * size).to(dt)
        else:
            t["s"] = (normal(m, d) * size).to(dt)
            t["dy"] = normal(m, d).to(dt)
            t["ds"] = normal(m, d, std=0.5).to(dt)
        return t
    k = case["din"]
    n = case["dout"] if case["op"] == "linear" else 2 * case["hidden"]
    x, w = normal(m, k), normal(n, k, std=1.0 / math.sqrt(k))
    t = {}
    if case["dtype"] == "e4m3":
        t["x"], t["x_scale"] = _rows8(x)
        t["weight"], t["w_scale"] = _rows8(w)
    else:
        t["x"], t["weight"] = x.to(dt), w.to(dt)
    if case["bias"]:
        t["bias"] = normal(n, std=0.1)
    if case["op"] == "linear":
        yt = DTYPES[case["y"]]
        shape = (n, m) if case["channel_major"] else (m, n)
        if case["dir"] == "bwd":
            t["dy"] = normal(*shape).to(yt)
        elif case["residual"]:
            t["residual"] = normal(*shape).to(yt)
    elif case["dir"] == "bwd":
        t["dh"] = normal(m, case["hidden"]).to(dt)
    return t


def prepare(case, seed):
    state = dict(case=dict(case), **_inputs(case, seed))
    if own:
        from differentiable_raster_amd import neural
        dt = DTYPES[case["dtype"]]
        if case["op"] == "norm":
            state["plan"] = neural.RmsNorm(case["rows"], case["width"], dt, eps=EPS, quantize=case["quantize"])
        elif case["op"] == "linear":
            state["plan"] = neural.Linear(case["rows"], case["din"], case["dout"], dt, act=case["act"],
                                          y_dtype=DTYPES[case["y"]], channel_major=case["channel_major"],
                                          backward=case["dir"] == "bwd")
        else:
            state["plan"] = neural.GatedUnit(case["rows"], case["din"], case["hidden"], dt, act=case["act"],
                                             y_dtype=torch.bfloat16 if case["dtype"] == "e4m3" else dt,
                                             backward=case["dir"] == "bwd")
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c, plan = s["case"], s["plan"]
    get = s.get
    if c["op"] == "norm":
        if c["dir"] == "bwd":
            dx, dw = plan.backward(s["s"], s["weight"], s["dy"], s["ds"])
            return {"dx": dx, "dweight": dw}
        if c["quantize"]:
            total, q, scale = plan.forward(s["x"], s["weight"], s["residual"])
            return {"sum": total, "q": q, "scale": scale}
        total, y = plan.forward(s["x"], s["weight"], s["residual"])
        return {"sum": total, "y": y}
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            return {"y": plan.forward(s["x"], s["weight"], get("bias"), get("residual"), get("x_scale"), get("w_scale"))}
        dx, dw, db = plan.backward(s["x"], s["weight"], s["dy"], get("bias"))
    else:
        if c["dir"] == "fwd":
            return {"h": plan.forward(s["x"], s["weight"], get("bias"), get("x_scale"), get("w_scale"))}
        dx, dw, db = plan.backward(s["x"], s["weight"], s["dh"], get("bias"))
    return {"dx": dx, "dweight": dw, **({"dbias": db} if c["bias"] else {})}


# ---- the plain forms: float32 throughout, rounded once at the end ----
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _dact(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))


def _wide(s):
    x, w = s["x"].float(), s["weight"].float()
    if "x_scale" in s:
        x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
    return x, w


def _run_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        w = s["weight"]
        if c["dir"] == "bwd":
            t, dy = s["s"].float(), s["dy"].float()
            r = 1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
            n, g = t * r, dy * w
            dx = s["ds"].float() + r * (g - n * (g * n).mean(1, keepdim=True))
            return {"dx": dx.to(dt), "dweight": (dy * n).sum(0)}
        t = s["x"].float() + s["residual"].float()
        y = t * (1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)) * w
        if c["quantize"]:
            q, scale = _rows8(y)
            return {"sum": t.to(dt), "q": q, "scale": scale}
        return {"sum": t.to(dt), "y": y.to(dt)}
    x, w = _wide(s)
    z = None
    if c["op"] == "gated" or c["dir"] == "fwd" or c["act"] != "none":
        z = torch.matmul(x, w.t())
        if "bias" in s:
            z = z + s["bias"]
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            y = _act(z, c["act"])
            y = y.t() if c["channel_major"] else y
            if "residual" in s:
                y = y + s["residual"].float()
            return {"y": y.to(DTYPES[c["y"]]).contiguous()}
        dz = s["dy"].float()
        dz = dz.t() if c["channel_major"] else dz
        if c["act"] != "none":
            dz = dz * _dact(z, c["act"])
    else:
        h = c["hidden"]
        gate, up = z[:, :h], z[:, h:]
        if c["dir"] == "fwd":
            return {"h": (_act(gate, c["act"]) * up).to(torch.bfloat16 if c["dtype"] == "e4m3" else dt)}
        dh = s["dh"].float()
        dz = torch.cat([dh * up * _dact(gate, c["act"]), dh * _act(gate, c["act"])], 1)
    out = {"dx": torch.matmul(dz, w).to(dt), "dweight": torch.matmul(dz.t(), x).to(dt)}
    if "bias" in s:
        out["dbias"] = dz.sum(0)
    return out


# ---- the definition in 64 bits ----
def exact(case, seed):
    """The operators written out in float64; gradients by differentiating the forward."""
    if work(case)["flops"] > 6e12:
        return None
    t = {k: v.to(torch.float64) for k, v in _inputs(case, seed).items()}
    f = torch.nn.functional
    acts = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v), "gelu": f.gelu}
    if case["op"] == "norm":
        norm = lambda v, w: v / (v.pow(2).sum(-1, keepdim=True) / case["width"] + EPS).sqrt() * w  # noqa: E731
        if case["dir"] == "fwd":
            total = t["x"] + t["residual"]
            y = norm(total, t["weight"])
            if not case["quantize"]:
                return {"sum": total, "y": y}
            scale = y.abs().max(1).values / E4M3_MAX
            return {"sum": total, "q": y / scale.unsqueeze(1), "scale": scale}
        v, w = t["s"].requires_grad_(), t["weight"].requires_grad_()
        dv, dw = torch.autograd.grad(norm(v, w), (v, w), t["dy"])
        return {"dx": dv + t["ds"], "dweight": dw}
    x, w = t["x"], t["weight"]
    if "x_scale" in t:
        x, w = x * t["x_scale"].unsqueeze(1), w * t["w_scale"].unsqueeze(1)
    bias = t.get("bias")
    wanted = [v.requires_grad_() for v in ([x, w] + ([bias] if bias is not None else []))] if case["dir"] == "bwd" else []

    def forward():
        z = f.linear(x, w, bias)
        if case["op"] == "gated":
            gate, up = z.split(case["hidden"], 1)
            return acts[case["act"]](gate) * up
        y = acts[case["act"]](z)
        return y.transpose(0, 1) if case["channel_major"] else y

    if case["dir"] == "fwd":
        y = forward()
        if case["op"] == "gated":
            return {"h": y}
        return {"y": (y + t["residual"] if "residual" in t else y).contiguous()}
    grads = torch.autograd.grad(forward(), wanted, t["dy"] if case["op"] == "linear" else t["dh"])
    return dict(zip(("dx", "dweight", "dbias"), grads))
