"""The neural decoder's operators on the GPU against their definitions in float64 (needs an MI355X).

Every bound is a sum of rounding errors, with u the unit roundoff of the type an element is rounded to
(2^-8 bfloat16, 2^-11 half, 2^-24 float32, 2^-4 for the 8-bit float):
  a product's float32 sum of K exact terms: (K + 8) 2^-23 sum |a||b| (the matrix unit may truncate);
  an activation: its slope (at most 1.13) times the error of z, plus 4e-6 (1 + |z|) for the exponential
  or error function; its derivative: 0.8 times the error of z plus the same;
  a gradient product: the error of its rounded operand dz through |weight| or |x|, plus its own sum.
"""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from differentiable_raster_amd import gsmi, neural
    gsmi.load()
    return torch, gsmi, neural


def dt(torch, name):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38, "e4m3": 2.0 ** -10}


def gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, std=1.0: torch.randn(*shape, generator=g, device="cuda") * std


def within(torch, got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    bad = ~(over <= 0)
    assert not bool(bad.any()), (what, int(bad.sum()), float(over[bad].max()), [int(v) for v in bad.nonzero()[0]])


def act64(torch, z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0 * z), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def strided(torch, t, pad):
    """The same values as a view with `pad` more elements per row, which hold NaN."""
    if pad == 0:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=t.device).to(t.dtype)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


# ---- norm -----------------------------------------------------------------------------------------
NORM = [(1, 1, "f32", 0), (3, 7, "bf16", 0), (257, 64, "bf16", 0), (65, 100, "f16", 4), (33, 128, "f32", 8), (1000, 256, "f16", 0),
        (130, 513, "bf16", 3), (17, 1024, "bf16", 8), (9, 2048, "f32", 0), (5, 2050, "f16", 0), (300, 4096, "bf16", 0),
        (3, 8192, "f32", 16), (2, 10001, "bf16", 0), (2, 32768, "f16", 0)]


def norm_reference(torch, s, w, eps):
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s * r * w, r


@pytest.mark.parametrize("rows,width,dtype,pad", NORM)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_forward(env, rows, width, dtype, pad, residual):
    torch, gsmi, neural = env
    t = dt(torch, dtype)
    normal = gen(torch, 100 + width)
    x = strided(torch, normal(rows, width).to(t), pad)
    r = strided(torch, normal(rows, width, std=2.0).to(t), 2 * pad) if residual else None
    w = 1 + normal(width, std=0.3)
    eps = 1e-5
    s64 = x.double() + (r.double() if residual else 0)
    y64, rstd = norm_reference(torch, s64, w.double(), eps)
    plan = neural.RmsNorm(rows, width, t, eps=eps)
    s, y = plan.forward(x, w, r)
    u = U[dtype]
    if residual:
        within(torch, s, s64, (u + 2.0 ** -24) * s64.abs() + TINY[dtype], "s")
    else:
        assert s is x
    # the float32 sum's rounding (2^-24 relative, but of a sum whose terms may cancel) moves y with rstd w;
    # mean square, root and products: (width / lanes + 20) roundings at most
    e_s = 2.0 ** -24 * s64.abs()
    within(torch, y, y64, (u + (40 + width / 8) * 2.0 ** -24) * y64.abs() + e_s * rstd * w.abs().double() + TINY[dtype], "y")
    plan8 = neural.RmsNorm(rows, width, t, eps=eps, quantize=True)
    _, q, scale = plan8.forward(x, w, r)
    amax = y64.abs().amax(1)
    tol = (60 + width / 8) * 2.0 ** -24
    within(torch, scale, amax / 448, tol * amax / 448 + 1e-38, "scale")
    step = torch.maximum(y64.abs() * 2.0 ** -4, (amax / 448)[:, None] * 2.0 ** -10)
    within(torch, q.double() * scale.double()[:, None], y64, step * (1 + 1e-3) + tol * y64.abs(), "q")
    assert float(q.double().abs().max()) <= 448


@pytest.mark.parametrize("rows,width,dtype,pad", NORM)
@pytest.mark.parametrize("through", [True, False])
def test_norm_backward(env, rows, width, dtype, pad, through):
    torch, gsmi, neural = env
    t = dt(torch, dtype)
    normal = gen(torch, 200 + width)
    s = strided(torch, normal(rows, width, std=1.5).to(t), pad)
    dy = strided(torch, normal(rows, width).to(t), pad)
    ds = strided(torch, normal(rows, width).to(t), 3 * pad) if through else None
    w = 1 + normal(width, std=0.3)
    eps = 1e-5
    s64, g64, w64 = s.double(), dy.double(), w.double()
    _, rstd = norm_reference(torch, s64, w64, eps)
    n = s64 * rstd
    mean = (g64 * w64 * n).mean(1, keepdim=True)
    dx64 = (ds.double() if through else 0) + rstd * (g64 * w64 - n * mean)
    dw64 = (g64 * n).sum(0)
    plan = neural.RmsNorm(rows, width, t, eps=eps)
    dx, dw = plan.backward(s, w, dy, ds)
    f = (60 + width / 8) * 2.0 ** -24
    mag = rstd * ((g64 * w64).abs() + n.abs() * (g64 * w64 * n).abs().mean(1, keepdim=True)) + (ds.double().abs() if through else 0)
    within(torch, dx, dx64, U[dtype] * dx64.abs() + f * mag + TINY[dtype], "dx")
    within(torch, dw, dw64, (f + (rows + 8) * 2.0 ** -24) * (g64 * n).abs().sum(0), "dweight")
    # against differences of the forward, in float64, along one direction
    v = normal(rows, width).double()
    h = 1e-5
    f64 = lambda z: (norm_reference(torch, z, w64, eps)[0] * g64).sum() + ((ds.double() * z).sum() if through else 0)  # noqa: E731
    diff = float((f64(s64 + h * v) - f64(s64 - h * v)) / (2 * h))
    bound = float(((U[dtype] * dx64.abs() + f * mag + TINY[dtype]) * v.abs()).sum()) + 1e-5 * (1 + float((mag * v.abs()).sum()))
    assert abs(float((dx.double() * v).sum()) - diff) <= bound


def test_norm_rows_past_one_axis(env):
    """More workgroups than one axis of a launch takes: short rows, 64 to a workgroup."""
    torch, gsmi, neural = env
    rows = (1 << 27) + 64 * 5 + 3
    x = torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w = torch.tensor([0.5, 2.0], device="cuda")
    _, y = neural.RmsNorm(rows, 2, torch.bfloat16, eps=1e-5).forward(x, w)
    at = torch.cat([torch.arange(0, 100), torch.arange((1 << 27) - 100, rows)]).cuda()
    y64, _ = norm_reference(torch, x[at].double(), w.double(), 1e-5)
    within(torch, y[at], y64, (2.0 ** -8 + 41 * 2.0 ** -24) * y64.abs() + 1e-38, "y")


def test_norm_special_rows(env):
    """Rows of zeros, a row with a NaN, one with an infinity: only those rows are touched."""
    torch, gsmi, neural = env
    x = gen(torch, 5)(6, 200)
    x[1] = 0
    x[2, 17] = float("nan")
    x[4, 3] = float("inf")
    ref, _ = norm_reference(torch, x.double(), 1.0, 0.0)
    for t in (torch.float32, torch.bfloat16):
        xt = x.to(t)
        s, y = neural.RmsNorm(6, 200, t, eps=1e-6).forward(xt)
        assert bool((y[1] == 0).all()) and bool(y[2].isnan().all()) and bool(y[4, 3].isnan())
        assert bool(y[[0, 3, 5]].isfinite().all())
        _, q, scale = neural.RmsNorm(6, 200, t, eps=1e-6, quantize=True).forward(xt)
        assert float(scale[1]) == 0 and bool((q[1].float() == 0).all())
        assert bool((q[2].float() * scale[2]).isnan().all())
        assert bool((q[[0, 3, 5]].float() * scale[[0, 3, 5], None]).isfinite().all())


def test_norm_in_place_and_quantize(env):
    torch, gsmi, neural = env
    normal = gen(torch, 6)
    x, r = normal(77, 640).to(torch.bfloat16), normal(77, 640).to(torch.bfloat16)
    w = 1 + normal(640, std=0.1)
    s, y = neural.RmsNorm(77, 640, torch.bfloat16).forward(x, w, r)
    x2, r2 = x.clone(), r.clone()
    d = gsmi.gs_norm_desc(77, 640, gsmi.GS_TYPE_BF16, 1e-6, 0, 0, 0, 0)
    gsmi.gs_rmsnorm(d, x2.data_ptr(), r2.data_ptr(), w.data_ptr(), r2.data_ptr(), x2.data_ptr(), None, None)
    assert torch.equal(r2, s) and torch.equal(x2, y)
    q, scale = neural.quantize_rows(x)
    amax = x.float().abs().amax(1)
    assert torch.allclose(scale, amax / 448, rtol=1e-6, atol=0)
    err = (q.float() * scale[:, None] - x.float()).abs()
    assert bool((err <= x.float().abs() * 2.0 ** -4 * 1.001 + scale[:, None] * 2.0 ** -10).all())


# ---- products -------------------------------------------------------------------------------------
def make_product(torch, rows, k, n, dtype, seed, bias, pad=0):
    normal = gen(torch, seed)
    t = dt(torch, dtype)
    x, w = normal(rows, k), normal(n, k, std=1 / math.sqrt(k))
    sx = sw = None
    if dtype == "e4m3":
        sx, sw = x.abs().amax(1) / 448, w.abs().amax(1) / 448
        x, w = (x / sx[:, None]).clamp(-448, 448).to(t), (w / sw[:, None]).clamp(-448, 448).to(t)
        x64, w64 = x.double() * sx.double()[:, None], w.double() * sw.double()[:, None]
    else:
        x, w = x.to(t), w.to(t)
        x64, w64 = x.double(), w.double()
    x, w = strided(torch, x, pad), strided(torch, w, pad)
    b = normal(n, std=0.5) if bias else None
    z = x64 @ w64.t() + (b.double() if bias else 0)
    mag = x64.abs() @ w64.abs().t() + (b.double().abs() if bias else 0)
    return normal, x, w, b, sx, sw, x64, w64, z, (k + 8) * 2.0 ** -23 * mag


LINEAR = [  # rows, in, out, dtype, y, act, bias, residual, channel_major, pad
    (1, 1, 1, "bf16", "bf16", "none", True, True, False, 0),
    (1, 4096, 1000, "bf16", "bf16", "none", True, True, False, 0),
    (3, 77, 130, "f16", "f16", "gelu", True, False, False, 0),
    (2, 4104, 64, "e4m3", "bf16", "none", True, True, False, 0),
    (4, 5000, 600, "f16", "f32", "none", True, True, True, 4),
    (4, 2100, 2100, "bf16", "bf16", "none", False, True, False, 0),
    (16, 640, 96, "f16", "f32", "silu", False, True, False, 8),
    (17, 512, 33, "bf16", "f32", "none", True, True, True, 0),
    (33, 130, 64, "e4m3", "bf16", "relu", True, True, False, 0),
    (64, 320, 200, "e4m3", "f32", "none", False, False, False, 16),
    (65, 64, 59, "bf16", "f32", "none", True, True, True, 0),
    (100, 1, 3, "f16", "f16", "silu", True, True, False, 0),
    (333, 72, 129, "bf16", "bf16", "silu", True, True, False, 0),
    (257, 1000, 300, "f16", "f16", "gelu", True, True, False, 5),
    (1024, 200, 11, "bf16", "f32", "none", True, True, True, 0),
    (4097, 64, 59, "f16", "f32", "none", True, True, True, 0),
    (700, 2000, 513, "bf16", "f32", "relu", False, True, False, 0),
    (300, 8192, 256, "bf16", "bf16", "none", False, True, False, 0),
    (600, 528, 512, "e4m3", "bf16", "none", True, True, False, 0),
    (513, 100, 700, "e4m3", "f16", "silu", False, False, False, 0),
    (2048, 256, 2048, "bf16", "bf16", "gelu", True, False, False, 0),
]


@pytest.mark.parametrize("rows,k,n,dtype,ytype,act,bias,residual,cm,pad", LINEAR)
def test_linear_forward(env, rows, k, n, dtype, ytype, act, bias, residual, cm, pad):
    torch, gsmi, neural = env
    normal, x, w, b, sx, sw, x64, w64, z, e_z = make_product(torch, rows, k, n, dtype, 7 * rows + k, bias, pad)
    v, _ = act64(torch, z, act)
    e_v = e_z if act == "none" else 1.13 * e_z + 4e-6 * (1 + z.abs())
    shape = (n, rows) if cm else (rows, n)
    yt = dt(torch, ytype)
    r = strided(torch, normal(*shape).to(yt), pad) if residual else None
    if cm:
        v, e_v = v.t(), e_v.t()
    want = v + (r.double() if residual else 0)
    bound = e_v + 2.0 ** -23 * (v.abs() + want.abs()) + U[ytype] * (want.abs() + e_v) + TINY[ytype]
    plan = neural.Linear(rows, k, n, dt(torch, dtype), act=act, y_dtype=yt, channel_major=cm)
    y = plan.forward(x, w, b, r, sx, sw)
    within(torch, y, want, bound, "y")
    first = y.clone()
    assert torch.equal(plan.forward(x, w, b, r, sx, sw), first)
    if residual:  # onto the residual itself
        out = r.clone()
        assert torch.equal(plan.forward(x, w, b, out, sx, sw, out=out), first)
    # rows of the result inside a wider array: what lies between them is left alone
    wide = torch.full((shape[0], shape[1] + 3), 7.0, device="cuda").to(yt)
    plan.forward(x, w, b, r, sx, sw, out=wide[:, :shape[1]])
    assert torch.equal(wide[:, :shape[1]], first) and bool((wide[:, shape[1]:] == 7).all())


def dz_bounds(torch, dy, z, e_z, act):
    _, d = act64(torch, z, act)
    dz = dy * d
    if act == "none":
        return dz, 0 * dz
    e = dy.abs() * (0.8 * e_z + 4e-6 * (1 + z.abs())) + 2.0 ** -22 * dz.abs()
    if act == "relu":
        e = torch.where(z.abs() <= e_z, dy.abs(), 0 * e)
    return dz, e


def check_grads(torch, dtype, gtype, x64, w64, dz, e_dz, dx, dw, db):
    r = U[dtype] * (dz.abs() + e_dz) + TINY[dtype] + e_dz  # the rounded operand
    m, n = dz.shape
    want = dz @ w64
    bound = r @ w64.abs() + (n + 8) * 2.0 ** -23 * ((dz.abs() + r) @ w64.abs())
    within(torch, dx, want, bound + U[dtype] * (want.abs() + bound) + TINY[dtype], "dx")
    want = dz.t() @ x64
    bound = r.t() @ x64.abs() + (m + 8) * 2.0 ** -23 * ((dz.abs() + r).t() @ x64.abs())
    within(torch, dw, want, bound + U[gtype] * (want.abs() + bound) + TINY[gtype], "dweight")
    if db is not None:
        within(torch, db, dz.sum(0), e_dz.sum(0) + (m + 8) * 2.0 ** -24 * (dz.abs() + e_dz).sum(0), "dbias")


LINEAR_BWD = [  # rows, in, out, dtype, y, grad, act, bias, channel_major, pad
    (1, 1, 1, "bf16", "bf16", "bf16", "none", True, False, 0),
    (1, 512, 64, "bf16", "bf16", "f32", "silu", True, False, 0),
    (5, 64, 59, "f16", "f32", "f16", "none", True, True, 0),
    (63, 100, 30, "bf16", "bf16", "bf16", "gelu", True, False, 0),
    (200, 256, 128, "bf16", "bf16", "bf16", "none", True, False, 8),
    (333, 77, 59, "f16", "f16", "f32", "relu", True, False, 3),
    (1000, 64, 59, "bf16", "f32", "f32", "none", True, True, 0),
    (2051, 64, 40, "bf16", "f32", "bf16", "silu", True, True, 0),
    (513, 520, 264, "f16", "f16", "f16", "silu", False, False, 0),
    (4099, 32, 300, "bf16", "bf16", "f32", "none", False, False, 0),
    (20000, 48, 24, "f16", "f16", "f16", "gelu", True, False, 0),
    (300, 2048, 777, "bf16", "bf16", "bf16", "none", True, False, 0),
    (67, 4104, 61, "f16", "f16", "f16", "silu", True, False, 0),
    (130, 5000, 64, "bf16", "f32", "f32", "gelu", True, True, 0),
]


@pytest.mark.parametrize("rows,k,n,dtype,ytype,gtype,act,bias,cm,pad", LINEAR_BWD)
def test_linear_backward(env, rows, k, n, dtype, ytype, gtype, act, bias, cm, pad):
    torch, gsmi, neural = env
    normal, x, w, b, _, _, x64, w64, z, e_z = make_product(torch, rows, k, n, dtype, 11 * rows + k, bias, pad)
    dy = strided(torch, normal(*((n, rows) if cm else (rows, n))).to(dt(torch, ytype)), pad)
    dz, e_dz = dz_bounds(torch, dy.double().t() if cm else dy.double(), z, e_z, act)
    plan = neural.Linear(rows, k, n, dt(torch, dtype), act=act, y_dtype=dt(torch, ytype), channel_major=cm,
                         grad_dtype=dt(torch, gtype), backward=True)
    dx, dw, db = plan.backward(x, w, dy, b)
    check_grads(torch, dtype, gtype, x64, w64, dz, e_dz, dx, dw, db)
    again = [g.clone() for g in (dx, dw) + ((db,) if bias else ())]
    for g in plan.backward(x, w, dy, b):
        if g is not None:
            assert torch.equal(g, again.pop(0))
    # against differences of the forward in float64 along one direction of x and of the weight
    vx, vw = normal(rows, k).double(), normal(n, k).double()
    h = 1e-5
    g64 = dy.double().t() if cm else dy.double()
    f = lambda a, c: (act64(torch, a @ c.t() + (b.double() if bias else 0), act)[0] * g64).sum()  # noqa: E731
    for got, diff, size in ((dx, f(x64 + h * vx, w64) - f(x64 - h * vx, w64), (dz.abs() @ w64.abs() * vx.abs()).sum()),
                            (dw, f(x64, w64 + h * vw) - f(x64, w64 - h * vw), (dz.abs().t() @ x64.abs() * vw.abs()).sum())):
        v = vx if got is dx else vw
        # roundings of dz and of the gradient, and relu's kinks inside the step
        assert abs(float((got.double() * v).sum()) - float(diff) / (2 * h)) <= (2.5 * U[dtype] + 1e-3) * float(size) + 1e-3


@pytest.mark.parametrize("rows,act,cm", [(270_011, "none", True), (270_011, "silu", False)])
def test_bias_gradient_of_many_rows(env, rows, act, cm):
    """More strips of rows than one launch adds up, and a map too wide for the one-pass kernel."""
    torch, gsmi, neural = env
    k, n = 136, 24
    normal, x, w, b, _, _, x64, w64, z, e_z = make_product(torch, rows, k, n, "bf16", 5, True)
    dy = normal(*((n, rows) if cm else (rows, n)))
    dz, e_dz = dz_bounds(torch, dy.double().t() if cm else dy.double(), z, e_z, act)
    plan = neural.Linear(rows, k, n, torch.bfloat16, act=act, y_dtype=torch.float32, channel_major=cm,
                         grad_dtype=torch.float32, backward=True)
    check_grads(torch, "bf16", "f32", x64, w64, dz, e_dz, *plan.backward(x, w, dy, b))


GATED = [  # rows, in, hidden, dtype, act, bias, pad
    (1, 1, 1, "bf16", "silu", True, 0),
    (4, 1024, 300, "bf16", "silu", False, 0),
    (3, 4104, 60, "bf16", "silu", True, 0),
    (1, 9000, 77, "f16", "gelu", True, 3),
    (2, 8208, 40, "e4m3", "silu", False, 0),
    (31, 77, 45, "f16", "gelu", True, 0),
    (50, 256, 96, "e4m3", "silu", True, 0),
    (65, 64, 128, "bf16", "silu", True, 0),
    (300, 100, 130, "f16", "relu", True, 5),
    (257, 1000, 333, "bf16", "none", False, 0),
    (1000, 64, 64, "bf16", "silu", True, 8),
    (4000, 256, 512, "f16", "gelu", False, 0),
    (333, 200, 260, "e4m3", "gelu", False, 0),
]


def gated_parts(torch, z, e_z, hidden, act):
    g, u, e_g, e_u = z[:, :hidden], z[:, hidden:], e_z[:, :hidden], e_z[:, hidden:]
    a, d = act64(torch, g, act)
    e_a = e_g if act == "none" else 1.13 * e_g + 4e-6 * (1 + g.abs())
    return g, u, a, d, e_g, e_u, e_a


@pytest.mark.parametrize("rows,k,hidden,dtype,act,bias,pad", GATED)
def test_gated_forward(env, rows, k, hidden, dtype, act, bias, pad):
    torch, gsmi, neural = env
    _, x, w, b, sx, sw, _, _, z, e_z = make_product(torch, rows, k, 2 * hidden, dtype, 13 * rows + k, bias, pad)
    g, u, a, _, _, e_u, e_a = gated_parts(torch, z, e_z, hidden, act)
    want = a * u
    e = e_a * (u.abs() + e_u) + a.abs() * e_u + 2.0 ** -23 * want.abs()
    yname = "bf16" if dtype == "e4m3" else dtype
    plan = neural.GatedUnit(rows, k, hidden, dt(torch, dtype), act=act)
    h = plan.forward(x, w, b, sx, sw)
    within(torch, h, want, e + U[yname] * (want.abs() + e) + TINY[yname], "h")


@pytest.mark.parametrize("rows,k,hidden,dtype,act,bias,pad", [c for c in GATED if c[3] != "e4m3"])
def test_gated_backward(env, rows, k, hidden, dtype, act, bias, pad):
    torch, gsmi, neural = env
    normal, x, w, b, _, _, x64, w64, z, e_z = make_product(torch, rows, k, 2 * hidden, dtype, 17 * rows + k, bias, pad)
    dh = strided(torch, normal(rows, hidden).to(dt(torch, dtype)), pad)
    g, u, a, _, e_g, e_u, e_a = gated_parts(torch, z, e_z, hidden, act)
    d64 = dh.double()
    dgate, e_gate = dz_bounds(torch, d64 * u, g, e_g, act)
    _, d = act64(torch, g, act)
    e_gate = e_gate + d64.abs() * e_u * (d.abs() + 0.8 * e_g + 4e-6 * (1 + g.abs())) + 2.0 ** -22 * dgate.abs()
    dup, e_up = d64 * a, d64.abs() * e_a + 2.0 ** -23 * (d64 * a).abs()
    dz, e_dz = torch.cat([dgate, dup], 1), torch.cat([e_gate, e_up], 1)
    for gtype in (dtype, "f32"):
        plan = neural.GatedUnit(rows, k, hidden, dt(torch, dtype), act=act, grad_dtype=dt(torch, gtype), backward=True)
        dx, dw, db = plan.backward(x, w, dh, b)
        check_grads(torch, dtype, gtype, x64, w64, dz, e_dz, dx, dw, db)
    vx, vw = normal(rows, k).double(), normal(2 * hidden, k).double()
    h = 1e-5

    def f(a64, c64):
        zz = a64 @ c64.t() + (b.double() if bias else 0)
        return (act64(torch, zz[:, :hidden], act)[0] * zz[:, hidden:] * d64).sum()

    for got, v, diff, size in ((dx, vx, f(x64 + h * vx, w64) - f(x64 - h * vx, w64), (dz.abs() @ w64.abs() * vx.abs()).sum()),
                               (dw, vw, f(x64, w64 + h * vw) - f(x64, w64 - h * vw), (dz.abs().t() @ x64.abs() * vw.abs()).sum())):
        assert abs(float((got.double() * v).sum()) - float(diff) / (2 * h)) <= (2.5 * U[dtype] + 1e-3) * float(size) + 1e-3


def test_values_outside_the_numbers(env):
    """A NaN or an infinity in one row of x, or in the padding after it, reaches that row's results alone."""
    torch, gsmi, neural = env
    for rows, k, n in ((8, 100, 50), (200, 100, 50), (300, 64, 256)):
        normal, x, w, b, *_ = make_product(torch, rows, k, n, "bf16", rows, True, 0)
        clean = neural.Linear(rows, k, n, torch.bfloat16, act="silu").forward(x, w, b).clone()
        big = torch.full((rows, k + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
        big[:, :k] = x
        big[3, k - 1] = float("nan")
        big[5, 0] = float("inf")
        y = neural.Linear(rows, k, n, torch.bfloat16, act="silu").forward(big[:, :k], w, b)
        keep = [r for r in range(rows) if r not in (3, 5)]
        assert torch.equal(y[keep], clean[keep]) and bool(y[3].isnan().all())
        assert not bool(y[5].isfinite().any() and y[5].abs().max() < 1e30)


def test_few_rows_equal_many(env):
    """The same rows through the kernel of few rows and through the tiled one."""
    torch, gsmi, neural = env
    normal, x, w, b, _, _, _, _, z, e_z = make_product(torch, 200, 256, 192, "bf16", 3, True)
    many = neural.Linear(200, 256, 192, torch.bfloat16, y_dtype=torch.float32).forward(x, w, b)
    for m in (1, 16, 40, 64):
        few = neural.Linear(m, 256, 192, torch.bfloat16, y_dtype=torch.float32).forward(x[:m], w, b)
        assert bool(((few - many[:m]).abs().double() <= 2 * e_z[:m]).all())


def test_no_rows(env):
    torch, gsmi, neural = env
    bf = torch.bfloat16
    e = lambda *s: torch.empty(*s, dtype=bf, device="cuda")  # noqa: E731
    w, b = torch.randn(24, 16, device="cuda").to(bf), torch.randn(24, device="cuda")
    assert neural.Linear(0, 16, 24, bf).forward(e(0, 16), w, b).shape == (0, 24)
    dx, dw, db = neural.Linear(0, 16, 24, bf, act="gelu", backward=True).backward(e(0, 16), w, e(0, 24), b)
    assert dx.shape == (0, 16) and bool((dw == 0).all()) and bool((db == 0).all())
    dx, dw, db = neural.GatedUnit(0, 16, 12, bf, backward=True).backward(e(0, 16), w, e(0, 12), b)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    nw = torch.ones(16, device="cuda")
    assert neural.RmsNorm(0, 16, bf).forward(e(0, 16), nw, e(0, 16))[1].shape == (0, 16)
    assert bool((neural.RmsNorm(0, 16, bf).backward(e(0, 16), nw, e(0, 16))[1] == 0).all())


def test_other_stream(env):
    """Operands made on one stream and used on another after an event; results read back there."""
    torch, gsmi, neural = env
    side = torch.cuda.Stream()
    x, w = torch.randn(500, 128, device="cuda").to(torch.bfloat16), torch.randn(256, 128, device="cuda").to(torch.bfloat16)
    plan = neural.Linear(500, 128, 256, torch.bfloat16)
    want = plan.forward(x, w).clone()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(want)
    plan.forward(x, w, out=got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_captured(env):
    """One forward and backward captured in a graph: every replay equals the eager results."""
    torch, gsmi, neural = env
    bf = torch.bfloat16
    x, w = torch.randn(300, 72, device="cuda").to(bf), torch.randn(96, 72, device="cuda").to(bf)
    dh = torch.randn(300, 48, device="cuda").to(bf)
    plan = neural.GatedUnit(300, 72, 48, bf, backward=True)
    h = plan.forward(x, w)
    dx, dw, _ = plan.backward(x, w, dh)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.forward(x, w)
        plan.backward(x, w, dh)
    for k in range(4):
        x.copy_(torch.randn(300, 72, device="cuda"))
        g.replay()
        got = [t.clone() for t in (h, dx, dw)]
        torch.cuda.synchronize()
        plan.forward(x, w)
        plan.backward(x, w, dh)
        assert all(torch.equal(a, b) for a, b in zip(got, (h, dx, dw)))


def test_large_offsets(env):
    """Rows whose byte offsets pass 32 bits, in the operand, the result and the summed axis."""
    torch, gsmi, neural = env
    rows = 34_000_000
    x = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    for c in x.chunk(8):
        c.normal_()
    w = (torch.randn(40, 64, device="cuda") / 8).to(torch.bfloat16)
    y = neural.Linear(rows, 64, 40, torch.bfloat16, y_dtype=torch.float32, channel_major=True).forward(x, w)
    at = torch.tensor([0, 1, rows // 2, 33_554_432, 33_554_433, rows - 2, rows - 1], device="cuda")
    want = w.double() @ x[at].double().t()
    within(torch, y[:, at], want, 72 * 2.0 ** -23 * (w.double().abs() @ x[at].double().abs().t()), "y")
    del y
    # a gradient that is zero but for the last rows: they alone make dweight
    dy = torch.zeros(rows, 40, dtype=torch.bfloat16, device="cuda")
    dy[at] = torch.randn(len(at), 40, device="cuda").to(torch.bfloat16)
    plan = neural.Linear(rows, 64, 40, torch.bfloat16, grad_dtype=torch.float32, backward=True)
    dx, dw, _ = plan.backward(x, w, dy)
    dz = dy[at].double()
    within(torch, dw, dz.t() @ x[at].double(), 100 * 2.0 ** -23 * (dz.abs().t() @ x[at].double().abs()), "dweight")
    want = dz @ w.double()
    within(torch, dx[at], want, (2.0 ** -8 + 50 * 2.0 ** -23) * (dz.abs() @ w.double().abs()) + 1e-38, "dx")


NARROW = [  # rows, in, out (hidden), gated, act, y, bias, channel_major
    (4096, 64, 59, False, "none", "f32", True, True),
    (5003, 64, 59, False, "none", "bf16", True, False),
    (4100, 8, 3, False, "silu", "bf16", True, False),
    (9001, 40, 100, False, "gelu", "bf16", True, False),
    (4130, 64, 250, False, "none", "f32", False, True),
    (4130, 56, 256, False, "relu", "bf16", True, False),
    (6007, 120, 60, False, "silu", "f16", False, False),
    (6007, 128, 128, False, "none", "f16", True, False),
    (4097, 72, 17, False, "gelu", "f32", True, True),
    (4099, 64, 128, True, "silu", "bf16", True, False),
    (4099, 64, 100, True, "none", "bf16", False, False),
    (4160, 24, 30, True, "gelu", "f16", True, False),
    (70000, 64, 16, True, "silu", "bf16", True, False),
    (4111, 128, 64, True, "relu", "f16", False, False),
    (4111, 96, 33, True, "silu", "bf16", True, False),
]


@pytest.mark.parametrize("rows,k,n,gated,act,ytype,bias,cm", NARROW)
def test_narrow_backward(env, rows, k, n, gated, act, ytype, bias, cm):
    """Many rows of a narrow map: the backward in one pass over the rows."""
    torch, gsmi, neural = env
    dtype = "f16" if ytype == "f16" else "bf16"
    w_rows = 2 * n if gated else n
    normal, x, w, b, _, _, x64, w64, z, e_z = make_product(torch, rows, k, w_rows, dtype, 19 * rows + k, bias)
    dy = normal(*((n, rows) if cm else (rows, n))).to(dt(torch, ytype))
    d64 = dy.double().t() if cm else dy.double()
    if gated:
        g, u, a, d, e_g, e_u, e_a = gated_parts(torch, z, e_z, n, act)
        dgate, e_gate = dz_bounds(torch, d64 * u, g, e_g, act)
        e_gate = e_gate + d64.abs() * e_u * (d.abs() + 0.8 * e_g + 4e-6 * (1 + g.abs())) + 2.0 ** -22 * dgate.abs()
        dz = torch.cat([dgate, d64 * a], 1)
        e_dz = torch.cat([e_gate, d64.abs() * e_a + 2.0 ** -23 * (d64 * a).abs()], 1)
        make = lambda gt: neural.GatedUnit(rows, k, n, dt(torch, dtype), act=act, grad_dtype=gt, backward=True)  # noqa: E731
    else:
        dz, e_dz = dz_bounds(torch, d64, z, e_z, act)
        make = lambda gt: neural.Linear(rows, k, n, dt(torch, dtype), act=act, y_dtype=dt(torch, ytype), channel_major=cm,  # noqa: E731
                                        grad_dtype=gt, backward=True)
    plan = make(torch.float32)
    dx, dw, db = plan.backward(x, w, dy, b)
    check_grads(torch, dtype, "f32", x64, w64, dz, e_dz, dx, dw, db)
    first = [t.clone() for t in (dx, dw)]
    assert all(torch.equal(p, q) for p, q in zip(first, plan.backward(x, w, dy, b)))
    assert torch.equal(make(dt(torch, dtype)).backward(x, w, dy, b)[1], dw.to(dt(torch, dtype)))
    # views with rows further apart, NaN between them
    xs, ws, dys = strided(torch, x, 8), strided(torch, w, 16), strided(torch, dy, 4)
    assert all(torch.equal(p, q) for p, q in zip(first, plan.backward(xs, ws, dys, b)))


NARROW_FWD = [  # rows, in, out (hidden), gated, act, y, bias, residual, channel_major
    (16384, 64, 59, False, "none", "f32", True, True, True),
    (16389, 63, 59, False, "none", "f32", False, False, True),
    (16385, 53, 48, False, "gelu", "bf16", True, True, False),
    (16411, 8, 3, False, "relu", "f32", True, False, False),
    (20001, 30, 64, False, "silu", "bf16", False, True, False),
    (16390, 64, 17, False, "none", "f16", True, True, False),
    (16391, 127, 64, False, "silu", "f16", True, False, False),
    (16400, 97, 33, False, "none", "f32", True, True, False),
    (70001, 36, 16, True, "gelu", "bf16", True, False, False),
    (16399, 64, 32, True, "silu", "bf16", True, False, False),
    (16399, 115, 27, True, "relu", "f16", False, False, False),
    (16384, 53, 31, True, "none", "f32", True, False, False),
]


@pytest.mark.parametrize("rows,k,n,gated,act,ytype,bias,residual,cm", NARROW_FWD)
def test_narrow_forward(env, rows, k, n, gated, act, ytype, bias, residual, cm):
    """Many rows of a narrow map: the forward straight from memory to fragments."""
    torch, gsmi, neural = env
    dtype = "f16" if ytype == "f16" else "bf16"
    yt = dt(torch, ytype)
    normal, x, w, b, _, _, x64, w64, z, e_z = make_product(torch, rows, k, 2 * n if gated else n, dtype, 23 * rows + k, bias)
    if gated:
        g, u, v, _, _, e_u, e_a = gated_parts(torch, z, e_z, n, act)
        want = v * u
        e = e_a * (u.abs() + e_u) + v.abs() * e_u + 2.0 ** -23 * want.abs()
        bound = e + U[ytype] * (want.abs() + e) + TINY[ytype]
        plan = neural.GatedUnit(rows, k, n, dt(torch, dtype), act=act, y_dtype=yt)
        run = lambda x, w, out=None: plan.forward(x, w, b, out=out)  # noqa: E731
        r = None
    else:
        v, _ = act64(torch, z, act)
        e = e_z if act == "none" else 1.13 * e_z + 4e-6 * (1 + z.abs())
        if cm:
            v, e = v.t(), e.t()
        r = normal(*((n, rows) if cm else (rows, n))).to(yt) if residual else None
        want = v + (r.double() if residual else 0)
        bound = e + 2.0 ** -23 * (v.abs() + want.abs()) + U[ytype] * (want.abs() + e) + TINY[ytype]
        plan = neural.Linear(rows, k, n, dt(torch, dtype), act=act, y_dtype=yt, channel_major=cm)
        run = lambda x, w, out=None: plan.forward(x, w, b, r, out=out)  # noqa: E731
    y = run(x, w).clone()
    within(torch, y, want, bound, "y")
    # views with rows further apart (NaN between them), and a result inside a wider array
    xs, ws = strided(torch, x, 3), strided(torch, w, 5)
    wide = torch.full((y.shape[0], y.shape[1] + 3), 7.0, device="cuda").to(yt)
    run(xs, ws, wide[:, :y.shape[1]])
    assert torch.equal(wide[:, :y.shape[1]], y) and bool((wide[:, y.shape[1]:] == 7).all())
    if residual:
        out = r.clone()
        plan.forward(x, w, b, out, out=out)
        assert torch.equal(out, y)
