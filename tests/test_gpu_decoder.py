"""The decoder of Gaussian parameters: its gradients against differentiation in float64, and a few training
steps that lower the rendering loss (needs an MI355X)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from differentiable_raster_amd import decoder, gsmi, pipeline, scenes
    gsmi.load()
    return torch, decoder, pipeline, scenes


@pytest.mark.parametrize("n,width,hidden,blocks", [(500, 32, 48, 1), (4200, 64, 128, 2), (777, 40, 33, 0)])
def test_gradients(env, n, width, hidden, blocks):
    torch, decoder, pipeline, scenes = env
    sc = scenes.random_scene(n, 64, 48, seed=3, sh_degree=1)
    dec = decoder.GaussianDecoder(pipeline.Renderer(sc, sc.settings()), width=width, hidden=hidden, blocks=blocks)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dec.masters[-2].copy_(torch.randn(dec.channels, width, generator=g, device="cuda") * 0.2)
    out = dec.forward().clone()
    dec.dparams.copy_(torch.randn(dec.channels, n, generator=g, device="cuda"))
    dec.backward()

    # the same network in float64, from the operands as they were rounded
    f = dec.features16.double().requires_grad_()
    ws = [w.double().requires_grad_() for w in dec.operands]
    norm = lambda s, w: s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    s = f
    for k in range(blocks):
        w_norm, w_in, b_in, w_down = ws[4 * k:4 * k + 4]
        z = norm(s, w_norm) @ w_in.t() + b_in
        h = torch.nn.functional.silu(z[:, :hidden]) * z[:, hidden:]
        s = s + h @ w_down.t()
    want = dec.base.double() + (norm(s, ws[-3]) @ ws[-2].t() + ws[-1]).t()
    grads = torch.autograd.grad(want, [f] + ws, dec.dparams.double())
    # each operator rounds its result once (2^-8 relative); a value passes 3 blocks + 2 of them on the way
    # forward and as many on the way back, and a sum of terms of both signs may double their weight
    tol = 2 * 2 * (3 * blocks + 2) * 2.0 ** -8
    rel = lambda a, b: float((a.double() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    assert rel(out - dec.base, want - dec.base.double()) <= tol
    for k, (got, ref) in enumerate(zip([dec.dfeatures] + dec.grads, grads)):
        assert rel(got, ref) <= tol, k


def test_training_lowers_the_loss(env):
    torch, decoder, pipeline, _ = env
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import neural_gaussians
    sc = neural_gaussians.disturbed_scene(3000, 128, 96)
    r = pipeline.Renderer(sc, sc.settings())
    # with the head at zero the decoder renders the base parameters
    r.project()
    r.bin()
    r.fused(image=False, loss_sum=True)
    before = float(r.loss_sum)
    dec = decoder.GaussianDecoder(r, width=32, hidden=64, blocks=1)
    first = float(dec.step())
    assert abs(first - before) <= 1e-3 * before
    for _ in range(60):
        last = dec.step()
    assert float(last) < 0.8 * first
