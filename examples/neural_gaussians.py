"""Train a decoder of Gaussian parameters on a small synthetic scene:

    python examples/neural_gaussians.py [--gaussians N] [--steps K]

A scene's images are the target; the decoder starts from the same Gaussians with their colours, sizes and
opacities disturbed and learns features and weights that undo it.  Prints the loss as it falls.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_raster_amd import decoder, pipeline, scenes  # noqa: E402


def disturbed_scene(n: int, width: int, height: int, views: int = 2, seed: int = 7):
    """A scene whose target images show its Gaussians as they were before the disturbance."""
    sc = scenes.random_scene(n, width, height, seed=seed, views=views, sh_degree=1)
    r = pipeline.Renderer(sc, sc.settings())
    r.project()
    r.bin()
    r.forward()
    torch.cuda.synchronize()
    sc.target = r.images_host()[0]
    rng = np.random.default_rng(seed)
    sc.sh = (sc.sh + 0.3 * rng.standard_normal(sc.sh.shape)).astype(np.float32)
    sc.opacity_logits = (sc.opacity_logits + rng.standard_normal(sc.opacity_logits.shape)).astype(np.float32)
    sc.log_scales = (sc.log_scales + 0.3 * rng.standard_normal(sc.log_scales.shape)).astype(np.float32)
    return sc


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gaussians", type=int, default=20_000)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    sc = disturbed_scene(a.gaussians, 320, 240)
    dec = decoder.GaussianDecoder(pipeline.Renderer(sc, sc.settings()), width=64, hidden=128, blocks=2)
    pixels = sc.target.size
    for k in range(a.steps):
        loss = dec.step()
        if k % 20 == 0 or k + 1 == a.steps:
            print(f"step {k:4d}  mean absolute error {float(loss) / pixels:.5f}", flush=True)


if __name__ == "__main__":
    main()
