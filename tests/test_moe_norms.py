"""The norm criterion for the experts' layer (moe_norms.py) on the CPU: arithmetic in fp32 keeps
it, and an output of zeros, inner values in one bfloat16 part, a piece of 128 columns left out
and a scale of the next group all break it."""
import numpy as np
import pytest
import torch

from moe_norms import UNIT, allowed, layer, rho, unpacked
from oracle import gptq_oracle as o

SIZES = [(8, 2048, 1408, 8, 8, 4, 128), (4, 512, 256, 4, 2, 8, 64), (16, 256, 384, 6, 3, 3, 128), (5, 704, 320, 6, 2, 4, 64)]


def experts(rng, E, rows, cols, bits, group):
    codes = o.pack(rng.integers(0, 2 ** bits, size=(E * rows, cols)).astype(np.uint8), bits)
    scales = (rng.random((E * rows, cols // group)) * 0.05 + 0.001).astype(np.float16)
    zeros = rng.integers(0, 2 ** bits, size=scales.shape).astype(np.float16)
    return unpacked(codes, scales, zeros, bits)


@pytest.mark.parametrize("n,d,f,E,k,bits,group", SIZES)
def test_the_criterion_can_fail(n, d, f, E, k, bits, group):
    rng = np.random.default_rng([n, d, f])
    up, down = experts(rng, E, 2 * f, d, bits, group), experts(rng, E, d, f, bits, group)
    c = allowed(d, f, k, rho(*up, bits), rho(*down, bits)) * UNIT
    Wu, Wd = (torch.from_numpy(S * (u - Z)) for S, u, Z in (up, down))
    x = (torch.from_numpy(rng.standard_normal((n, d))) * 0.1).to(torch.bfloat16)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(n)]))
    w = torch.softmax(torch.from_numpy(rng.standard_normal((n, k))), 1).float()
    ref = layer(x, ids, w, Wu.view(E, 2 * f, d), Wd.view(E, d, f))

    def off(y):
        return float((y - ref).norm() / ref.norm())

    def fp32(part=lambda h: h, Wu=Wu, Wd=Wd):
        """The layer in 32 bits, the inner values passed through ``part``."""
        y = torch.zeros(n, d)
        for t in range(n):
            for j in range(k):
                e = int(ids[t, j])
                gu = Wu[2 * f * e:2 * f * (e + 1)].float() @ x[t].float()
                h = part(gu[:f] / (1 + torch.exp(-gu[:f])) * gu[f:] * w[t, j])
                y[t] += Wd[d * e:d * (e + 1)].float() @ h
        return y.double()

    assert off(fp32()) <= c < 2.0 ** -13
    assert off(torch.zeros_like(ref)) > c
    assert off(fp32(lambda h: h.bfloat16().float())) > 4 * c
    for W in ("Wu", "Wd"):
        S, u, Z = up if W == "Wu" else down
        less = S * (u - Z)
        less[:, :128] = 0
        assert off(fp32(**{W: torch.from_numpy(less)})) > 4 * c
        moved = np.roll(S, group, axis=1) * (u - Z)
        assert off(fp32(**{W: torch.from_numpy(moved)})) > 4 * c
