"""How far, in the 2-norm, an experts' layer in fp32 may be from its definition.

The elementwise bounds of the parity tests add up worst cases and are as large as the values
at real widths.  In the norm, over many outputs of random data, a partial sum is no larger
than the whole, so with every rounding at one unit, 2^-23, and all of them in one direction:

 * gate and up: a term passes at most r(d) roundings: 4 products of 32 columns per piece of
   128, 2 to scale it and take its zero's rest off, one per piece of the wave's eighth of the
   row, and the 8 waves' sums.  What is added up is u x and z x in place of (u - z) x (the
   whole part zc of z enters the operand for 8-bit codes): larger by rho = (|S (u - zc)| + |S
   (z - zc)|) / |S (u - z)|.  So g and u are off by r(d) rho units.
 * h = silu(g) u w: |silu'| <= 1.1 and |silu(g)| is at least half of |g| in the norm, so 3.2
   times that, and 16 units for its own operations.
 * y: r(f) rho + the sum over the choices, k, + 2 for the parts' sums."""
import numpy as np
import torch

from oracle import gptq_oracle as o

UNIT = 2.0 ** -23


def unpacked(codes, scales, zeros, bits):
    """S, u, z of every weight in 64 bits."""
    u = o.unpack(codes, bits).astype(np.float64)
    S, Z = (np.repeat(a.astype(np.float64), u.shape[1] // a.shape[1], axis=1) for a in (scales, zeros))
    return S, u, Z


def rho(S, u, Z, bits):
    zc = np.clip(np.rint(Z), -1, 255) if bits == 8 else 0.0
    return (np.linalg.norm(S * (u - zc)) + np.linalg.norm(S * (Z - zc))) / np.linalg.norm(S * (u - Z))


def roundings(d):
    return 4 + 2 + -(-d // 1024) + 8


def allowed(d, f, k, rho_up, rho_down):
    """|y - ref| / |ref| of an fp32 y, in units."""
    return 3.2 * roundings(d) * rho_up + 16 + roundings(f) * rho_down + k + 2


def layer(x, ids, w, up, down):
    """y = sum_j w_j D_j (silu(G_j x) u_j) in 64 bits; up[e] = 2 f x d, down[e] = d x f."""
    y = torch.zeros(x.shape[0], x.shape[1], dtype=torch.float64)
    for e in sorted(set(ids.reshape(-1).tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t].double() @ up[e].t()
        f = gu.shape[1] // 2
        h = gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:] * w[t, j].double()[:, None]
        y.index_add_(0, t, h @ down[e].t())
    return y
