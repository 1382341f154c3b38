"""2-norm criteria for the tuning operators' fp32 gradients, which a dropped second part breaks (an
element's worst case grows with the number of summed rows and lets it through at real widths).

A sum of R products: its roundings are at most 2^-23 of the partial sums, of independent signs for
random data, and partial sums are no larger than the whole in the norm; a weight in two parts is
off by 2^-23 of it: 2^-22 sqrt(R + 64) of the result.  A softmax value is off by its logit's error
more: 2^-22 sqrt(d + 64) of logits of at most ``largest``."""
import torch


def sum_criterion(rows):
    return 2.0 ** -22 * (rows + 64) ** 0.5


def softmax_criterion(words, d, largest):
    return sum_criterion(words) + sum_criterion(d) * largest


def one_part(v):
    """v (in 64 bits) as the nearest fp16 number."""
    return v.half().double()


def unit_rows(What, S):
    """What's rows times the power of two with which their largest scale is in 16 .. 32, and that power."""
    p2 = 2.0 ** (torch.floor(torch.log2(S.abs().amax(1, keepdim=True))) - 4)
    return What / p2, p2


def relative(got, want):
    return float((got - want).norm() / want.norm())


def random_layer(rows, cols, bits, group, seed, device="cpu"):
    """u, S and z of a random layer with whole zeros, and What, in 64 bits."""
    gen = torch.Generator().manual_seed(seed)
    u = torch.randint(0, 2 ** bits, (rows, cols), generator=gen).to(device)
    S = (torch.rand(rows, cols // group, generator=gen) * 0.05 + 0.001).half().to(device)
    z = torch.randint(0, 2 ** bits, S.shape, generator=gen).half().to(device)
    s, o = S.double().repeat_interleave(group, 1), z.double().repeat_interleave(group, 1)
    return u, S, z, s * (u.double() - o)


def packed(u, bits):
    """Codes as stored (4 or 8 bits)."""
    return u.to(torch.uint8) if bits == 8 else (u[:, 0::2] | (u[:, 1::2] << 4)).to(torch.uint8)
