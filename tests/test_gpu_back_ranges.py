"""The gradient through stored layers, and the losses' gradients, at the ends of what scales and
zeros hold.

In the kernel a row's weights are S (u - z) 2^-e with e the largest over its groups of the scale's
exponent, and 2 more where a zero is beyond 32000.  A weight is off by half an fp16 step: 2^-11 of
it in one part; in two 2^-23 (the second part is half a step off what the first leaves, at most
2^-11); and by half a subnormal step, 2^-25 2^e, at least.  The other terms as in tuning_helpers."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import out_rounding, stored, weights
from tuning_helpers import BF, F32, HF, U

pytestmark = pytest.mark.gpu


def with_values(q, S, Z):
    """q with scales and zeros replaced, and its What in 64 bits."""
    q.scales.copy_(S.half())
    q.zeros.copy_(Z.half())
    return torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(), q.bits, q.group_size))


def units(q):
    """2^e of every row."""
    S, Z = q.scales.cpu().double(), q.zeros.cpu().double().abs()
    e = torch.floor(torch.log2(S.abs())) + torch.where(Z <= 32000, 0.0, 2.0)
    return 2.0 ** e.amax(1)


def near(got, ref, bound, t, what):
    err, bound = (got.cpu().double() - ref).abs(), bound * (1 + 2.0 ** -10) + out_rounding(ref, t)
    log(f"  {what}: max |err| / bound = {float((err / bound).max()):.3f}")
    assert got.dtype == t and bool((err <= bound).all())


def gradient(q, What, dy, t):
    """dx and its bound."""
    dy, unit = dy.cpu().double(), units(q)
    rel = 2.0 ** -11 if t == BF else 2.0 ** -23
    bound = ((What.shape[0] + 64) * U + rel) * (dy.abs() @ What.abs()) + 2.0 ** -25 * (dy.abs() @ unit)[:, None]
    bound += 2.0 ** -39 * (dy.abs() * unit).amax(1)[:, None] * (What.abs() / unit[:, None]).sum(0)[None]
    return dy @ What, bound


@pytest.mark.parametrize("bits,group,d_row,d_col", [(4, 32, 130, 256), (8, 0, 333, 200), (3, 64, 97, 128), (8, 128, 64, 384)])
@pytest.mark.parametrize("n", [3, 130, 1100])
@pytest.mark.parametrize("t", [BF, F32])
def test_any_zero(bits, group, d_row, d_col, n, t):
    """Zeros up to fp16's largest, in some groups of a row, in all, in none."""
    import post_weight_quantization_25_amd as g
    q, _ = stored(d_row, d_col, bits, group, 1)
    gen = torch.Generator().manual_seed(2)
    S = torch.rand(q.scales.shape, generator=gen) * 0.05 + 0.001
    Z = torch.randint(0, 2 ** bits, q.zeros.shape, generator=gen).float()
    far = torch.tensor([65504.0, -65504.0, 32000.0, -32000.0, 32016.0, -40000.0, 1025.0, -1024.0])
    Z = torch.where(torch.rand(Z.shape, generator=gen) < 0.3, far[torch.randint(0, 8, Z.shape, generator=gen)], Z)
    Z[: d_row // 3] = torch.randint(0, 2 ** bits, Z[: d_row // 3].shape, generator=gen).float()
    Z[0], Z[1], S[2] = 65504.0, -65504.0, 1.999
    What = with_values(q, S, Z)
    dy = (torch.randn(n, d_row, generator=gen) * 1e-3).to(BF)
    log(f"zeros to 65504: {d_row}x{d_col} bits={bits} g={group} n={n} {t}")
    got = g.linear_grouped_backward(q, dy.cuda(), out_dtype=t)
    ref, bound = gradient(q, What, dy, t)
    near(got, ref, bound, t, "dx")


@pytest.mark.parametrize("n", [5, 150])
@pytest.mark.parametrize("gt", [BF, F32])
def test_any_zero_of_a_head(n, gt):
    """A head with such zeros in every fourth word: finite gradients within 2^-8 of what they add up
    (weights and exponentials to 2^-11 each, a logit of sums of 10^3 to 2^-10)."""
    import post_weight_quantization_25_amd as g
    V, d = 600, 64
    q, _ = stored(V, d, 4, 32, 3)
    gen = torch.Generator().manual_seed(4)
    S = torch.rand(q.scales.shape, generator=gen) * 0.02 + 0.01
    Z = torch.randint(0, 16, q.zeros.shape, generator=gen).float()
    S[::4], Z[::4] = 1.75 * 2.0 ** -16, torch.where(torch.rand(Z[::4].shape, generator=gen) < 0.5, 65504.0, -50000.0)
    What = with_values(q, S, Z)
    x = torch.randn(n, d, generator=gen).to(HF)
    t = torch.randint(0, V, (n,), generator=gen)
    loss, dx = g.cross_entropy(q, x.cuda(), t.int().cuda(), dx_dtype=gt)
    z = x.double() @ What.t()
    p = torch.softmax(z, 1)
    p[torch.arange(n), t] -= 1.0
    ref = p @ What
    assert bool(((dx.cpu().double() - ref).abs() <= 2.0 ** -8 * (p.abs() @ What.abs()) + out_rounding(ref, gt)).all())


@pytest.mark.parametrize("bits,group", [(4, 32), (8, 64), (3, 128)])
@pytest.mark.parametrize("n", [3, 130, 1100])
@pytest.mark.parametrize("t", [BF, F32])
def test_small_scales_beside_large_ones(bits, group, n, t):
    """Columns whose scales are 2^-14 to 2^-18 in rows that have one of 2 to 31 elsewhere.  With zeros
    up to 1024 a row's largest scale enters as 16 to 32, so 2^e is 2^-4 of the scale's power of two:
    the scales keep their bits, and those columns' weights are off by 2^-23 (one part 2^-11) and
    2^-25 2^e."""
    import post_weight_quantization_25_amd as g
    d_row, d_col = 150, 4 * group
    q, _ = stored(d_row, d_col, bits, group, 1, "fraction")
    gen = torch.Generator().manual_seed(3)
    S = (1 + torch.rand(q.scales.shape, generator=gen)) * 2.0 ** torch.randint(-18, -14, q.scales.shape, generator=gen)
    S[:, 1] = 2 + 29 * torch.rand(d_row, generator=gen)
    Z = torch.randint(0, 2 ** bits, q.zeros.shape, generator=gen).float()
    Z[::5] += 0.25                                                   # decoded in another way
    What = with_values(q, S, Z)
    unit = units(q) / 16
    dy = torch.randn(n, d_row, generator=gen).to(HF)
    got = g.linear_grouped_backward(q, dy.cuda(), out_dtype=t)
    a = dy.double().abs()
    ref, rel = dy.double() @ What, 2.0 ** -11 if t == BF else 2.0 ** -23
    bound = ((d_row + 64) * U + rel) * (a @ What.abs()) + 2.0 ** -25 * (a @ unit)[:, None]
    bound += 2.0 ** -39 * (a * unit).amax(1)[:, None] * (What.abs() / unit[:, None]).sum(0)[None]
    near(got, ref, bound, t, "dx")
