"""Products grouped by expert where x has infinities, NaNs and numbers near the type's largest:
the definition's sum of the row, whatever kernel the batch takes.

Elements that are not finite decide their row alone (the others add something finite): an infinity
with the weights' sign, NaN of a zero weight, of both signs or of a NaN.  Finite sums: (d_col + 64)
additions of what the products add up (tuning_helpers)."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import stored
from test_gpu_back_infinities import alike, spoil
from tuning_helpers import BF, F32, HF, U, segments

pytestmark = pytest.mark.gpu
INF = float("inf")


def definition(x, What):
    out = torch.empty(x.shape[0], What.shape[0], dtype=torch.float64)
    for t in range(x.shape[0]):
        at = ~torch.isfinite(x[t])
        out[t] = (What[:, at] * x[t][at].double()[None]).sum(1)
    return out


# (tests/test_tuning_rules.py: 17000 rows take the tiles of 64 tokens up to 96, of 128 beyond)
SIZES = [(300, 3), (17000, 64), (17003, 130), (16999, 300)]


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("cols,bits,group,zeros,dt,yt", [
    (128, 4, 32, "fraction", BF, F32), (136, 3, 0, "fraction", BF, BF), (320, 8, 64, "far", HF, HF), (258, 4, 0, "far", BF, F32),
    (256, 8, 128, "fraction", HF, F32), (128, 4, 128, "whole", HF, BF),
])
def test_rows_of_infinities(rows, n, cols, bits, group, zeros, dt, yt):
    import post_weight_quantization_25_amd as g
    log(f"infinite x {rows}x{cols} bits={bits} g={group} n={n} {dt}->{yt} zeros={zeros}")
    q, What = stored(rows, cols, bits, group, 1, zeros)
    wide = torch.randn(n, cols + 3, generator=torch.Generator().manual_seed(n)).to(dt)
    plain = wide[:, 1:1 + cols]
    bad = plain.clone()
    k = spoil(bad)
    spoilt = wide.clone()
    spoilt[:, 1:1 + cols] = bad
    want = g.linear_grouped(q, plain.contiguous().cuda(), out_dtype=yt)
    got = g.linear_grouped(q, spoilt.cuda()[:, 1:1 + cols], out_dtype=yt)
    torch.cuda.synchronize()
    assert torch.equal(got[k:], want[k:])
    assert alike(got[:k], definition(bad[:k], What))


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("zeros", ["fraction", "far", "symmetric"])
def test_numbers_near_the_largest(rows, n, zeros):
    """u x beyond fp32's range where S (u - z) x is within it."""
    import post_weight_quantization_25_amd as g
    q, What = stored(rows, 256, 8, 64, 2, zeros)
    x = torch.randn(n, 256, generator=torch.Generator().manual_seed(1)).to(BF)
    for t in range(min(n, 5)):
        x[t, 50 * t] = 2.0 ** 127 * (-1) ** t
    y = g.linear_grouped(q, x.cuda())[:5].cpu().double()
    x = x[:5].double()
    ref, mag = x @ What.t(), x.abs() @ What.abs().t()
    top = float(torch.finfo(F32).max)
    bound = (256 + 64) * U * mag
    inside, outside = ref.abs() + bound < top, ref.abs() - bound > top
    assert bool(inside[:min(n, 5)].any())
    assert bool(((y - ref).abs() <= bound)[inside].all())
    assert torch.equal(y[outside], torch.sign(ref[outside]) * INF)


def test_experts():
    """In every expert its own weights, rows of no expert as they were."""
    import post_weight_quantization_25_amd as g
    E, rows, cols, n = 3, 5666, 64, 700
    q, What = stored(E * rows, cols, 4, 32, 3, "fraction")
    x = torch.randn(n, cols, generator=torch.Generator().manual_seed(1)).to(BF)
    lost = torch.arange(0, n, 70)
    x[lost, 5] = INF
    at = [30, 200, 201, 690]
    out = torch.full((n, rows), 7.0, device="cuda")
    got = g.linear_grouped(q, x.cuda(), torch.tensor(at, dtype=torch.int32).cuda(), out=out)
    torch.cuda.synchronize()
    for e, r0, r1 in segments(at, n):
        pick = lost[(lost >= r0) & (lost < r1)]
        if pick.numel():
            assert alike(got[pick.cuda()], definition(x[pick], What[e * rows:(e + 1) * rows]))
    assert bool((got[:30] == 7.0).all()) and bool((got[690:] == 7.0).all())


@pytest.mark.parametrize("zeros", ["whole", "fraction"])
def test_large_calls(zeros):
    """The tiles of large calls, and the kernel that they leave other zeros to."""
    import post_weight_quantization_25_amd as g
    q, What = stored(4096, 2048, 4, 128, 7, zeros)
    x = torch.randn(4096, 2048, generator=torch.Generator().manual_seed(8)).to(BF)
    spoil(x)
    y = g.linear_grouped(q, x.cuda())
    assert alike(y[:7], definition(x[:7], What)) and bool(torch.isfinite(y[7:]).all())
