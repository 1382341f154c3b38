"""gptqt_linear_grouped and its backward against their definitions in 64 bits (tolerances:
tuning_helpers; the forward product as the serving products: (d_col + 64) additions of
S sum |x| (|u - zc| + |z - zc|))."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import part, stored
from tuning_helpers import BF, F32, HF, U, back_reference, out_rounding, segments, zero_parts

pytestmark = pytest.mark.gpu


def ragged(n, E, seed):
    """Offsets over n rows: some experts without a row, the last segment may end before n."""
    gen = torch.Generator().manual_seed(seed)
    cut = torch.sort(torch.randint(0, n + 1, (E + 1,), generator=gen)).values
    if E > 2:
        cut[1] = cut[2]
    return cut.to(torch.int32)


def check(y, ref, bound, yt, rows):
    err = (y.cpu().double()[rows] - ref).abs()
    bound = bound * (1 + 2.0 ** -10) + out_rounding(ref, yt)
    log(f"  max |err| / bound = {float((err / bound.clamp_min(1e-300)).max()) if err.numel() else 0:.3f}")
    assert y.dtype == yt and bool((err <= bound).all())


CASES = [
    # d_row, d_col, bits, group, n, experts (0: none, all rows), dtype, out dtype, zeros
    (17, 64, 4, 32, 1, 0, HF, F32, "whole"), (100, 256, 4, 128, 3, 0, BF, F32, "whole"),
    (129, 136, 3, 0, 70, 0, BF, BF, "symmetric"), (64, 192, 8, 64, 65, 0, HF, HF, "whole"),
    (300, 130, 4, 0, 33, 0, BF, F32, "fraction"), (50, 96, 4, 32, 20, 0, BF, F32, "far"),
    (333, 333, 8, 0, 129, 0, HF, F32, "whole"), (65, 128, 3, 128, 257, 0, HF, HF, "whole"),
    (200, 512, 4, 128, 300, 5, BF, BF, "whole"), (90, 160, 4, 32, 100, 70, HF, F32, "whole"),
    (40, 64, 8, 32, 9, 130, BF, F32, "fraction"), (130, 320, 4, 64, 1000, 3, HF, HF, "far"),
    (70, 384, 3, 64, 400, 20, BF, F32, "whole"), (257, 258, 4, 0, 500, 2, BF, BF, "whole"),
    (64, 128, 8, 128, 1, 64, BF, BF, "whole"), (1, 8, 3, 0, 5, 4, HF, F32, "whole"),
    # many rows per expert: every width and group, rows that end in a slab, a turn, a chunk and a tile
    (300, 128, 4, 128, 300, 0, BF, F32, "whole"), (257, 320, 4, 64, 513, 0, HF, F32, "whole"),
    (64, 96, 4, 32, 161, 0, BF, BF, "whole"), (100, 160, 4, 32, 700, 3, HF, F32, "symmetric"),
    (520, 256, 8, 128, 400, 0, HF, HF, "whole"), (33, 192, 8, 64, 600, 2, BF, F32, "whole"), (300, 352, 8, 32, 300, 0, BF, F32, "whole"),
    (130, 384, 3, 128, 520, 0, BF, F32, "whole"), (90, 448, 3, 64, 260, 0, HF, F32, "symmetric"), (77, 128, 3, 32, 300, 0, BF, BF, "whole"),
    (300, 416, 4, 0, 300, 0, BF, F32, "symmetric"), (70, 48, 8, 0, 333, 0, HF, F32, "whole"), (260, 128, 3, 0, 270, 0, BF, F32, "whole"),
    (90, 250, 4, 0, 500, 2, BF, F32, "whole"), (300, 256, 4, 64, 290, 0, BF, F32, "fraction"), (64, 160, 8, 32, 700, 3, HF, F32, "far"),
    (2000, 64, 4, 32, 2100, 9, BF, F32, "whole"),
    # many weight rows: the forward product's tiles of 64 and 128 tokens, every width and group, odd rows and ends
    (17000, 128, 4, 128, 64, 0, BF, F32, "whole"), (17001, 64, 4, 64, 97, 0, HF, HF, "whole"), (17003, 96, 4, 32, 65, 0, BF, BF, "symmetric"),
    (17000, 130, 4, 0, 130, 0, BF, F32, "whole"), (17000, 128, 8, 128, 300, 0, BF, BF, "whole"), (17001, 64, 8, 64, 40, 0, HF, F32, "whole"),
    (17003, 96, 8, 32, 96, 0, HF, HF, "fraction"), (17000, 100, 8, 0, 130, 0, BF, F32, "whole"), (17000, 128, 3, 128, 64, 0, HF, F32, "whole"),
    (17001, 64, 3, 64, 130, 0, BF, BF, "symmetric"), (17003, 96, 3, 32, 300, 0, BF, F32, "whole"), (17000, 136, 3, 0, 65, 0, HF, F32, "whole"),
    (17000, 128, 4, 64, 130, 0, HF, F32, "far"), (5666, 64, 4, 32, 700, 3, BF, F32, "far"),
    # more than 1024 rows: the gradient's 256 x 256 tiles, with codes of whole 16 bytes and others
    (300, 256, 4, 128, 1100, 0, BF, BF, "whole"), (70, 384, 3, 64, 1030, 0, HF, BF, "symmetric"), (513, 128, 8, 32, 1200, 0, BF, BF, "whole"),
    (33, 288, 4, 32, 1025, 0, BF, BF, "fraction"), (90, 250, 4, 0, 1100, 0, HF, BF, "whole"), (64, 100, 8, 0, 1100, 0, BF, BF, "whole"),
    (700, 520, 3, 0, 1300, 0, BF, BF, "symmetric"), (1500, 128, 4, 128, 2500, 2, BF, BF, "far"), (1000, 64, 4, 64, 99, 0, HF, HF, "whole"),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("d_row,d_col,bits,group,n,E,dt,yt,zeros", CASES)
def test_parity(d_row, d_col, bits, group, n, E, dt, yt, zeros, back):
    import post_weight_quantization_25_amd as g
    log(f"grouped {d_row}x{d_col} bits={bits} g={group} n={n} E={E} {dt}->{yt} zeros={zeros} back={back}")
    q, What = stored(max(E, 1) * d_row, d_col, bits, group, 1, zeros)
    width = d_row if back else d_col
    gen = torch.Generator().manual_seed(n + d_row)
    a = torch.randn(n, width, generator=gen)
    if back:
        a *= torch.exp(3 * torch.randn(n, 1, generator=gen)) * 1e-3
    a = a.to(dt).cuda()
    offs = ragged(n, E, n) if E else None
    f = g.linear_grouped_backward if back else g.linear_grouped
    out = torch.full((n, d_col if back else d_row), 7.0, dtype=yt, device="cuda")
    y = f(q, a, None if offs is None else offs.cuda(), out=out)
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr()
    inside = torch.zeros(n, dtype=torch.bool)
    for e, r0, r1 in segments(None if offs is None else offs.tolist(), n):
        inside[r0:r1] = True
        if r1 > r0:
            qe, We = part(q, e * d_row, (e + 1) * d_row), What[e * d_row:(e + 1) * d_row]
            x = a[r0:r1].cpu().double()
            if back:
                ref, bound = back_reference(qe, We, x, yt)
            else:
                ref, bound = x @ We.t(), (d_col + 64) * U * zero_parts(qe, x)
                # bfloat16 as fp16 rows: what is below 2^-28 of a row's largest
                bound = bound + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * We.abs().sum(1)[None]
            check(y, ref, bound, yt, slice(r0, r1))
    assert bool((y.cpu()[~inside] == 7.0).all())
    again = f(q, a, None if offs is None else offs.cuda(), out_dtype=yt)
    assert torch.equal(again.cpu()[inside], y.cpu()[inside])


@pytest.mark.parametrize("back", [False, True])
def test_offsets_that_fall_or_leave_the_rows(back):
    """Any int32 is taken: clamped to the rows, never falling."""
    import post_weight_quantization_25_amd as g
    E, d, n = 7, 64, 50
    q, What = stored(E * d, d, 4, 32, 3)
    a = torch.randn(n, d, generator=torch.Generator().manual_seed(0)).to(BF).cuda()
    offs = [-2 ** 31, 5, 3, 2 ** 31 - 1, 20, -1, 60, 0]
    f = g.linear_grouped_backward if back else g.linear_grouped
    out = torch.full((n, d), 7.0, dtype=F32, device="cuda")
    y = f(q, a, torch.tensor(offs, dtype=torch.int32).cuda(), out=out)
    for e, r0, r1 in segments(offs, n):
        x, qe, We = a[r0:r1].cpu().double(), part(q, e * d, (e + 1) * d), What[e * d:(e + 1) * d]
        if r1 > r0:
            ref, bound = back_reference(qe, We, x, F32) if back else (x @ We.t(), (d + 64) * U * zero_parts(qe, x))
            check(y, ref, bound, F32, slice(r0, r1))


@pytest.mark.parametrize("n", [4, 200, 500])
@pytest.mark.parametrize("back", [False, True])
def test_strided_rows(n, back):
    """Rows of an odd pitch, as views of wider matrices."""
    import post_weight_quantization_25_amd as g
    q, _ = stored(96, 128, 4, 64, 2)
    width = 96 if back else 128
    wide = torch.randn(n, width + 7, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    x = wide[:, 3:3 + width]
    f = g.linear_grouped_backward if back else g.linear_grouped
    assert torch.equal(f(q, x), f(q, x.contiguous()))


def test_backward_against_differences():
    """sum(y dy) along a direction of x, by central differences of the 64-bit product (which is
    linear: to the bound of dx itself)."""
    import post_weight_quantization_25_amd as g
    q, What = stored(150, 192, 4, 64, 9)
    gen = torch.Generator().manual_seed(5)
    dy = torch.randn(40, 150, generator=gen).to(HF)
    v, x = torch.randn(40, 192, generator=gen).double(), torch.randn(40, 192, generator=gen).double()
    dx = g.linear_grouped_backward(q, dy.cuda(), out_dtype=F32).cpu().double()
    f = lambda t: (((x + t * v) @ What.t()) * dy.double()).sum()  # noqa: E731
    slope = (f(0.5) - f(-0.5))
    _, bound = back_reference(q, What, dy, F32)
    assert abs(float((dx * v).sum() - slope)) <= float((bound * v.abs()).sum()) + 1e-9 * float((What.abs().sum()))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n", [3, 150, 300])
def test_infinities_stay_in_their_rows(n, back):
    import post_weight_quantization_25_amd as g
    q, _ = stored(128, 128, 4, 128, 4)
    x = torch.randn(n, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    f = g.linear_grouped_backward if back else g.linear_grouped
    want = f(q, x)
    bad = x.clone()
    bad[1, 5] = float("inf")
    bad[2, 7] = float("nan")
    y = f(q, bad)
    keep = torch.arange(n, device="cuda") % n
    keep = keep[(keep != 1) & (keep != 2)]
    assert torch.equal(y[keep], want[keep])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()


def test_backward_of_far_apart_magnitudes():
    """Elements of dy from 2^-20 to 2^20 of each other and scales from 2^-14 to 2^10: the bound
    counts what the parts cannot hold."""
    import post_weight_quantization_25_amd as g
    q, _ = stored(200, 128, 4, 32, 6)
    gen = torch.Generator().manual_seed(2)
    q.scales.copy_((2.0 ** torch.randint(-14, 11, q.scales.shape, generator=gen).double()).half())
    from serving_helpers import weights
    What = torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(), 4, 32))
    dy = (torch.randn(30, 200, generator=gen) * 2.0 ** torch.randint(-20, 21, (30, 200), generator=gen)).to(BF)
    dy[3] = 0
    for t in (BF, F32):
        y = g.linear_grouped_backward(q, dy.cuda(), out_dtype=t)
        ref, bound = back_reference(q, What, dy, t)
        check(y, ref, bound, t, slice(None))
    assert bool((y[3] == 0).all())


@pytest.mark.parametrize("n", [5, 300])
def test_scales_of_zero_and_far_apart(n):
    """Groups without a scale give nothing, whatever their codes; scales from 2^-14 to 2^10 in a row."""
    import post_weight_quantization_25_amd as g
    from serving_helpers import weights
    for dead in (False, True):
        q, _ = stored(150, 256, 4, 32, 8)
        gen = torch.Generator().manual_seed(7)
        S = 2.0 ** torch.randint(-14, 11, q.scales.shape, generator=gen).double()
        if dead:
            S[3] = 0
            S[5, 2] = 0
            S[6, 0] = 0
            S[7, -1] = 0
        q.scales.copy_(S.half())
        What = torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(), 4, 32))
        x = torch.randn(n, 256, generator=gen).to(BF)
        y = g.linear_grouped(q, x.cuda())
        check(y, x.double() @ What.t(), (256 + 64) * U * zero_parts(q, x.double()), F32, slice(None))
        assert not dead or bool((y[:, 3] == 0).all())


def test_forward_of_far_apart_magnitudes():
    """Elements of x from 2^-20 to 2^20 of each other, rows of zeros and of subnormals: bfloat16
    elements below 2^-28 of their row's largest are off by 2^-39 of it."""
    import post_weight_quantization_25_amd as g
    q, What = stored(200, 256, 4, 64, 6)
    gen = torch.Generator().manual_seed(2)
    x = (torch.randn(300, 256, generator=gen) * 2.0 ** torch.randint(-20, 21, (300, 256), generator=gen)).to(BF)
    x[3] = 0
    x[4] *= 2.0 ** -126
    x[5] *= 2.0 ** 100
    y = g.linear_grouped(q, x.cuda())
    d = x.double()
    bound = (256 + 64) * U * zero_parts(q, d) + 2.0 ** -39 * d.abs().amax(1, keepdim=True) * What.abs().sum(1)[None]
    check(y, d @ What.t(), bound, F32, slice(None))
    assert bool((y[3] == 0).all())


def test_no_rows():
    import post_weight_quantization_25_amd as g
    q, _ = stored(64, 64, 4, 32, 1)
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    assert g.linear_grouped(q, x).shape == (0, 64) and g.linear_grouped_backward(q, x).shape == (0, 64)
    x = torch.ones(5, 64, dtype=BF, device="cuda")
    out = torch.full((5, 64), 7.0, dtype=BF, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    q2, _ = stored(128, 64, 4, 32, 1)
    assert bool((g.linear_grouped(q2, x, none, out=out) == 7).all())
    assert bool((g.linear_grouped_backward(q2, x, none, out=out) == 7).all())


def test_refusals():
    import post_weight_quantization_25_amd as g
    q, _ = stored(128, 64, 4, 32, 1)
    x = torch.ones(5, 64, dtype=BF, device="cuda")
    offs = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        g.linear_grouped(q, x[:, :32], offs)
    with pytest.raises(ValueError):
        g.linear_grouped(q, x.float(), offs)
    with pytest.raises(ValueError):
        g.linear_grouped(q, x, offs.long())
    with pytest.raises(ValueError):
        g.linear_grouped(q, x, torch.tensor([0, 1, 2, 5], dtype=torch.int32, device="cuda"))   # 128 rows, 3 experts
    with pytest.raises(ValueError):
        g.linear_grouped(q, x, offs.cpu())
    with pytest.raises(ValueError):
        g.linear_grouped(q, x, offs, out=torch.empty(5, 128, dtype=BF, device="cuda"))         # 64 rows each
    with pytest.raises(ValueError):
        g.linear_grouped_backward(q, x, None)                                                  # 128 columns are due
    buf = torch.ones(5, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        g.linear_grouped(q, buf, offs, out=buf)
    with pytest.raises(ValueError):
        g.linear_grouped_backward(q, buf, offs, out=buf)
