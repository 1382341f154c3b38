"""The gradient through stored layers where dy has infinities and NaNs: the definition's sum of the
row, whatever the weights' parts, the tile and the place of the element in the slabs.

The elements that are not finite decide the row alone (the others add something finite), so the
result is exact: an infinity of some sign, or NaN of a zero weight, of both signs or of a NaN."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import stored
from tuning_helpers import BF, F32, HF, segments

pytestmark = pytest.mark.gpu
INF = float("inf")


def definition(dy, What):
    """Row by row the sum over the elements that are not finite, in 64 bits."""
    out = torch.empty(dy.shape[0], What.shape[1], dtype=torch.float64)
    for t in range(dy.shape[0]):
        at = ~torch.isfinite(dy[t])
        out[t] = (dy[t][at][:, None].double() * What[at]).sum(0)
    return out


def alike(got, want):
    got = got.cpu().double()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(0.0, 1.0, -1.0), want.nan_to_num(0.0, 1.0, -1.0))


def spoil(dy):
    """Infinities first, last, alone, in pairs of one sign and of both, a NaN, and a whole row."""
    d = dy.shape[1]
    dy[0, d - 1] = INF
    if dy.shape[0] > 2:
        dy[1, 0] = -INF
        dy[2, d // 2], dy[2, d - 1] = INF, INF
    if dy.shape[0] > 6:
        dy[3, 0], dy[3, d - 1] = INF, -INF
        dy[4, d - 1] = float("nan")
        dy[5, :] = -INF
        dy[6, d - 1], dy[6, 0] = -INF, float("nan")
    return min(dy.shape[0], 7) if dy.shape[0] > 6 else min(dy.shape[0], 3) if dy.shape[0] > 2 else 1


@pytest.mark.parametrize("dt,yt", [(BF, BF), (BF, F32), (HF, HF)])
@pytest.mark.parametrize("d_row,d_col,bits,group,n,zeros", [
    (33, 64, 4, 32, 1, "whole"), (130, 136, 3, 0, 9, "symmetric"), (290, 333, 8, 0, 40, "whole"), (161, 128, 4, 64, 130, "fraction"),
    (2017, 256, 8, 128, 100, "far"), (65, 2056, 8, 0, 20, "fraction"), (300, 512, 4, 128, 1100, "whole"),
])
def test_rows_of_infinities(d_row, d_col, bits, group, n, zeros, dt, yt):
    import post_weight_quantization_25_amd as g
    log(f"infinite dy {d_row}x{d_col} bits={bits} g={group} n={n} {dt}->{yt} zeros={zeros}")
    q, What = stored(d_row, d_col, bits, group, 1, zeros)
    wide = torch.randn(n, d_row + 3, generator=torch.Generator().manual_seed(n)).to(dt)
    plain = wide[:, 1:1 + d_row]
    bad = plain.clone()
    rows = spoil(bad)
    want = g.linear_grouped_backward(q, plain.contiguous().cuda(), out_dtype=yt)
    spoilt = wide.clone()
    spoilt[:, 1:1 + d_row] = bad
    got = g.linear_grouped_backward(q, spoilt.cuda()[:, 1:1 + d_row], out_dtype=yt)
    torch.cuda.synchronize()
    assert torch.equal(got[rows:], want[rows:])
    assert alike(got[:rows], definition(bad[:rows], What))


def test_rows_of_experts():
    """In every expert its own weights; rows of no expert stay as they were."""
    import post_weight_quantization_25_amd as g
    E, d_row, d_col, n = 5, 97, 192, 60
    q, What = stored(E * d_row, d_col, 4, 64, 3)
    dy = torch.randn(n, d_row, generator=torch.Generator().manual_seed(1)).to(BF)
    dy[:, d_row - 1] = torch.where(torch.arange(n) % 3 == 0, INF, dy[:, d_row - 1].float()).to(BF)
    at = [2, 20, 20, 31, 50, 57]
    out = torch.full((n, d_col), 7.0, device="cuda")
    got = g.linear_grouped_backward(q, dy.cuda(), torch.tensor(at, dtype=torch.int32).cuda(), out=out)
    torch.cuda.synchronize()
    for e, r0, r1 in segments(at, n):
        lost = torch.arange(r0, r1)[torch.arange(r0, r1) % 3 == 0]
        assert alike(got[lost.cuda()], definition(dy[lost], What[e * d_row:(e + 1) * d_row]))
        rest = torch.arange(r0, r1)[torch.arange(r0, r1) % 3 != 0]
        assert bool(torch.isfinite(got[rest.cuda()]).all())
    assert bool((got[:2] == 7.0).all()) and bool((got[57:] == 7.0).all())
