"""Products and gradients in captured graphs whose rows become infinite, are replayed, and become
finite again: each replay as the eager call on the same values, in one workspace."""
import pytest

torch = pytest.importorskip("torch")

from serving_helpers import stored
from tuning_helpers import BF, F32, HF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("yt", [BF, F32, HF])
@pytest.mark.parametrize("rows,cols,n,E", [(17000, 64, 130, 1), (300, 192, 40, 3), (2017, 256, 300, 1)])
def test_replays(rows, cols, n, E, yt):
    import post_weight_quantization_25_amd as g
    q, _ = stored(E * rows, cols, 4, 32, 1, "fraction")
    gen = torch.Generator().manual_seed(2)
    x, dy = torch.randn(n, cols, generator=gen).to(BF).cuda(), torch.randn(n, rows, generator=gen).to(BF).cuda()
    at = None if E == 1 else torch.tensor([0, 11, 12, n], dtype=torch.int32, device="cuda")
    need = max(g.linear_grouped_workspace_size(n, E, rows, cols, 32), g.linear_grouped_backward_workspace_size(n, E, rows, cols, 32))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y, dx = torch.empty(n, rows, dtype=yt, device="cuda"), torch.empty(n, cols, dtype=yt, device="cuda")

    def call():
        g.linear_grouped(q, x, at, out=y, ws=ws)
        g.linear_grouped_backward(q, dy, at, out=dx, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    plain = x.clone(), dy.clone()
    for turn in range(6):
        x.copy_(plain[0])
        dy.copy_(plain[1])
        if turn % 3 == 1:
            x[3, 5], x[n - 1, cols - 1] = float("inf"), float("nan")
            dy[4, rows - 1], dy[n - 2, 0] = -float("inf"), float("nan")
        elif turn % 3 == 2:
            x[7], dy[8] = float("inf"), -float("inf")
        want = g.linear_grouped(q, x, at, out_dtype=yt), g.linear_grouped_backward(q, dy, at, out_dtype=yt)
        y.fill_(3.0)
        dx.fill_(3.0)
        ws.fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, dx), want):
            assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got.nan_to_num(0.0), ref.nan_to_num(0.0)), turn
        lost = (~torch.isfinite(y)).any(1).sum().item(), (~torch.isfinite(dx)).any(1).sum().item()
        assert lost == {0: (0, 0), 1: (2, 2), 2: (1, 1)}[turn % 3]
