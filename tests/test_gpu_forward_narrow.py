"""The large forward tiles on rows of few columns: of a single group, of groups that do not fill a
turn of four slabs, and of one scale (tests/test_forward_tables.py: these sizes take them).

Element by element against the definition in 64 bits: (d_col + 64) additions of what the products
add up (tests/test_gpu_forward.py)."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import BF, F32, HF
from test_gpu_forward import compare, layer

pytestmark = pytest.mark.gpu


def sampled(n, seed):
    """Rows at both ends, around a tile's end, and between."""
    gen = torch.Generator().manual_seed(seed)
    some = torch.randint(0, n, (400,), generator=gen)
    return torch.cat([torch.tensor([0, 1, 255, 256, 257, n - 2, n - 1]), some]).unique().cuda()


@pytest.mark.parametrize("bits,group,cols,n,rows,dt", [
    (4, 64, 64, 32768, 20480, BF), (8, 64, 64, 32768, 20480, HF), (4, 32, 32, 65536, 20480, HF), (8, 32, 32, 65536, 20480, BF),
    (4, 32, 96, 32768, 20480, BF), (8, 32, 96, 32768, 20480, HF), (4, 0, 64, 32768, 20480, BF), (8, 0, 64, 32768, 20480, HF),
])
def test_one_expert(bits, group, cols, n, rows, dt):
    import post_weight_quantization_25_amd as g
    log(f"narrow forward bits={bits} g={group} cols={cols} n={n} rows={rows} {dt}")
    q, What, parts = layer(rows, cols, bits, group, 1)
    x = torch.randn(n, cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dt)
    need = g.linear_grouped_workspace_size(n, 1, rows, cols, group)
    room = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")      # NaNs behind the tables, too
    y = g.linear_grouped(q, x, ws=room[:need])
    pick = sampled(n, 3)
    compare(y[pick], x[pick], What, parts, F32)


@pytest.mark.parametrize("bits,group,cols,n,rows,dt", [(4, 64, 64, 40000, 20001, BF), (8, 32, 32, 65536, 24001, HF)])
def test_experts(bits, group, cols, n, rows, dt):
    """Three experts of an odd number of rows, the second with few tokens: the last one's tables end
    the workspace."""
    import post_weight_quantization_25_amd as g
    log(f"narrow forward of experts bits={bits} g={group} cols={cols} n={n} rows={rows} {dt}")
    E, at = 3, [5, n // 2, n // 2 + 3, n - 2]
    q, What, parts = layer(E * rows, cols, bits, group, 4)
    x = torch.randn(n, cols, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(dt)
    need = g.linear_grouped_workspace_size(n, E, rows, cols, group)
    room = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((n, rows), 7.0, device="cuda")
    y = g.linear_grouped(q, x, torch.tensor(at, dtype=torch.int32, device="cuda"), out=out, ws=room[:need])
    for e in range(E):
        pick = at[e] + sampled(at[e + 1] - at[e], e) if at[e + 1] - at[e] > 300 else torch.arange(at[e], at[e + 1], device="cuda")
        s = slice(e * rows, (e + 1) * rows)
        compare(y[pick], x[pick], What[s], parts[s], F32)
    assert bool((y[:at[0]] == 7.0).all()) and bool((y[at[-1]:] == 7.0).all())
