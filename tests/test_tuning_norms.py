"""On the CPU: the 2-norm criteria of tuning_norms are broken by weights or exponentials in one part,
a dropped slab of rows and a neighbour's scale, and kept by what the kernels do."""
import pytest

torch = pytest.importorskip("torch")

from tuning_norms import one_part, random_layer, relative, softmax_criterion, sum_criterion, unit_rows


def two_parts(v):
    hi = one_part(v)
    return hi + one_part(v - hi)


@pytest.mark.parametrize("rows,bits,group", [(11008, 4, 32), (4001, 8, 64)])
def test_the_sums_criterion(rows, bits, group):
    _, S, _, What = random_layer(rows, 64, bits, group, 1)
    dy = torch.randn(40, rows, generator=torch.Generator().manual_seed(2)).double()
    want, limit = dy @ What, sum_criterion(rows)
    W, p2 = unit_rows(What, S.double())
    assert relative(dy @ (two_parts(W) * p2), want) <= limit / 8
    assert relative((dy.float() @ What.float()).double(), want) <= limit       # fp32 sums
    assert relative(dy @ (one_part(W) * p2), want) > 2 * limit                 # no second part
    assert relative(dy[:, :-32] @ What[:-32], want) > limit                    # the last slab
    other = What.clone()
    other[7] = What[7] * (S[8].double() / S[7].double()).repeat_interleave(group)
    assert relative(dy @ other, want) > limit                                  # a neighbour's scales


def test_the_softmax_criterion():
    """Few words of many columns, whose sum is no larger than its parts: with many words roundings
    average out against it."""
    V, d = 200, 2048
    _, S, _, What = random_layer(V, d, 8, 64, 3)
    What /= float(What.pow(2).sum(1).mean().sqrt())
    z = torch.randn(20, d, generator=torch.Generator().manual_seed(4)).double() @ What.t()
    assert float(z.abs().max()) <= 5.0
    limit = softmax_criterion(V, d, 5.0)
    e = torch.exp(z - z.amax(1, keepdim=True))
    want = e @ What
    W, p2 = unit_rows(What, torch.ones_like(S, dtype=torch.float64))
    assert relative(two_parts(e * 2.0 ** 14) * 2.0 ** -14 @ (two_parts(W) * p2), want) <= limit / 8
    assert relative(one_part(e * 2.0 ** 14) * 2.0 ** -14 @ What, want) > 2 * limit   # exponentials in one part
    assert relative(e @ (one_part(W) * p2), want) > 2 * limit                        # weights in one part
    assert relative(e[:, :-8] @ What[:-8], want) > limit                             # the last words
