"""Arguments of the tuning operators that a program's views give them."""
import pytest

torch = pytest.importorskip("torch")

from serving_helpers import stored
from tuning_helpers import BF

pytestmark = pytest.mark.gpu


def test_the_last_token_of_a_long_sequence():
    """hidden[:, -1] of one long sequence: a single row whose pitch is the whole sequence, more than
    the 2^23 elements that rows may lie apart."""
    import post_weight_quantization_25_amd as g
    q, _ = stored(300, 128, 4, 64, 1)
    hidden = torch.randn(1, 70000, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    x = hidden[:, -1]
    assert x.shape == (1, 128) and x.stride(0) > 1 << 23
    row, t = x.contiguous(), torch.tensor([7], dtype=torch.int32, device="cuda")
    ids, top = t[:, None].contiguous(), torch.zeros(1, 1, device="cuda")
    assert torch.equal(g.linear_grouped(q, x), g.linear_grouped(q, row))
    for a, b in ((g.cross_entropy(q, x, t), g.cross_entropy(q, row, t)), (g.distill(q, x, ids, top), g.distill(q, row, ids, top))):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(g.GptqError):                       # two rows that far apart are refused, as documented
        g.linear_grouped(q, torch.empty(2, 1 << 24, dtype=BF, device="cuda")[:, :128])
