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


def test_outputs_that_are_inputs_are_refused():
    """A loss or a gradient in the buffer of the weights, the entries, the activations or of each
    other; next to one another they are taken."""
    import post_weight_quantization_25_amd as g
    q, _ = stored(300, 128, 4, 64, 1)
    n = 6
    x = torch.randn(n, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    ids, top = t[:, None].repeat(1, 2).contiguous(), torch.zeros(n, 2, device="cuda")
    room = torch.zeros(n * 128 + 2 * n, device="cuda")
    w, loss, dx = room[:n], room[n:2 * n], room[2 * n:].view(n, 128)
    w.fill_(0.5)
    want = g.cross_entropy(q, x, t, w.clone(), dx_dtype=torch.float32)
    got = g.cross_entropy(q, x, t, w, loss=loss, dx=dx)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bool((w == 0.5).all())
    kept = x.clone()
    for bad in (dict(weights=w, loss=w), dict(weights=w, loss=room[3:3 + n]), dict(loss=t.view(torch.float32)),
                dict(loss=room[5 * n:6 * n], dx=dx), dict(weights=room[n * 128:n * 129], dx=dx), dict(loss=x.view(-1).view(torch.float32)[:n])):
        with pytest.raises(ValueError, match="overlaps"):
            g.cross_entropy(q, x, t, **bad)
    for bad in (dict(loss=top.view(-1)[n:]), dict(loss=ids.view(-1)[:n].view(torch.float32))):
        with pytest.raises(ValueError, match="overlaps"):
            g.distill(q, x, ids, top, **bad)
    assert torch.equal(x, kept) and bool((w == 0.5).all()) and bool((top == 0).all())
