"""Losses at a stored head where finite logits lie further apart than fp32's range: words that far
below the largest count as nothing, in the loss and in its gradient."""
import pytest

torch = pytest.importorskip("torch")

from serving_helpers import weights
from tuning_helpers import BF, F32, out_rounding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [700, 9000])
@pytest.mark.parametrize("n", [4, 150])
@pytest.mark.parametrize("gt", [BF, F32])
def test_logits_further_apart_than_the_range(vocab, n, gt):
    """One column decides: z = x_0 w with w a multiple of 2^-6 from -2 on.  Words of one w tie, so
    that the loss of a target among the largest is the logarithm of their number, and of another one
    the distance."""
    import post_weight_quantization_25_amd as g
    d = 64
    gen = torch.Generator().manual_seed(vocab)
    codes = torch.randint(0, 256, (vocab, d), generator=gen, dtype=torch.uint8)
    S, Z = torch.full((vocab, 1), 2.0 ** -6).half(), torch.full((vocab, 1), 128.0).half()
    What = torch.from_numpy(weights(codes.numpy(), S.numpy(), Z.numpy(), 8, 64))
    q = g.Quantized(codes.cuda(), S.cuda(), Z.cuda(), None, 8, 64, d)
    x = torch.zeros(n, d)
    x[:, 0] = 2.0 ** 126 * torch.where(torch.arange(n) % 2 == 0, 1.9, -1.5)
    x = x.to(BF)
    z = x.double() @ What.t()
    assert float((z.amax(1) - z.amin(1)).min()) > 2.0 ** 128
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    t = order[torch.arange(n), torch.where(torch.arange(n) % 4 < 2, 0, vocab // 4)]
    loss, dx = g.cross_entropy(q, x.cuda(), t.int().cuda(), dx_dtype=gt)
    only, _ = g.cross_entropy(q, x.cuda(), t.int().cuda(), grad=False)
    ref = torch.logsumexp(z - z[torch.arange(n), t][:, None], 1)      # (z of 10^38 would absorb a logarithm in 64 bits, too)
    p = torch.softmax(z, 1)
    p[torch.arange(n), t] -= 1.0
    want = p @ What
    # logits: one product, an fp32 rounding each; a logarithm of up to 100 words: 2^-18 (tuning_helpers)
    bound = 2.0 ** -22 * z.abs().amax(1) * (ref > 1e30) + 2.0 ** -18
    assert bool(((loss.cpu().double() - ref).abs() <= bound).all()) and bool(((only.cpu().double() - ref).abs() <= bound).all())
    # weights and exponentials in one fp16 part (2^-11 each) or two, 2^-16 for the sums and softmax
    rel = (2.0 ** -10 if gt == BF else 0.0) + 2.0 ** -16
    assert bool(((dx.cpu().double() - want).abs() <= rel * (p.abs() @ What.abs()) + out_rounding(want, gt)).all())
    assert bool(torch.isfinite(dx).all())
