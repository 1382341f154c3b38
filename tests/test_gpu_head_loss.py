"""gptqt_cross_entropy and gptqt_distill against their definitions in 64 bits (tolerances:
tuning_helpers)."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import stored
from tuning_helpers import BF, F32, HF, U, head_reference, out_rounding, teacher_weights

pytestmark = pytest.mark.gpu


def head(vocab, d, bits, group, zeros="whole", spread=2.0):
    """A stored head whose logits spread by about ``spread`` for standard normal x."""
    from serving_helpers import weights
    q, What = stored(vocab, d, bits, group, 11, zeros)
    q.scales.mul_(spread / float(What.pow(2).sum(1).mean().sqrt()))
    return q, torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(), bits, group))


def tokens(n, d, dt, seed):
    return torch.randn(n, d, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


def near(got, ref, bound, t, what):
    err = (got.cpu().double() - ref).abs()
    bound = bound * (1 + 2.0 ** -10) + out_rounding(ref, t)
    log(f"  {what}: max |err| / bound = {float((err / bound.clamp_min(1e-300)).max()):.3f}, err {float(err.max()):.2e}")
    assert got.dtype == t and bool((err <= bound).all())


CASES = [
    # vocab, d, bits, group, n, dtype, dx dtype, zeros
    (1, 64, 4, 32, 3, BF, F32, "whole"), (2, 64, 8, 64, 1, HF, HF, "whole"), (100, 64, 4, 64, 5, BF, BF, "whole"),
    (1000, 128, 4, 128, 33, HF, F32, "whole"), (777, 136, 3, 0, 130, BF, F32, "symmetric"),
    (8192, 64, 8, 32, 20, BF, BF, "whole"), (8193, 64, 4, 32, 17, HF, HF, "whole"), (20000, 96, 4, 32, 129, BF, F32, "fraction"),
    (9001, 130, 4, 0, 300, BF, BF, "whole"), (30000, 64, 8, 0, 2, BF, F32, "whole"), (300, 256, 8, 128, 64, HF, F32, "far"),
    (3000, 256, 4, 128, 200, BF, BF, "whole"), (500, 128, 8, 64, 130, HF, F32, "whole"), (700, 128, 4, 64, 1100, BF, BF, "whole"),
    (999, 64, 3, 64, 99, HF, HF, "symmetric"), (640, 100, 8, 0, 1030, BF, BF, "whole"),
    # few tokens of many columns, which several workgroups finish
    (600, 522, 4, 0, 7, BF, F32, "whole"), (9000, 1024, 8, 64, 33, HF, HF, "whole"), (400, 768, 3, 128, 1, BF, BF, "whole"),
    (500, 2051, 8, 0, 130, BF, BF, "fraction"),
]


@pytest.mark.parametrize("vocab,d,bits,group,n,dt,gt,zeros", CASES)
def test_cross_entropy(vocab, d, bits, group, n, dt, gt, zeros):
    import post_weight_quantization_25_amd as g
    log(f"cross_entropy V={vocab} d={d} bits={bits} g={group} n={n} {dt}->{gt} zeros={zeros}")
    q, What = head(vocab, d, bits, group, zeros)
    x = tokens(n, d, dt, n)
    gen = torch.Generator().manual_seed(4)
    t = torch.randint(0, vocab, (n,), generator=gen, dtype=torch.int32)
    t[::2] = (x.cpu().double() @ What.t()).argmax(1)[::2].int()      # half of them the model's own choice
    w = torch.rand(n, generator=gen) + 0.5
    masked = torch.zeros(n, dtype=torch.bool)
    if n > 4:
        t[1], t[2], t[3], w[4] = -100, vocab, -2 ** 31, 0.0
        masked[1:5] = True
        x[1] = float("nan")                                          # what a masked token holds does not count
        x[4] = float("inf")
    loss, dx = g.cross_entropy(q, x, t.cuda(), w.cuda(), dx_dtype=gt)
    only, none = g.cross_entropy(q, x, t.cuda(), w.cuda(), grad=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(only, loss) or float((only - loss).abs().max()) <= 1e-5 * float(loss.abs().max())
    assert bool((loss.cpu()[masked] == 0).all()) and bool((dx.cpu()[masked] == 0).all())
    ok = ~masked
    ids = t.long()[ok][:, None]
    l, bl, r, br = head_reference(q, What, x.cpu()[ok], torch.ones(int(ok.sum()), 1).double(), ids, w[ok].double(), 1.0, gt)
    near(loss[ok.cuda()], l, bl, F32, "loss")
    near(dx[ok.cuda()], r, br, gt, "dx")
    l2, d2 = g.cross_entropy(q, x, t.cuda(), w.cuda(), dx_dtype=gt)
    assert torch.equal(l2, loss) and torch.equal(d2, dx)


@pytest.mark.parametrize("k,T,tt", [(1, 1.0, F32), (7, 2.0, BF), (64, 0.7, HF), (300, 1.5, F32)])
@pytest.mark.parametrize("vocab,d,bits,group,n,dt,gt,zeros", [CASES[2], CASES[3], CASES[4], CASES[6], CASES[7], CASES[-4], CASES[-3], CASES[-1]])
def test_distill(vocab, d, bits, group, n, dt, gt, zeros, k, T, tt):
    import post_weight_quantization_25_amd as g
    log(f"distill V={vocab} d={d} bits={bits} g={group} n={n} {dt}->{gt} k={k} T={T}")
    q, What = head(vocab, d, bits, group, zeros)
    x = tokens(n, d, dt, n + k)
    gen = torch.Generator().manual_seed(k)
    ids = torch.randint(-3, vocab + 3, (n, k), generator=gen, dtype=torch.int32)   # some outside, some twice
    ids[0] = int(ids[0, 0])                                          # one word k times
    top = (torch.randn(n, k, generator=gen) * 2).to(tt)
    if k > 3:
        top[:, 3] = -float("inf")                                    # an entry of no weight
    w = torch.rand(n, generator=gen) + 0.5
    if n > 4:
        ids[1] = -1                                                  # no entry
        top[2] = -float("inf")                                       # none with a weight
        w[3] = 0.0
        x[1] = float("nan")
    p, at, live = teacher_weights(ids, top, T, vocab)
    ok = live & (w != 0)
    loss, dx = g.distill(q, x, ids.cuda(), top.cuda(), T, w.cuda(), dx_dtype=gt)
    torch.cuda.synchronize()
    assert bool((loss.cpu()[~ok] == 0).all()) and bool((dx.cpu()[~ok] == 0).all())
    l, bl, r, br = head_reference(q, What, x.cpu()[ok], p[ok], at[ok], w[ok].double(), T, gt)
    near(loss[ok.cuda()], l, bl, F32, "loss")
    near(dx[ok.cuda()], r, br, gt, "dx")
    only, _ = g.distill(q, x, ids.cuda(), top.cuda(), T, w.cuda(), grad=False)
    near(only[ok.cuda()], l, bl, F32, "loss alone")


def test_sure_tokens():
    """Tokens whose target the model is all but sure of, 1 - p from 1e-2 to 1e-9: loss and
    gradient to 2% of themselves (an fp32 logit of 30 is off by up to (256 + 64) 2^-23 times
    what its products add up, about 60: 2.3e-3 as a worst case, which both sums follow; bfloat16 dx 2^-9; the rest 2^-10)."""
    import post_weight_quantization_25_amd as g
    q, What = head(500, 256, 4, 64, "symmetric")
    gen = torch.Generator().manual_seed(1)
    t = torch.randint(0, 500, (40,), generator=gen)
    x = 0.3 * torch.randn(40, 256, generator=gen).double()
    row = What[t]
    gain = torch.linspace(12.0, 30.0, 40).double()
    x = (x + gain[:, None] * row / (row * row).sum(1, keepdim=True)).to(BF)
    z = x.double() @ What.t()
    rest = z.clone()
    rest.scatter_(1, t[:, None], -float("inf"))
    miss = torch.sigmoid(torch.logsumexp(rest, 1) - z.gather(1, t[:, None])[:, 0])
    assert float(miss.min()) < 1e-8 and float(miss.max()) > 1e-4
    loss, dx = g.cross_entropy(q, x.cuda(), t.int().cuda())
    ref = -torch.log1p(-miss)
    assert bool(((loss.cpu().double() - ref).abs() <= 0.02 * ref).all())
    soft = torch.softmax(rest, 1) * miss[:, None]
    soft.scatter_(1, t[:, None], -miss[:, None])
    want = soft @ What
    err = (dx.cpu().double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(err.max()) <= 0.02


def test_against_differences():
    """The gradient along random directions against central differences of the 64-bit losses."""
    import post_weight_quantization_25_amd as g
    q, What = head(300, 64, 4, 32)
    gen = torch.Generator().manual_seed(8)
    n, k, T = 12, 5, 1.7
    x = torch.randn(n, 64, generator=gen).to(HF)
    t = torch.randint(0, 300, (n,), generator=gen, dtype=torch.int32)
    ids = torch.randint(0, 300, (n, k), generator=gen, dtype=torch.int32)
    top = torch.randn(n, k, generator=gen)
    w = torch.rand(n, generator=gen)
    p, at, _ = teacher_weights(ids, top, T, 300)
    v = torch.randn(n, 64, generator=gen).double()

    def ce(y):
        z = y @ What.t()
        return (w.double() * (torch.logsumexp(z, 1) - z.gather(1, t.long()[:, None])[:, 0])).sum()

    def kd(y):
        z = y @ What.t() / T
        return (w.double() * T * T * (p * (p.log() - z.gather(1, at) + torch.logsumexp(z, 1)[:, None])).sum(1)).sum()

    _, a = g.cross_entropy(q, x.cuda(), t.cuda(), w.cuda(), dx_dtype=F32)
    _, b = g.distill(q, x.cuda(), ids.cuda(), top.cuda(), T, w.cuda(), dx_dtype=F32)
    for dx, f in ((a, ce), (b, kd)):
        h = 1e-4
        slope = float((f(x.double() + h * v) - f(x.double() - h * v)) / (2 * h))
        size = float((dx.cpu().double().abs() * v.abs()).sum())
        assert abs(float((dx.cpu().double() * v).sum()) - slope) <= 1e-4 * size   # 128 2^-23 of sums 5 times as large; h^2


def test_nan_in_a_live_token():
    """A NaN in a token's x, or among a teacher's logits, is that token's alone."""
    import post_weight_quantization_25_amd as g
    q, _ = head(400, 64, 4, 32)
    x = tokens(150, 64, BF, 1)
    t = torch.arange(150, dtype=torch.int32, device="cuda")
    l0, d0 = g.cross_entropy(q, x, t)
    x[7, 3] = float("nan")
    l1, d1 = g.cross_entropy(q, x, t)
    keep = torch.arange(150, device="cuda") != 7
    assert torch.equal(l0[keep], l1[keep]) and torch.equal(d0[keep], d1[keep])
    assert bool(torch.isnan(l1[7])) and bool(torch.isnan(d1[7]).all())
    ids = torch.stack([t, t + 1, t + 2], 1).contiguous()
    top = torch.zeros(150, 3, device="cuda")
    top[9, 1] = float("nan")
    top[10] = float("nan")
    loss, dx = g.distill(q, tokens(150, 64, BF, 1), ids, top)
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[9:11] = True
    assert torch.equal(torch.isnan(loss), bad) and torch.equal(torch.isnan(dx).all(1), bad)
    assert torch.equal(torch.isnan(dx).any(1), bad)


@pytest.mark.parametrize("gt", [BF, F32])
def test_more_tokens_than_a_chunk(gt):
    """Batches longer than the tokens taken at a time give each token what a short batch does, to
    the order of fp32 sums."""
    import post_weight_quantization_25_amd as g
    q, What = head(9000, 64, 4, 32)
    n = 4096 + 4096 + 5
    x = tokens(n, 64, BF, 3)
    t = (torch.arange(n) % 9000).int().cuda()
    loss, dx = g.cross_entropy(q, x, t, dx_dtype=gt)
    pick = torch.tensor([0, 1, 4095, 4096, 8191, 8192, n - 1])
    l, bl, r, br = head_reference(q, What, x.cpu()[pick], torch.ones(7, 1).double(), t.cpu().long()[pick][:, None],
                                  torch.ones(7).double(), 1.0, gt)
    near(loss[pick.cuda()], l, bl, F32, "loss")
    near(dx[pick.cuda()], r, br, gt, "dx")


def test_one_workspace_for_smaller_batches():
    import post_weight_quantization_25_amd as g
    q, _ = head(9000, 64, 4, 32)
    need = g.cross_entropy_workspace_size(600, 64, 9000, 32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")       # NaNs
    for n in (600, 1, 129, 30):
        x = tokens(n, 64, BF, n)
        t = torch.zeros(n, dtype=torch.int32, device="cuda")
        l0, d0 = g.cross_entropy(q, x, t)
        l1, d1 = g.cross_entropy(q, x, t, ws=ws)
        assert torch.equal(l0, l1) and torch.equal(d0, d1)


def test_strided_rows_and_given_outputs():
    import post_weight_quantization_25_amd as g
    q, _ = head(500, 64, 4, 32)
    wide = tokens(20, 71, BF, 2)
    x = wide[:, 5:69]
    t = torch.arange(20, dtype=torch.int32, device="cuda")
    l0, d0 = g.cross_entropy(q, x.contiguous(), t)
    loss, dx = torch.empty(20, device="cuda"), torch.empty(20, 64, dtype=BF, device="cuda")
    l1, d1 = g.cross_entropy(q, x, t, loss=loss, dx=dx)
    assert l1 is loss and d1 is dx and torch.equal(l0, l1) and torch.equal(d0, d1)


def test_no_tokens():
    import post_weight_quantization_25_amd as g
    q, _ = head(500, 64, 4, 32)
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    loss, dx = g.cross_entropy(q, x, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert loss.shape == (0,) and dx.shape == (0, 64)


def test_refusals():
    import post_weight_quantization_25_amd as g
    q, _ = head(100, 64, 4, 32)
    x = tokens(4, 64, BF, 0)
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    ids, top = t[:, None].repeat(1, 3).contiguous(), torch.zeros(4, 3, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(targets=t.long()), dict(targets=t[:3]), dict(targets=t.cpu()),
                dict(weights=torch.ones(4, dtype=BF, device="cuda")), dict(dx=x), dict(grad=False, dx=torch.empty_like(x)),
                dict(loss=torch.empty(3, device="cuda"))):
        with pytest.raises(ValueError):
            g.cross_entropy(**{"q": q, "x": x, "targets": t, **bad})
    for bad in (dict(ids=ids[:, 0]), dict(top=top[:, :2]), dict(ids=ids.long()), dict(top=top.double())):
        with pytest.raises(ValueError):
            g.distill(**{"q": q, "x": x, "ids": ids, "top": top, **bad})
    for T in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(g.GptqError):
            g.distill(q, x, ids, top, temperature=T)
    with pytest.raises(g.GptqError):
        g.distill(q, x, ids[:, :0].contiguous(), top[:, :0].contiguous())
