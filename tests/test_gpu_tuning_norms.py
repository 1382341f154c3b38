"""The tuning operators' fp32 gradients in the 2-norm (tuning_norms; tests/test_tuning_norms.py: the
criteria fail without a second part), the losses with and without a gradient, and the losses'
gradients of codes that begin at any address, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from test_gpu_head_loss import head, near, tokens
from tuning_helpers import BF, F32, HF, head_reference
from tuning_norms import packed, random_layer, softmax_criterion, sum_criterion

pytestmark = pytest.mark.gpu


def layer(rows, cols, bits, group, seed, size=None):
    """A random layer as a Quantized, and its What in 64 bits on the device."""
    import post_weight_quantization_25_amd as g
    u, S, z, What = random_layer(rows, cols, bits, group, seed, "cuda")
    if size is not None:
        S = (S.double() * size / float(What.pow(2).sum(1).mean().sqrt())).half()
        What = S.double().repeat_interleave(group, 1) * (u.double() - z.double().repeat_interleave(group, 1))
    return g.Quantized(packed(u, bits).contiguous(), S, z, None, bits, group, cols), What


@pytest.mark.parametrize("rows,cols,bits,group,n", [(11008, 4096, 4, 128, 64), (11008, 4096, 4, 32, 300), (4001, 2816, 8, 64, 100),
                                                    (4096, 5504, 4, 128, 1100), (4096, 4096, 8, 128, 20)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_gradient(rows, cols, bits, group, n, dt):
    import post_weight_quantization_25_amd as g
    q, What = layer(rows, cols, bits, group, 1)
    dy = (torch.randn(n, rows, generator=torch.Generator().manual_seed(2)) * 1e-2).to(dt).cuda()
    dx = g.linear_grouped_backward(q, dy, out_dtype=F32)
    ref = dy.double() @ What
    rel = float((dx.double() - ref).norm() / ref.norm())
    log(f"gradient {rows}x{cols} bits={bits} g={group} n={n}: {rel:.2e} of {sum_criterion(rows):.2e}")
    assert rel <= sum_criterion(rows)
    if dt is HF:
        # experts: the same rows in three, the middle one of one token
        at = torch.tensor([0, n // 2, n // 2 + 1, n], dtype=torch.int32, device="cuda")
        q3 = g.Quantized(*(torch.cat([t, t.flip(0), t]) for t in (q.codes, q.scales, q.zeros)), None, bits, group, cols)
        ref[n // 2] = dy[n // 2].double() @ What.flip(0)
        dx = g.linear_grouped_backward(q3, dy, at, out_dtype=F32)
        assert float((dx.double() - ref).norm() / ref.norm()) <= sum_criterion(rows)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [20, 130])
@pytest.mark.parametrize("k", [1, 5])
def test_losses_gradient(bits, n, k):
    """The large sum alone is what the criterion is taken of: the entries' own words, in fp32, are
    most of dx."""
    import post_weight_quantization_25_amd as g
    V, d = 200, 2048
    q, What = layer(V, d, bits, 64, 3, 1.0)
    gen = torch.Generator().manual_seed(n + k)
    x = torch.randn(n, d, generator=gen).to(HF).cuda()
    ids = torch.stack([torch.randperm(V, generator=gen)[:k] for _ in range(n)]).cuda()
    top = torch.randn(n, k, generator=gen).cuda()
    if k == 1:
        _, dx = g.cross_entropy(q, x, ids[:, 0].int(), dx_dtype=F32)
    else:
        _, dx = g.distill(q, x, ids.int(), top, dx_dtype=F32)
    z = x.double() @ What.t()
    assert float(z.abs().max()) <= 5.0
    soft = torch.softmax(z, 1)
    own = torch.zeros_like(soft).scatter_(1, ids, soft.gather(1, ids) - torch.softmax(top.double(), 1))
    rest = soft.scatter(1, ids, 0.0) @ What
    ref = rest + own @ What
    rel, share = float((dx.double() - ref).norm() / rest.norm()), float((own @ What).norm() / rest.norm())
    limit = softmax_criterion(V, d, 5.0) * (1 + 2.0 ** -3) + 2.0 ** -21 * share      # own: their softmax values, and fp32 roundings
    log(f"losses' gradient bits={bits} n={n} k={k}: {rel:.2e} of {limit:.2e}, entries {share:.1f} times the rest")
    assert rel <= limit


@pytest.mark.parametrize("n", [3, 130])
def test_losses_alone(n):
    import post_weight_quantization_25_amd as g
    V, d = 9000, 128
    q, What = head(V, d, 4, 64)
    x, gen = tokens(n, d, BF, 1), torch.Generator().manual_seed(2)
    t, w = torch.randint(0, V, (n,), generator=gen), torch.rand(n, generator=gen) + 0.5
    l, bl, _, _ = head_reference(q, What, x, torch.ones(n, 1).double(), t[:, None], w.double(), 1.0, F32)
    both, dx = g.cross_entropy(q, x, t.int().cuda(), w.cuda())
    only, none = g.cross_entropy(q, x, t.int().cuda(), w.cuda(), grad=False)
    assert dx is not None and none is None
    near(both, l, bl, F32, "loss")
    near(only, l, bl, F32, "loss alone")


@pytest.mark.parametrize("n,rows", [(3, 300), (130, 300), (1100, 300)])
@pytest.mark.parametrize("dt,gt", [(HF, HF), (BF, BF), (BF, F32)])
def test_losses_of_codes_at_any_address(n, rows, dt, gt):
    """Some tokens against the definition: the kernels that load whole aligned pieces, and those that
    they leave such a head to."""
    import post_weight_quantization_25_amd as g
    q, What = head(rows, 128, 4, 64)
    room = torch.empty(q.codes.numel() + 1, dtype=torch.uint8, device="cuda")
    codes = room[1:].view(q.codes.shape)
    codes.copy_(q.codes)
    x, t = tokens(n, 128, dt, 3), torch.arange(n) * 7 % rows
    pick = torch.tensor(sorted({0, 1, n // 2, n - 1}))
    l, bl, r, br = head_reference(q, What, x.cpu()[pick], torch.ones(pick.numel(), 1).double(), t[pick][:, None],
                                  torch.ones(pick.numel()).double(), 1.0, gt)
    for layer_ in (q, g.Quantized(codes, q.scales, q.zeros, None, 4, 64, 128)):
        loss, dx = g.cross_entropy(layer_, x, t.int().cuda(), dx_dtype=gt)
        near(loss[pick.cuda()], l, bl, F32, "loss")
        near(dx[pick.cuda()], r, br, gt, "dx")
