"""Products of many tokens on stored layers (the 256 x 256 tiles, which large calls take): every
width and group, rows that end in a slab, a chunk, a turn of slabs and a tile, experts, and the
layers that they leave to the other kernel.

Against the definition in 64 bits on the device.  Element by element (d_col + 64) additions of
what the products add up (tuning_helpers), and in the 2-norm 2^-22 sqrt(d_col + 64) of the
result: a sum's roundings, at most 2^-23 of it each, have independent signs for random data."""
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import BF, F32, HF, out_rounding

pytestmark = pytest.mark.gpu


def layer(rows, cols, bits, group, seed, zeros="whole"):
    """Random codes, scales and zeros, What and S (|u - zc| + |z - zc|) in 64 bits on the device (zc
    the whole part of the zero that small batches leave out: 0, or for 8-bit codes all of it)."""
    import post_weight_quantization_25_amd as g
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ng = cols // group if group else 1
    codes = torch.randint(0, 256, (rows, g.code_bytes(bits, cols)), generator=gen, device="cuda", dtype=torch.uint8)
    S = (torch.rand(rows, ng, generator=gen, device="cuda") * 0.05 + 0.001).half()
    Z = torch.randint(0, 2 ** bits, (rows, ng), generator=gen, device="cuda").half()
    if zeros == "fraction":
        Z = (torch.rand(rows, ng, generator=gen, device="cuda") * 2 ** bits).half()
    q = g.Quantized(codes, S, Z, None, bits, group, cols)
    if bits == 8:
        u = codes
    elif bits == 4:
        u = torch.stack([codes & 15, codes >> 4], -1).view(rows, cols)
    else:
        b = codes.view(rows, -1, 3).int()
        w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        u = ((w[..., None] >> torch.arange(0, 24, 3, device="cuda", dtype=torch.int32)) & 7).view(rows, cols)
    rep = cols // ng
    s, z = S.double().repeat_interleave(rep, 1), Z.double().repeat_interleave(rep, 1)
    u = u.double()
    return q, s * (u - z), s * (u + z.abs() if bits != 8 else (u - z).abs() + 1.0)


def compare(y, x, What, parts, t):
    ref = x.double() @ What.t()
    d = x.shape[1]
    bound = (d + 64) * 2.0 ** -23 * (x.double().abs() @ parts.t())
    bound += 2.0 ** -39 * x.double().abs().amax(1, keepdim=True) * What.abs().sum(1)[None]
    bound = bound * (1 + 2.0 ** -10) + out_rounding(ref, t)
    err = (y.double() - ref).abs()
    rel = float(err.norm() / ref.norm())
    log(f"  max |err| / bound = {float((err / bound).max()):.3f}, 2-norm {rel:.2e}")
    assert y.dtype == t and bool((err <= bound).all())
    assert rel <= 2.0 ** -22 * (d + 64) ** 0.5 + (torch.finfo(t).eps / 2 if t != F32 else 0.0)


CASES = [(4, 128, 4096, BF, F32), (4, 64, 4032, HF, F32), (4, 32, 4000, BF, F32), (4, 0, 4128, HF, F32),
         (8, 128, 4224, HF, BF), (8, 64, 3904, BF, F32), (8, 32, 4128, HF, F32), (8, 0, 4112, BF, F32),
         (3, 128, 4096, HF, HF), (3, 64, 4096, BF, F32), (3, 32, 4096, BF, BF), (3, 0, 4224, HF, F32)]


@pytest.mark.parametrize("bits,group,cols,dt,yt", CASES)
def test_large(bits, group, cols, dt, yt):
    import post_weight_quantization_25_amd as g
    log(f"forward bits={bits} g={group} cols={cols} {dt}->{yt}")
    rows, n = 4083, 4090                                   # 16 x 16 tiles, the last ones not whole
    q, What, parts = layer(rows, cols, bits, group, 1)
    x = torch.randn(n, cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dt)
    y = g.linear_grouped(q, x, out_dtype=yt)
    compare(y, x, What, parts, yt)
    assert torch.equal(g.linear_grouped(q, x, out_dtype=yt), y)


@pytest.mark.parametrize("bits,group,cols", [(4, 32, 288), (8, 64, 320), (3, 128, 384)])
def test_few_columns(bits, group, cols):
    """Short sums, whose bound is tight: tens of thousands of rows and tokens."""
    import post_weight_quantization_25_amd as g
    q, What, parts = layer(17000, cols, bits, group, 3)
    x = torch.randn(17001, cols, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF)
    y = g.linear_grouped(q, x)
    for a in range(0, 17001, 4000):
        compare(y[a:a + 4000], x[a:a + 4000], What, parts, F32)


def test_experts():
    """Experts of very different numbers of rows, one with none, rows of none, a strided x."""
    import post_weight_quantization_25_amd as g
    E, rows, cols = 5, 4000, 2048                          # (tests/test_tuning_rules.py: all these sizes take the large tiles)
    q, What, parts = layer(E * rows, cols, 4, 128, 5)
    at = [7, 1500, 1500, 1501, 9000, 15990]
    x = torch.randn(16000, cols + 5, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(BF)[:, 3:3 + cols]
    out = torch.full((16000, rows), 7.0, device="cuda")
    y = g.linear_grouped(q, x, torch.tensor(at, dtype=torch.int32, device="cuda"), out=out)
    for e in range(E):
        if at[e + 1] > at[e]:
            s = slice(e * rows, (e + 1) * rows)
            compare(y[at[e]:at[e + 1]], x[at[e]:at[e + 1]], What[s], parts[s], F32)
    assert bool((y[:at[0]] == 7.0).all()) and bool((y[at[-1]:] == 7.0).all())


@pytest.mark.parametrize("how", ["fraction", "zero scale", "infinite x"])
def test_what_the_large_tiles_leave(how):
    """Zeros that are no whole numbers and scales of zero (the other kernel), and infinities in x,
    which stay in their rows."""
    import post_weight_quantization_25_amd as g
    q, What, parts = layer(4096, 4096, 4, 128, 7, "fraction" if how == "fraction" else "whole")
    x = torch.randn(4096, 4096, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").to(BF)
    if how == "zero scale":
        for s in (q.scales, ):
            s[5] = 0
            s[6, 3] = 0
        rep = q.scales.double().repeat_interleave(128, 1)
        for m in (What, parts):
            m[5] = 0
            m[6, 384:512] = 0
        del rep
    if how == "infinite x":
        want = g.linear_grouped(q, x)
        bad = x.clone()
        bad[3, 100], bad[9, 5] = float("inf"), float("nan")
        y = g.linear_grouped(q, bad)
        keep = torch.ones(4096, dtype=torch.bool, device="cuda")
        keep[3] = keep[9] = False
        assert torch.equal(y[keep], want[keep]) and not torch.isfinite(y[3]).any() and torch.isnan(y[9]).all()
        return
    y = g.linear_grouped(q, x)
    if how == "fraction":      # the other kernel's operand holds the whole number next to z, the rest comes on top: no larger than u and z
        compare(y, x, What, parts, F32)
    else:
        compare(y, x, What, parts, F32)
        assert bool((y[:, 5] == 0).all())


def test_logits_of_a_large_batch():
    """The losses on them: 4096 tokens at a head of 16384 words; loss and gradient of some tokens
    against the formulas."""
    import post_weight_quantization_25_amd as g
    V, d, n = 16384, 2048, 4096
    q, What, _ = layer(V, d, 8, 128, 9)
    k = 2.0 / float(What.pow(2).sum(1).mean().sqrt())
    q.scales.mul_(k)
    What = (q.scales.double().repeat_interleave(128, 1)) * (q.codes.double() - q.zeros.double().repeat_interleave(128, 1))
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(10), device="cuda").to(BF)
    t = (torch.arange(n, device="cuda") * 7 % V).int()
    t[5] = -100
    loss, dx = g.cross_entropy(q, x, t)
    only, _ = g.cross_entropy(q, x, t, grad=False)
    pick = torch.tensor([0, 1, 255, 256, 2047, 4095], device="cuda")
    z = x[pick].double() @ What.t()
    lse = torch.logsumexp(z, 1)
    want = lse - z.gather(1, t[pick].long()[:, None])[:, 0]
    p = torch.softmax(z, 1)
    p.scatter_add_(1, t[pick].long()[:, None], torch.full((6, 1), -1.0, dtype=torch.float64, device="cuda"))
    # a logit: (d + 64) additions of what 2048 products add up, about 2048 times 0.8 |x| |w|
    dz = (d + 64) * 2.0 ** -23 * float((x[pick].double().abs() @ What.abs().t()).max())
    for got in (loss, only):
        assert float((got[pick].double() - want).abs().max()) <= 2 * dz + 2.0 ** -18
        assert float((got[pick].double() - want).abs().max()) <= 1e-4       # and as measured for random signs
    ref = p @ What
    err = (dx[pick].double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert float(err.max()) <= 2.0 ** -8
    assert float(loss[5]) == 0 and bool((dx[5] == 0).all())
