"""gptqs_rmsnorm_int8 against its definition in 64 bits.

Tolerances.  Codes of 16-bit rows with 16-bit weights: none, they are exact roundings of
127 p / am, decided here from the exact remainder.  fp32 rows or weights: the kernel rounds
a quotient in 64 bits (relative 2^-52), so a code may differ only where 127 |p| / am lies
within 127 * 2^-50 of a half-integer.  Scale: am rstd / 127 in 64 bits, rounded once to
fp32: 2^-24 relative, plus d * 2^-52 for the sum.  Normalised rows: p (exact for 16 bits)
times rstd rounded to fp32, rounded to fp32: 2 * 2^-24, then to the row's type (half a
step, at least half the smallest subnormal)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(x, w, r, eps):
    """(h in T, |127 p / am| decided exactly or None, scale, normalised) on the CPU in 64 bits."""
    h = x if r is None else (x.double() + r.double()).to(x.dtype)   # one rounding: the sum of two fits 64 bits
    v = h.double()
    p = v * w.double()
    am = p.abs().amax(1, keepdim=True)
    one = torch.ones_like(am)
    safe = torch.where(am > 0, am, one)
    rest = torch.fmod(254.0 * p.abs() + safe, 2.0 * safe)
    k = torch.round((254.0 * p.abs() + safe - rest) / (2.0 * safe))
    k = k - ((rest == 0) & (k % 2 == 1)).double()
    rstd = 1.0 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + eps)
    scale = torch.where(am > 0, am * rstd / 127.0, one)
    near = (torch.fmod(127.0 * p.abs() / safe, 1.0) - 0.5).abs()
    return h, k * torch.sign(p), scale[:, 0], p * rstd, near


def check(x, w, r, eps, rows, h, normed):
    hr, k, scale, y, near = reference(x.cpu(), w.cpu(), None if r is None else r.cpu(), eps)
    assert torch.equal(h.cpu().float(), hr.float())
    q = rows.q.cpu().double()
    wide = x.dtype == F32 or w.dtype == F32
    ok = (q == k) | (near <= 127 * 2.0 ** -50) if wide else q == k
    assert bool(ok.all()), f"{int((~ok).sum())} codes differ"
    d = x.shape[1]
    rel = ((rows.scale.cpu().double() - scale).abs() / scale).max().item()
    log(f"  scale rel {rel:.2e}")
    assert rel <= 2.0 ** -24 * (1 + 2.0 ** -20) + d * 2.0 ** -52
    if normed is not None:
        fi = torch.finfo(x.dtype)
        err = (normed.cpu().double() - y).abs()
        bound = (2.0 ** -23 + fi.eps / 2 * (1 + 2.0 ** -20)) * y.abs() + fi.smallest_normal * fi.eps / 2
        assert bool((err <= bound).all()), float((err / bound).max())


def inputs(n, d, dt, wt, residual, seed=0):
    gen = torch.Generator().manual_seed(1000 * n + d + seed)
    x = torch.randn(n, d, generator=gen)
    x[:, :: max(1, d // 4)] *= 20
    r = torch.randn(n, d, generator=gen).to(dt).cuda() if residual else None
    return x.to(dt).cuda(), (1 + 0.1 * torch.randn(d, generator=gen)).to(wt).cuda(), r


CASES = [
    # n, d, x dtype, weight dtype, residual, normed
    (1, 1, BF, BF, False, True), (1, 1, HF, F32, True, True), (5, 7, F32, F32, True, True), (3, 8, HF, HF, False, False),
    (9, 64, BF, BF, True, True), (6, 511, BF, BF, True, False), (7, 512, HF, HF, True, True),   # a wave per row
    (4, 513, BF, F32, True, True), (1, 2048, BF, BF, True, False), (33, 2047, HF, HF, False, True),
    (1, 4096, BF, BF, True, True), (65, 4096, HF, HF, True, True), (3, 4095, F32, F32, True, True),
    (3, 4097, BF, BF, False, True), (17, 8192, BF, BF, True, True), (5, 8193, HF, F32, True, True),
    (3, 11008, HF, HF, False, True), (2, 16384, F32, F32, True, True), (2, 16385, BF, BF, True, True),
    (1, 49152, BF, BF, True, True), (3, 20001, HF, HF, False, False), (2, 65537, F32, F32, True, True),
    (4100, 4096, BF, BF, True, True),
]


@pytest.mark.parametrize("n,d,dt,wt,residual,with_normed", CASES)
def test_norm_parity(n, d, dt, wt, residual, with_normed):
    import post_weight_quantization_25_amd as g
    log(f"norm {n}x{d} {dt} w={wt} residual={residual}")
    x, w, r = inputs(n, d, dt, wt, residual)
    normed = torch.empty_like(x) if with_normed else None
    rows, h = g.rmsnorm_int8(x, w, r, 1e-5, normed=normed)
    torch.cuda.synchronize()
    check(x, w, r, float(np.float32(1e-5)), rows, h, normed)
    again, _ = g.rmsnorm_int8(x, w, r, 1e-5)
    assert torch.equal(again.q, rows.q) and torch.equal(again.scale, rows.scale)


@pytest.mark.parametrize("dt", [BF, HF])
def test_norm_ties_are_exact(dt):
    """Rows made of half-integer multiples of am / 127: every product is a tie or next to one."""
    import post_weight_quantization_25_amd as g
    top = 127.0
    v = torch.tensor([[top] + [k + 0.5 for k in range(60)] + [-(k + 0.5) for k in range(60)] + [k + 0.5 + 2 ** -2 for k in range(7)]])
    x = v.to(dt).cuda()
    w = torch.ones(v.shape[1], dtype=dt, device="cuda")
    rows, _ = g.rmsnorm_int8(x, w)
    assert torch.equal(rows.q.cpu().double(), torch.round(x.cpu().double()))   # torch rounds ties to even too
    # the same at a maximum that is no power of two times 127: random weights, exact remainders
    gen = torch.Generator().manual_seed(5)
    x = (torch.randint(-255, 256, (64, 4096), generator=gen)).float().to(dt).cuda()
    w = (torch.randint(1, 16, (4096,), generator=gen)).float().to(dt).cuda()
    rows, h = g.rmsnorm_int8(x, w)
    check(x, w, None, float(np.float32(1e-6)), rows, h, None)


@pytest.mark.parametrize("d", [40, 1000, 4096, 20000])
def test_norm_special_rows(d):
    """Zero rows, rows whose products underflow or overflow fp32, infinities and NaNs; each
    row only changes its own outputs."""
    import post_weight_quantization_25_amd as g
    x, w, _ = inputs(8, d, BF, BF, False, 3)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[5, d // 2] = float("inf")
    x[6, d - 1] = float("nan")
    w = w * 1e10
    normed = torch.empty_like(x)
    rows, _ = g.rmsnorm_int8(x, w, eps=1e-6, normed=normed)
    fine = [0, 1, 2, 3, 4, 7]
    sub = g.Int8Rows(rows.q[fine], rows.scale[fine])
    check(x[fine], w, None, float(np.float32(1e-6)), sub, x[fine], normed[fine])
    assert float(rows.scale[1]) == 1.0 and not rows.q[1].any()
    assert torch.isnan(rows.scale[[5, 6]]).all() and not rows.q[[5, 6]].any()
    assert torch.isnan(normed[6]).any()


@pytest.mark.parametrize("n,d", [(3, 100), (5, 4096), (2, 18000)])
def test_norm_strides_and_in_place(n, d):
    """Odd pitches, and h or the normalised rows written over x or the residual."""
    import post_weight_quantization_25_amd as g
    x, w, r = inputs(n, d, HF, HF, True, 7)
    wantn = torch.empty_like(x)
    want, wanth = g.rmsnorm_int8(x, w, r, normed=wantn)

    def strided(t, pad, fill):
        b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
        b[:, 1:1 + t.shape[1]] = t
        return b, b[:, 1:1 + t.shape[1]]
    xb, xs = strided(x, 3, 9.0)
    rb, rs = strided(r, 5, 9.0)
    qb = torch.full((n, d + 3), 77, dtype=torch.int8, device="cuda")
    rows, h = g.rmsnorm_int8(xs, w, rs, residual_out=rs, normed=xs, out=g.Int8Rows(qb[:, 2:2 + d], torch.empty(n, device="cuda")))
    assert torch.equal(rows.q, want.q) and torch.equal(rows.scale, want.scale)
    assert torch.equal(rs, wanth) and torch.equal(xs, wantn) and h is rs
    assert bool((xb[:, 0] == 9).all()) and bool((xb[:, d + 1:] == 9).all()) and bool((rb[:, d + 1:] == 9).all())
    assert bool((qb[:, :2] == 77).all()) and bool((qb[:, d + 2:] == 77).all())
    x2, r2 = x.clone(), r.clone()
    rows, h = g.rmsnorm_int8(x2, w, r2, residual_out=x2, normed=r2)
    assert torch.equal(x2, wanth) and torch.equal(r2, wantn) and torch.equal(rows.q, want.q)


def test_norm_empty():
    import post_weight_quantization_25_amd as g
    w = torch.ones(16, dtype=BF, device="cuda")
    rows, h = g.rmsnorm_int8(torch.zeros(0, 16, dtype=BF, device="cuda"), w)
    assert tuple(rows.q.shape) == (0, 16) and tuple(rows.scale.shape) == (0,)
