"""The serving operators as a program uses them: one after another through a layer, on
streams of their own, captured and replayed, with buffers that hold something else."""
import threading

import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import BF, F32, HF, stored

pytestmark = pytest.mark.gpu


class Block:
    """A decoder block's products: norm to 8-bit rows, a projection on them, a projection with
    adapters, experts."""

    def __init__(self, d=256, f=128, experts=6, k=2, rank=16, m=4, dt=BF, seed=0):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dt).cuda()  # noqa: E731
        self.d, self.k, self.m, self.dt = d, k, m, dt
        self.w = (1 + 0.1 * torch.randn(d, generator=gen)).to(dt).cuda()
        self.q8, _ = stored(d, d, 4, 128, 1 + seed)
        self.ql, _ = stored(d, d, 4, 64, 2 + seed)
        for q in (self.q8, self.ql):
            q.scales.mul_(0.05)
        self.A, self.B = rand(m, rank, d, std=d ** -0.5), rand(m, d, rank, std=0.1)
        self.s = (0.5 + torch.rand(m, generator=gen)).cuda()
        self.router = rand(experts, d, std=d ** -0.5)
        self.up, _ = stored(experts * 2 * f, d, 4, 32, 3 + seed)
        self.down, _ = stored(experts * d, f, 4, 32, 4 + seed)
        self.up.scales.mul_(0.05)
        self.down.scales.mul_(0.05)

    def inputs(self, n, seed=0):
        gen = torch.Generator().manual_seed(77 + seed)
        return (torch.randn(n, self.d, generator=gen).to(self.dt).cuda(), torch.randn(n, self.d, generator=gen).to(self.dt).cuda(),
                torch.randint(-1, self.m, (n,), generator=gen, dtype=torch.int32).cuda())

    def run(self, x, r, ids, stream=None):
        import post_weight_quantization_25_amd as g
        rows, h = g.rmsnorm_int8(x, self.w, r, stream=stream)
        y1 = g.linear_int8(self.q8, rows, out_dtype=self.dt, stream=stream)
        y2 = g.linear_lora(self.ql, y1, self.A, self.B, ids, self.s, out_dtype=self.dt, stream=stream)
        y3, chosen, w = g.moe(y2, self.router, self.up, self.down, self.k, out_dtype=self.dt, stream=stream)
        return rows.q, rows.scale, h, y1, y2, y3, chosen, w


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n", [1, 20, 100])
@pytest.mark.parametrize("dt", [BF, HF])
def test_run_together(n, dt):
    """Through the block, each step against its plain form in 64 bits on the step's own input,
    to twice the output type's half step of the largest magnitude of a row."""
    from serving_helpers import weights
    b = Block(dt=dt)
    x, r, ids = b.inputs(n)
    q, scale, h, y1, y2, y3, chosen, w = (t.cpu() for t in b.run(x, r, ids))
    eps = torch.finfo(dt).eps

    def what(l):
        return torch.from_numpy(weights(l.codes.cpu().numpy(), l.scales.cpu().numpy(), l.zeros.cpu().numpy(), l.bits, l.group_size))

    def near(y, ref, mag):
        # half a step of the type, and 2^-13 of what a row adds up for fp32's sums and parts
        assert bool(((y.double() - ref).abs() <= eps / 2 * ref.abs() + 2.0 ** -13 * mag).all())

    v = h.double()
    assert torch.equal(h, (x.cpu().double() + r.cpu().double()).to(dt))
    norm = v * b.w.cpu().double() / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert bool(((q.double() * scale.double()[:, None] - norm).abs() <= 0.5001 * scale.double()[:, None]).all())
    W = what(b.q8)
    xr = q.double() * scale.double()[:, None]
    near(y1, xr @ W.t(), xr.abs() @ W.abs().t())
    W, a = what(b.ql), y1.double()
    ref, mag = a @ W.t(), a.abs() @ W.abs().t()
    for t in range(n):
        j = int(ids[t])
        if j >= 0:
            A, B, s = b.A[j].cpu().double(), b.B[j].cpu().double(), float(b.s[j])
            ref[t] += s * (B @ (A @ a[t]))
            mag[t] += s * (B.abs() @ (A.abs() @ a[t].abs()))
    near(y2, ref, mag)
    a, d, f = y2.double(), b.d, b.down.d_col
    U, D = what(b.up), what(b.down)
    logits = a @ b.router.cpu().double().t()
    ref, mag = torch.zeros(n, d).double(), torch.zeros(n, d).double()
    for t in range(n):
        top = torch.softmax(logits[t][chosen[t].long()], 0)
        assert bool((logits[t].topk(b.k).values.min() - logits[t][chosen[t].long()] <= 1e-4).all())
        for j, e in enumerate(chosen[t].tolist()):
            g, u = U[2 * f * e:2 * f * e + f] @ a[t], U[2 * f * e + f:2 * f * (e + 1)] @ a[t]
            hid = top[j] * g * torch.sigmoid(g) * u
            ref[t] += D[d * e:d * (e + 1)] @ hid
            # the inner sums' magnitudes stand for their errors
            gm = U[2 * f * e:2 * f * e + f].abs() @ a[t].abs()
            um = U[2 * f * e + f:2 * f * (e + 1)].abs() @ a[t].abs()
            mag[t] += D[d * e:d * (e + 1)].abs() @ (top[j] * 1.1 * gm * um)
    near(y3, ref, mag)


@pytest.mark.parametrize("n", [1, 30, 100])
def test_own_stream(n):
    """On a stream that is not the current one, with the buffers made inside: the default
    stream is kept busy with other allocations meanwhile."""
    b = Block()
    x, r, ids = b.inputs(n)
    want = b.run(x, r, ids)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append(b.run(x, r, ids, stream=s))
        junk = [torch.full((n, 256), float("nan"), device="cuda") for _ in range(20)]   # freed memory is taken at once
        del junk
    s.synchronize()
    torch.cuda.synchronize()
    assert all(same(want, g) for g in got)


@pytest.mark.parametrize("n", [1, 30, 100])
def test_captured_and_replayed(n):
    """Two graphs of the block on inputs of their own, replayed in turn with eager work between;
    every replay equals the eager result."""
    b = Block()
    sets = [b.inputs(n, seed=i) for i in range(2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            b.run(*s)
    torch.cuda.current_stream().wait_stream(side)
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.run(*s))
        graphs.append(g)
    for step in range(4):
        for i, s in enumerate(sets):
            new = b.inputs(n, seed=10 * step + i)
            for t, v in zip(s, new):
                t.copy_(v)
            for o in outs[i]:
                o.fill_(3)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(b.run(*new), outs[i]), (step, i)


def test_two_threads():
    """Calls from two host threads, each on a stream of its own."""
    b = Block()
    data = [b.inputs(40, seed=i) for i in range(2)]
    want = [b.run(*d) for d in data]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(10):
            got[i].append(b.run(*data[i], stream=s))
        s.synchronize()
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 10 and all(same(want[i], g) for g in got[i])


def test_caller_buffers_are_used_and_checked():
    import post_weight_quantization_25_amd as g
    b = Block()
    x, r, ids = b.inputs(9)
    want = b.run(x, r, ids)
    rows = g.Int8Rows(torch.empty(9, 256, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda"))
    got, h = g.rmsnorm_int8(x, b.w, r, residual_out=r, out=rows)
    assert got is rows and h is r and torch.equal(r, want[2]) and torch.equal(rows.q, want[0])
    out = torch.empty(9, 256, dtype=BF, device="cuda")
    assert g.linear_int8(b.q8, rows, out=out) is out and torch.equal(out, want[3])
    with pytest.raises(ValueError):
        g.linear_int8(b.q8, rows, out=out.float()[:, :255])
    with pytest.raises(ValueError):
        g.linear_int8(b.q8, rows, out=out.cpu())
    with pytest.raises(ValueError):
        g.rmsnorm_int8(x, b.w[:-1], r)
    with pytest.raises(ValueError):
        g.rmsnorm_int8(x, b.w, r[:5])
    with pytest.raises(ValueError):
        g.rmsnorm_int8(x, b.w, r, residual_out=out, normed=out)
    with pytest.raises(ValueError):
        g.rmsnorm_int8(x.cpu(), b.w, r)
    with pytest.raises(ValueError):
        g.linear_int8(g.Quantized(b.q8.codes, b.q8.scales, b.q8.zeros, None, 4, 128, 256, fp4=True), rows)
    with pytest.raises(g.GptqError):
        g.rmsnorm_int8(x, b.w, r, eps=-1.0)
    log("buffers and refusals done")
