"""The tuning operators as a tuning step uses them: experts up and down, the loss at the head, and
the gradient back through both; on streams of their own, captured, from two threads, and in
workspaces of larger batches.  Against the same chain in 64 bits, and against themselves."""
import threading

import pytest

torch = pytest.importorskip("torch")

from gpu_helpers import log
from serving_helpers import part, stored, zero_parts
from tuning_helpers import BF, F32, HF, U, back_reference, head_reference, out_rounding, segments

pytestmark = pytest.mark.gpu


class Step:
    """relu(up x) -> down -> + x -> loss at the head, and the gradient of x, with E experts."""

    def __init__(self, n, E=4, d=128, f=192, vocab=1000, dt=HF, seed=1):
        gen = torch.Generator().manual_seed(seed)
        self.E, self.d, self.f, self.n = E, d, f, n
        (self.up, self.Wu), (self.down, self.Wd) = stored(E * f, d, 4, 64, 1), stored(E * d, f, 8, 64, 2)
        self.head, _ = stored(vocab, d, 4, 32, 3)
        for q, W in ((self.up, self.Wu), (self.down, self.Wd), (self.head, _)):
            q.scales.mul_(1.0 / float(W.pow(2).sum(1).mean().sqrt()))
        from serving_helpers import weights
        self.Wu, self.Wd, self.Wh = (torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(),
                                                              q.bits, q.group_size)) for q in (self.up, self.down, self.head))
        self.x = torch.randn(n, d, generator=gen).to(dt).cuda()
        cut = torch.sort(torch.randint(0, n + 1, (E - 1,), generator=gen)).values.tolist()
        self.cut = [0] + cut + [n]
        self.offsets = torch.tensor(self.cut, dtype=torch.int32).cuda()
        self.targets = torch.randint(-5, vocab, (n,), generator=gen, dtype=torch.int32).cuda()
        self.ids = torch.randint(0, vocab, (n, 8), generator=gen, dtype=torch.int32).cuda()
        self.top = torch.randn(n, 8, generator=gen).cuda()
        self.dt = dt

    def run(self, x=None, ws=None, kind="ce", n=None, offsets=None):
        """All that the step computes; ws: one workspace for every call, or None."""
        import post_weight_quantization_25_amd as g
        x = self.x if x is None else x
        o = self.offsets if offsets is None else offsets
        n = x.shape[0]
        a = g.linear_grouped(self.up, x, o, out_dtype=self.dt, ws=ws)
        h = torch.relu(a)
        b = g.linear_grouped(self.down, h, o, out_dtype=self.dt, ws=ws)
        y = x + b
        if kind == "ce":
            loss, dy = g.cross_entropy(self.head, y, self.targets[:n], ws=ws)
        else:
            loss, dy = g.distill(self.head, y, self.ids[:n], self.top[:n], 2.0, ws=ws)
        dh = g.linear_grouped_backward(self.down, dy, o, ws=ws)
        da = dh * (a > 0)
        dx = dy + g.linear_grouped_backward(self.up, da, o, ws=ws)
        return dict(a=a, h=h, b=b, y=y, loss=loss, dy=dy, dh=dh, da=da, dx=dx)

    def workspace(self, kind="ce", n=None):
        import post_weight_quantization_25_amd as g
        n, E, d, f, V = n or self.n, self.E, self.d, self.f, self.head.codes.shape[0]
        need = max(g.linear_grouped_workspace_size(n, E, f, d, 64), g.linear_grouped_workspace_size(n, E, d, f, 64),
                   g.linear_grouped_backward_workspace_size(n, E, f, d, 64), g.linear_grouped_backward_workspace_size(n, E, d, f, 64),
                   g.cross_entropy_workspace_size(n, d, V, 32) if kind == "ce" else g.distill_workspace_size(n, d, V, 8, 32))
        return torch.full((need,), 255, dtype=torch.uint8, device="cuda")


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("n", [1, 5, 40, 700])
def test_step_in_parts(n):
    """Each operator of the step on what the one before it gave, against its own definition."""
    s = Step(n)
    r = {k: v.cpu() for k, v in s.run().items()}
    x = s.x.cpu()

    def near(got, ref, bound, t, what):
        err, bound = (got.double() - ref).abs(), bound * (1 + 2.0 ** -10) + out_rounding(ref, t)
        log(f"  {what}: {float((err / bound.clamp_min(1e-300)).max()) if err.numel() else 0:.3f}")
        assert bool((err <= bound).all()), what

    for e, r0, r1 in segments(s.cut, n):
        if r0 == r1:
            continue
        at = slice(r0, r1)
        for q, W, rows, i, o in ((s.up, s.Wu, s.f, x, r["a"]), (s.down, s.Wd, s.d, r["h"], r["b"])):
            qe, We = part(q, e * rows, (e + 1) * rows), W[e * rows:(e + 1) * rows]
            near(o[at], i[at].double() @ We.t(), (We.shape[1] + 64) * U * zero_parts(qe, i[at].double()), HF, "forward")
        for q, W, rows, i, o in ((s.down, s.Wd, s.d, r["dy"], r["dh"]), (s.up, s.Wu, s.f, r["da"], None)):
            qe, We = part(q, e * rows, (e + 1) * rows), W[e * rows:(e + 1) * rows]
            ref, bound = back_reference(qe, We, i[at], HF)
            if o is not None:
                near(o[at], ref, bound, HF, "backward")
            else:                                              # added to dy in fp16: rounded once more
                total = ref + r["dy"][at].double()
                near(r["dx"][at], total, bound + out_rounding(ref, HF), HF, "dx")
    t = s.targets.cpu().long()
    ok = (t >= 0)
    loss, bl, dy, bd = head_reference(s.head, s.Wh, r["y"][ok], torch.ones(int(ok.sum()), 1).double(), t[ok][:, None],
                                      torch.ones(int(ok.sum())).double(), 1.0, HF)
    near(r["loss"][ok], loss, bl, F32, "loss")
    near(r["dy"][ok], dy, bd, HF, "dy")
    assert bool((r["loss"][~ok] == 0).all()) and bool((r["dy"][~ok] == 0).all())


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_one_workspace_and_another_stream(kind):
    """One workspace for all of a step's calls, filled with NaNs; a stream of its own."""
    s = Step(300)
    want = s.run(kind=kind)
    assert same(want, s.run(ws=s.workspace(kind), kind=kind))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.run(ws=s.workspace(kind), kind=kind)
    side.synchronize()
    assert same(want, got)


def test_stream_argument():
    """The stream given with the call, while another is the current one."""
    import post_weight_quantization_25_amd as g
    s = Step(200)
    want = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = g.linear_grouped(s.up, s.x, s.offsets, out_dtype=HF, stream=side)
    loss, dy = g.cross_entropy(s.head, want["y"], s.targets, stream=side)
    dh = g.linear_grouped_backward(s.down, dy, s.offsets, stream=side)
    side.synchronize()
    assert torch.equal(y, want["a"]) and torch.equal(loss, want["loss"]) and torch.equal(dh, want["dh"])


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_captured(kind):
    """Two graphs of the step on inputs of their own that share one workspace, replayed in turn
    with eager work in it between."""
    import post_weight_quantization_25_amd as g  # noqa: F401
    steps = [Step(300, seed=1), Step(130, seed=2)]
    ws = steps[0].workspace(kind)
    eager = [s.run(ws=ws, kind=kind) for s in steps]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in steps:
            s.run(ws=ws, kind=kind)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for s in steps:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(s.run(ws=ws, kind=kind))
        graphs.append(gr)
    for turn in range(4):
        for i in (0, 1, 0):
            for v in outs[i].values():
                v.fill_(float("nan"))
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(eager[i], outs[i]), (turn, i)
            ws.fill_(255)
            assert same(eager[1 - i], steps[1 - i].run(ws=ws, kind=kind))
    # new inputs in place: nothing of the last call is kept
    for i, s in enumerate(steps):
        s.x.copy_(torch.randn(s.x.shape, generator=torch.Generator().manual_seed(9 + i)).to(s.dt))
        s.targets.copy_(s.targets.flip(0))
        want = s.run(kind=kind)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same(want, outs[i])


def test_captured_large_tiles():
    """The large calls, with layers that those tiles leave to the other kernel and back: the kernel
    that does the work is chosen on the device at each replay."""
    import post_weight_quantization_25_amd as g
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (4096, 2048), generator=gen, device="cuda", dtype=torch.uint8)
    S = torch.rand(4096, 32, generator=gen, device="cuda").half()
    Z = torch.randint(0, 16, (4096, 32), generator=gen, device="cuda").half()
    x = torch.randn(4096, 4096, generator=gen, device="cuda").to(BF)
    q = g.Quantized(codes, S, Z, None, 4, 128, 4096)
    ws = torch.zeros(g.linear_grouped_workspace_size(4096, 1, 4096, 4096, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(4096, 4096, device="cuda")
    g.linear_grouped(q, x, out=out, ws=ws)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        g.linear_grouped(q, x, out=out, ws=ws)
    for turn in range(4):
        Z.copy_(torch.randint(0, 16, (4096, 32), generator=gen, device="cuda").half())
        if turn % 2:
            Z[17, 3] = 2.5
        want = g.linear_grouped(q, x)
        out.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), turn


def test_two_threads():
    """Calls from two host threads, each on a stream and in a workspace of its own."""
    steps = [Step(300, seed=1), Step(300, seed=2)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    bad, errors = [], []

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                ws = steps[i].workspace()
                for _ in range(20):
                    got = steps[i].run(ws=ws)
                    side.synchronize()
                    if not same(want[i], got):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert bad == [] and errors == []


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_smaller_batches_in_a_larger_workspace(kind):
    """The sizes made for the largest batch serve every smaller one, of the same numbers."""
    s = Step(1500)
    ws = s.workspace(kind)
    for n in (1500, 641, 160, 33, 7, 1):
        x = s.x[:n].contiguous()
        want = s.run(x=x, kind=kind)
        ws.fill_(255)
        assert same(want, s.run(x=x, ws=ws, kind=kind)), n


def test_only_the_outputs_are_written():
    """Inputs, and what lies behind the outputs and the workspace, stay as they were."""
    import post_weight_quantization_25_amd as g
    s = Step(333)
    n, V = 333, s.head.codes.shape[0]
    keep = [t.clone() for q in (s.up, s.down, s.head) for t in (q.codes, q.scales, q.zeros)] + [s.x.clone(), s.targets.clone()]

    def guarded(shape, dt):
        size = torch.Size(shape).numel()
        b = torch.full((size + 512,), 7, dtype=dt, device="cuda")
        return b, b[256:256 + size].view(shape)

    def work(need):
        b = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
        return b, b[256:256 + need]

    for dt in (BF, HF, F32):
        pads = []
        for fn, args, shape, need in (
                (g.linear_grouped, (s.up, s.x, s.offsets), (n, s.f), g.linear_grouped_workspace_size(n, s.E, s.f, s.d, 64)),
                (g.linear_grouped_backward, (s.down, s.x, s.offsets), (n, s.f),
                 g.linear_grouped_backward_workspace_size(n, s.E, s.d, s.f, 64))):
            a, out = guarded(shape, dt)
            b, ws = work(need)
            fn(*args, out=out, ws=ws)
            pads += [a[:256], a[-256:], b[:256], b[-256:]]
        a, dx = guarded((n, s.d), dt)
        c, loss = guarded((n,), F32)
        b, ws = work(g.cross_entropy_workspace_size(n, s.d, V, 32))
        g.cross_entropy(s.head, s.x, s.targets, loss=loss, dx=dx, ws=ws)
        pads += [a[:256], a[-256:], b[:256], b[-256:], c[:256], c[-256:]]
        b, ws = work(g.distill_workspace_size(n, s.d, V, 8, 32))
        g.distill(s.head, s.x, s.ids, s.top, loss=loss, dx=dx, ws=ws)
        pads += [a[:256], a[-256:], b[:256], b[-256:], c[:256], c[-256:]]
        torch.cuda.synchronize()
        assert all(bool((p == 7).all()) for p in pads)
    now = [t for q in (s.up, s.down, s.head) for t in (q.codes, q.scales, q.zeros)] + [s.x, s.targets]
    assert all(torch.equal(a, b) for a, b in zip(keep, now))


def test_more_than_2_to_31_elements():
    """Outputs, gradients and the planes between them beyond 32-bit offsets: rows at both ends and
    around the 2^31st element against the definition."""
    import post_weight_quantization_25_amd as g
    rows, cols, n = 32000, 64, 70001
    q, What = stored(rows, cols, 4, 32, 5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, cols, generator=gen, device="cuda").to(HF)
    pick = torch.tensor([0, 1, 67107, 67108, 67109, 69888, n - 1])
    y = g.linear_grouped(q, x, out_dtype=HF)
    xp = x[pick.cuda()].cpu().double()
    ref = xp @ What.t()
    assert bool(((y[pick.cuda()].cpu().double() - ref).abs() <= ((cols + 64) * U * zero_parts(q, xp)) * (1 + 2.0 ** -10) + out_rounding(ref, HF)).all())
    dx = g.linear_grouped_backward(q, y)                   # y as any other gradient
    r, bound = back_reference(q, What, y[pick.cuda()], HF)
    assert bool(((dx[pick.cuda()].cpu().double() - r).abs() <= bound * (1 + 2.0 ** -10) + out_rounding(r, HF)).all())


def test_no_rows():
    import post_weight_quantization_25_amd as g
    s = Step(5)
    x = torch.empty(0, s.d, dtype=BF, device="cuda")
    offs = torch.zeros(s.E + 1, dtype=torch.int32, device="cuda")
    assert g.linear_grouped(s.up, x, offs).shape == (0, s.f)
    assert g.linear_grouped_backward(s.down, x, offs).shape == (0, s.f)
    y = torch.full((7, s.f), 3.0, device="cuda")           # rows, but none of an expert
    x = torch.randn(7, s.d, device="cuda").to(BF)
    assert bool((g.linear_grouped(s.up, x, offs, out=y) == 3.0).all())
    assert bool((g.linear_grouped_backward(s.down, x, offs, out=y) == 3.0).all())


@pytest.mark.parametrize("vocab", [30, 5000])
def test_the_most_entries(vocab):
    """1024 entries a token, every word several times among 30."""
    import post_weight_quantization_25_amd as g
    from tuning_helpers import teacher_weights
    q, What = stored(vocab, 64, 8, 32, 4)
    q.scales.mul_(2.0 / float(What.pow(2).sum(1).mean().sqrt()))
    from serving_helpers import weights
    What = torch.from_numpy(weights(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(), 8, 32))
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(3, 64, generator=gen).to(HF)
    ids = torch.randint(0, vocab, (3, 1024), generator=gen, dtype=torch.int32)
    top = torch.randn(3, 1024, generator=gen)
    loss, dx = g.distill(q, x.cuda(), ids.cuda(), top.cuda(), 1.5, dx_dtype=F32)
    p, at, _ = teacher_weights(ids, top, 1.5, vocab)
    l, bl, r, br = head_reference(q, What, x, p, at, torch.ones(3).double(), 1.5, F32)
    for got, ref, bound in ((loss, l, bl), (dx, r, br)):
        assert bool(((got.cpu().double() - ref).abs() <= bound * (1 + 2.0 ** -10) + out_rounding(ref, F32)).all())


@pytest.mark.parametrize("n", [3, 130, 4096])
def test_codes_at_any_address(n):
    """A layer whose codes begin at an odd byte: the kernels that load whole aligned pieces leave it
    to the others."""
    import post_weight_quantization_25_amd as g
    from tuning_helpers import layer_parts
    rows = 4096 if n == 4096 else 300
    q, _ = stored(rows, 128, 4, 64, 6)
    room = torch.empty(q.codes.numel() + 1, dtype=torch.uint8, device="cuda")
    codes = room[1:].view(q.codes.shape)
    codes.copy_(q.codes)
    odd = g.Quantized(codes, q.scales, q.zeros, None, 4, 64, 128)
    x = torch.randn(n, 128, generator=torch.Generator().manual_seed(3)).to(HF).cuda()
    a, b = g.linear_grouped(q, x), g.linear_grouped(odd, x)
    size = (x.double().abs() @ torch.ones(128, rows, dtype=torch.float64, device="cuda")) * layer_parts(q)[0].max() * 32
    assert bool(((a - b).double().abs() <= 2 * (128 + 64) * U * size).all())
    dy = torch.randn(n, rows, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    assert torch.equal(g.linear_grouped_backward(q, dy), g.linear_grouped_backward(odd, dy))
    t = torch.arange(n, dtype=torch.int32, device="cuda") % rows
    (l0, d0), (l1, d1) = g.cross_entropy(q, x, t), g.cross_entropy(odd, x, t)
    assert float((l0 - l1).abs().max()) <= 1e-3 * float(l0.abs().max()) and d0.isfinite().all() and d1.isfinite().all()
