"""GPU tests of moe_forward_few against the layer's formula in 64 bits.

The bound of an output element is computed with it, from what the kernels
round (u = 2^-24 for fp32, half a step of bf16 = 2^-8):

  logits   a sum of H products in fp32: |d l| <= (H + 8) u sum |x r|.  Softmax
           weights move by a factor of at most exp(2 max |d l|), plus the
           roundings of exp and the division (8 u).
  g, u     sums of H products (fp8: codes times a scale per 128, 2 more
           roundings a block): |d g| <= (H + H / 64 + 8) u sum |x w|.
  h        SiLU has slope at most 1.1; expf, its sum, the division and the
           products: 12 u |h|.
  h'       h times the weight, kept in two bf16: 2^-16 of it.
  out      one sum over all n = (experts chosen) I columns: (n + n / 64 + 16) u
           of the sum of the magnitudes, then half a step of bf16.

Rows are drawn so that the k-th and (k + 1)-th logit differ by more than their
rounding, so that both sides choose the same experts."""
import math

import pytest
import torch

import expert_layer_moe_amd as moe

pytestmark = pytest.mark.gpu
U, BF16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _codes(gen, *shape):
    """Random finite e4m3fn codes."""
    c = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
    return torch.where(c % 128 == 127, c - 1, c)


class Layer:
    """Random weights, the device layer, and the weights in 64 bits."""

    def __init__(self, seed, H, E, I, k, ns=0, fp8=False, packed=False):
        g = torch.Generator().manual_seed(seed)
        self.H, self.E, self.I, self.k, self.ns, self.g = H, E, I, k, ns, g
        n = E + ns
        self.router = (torch.randn(E, H, generator=g) / math.sqrt(H)).bfloat16()
        s13 = s2 = None
        if fp8:
            w13, w2 = _codes(g, n, 2 * I, H), _codes(g, n, H, I)
            s13 = torch.rand(n, 2 * I // 128, H // 128, generator=g) / (100 * math.sqrt(H))
            s2 = torch.rand(n, H // 128, I // 128, generator=g) / (100 * math.sqrt(I))
            wide = lambda s: s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)  # noqa: E731
            self.w13 = w13.view(torch.float8_e4m3fn).double() * wide(s13)
            self.w2 = w2.view(torch.float8_e4m3fn).double() * wide(s2)
        else:
            w13 = (torch.randn(n, 2 * I, H, generator=g) / math.sqrt(H)).bfloat16()
            w2 = (torch.randn(n, H, I, generator=g) / math.sqrt(I)).bfloat16()
            self.w13, self.w2 = w13.double(), w2.double()
        self.dev = moe.DeviceLayer(self.router, w13, w2, k, ns, s13, s2, packed=packed)

    def rows(self, T):
        """T rows whose choice of experts no rounding changes."""
        out = []
        while len(out) < T:
            x = torch.randn(self.H, generator=self.g).bfloat16()
            l = self.router.double() @ x.double()
            top = l.sort(descending=True).values
            noise = (self.H + 8) * U * (self.router.double().abs() @ x.double().abs()).max()
            if self.k == self.E or top[self.k - 1] - top[self.k] > 4 * noise:
                out.append(x)
        return torch.stack(out)

    def reference(self, x, valid):
        """(out, bound) in 64 bits."""
        H, I, k = self.H, self.I, self.k
        T = x.shape[0]
        out, err = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
        chosen = set()
        mags = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            if not valid[t]:
                continue
            xr = x[t].double()
            l = self.router.double() @ xr
            dl = (H + 8) * U * (self.router.double().abs() @ xr.abs()).max()
            top = l.topk(k)
            w = torch.softmax(top.values, 0)
            picks = [(int(e), float(p)) for e, p in zip(top.indices, w)]
            if self.ns:
                picks.append((self.E, 1.0))
            for e, p in picks:
                chosen.add(e)
                gu, mag = self.w13[e] @ xr, self.w13[e].abs() @ xr.abs()
                d = (H + H / 64 + 8) * U * mag
                g, u = gu[:I], gu[I:]
                silu = g * torch.sigmoid(g)
                h = silu * u
                dh = 1.1 * d[:I] * (u.abs() + d[I:]) + silu.abs() * d[I:] + 12 * U * h.abs()
                dw = 0.0 if e == self.E else math.expm1(2 * float(dl)) + 8 * U
                out[t] += p * (self.w2[e] @ h)
                hp = p * h.abs()
                err[t] += self.w2[e].abs() @ (p * dh * (1 + dw) + hp * (dw + BF16 * BF16))
                mags[t] += self.w2[e].abs() @ (hp + p * dh)
        n = len(chosen) * I
        err += (n + n / 64 + 16) * U * mags
        return out, err * 1.01 + BF16 * (out.abs() + err) + 1e-30


def _check(layer, T, padding=()):
    x = layer.rows(T)
    valid = torch.ones(T, dtype=torch.uint8)
    for t in padding:
        valid[t] = 0
        x[t] = float("nan")
    given = valid.cuda() if padding else None
    out = layer.dev.forward_few(x.cuda(), given)
    ref, tol = layer.reference(x, valid)
    got = out.double().cpu()
    off = (got - ref).abs()
    assert torch.isfinite(got).all()
    assert (off <= tol).all(), float((off / tol).max())
    for t in padding:
        assert (got[t] == 0).all()
    again = layer.dev.forward_few(x.cuda(), given)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    return x, out


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T, H, E, I, k, ns", [
    (1, 128, 4, 32, 1, 0),        # the smallest sizes
    (1, 128, 1, 32, 1, 1),        # one expert
    (1, 1024, 48, 96, 3, 0),
    (2, 256, 5, 64, 5, 1),        # every expert chosen
    (3, 384, 17, 160, 4, 0),
    (5, 2048, 33, 32, 16, 1),     # most experts a row
    (7, 4224, 8, 96, 2, 0),       # down blocks of 32 columns, I not of 64
    (16, 4224, 8, 64, 2, 1),
    (9, 1152, 256, 32, 8, 1),     # most segments
    (16, 2048, 24, 128, 3, 0),
    (16, 128, 2, 32, 2, 0),
    (3, 640, 64, 256, 8, 1),      # several units to a block's share, rows on chip
    (1, 16256, 3, 32, 2, 0),      # the longest row that is kept on chip
    (1, 16384, 3, 32, 2, 0),      # and the first that is not
])
def test_bf16(T, H, E, I, k, ns, packed):
    _check(Layer(T * 1000 + H, H, E, I, k, ns, packed=packed), T)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T, H, E, I, k, ns", [
    (1, 128, 4, 128, 2, 0),
    (1, 1024, 12, 256, 3, 1),
    (2, 4224, 6, 128, 2, 0),
    (6, 2176, 16, 128, 4, 1),
    (16, 640, 8, 256, 2, 1),
    (16, 4224, 4, 128, 1, 0),
    (3, 640, 64, 256, 8, 1),
    (1, 16256, 3, 128, 2, 0),
    (4, 384, 64, 128, 8, 1),
])
def test_fp8(T, H, E, I, k, ns, packed):
    _check(Layer(T * 1000 + H + 1, H, E, I, k, ns, fp8=True, packed=packed), T)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T, padding", [(1, (0,)), (2, (0,)), (5, (1, 4)), (16, (0, 3, 15)),
                                        (16, tuple(range(16))), (16, tuple(range(1, 16)))])
def test_padding_rows_are_not_read(T, padding, fp8):
    """Rows marked padding, here NaN: zeros in the output, no part in the
    others; also when nothing but padding is left."""
    layer = Layer(77 + T, 256, 6, 128, 2, 1, fp8=fp8)
    _check(layer, T, padding)


@pytest.mark.parametrize("T", [1, 4, 16])
def test_rows_of_nan_logits_are_nan_alone(T):
    """A NaN or an infinity in a row makes its logits NaN: that row is NaN, the
    others keep their values."""
    layer = Layer(5, 512, 12, 64, 3)
    x = layer.rows(T)
    for t, bad in ((T - 1, float("nan")), (T // 2, float("inf"))):
        y = x.clone()
        y[t, 17] = bad
        if bad == float("inf"):
            y[t, 18] = -bad       # both signs of infinity: no logit is a number
            layer.dev.router[:, 17] = layer.dev.router[:, 18] = 1
        out = layer.dev.forward_few(y.cuda()).double().cpu()
        assert torch.isnan(out[t]).all()
        assert torch.isfinite(out[torch.arange(T) != t]).all()


def test_equal_logits_take_the_lowest_experts():
    """Ties, by moe_route's rule; also all-zero rows, whose logits all tie."""
    layer = Layer(6, 256, 64, 32, 8)
    layer.dev.router[1::2] = layer.dev.router[::2]     # every logit twice
    x = layer.rows(6)
    x[2] = 0
    few = layer.dev.forward_few(x.cuda())
    ids, w, _ = layer.dev.route(x.cuda())
    assert ids[2].tolist() == list(range(8))
    # the formula on the routed experts
    for t in range(6):
        want = torch.zeros(256, dtype=torch.float64)
        mags = torch.zeros(256, dtype=torch.float64)
        for e, p in zip(ids[t].tolist(), w[t].double().tolist()):
            gu = layer.w13[e] @ x[t].double()
            h = gu[:32] * torch.sigmoid(gu[:32]) * gu[32:]
            want += p * (layer.w2[e] @ h)
            mags += p * (layer.w2[e].abs() @ h.abs())
        # 2^-16 of h' and some 600 roundings of 2^-24 of sums and logits
        tol = BF16 * want.abs() * 1.01 + 2.0 ** -12 * mags + 1e-30
        assert ((few[t].double().cpu() - want).abs() <= tol).all()


def test_matches_forward_on_rows_alone_and_together():
    """moe_forward, which keeps h in bf16: half a step of h and the output."""
    layer = Layer(8, 1024, 48, 96, 3, packed=True)
    x = layer.rows(16).cuda()
    whole = layer.dev.forward(x)
    mags = layer.reference(x.cpu(), [1] * 16)[0].abs().max()
    for T in (1, 2, 16):
        out = layer.dev.forward_few(x[:T].contiguous())
        # two output roundings and the rounding of h, whose sum of 96 x 3 terms
        # stays below the largest output times 8
        assert (out.double() - whole[:T].double()).abs().max() <= (2 + 8) * BF16 * mags


def test_output_and_workspace_stay_in_their_bounds():
    layer = Layer(9, 256, 6, 64, 2)
    for T in (1, 3, 16):
        x = layer.rows(T).cuda()
        n = moe.moe_few_workspace_size(layer.dev.desc(T), 2)
        ws = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")
        out = torch.full((T + 2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        layer.dev.forward_few(x, out=out[1:T + 1], workspace=ws[:n])
        assert (ws[n:] == 0xAB).all() and (out[0] == 7).all() and (out[T + 1] == 7).all()
        assert torch.equal(out[1:T + 1], layer.dev.forward_few(x))


@pytest.mark.parametrize("T", [1, 16])
def test_streams_at_once(T):
    """Calls on two streams, which run at the same time: each its workspace."""
    layer = Layer(10, 2048, 24, 128, 3, packed=True)
    xs = [layer.rows(T).cuda() for _ in range(2)]
    want = [layer.dev.forward_few(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            outs[i].append(layer.dev.forward_few(xs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


@pytest.mark.parametrize("T", [1, 5])
def test_two_graphs_of_a_layer(T):
    """Two captured graphs and eager calls of one layer, in turn, with new
    rows: each replay equals the eager call on the same rows."""
    layer = Layer(11, 1024, 12, 64, 3, 1)
    xs = [layer.rows(T).cuda() for _ in range(2)]
    outs = [torch.empty_like(x) for x in xs]
    layer.dev.forward_few(xs[0])
    graphs = []
    side = torch.cuda.Stream()
    for x, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer.dev.forward_few(x, out=o)
        graphs.append(g)
    for step in range(4):
        fresh = [layer.rows(T).cuda() for _ in range(2)]
        for x, f in zip(xs, fresh):
            x.copy_(f)
        for g in (graphs if step % 2 else graphs[::-1]):
            g.replay()
        eager = [layer.dev.forward_few(f) for f in fresh]
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)


def test_graph_captured_on_a_stream_given_by_name():
    """A capture on a stream that is passed along while it is not the current
    one: its workspace is not the one of eager calls there."""
    layer = Layer(13, 1024, 12, 64, 3)
    x = layer.rows(5).cuda()
    s = torch.cuda.Stream()
    want = layer.dev.forward_few(x)
    layer.dev.forward_few(x, stream=s)
    torch.cuda.synchronize()
    out = torch.empty_like(x)
    eager_ws = layer.dev.few_workspace(5, s).data_ptr()
    seen = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ws = layer.dev.few_workspace(5, s)
        seen.append(ws.data_ptr())
        layer.dev.forward_few(x, out=out, workspace=ws, stream=s)
    assert seen[0] != eager_ws
    for _ in range(3):
        out.zero_()
        graph.replay()
        other = layer.dev.forward_few(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)


def test_threads_on_one_stream():
    """Calls of one layer from several threads, all on one stream."""
    import threading
    layer = Layer(14, 1024, 24, 96, 3, packed=True)
    xs = [layer.rows(4).cuda() for _ in range(4)]
    want = [layer.dev.forward_few(x) for x in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]

    def work(i):
        for _ in range(50):
            got[i].append(layer.dev.forward_few(xs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert len(got[i]) == 50 and all(torch.equal(o, want[i]) for o in got[i])


def test_binding_call():
    """moe_forward_few as the C ABI has it: descriptor, weights, workspace."""
    layer = Layer(12, 256, 6, 64, 2, 1)
    d = layer.dev
    x = layer.rows(3).cuda()
    desc = d.desc(3)
    ws = moe.alloc_few_workspace(desc, 2)
    out = torch.empty_like(x)
    moe.moe_forward_few(desc, x, None, d.router, d.w13, d.w2, 2, out, ws)
    assert torch.equal(out, d.forward_few(x))
    with pytest.raises(moe.MoeError):
        moe.moe_forward_few(desc, x, None, d.router, d.w13, d.w2, 2, out, ws[:256])
    with pytest.raises(ValueError):
        d.forward_few(x.cpu())
    with pytest.raises(moe.MoeError):
        d.forward_few(torch.zeros(17, 256, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", ["bf16 nan", "bf16 inf", "fp8 nan", "fp8 scale inf", "fp8 scale nan"])
@pytest.mark.parametrize("T, H, I", [
    (2, 256, 128),       # on chip
    (5, 4224, 128),      # a down launch of 32 columns a block
    (16, 2048, 256),     # and one of 16
])
def test_weights_that_are_not_finite_stay_with_their_rows(T, H, I, kind, packed):
    """A down weight or scale of one expert that is NaN or infinite: rows that
    chose the expert take the formula's value in its columns, the others and
    padding rows what they had (to the rounding of a sum in any order)."""
    E, k, fp8 = 32, 3, kind.startswith("fp8")
    layer = Layer(300 + T, H, E, I, k, fp8=fp8)
    x = layer.rows(T)
    valid = torch.ones(T, dtype=torch.uint8)
    valid[T - 1] = 0
    picks = [set((layer.router.double() @ r.double()).topk(k).indices.tolist()) for r in x]
    chosen = [e for t in range(T - 1) for e in picks[t]]
    e = min(c for c in chosen if chosen.count(c) == 1)
    owner = next(t for t in range(T - 1) if e in picks[t])
    ref, tol = layer.reference(x, valid)
    xr = x[owner].double()
    g, u = (layer.w13[e] @ xr).split(I)
    h = g * torch.sigmoid(g) * u
    dev, n, c = layer.dev, 77, 21
    cols = slice(n, n + 1)
    want = torch.tensor(float("nan"))
    if kind == "bf16 nan":
        dev.w2[e, n, c] = float("nan")
    elif kind == "bf16 inf":
        dev.w2[e, n, c] = float("inf")
        want = torch.sign(h[c]) * float("inf")
    elif kind == "fp8 nan":
        dev.w2[e, n, c] = 0xFF
    else:
        dev.s2[e, 1, 0] = float(kind.split()[-1])
        cols = slice(128, 256)
    if packed:
        dev = moe.DeviceLayer(dev.router, dev.w13, dev.w2, k, 0, dev.s13, dev.s2, packed=True)
    x[T - 1] = float("nan")
    got = dev.forward_few(x.cuda(), valid.cuda()).double().cpu()
    inside = torch.zeros(T, H, dtype=torch.bool)
    inside[owner, cols] = True
    off = (got - ref).abs()
    assert (off <= tol)[~inside].all()
    assert (got[T - 1] == 0).all()
    bad = got[inside]
    if kind == "fp8 scale inf":
        # a block's sum of either sign, times infinity
        assert (~torch.isfinite(bad)).all()
    else:
        assert torch.equal(bad.isnan(), want.isnan().expand(bad.shape))
        assert want.isnan() or (bad == want).all()


def test_scales_put_in_place_after_a_call():
    layer = Layer(15, 512, 8, 128, 2, fp8=True)
    x = layer.rows(3).cuda()
    first = layer.dev.forward_few(x)
    layer.dev.s13, layer.dev.s2 = layer.dev.s13.clone(), 4 * layer.dev.s2
    assert torch.equal(layer.dev.forward_few(x), 4 * first)


@pytest.mark.parametrize("T, H, E, I, k, ns, fp8, packed", [
    # 32 columns a block: rings of 4, row-major of 3, of one or two 32-wide steps
    (16, 4224, 32, 256, 4, 0, False, True), (16, 4224, 32, 160, 4, 1, False, True),
    (16, 4224, 32, 256, 4, 0, False, False), (16, 4224, 40, 192, 4, 1, False, False),
    (16, 4224, 32, 160, 4, 0, False, False),
    (16, 4224, 32, 256, 4, 1, True, True), (16, 4224, 32, 384, 4, 0, True, False),
    # 16 columns a block: rings of 8, row-major and fp8 of 4
    (16, 1024, 64, 256, 4, 0, False, True), (13, 1152, 64, 160, 5, 1, False, True),
    (16, 1024, 64, 256, 4, 0, False, False), (16, 1024, 64, 224, 4, 0, False, False),
    (16, 1024, 64, 256, 4, 1, True, True), (13, 1152, 48, 384, 5, 0, True, False),
])
def test_down_launch_of_many_experts(T, H, E, I, k, ns, fp8, packed):
    """Every wave of the down launch goes round its ring and on into a part of a
    round, over several experts, whose columns end inside a round or at its end."""
    layer = Layer(T + H + I + k, H, E, I, k, ns, fp8=fp8, packed=packed)
    x, _ = _check(layer, T)
    chosen = (layer.router.double() @ x.double().T).topk(k, 0).indices.unique().numel() + ns
    wide = not fp8 and not packed and I % 64 == 0
    steps = chosen * I // (64 if fp8 or wide else 32)
    ring = (3 if H > 4096 else 4) if wide else 4 if fp8 or H > 4096 else 8
    assert steps // (12 if wide else 16) > ring


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T, H, I", [(1, 32640, 32768), (5, 32640, 32768), (3, 128, (1 << 23) - 128)])
def test_experts_of_the_largest_size(T, H, I, fp8, packed):
    """H I just below 2^30: offsets beyond 32 bits between experts and rows of h',
    and up to them inside an expert.  Only 64 columns of h', from the first to the
    last, are not zero; the reference has those (and zeros for 128 more, as for
    fp8 each is a block of its own, with two roundings beside the sum's)."""
    E, k = 3, 2
    g = torch.Generator().manual_seed(T + H)
    cols = torch.linspace(0, I - 1, 64).long()
    ref = Layer.__new__(Layer)
    ref.H, ref.E, ref.I, ref.k, ref.ns, ref.g = H, E, 192, k, 0, g
    ref.router = (torch.randn(E, H, generator=g) / math.sqrt(H)).bfloat16()
    ref.w13 = torch.zeros(E, 384, H, dtype=torch.float64)
    ref.w2 = torch.zeros(E, H, 192, dtype=torch.float64)
    dt = torch.uint8 if fp8 else torch.bfloat16
    w13 = torch.zeros(E, 2 * I, H, dtype=dt, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=dt, device="cuda")
    s13 = s2 = None
    if fp8:
        s13 = torch.rand(E, 2 * I // 128, H // 128, generator=g) / (100 * math.sqrt(H))
        s2 = torch.rand(E, H // 128, I // 128, generator=g) / 800
    for e in range(E):
        for half, first in ((0, 0), (192, I)):
            if fp8:
                w = _codes(g, 64, H)
                scale = s13[e, (first + cols) // 128].double().repeat_interleave(128, 1)
                ref.w13[e, half:half + 64] = w.view(torch.float8_e4m3fn).double() * scale
            else:
                w = (torch.randn(64, H, generator=g) / math.sqrt(H)).bfloat16()
                ref.w13[e, half:half + 64] = w.double()
            w13[e, (first + cols).cuda()] = w.cuda()
        if fp8:
            w = _codes(g, H, 64)
            scale = s2[e][:, cols // 128].double().repeat_interleave(128, 0)
            ref.w2[e, :, :64] = w.view(torch.float8_e4m3fn).double() * scale
        else:
            w = (torch.randn(H, 64, generator=g) / 8).bfloat16()
            ref.w2[e, :, :64] = w.double()
        w2[e, :, cols.cuda()] = w.cuda()
    ref.dev = moe.DeviceLayer(ref.router, w13, w2, k, 0, s13, s2, packed=packed)
    del w13, w2
    _check(ref, T)
    ref.dev = None
    torch.cuda.empty_cache()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", ["bf16 nan", "bf16 inf", "fp8 nan", "fp8 scale inf"])
@pytest.mark.parametrize("T, H, I", [(2, 256, 128), (5, 4224, 128), (16, 2048, 256)])
def test_gate_and_up_weights_that_are_not_finite_stay_with_their_rows(T, H, I, kind, packed):
    """The same of the first product: a row that chose the expert has an h' that is
    not a number, and with it no output that is finite; the others keep theirs."""
    E, k, fp8 = 32, 3, kind.startswith("fp8")
    layer = Layer(400 + T, H, E, I, k, fp8=fp8)
    x = layer.rows(T)
    valid = torch.ones(T, dtype=torch.uint8)
    valid[T - 1] = 0
    picks = [(layer.router.double() @ r.double()).topk(k).indices.tolist() for r in x]
    chosen = [e for t in range(T - 1) for e in picks[t]]
    e = min(c for c in chosen if chosen.count(c) == 1)
    owner = next(t for t in range(T - 1) if e in picks[t])
    ref, tol = layer.reference(x, valid)
    dev = layer.dev
    if kind == "fp8 scale inf":
        dev.s13[e, 0, 0] = float("inf")
    else:
        dev.w13[e, 5, 9] = {"bf16 nan": float("nan"), "bf16 inf": float("inf"), "fp8 nan": 0x7F}[kind]
    if packed:
        dev = moe.DeviceLayer(dev.router, dev.w13, dev.w2, k, 0, dev.s13, dev.s2, packed=True)
    x[T - 1] = float("nan")
    got = dev.forward_few(x.cuda(), valid.cuda()).double().cpu()
    others = torch.arange(T) != owner
    assert ((got - ref).abs() <= tol)[others].all() and (got[T - 1] == 0).all()
    if kind.endswith("nan"):
        assert got[owner].isnan().all()
    # SiLU(-inf) is NaN, SiLU(inf) infinite: times a weight, and 0 in fp8, never finite
    if kind == "fp8 scale inf" or (kind == "bf16 inf"):
        assert not torch.isfinite(got[owner]).any()
