"""GPU tests of the fp8 block-scale product, the token quantisations and the
dense layer made of them, against their formulas in 64 bits.

Bounds (u = 2^-24 for fp32, half a step of bf16 2^-8, of e4m3 2^-4):
  product  S = sum over blocks of sa sb sum |a b|.  fp32 results: products of
           codes are exact, K + 2 ceil(K / 128) + 8 roundings of u of at most S.
           bf16 results: half a step of the result, plus 2^-12 S for the fp8
           matrix unit, which lines the 128 products of a block up to the
           largest and keeps no less than 12 bits below it.
  codes    a function of the input, equal bit by bit: the quotients are
           rounded to fp32 and then to e4m3.
  SiLU     v to 16 u, so that a code may be the other neighbour of a tie:
           half a step of e4m3 and of its smallest values (2^-10 scale), plus
           that much of v and of the scale."""
import math

import pytest
import torch

import expert_layer_moe_amd as moe

pytestmark = pytest.mark.gpu
U, BF16, E4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _blocks(n):
    return (n + 127) // 128


def _codes(gen, *shape):
    c = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
    return torch.where(c % 128 == 127, c - 1, c)


def _operands(seed, M, N, K):
    g = torch.Generator().manual_seed(seed)
    return (_codes(g, M, K), torch.rand(M, _blocks(K), generator=g) + 0.01, _codes(g, N, K),
            torch.rand(_blocks(N), _blocks(K), generator=g) + 0.01)


def _product(a, sa, b, sb):
    """(product, sum of magnitudes) in 64 bits."""
    N, K = b.shape
    a64 = a.view(F8).double() * sa.double().repeat_interleave(128, 1)[:, :K]
    b64 = b.view(F8).double() * sb.double().repeat_interleave(128, 0)[:N] \
        .repeat_interleave(128, 1)[:, :K]
    return a64 @ b64.T, a64.abs() @ b64.abs().T


def _check_product(out, a, sa, b, sb):
    K = a.shape[1]
    ref, mag = _product(a, sa, b, sb)
    if out.dtype == torch.float32:
        tol = (K + 2 * _blocks(K) + 8) * U * mag
    else:
        tol = BF16 * ref.abs() + (1 + BF16) * 2.0 ** -12 * mag
    off = (out.double().cpu() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", [
    (1, 1, 16), (1, 16, 128), (1, 130, 144), (2, 127, 1024), (15, 129, 400), (16, 128, 2048),
    (17, 1, 272), (31, 65, 128), (33, 1001, 656), (64, 64, 112), (65, 257, 1152),
    (100, 384, 1040), (129, 640, 512), (257, 255, 912), (300, 2048, 256), (1000, 520, 368),
    (2049, 130, 160), (520, 4100, 144),
    (4096, 4090, 272),            # the largest tiles
    (16, 9000, 2064), (1, 600, 2320), (40, 1000, 1040),
])
def test_product(M, N, K, dtype):
    a, sa, b, sb = _operands(M * 7 + N * 3 + K, M, N, K)
    out = moe.moe_gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
    _check_product(out, a, sa, b, sb)
    again = moe.moe_gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", [(3, 50, 272), (70, 131, 400), (260, 300, 128)])
def test_product_of_strided_rows(M, N, K, dtype):
    """Row strides of every operand; the gaps of the output and the rows
    around it stay as they were, also at an odd first column."""
    a, sa, b, sb = _operands(1, M, N, K)
    wide = lambda t, pad: torch.cat([t, t.new_full((t.shape[0], pad), 126 if t.dtype == torch.uint8  # noqa: E731
                                                   else float("nan"))], 1).cuda()[:, :t.shape[1]]
    big = torch.full((M + 2, N + 9), 5.0, dtype=dtype, device="cuda")
    out = big[1:M + 1, 3:N + 3]
    moe.moe_gemm_fp8(wide(a, 48), wide(sa, 3), wide(b, 16), sb.cuda(), out=out)
    _check_product(out, a, sa, b, sb)
    big[1:M + 1, 3:N + 3] = 5.0
    assert (big == 5.0).all()


def test_product_rows_do_not_depend_on_each_other():
    a, sa, b, sb = [t.cuda() for t in _operands(2, 200, 256, 512)]
    want = moe.moe_gemm_fp8(a, sa, b, sb)
    a2 = a.clone()
    a2[100] = 0x7F   # NaN
    got = moe.moe_gemm_fp8(a2, sa, b, sb)
    assert torch.isnan(got[100]).all()
    keep = torch.arange(200, device="cuda") != 100
    assert torch.equal(got[keep], want[keep])
    b2 = b.clone()
    b2[7, 300] = 0xFF
    got = moe.moe_gemm_fp8(a, sa, b2, sb)
    assert torch.isnan(got[:, 7]).all()
    keep = torch.arange(256, device="cuda") != 7
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_largest_codes_and_scales(dtype):
    """448 x 448 in every place, scales far apart from block to block."""
    M, N, K = 40, 80, 640
    a, b = torch.full((M, K), 0x7E, dtype=torch.uint8), torch.full((N, K), 0xFE, dtype=torch.uint8)
    sa = torch.tensor([2.0 ** e for e in (0, 20, -20, 3, 10)]).repeat(M, 1)
    sb = torch.tensor([2.0 ** e for e in (0, 5, 30, -9, 1)]).repeat(1, 1)
    out = moe.moe_gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
    _check_product(out, a, sa, b, sb)


def _quant64(x):
    """Codes and scales of the definition: quotients rounded to fp32 (from 64
    bits, which rounds a quotient of fp32 values once), then to e4m3."""
    M, K = x.shape
    nb = _blocks(K)
    wide = torch.nn.functional.pad(x.double(), (0, nb * 128 - K)).view(M, nb, 128)
    tiny = torch.tensor(1e-12, dtype=torch.float32).double()
    scale = (torch.maximum(wide.abs().amax(2), tiny) / 448).float()
    q = (wide / scale.double()[..., None]).float().to(F8).view(torch.uint8)
    return q.view(M, nb * 128)[:, :K], scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, K", [(1, 16), (1, 128), (2, 144), (7, 112), (33, 1040), (16, 2048),
                                  (300, 256), (5, 4080)])
def test_quantisation(M, K, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(4 * torch.randn(M, K, generator=g))).to(dtype)
    codes, scales = moe.moe_quant_fp8(x.cuda())
    want, scale = _quant64(x)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(codes.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantisation_of_every_bf16(dtype):
    """All finite bf16 values below 2^120, a block each with a value of 448
    times a power of two near it: ties and subnormal codes among them."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[bits.float().abs() < 2.0 ** 120]
    bits = bits[: bits.numel() // 112 * 112].view(-1, 112)
    top = bits.float().abs().amax(1).clamp(min=2.0 ** -100)
    x = torch.cat([bits.float(), (448 * torch.exp2(torch.floor(torch.log2(top)) - 8))[:, None]
                   .expand(-1, 16)], 1).to(dtype)
    codes, scales = moe.moe_quant_fp8(x.cuda())
    want, scale = _quant64(x.float())
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(codes.cpu(), want)


def test_quantisation_of_special_values():
    """Zeros (also negative ones), tiny blocks, NaN and infinities."""
    x = torch.zeros(6, 256)
    x[1, ::2] = -0.0
    x[2] = 1e-30
    x[3] = torch.linspace(-3, 3, 256)
    x[3, 5] = float("nan")
    x[4] = torch.linspace(-3, 3, 256)
    x[4, 200] = float("-inf")
    x[5] = 3e38
    codes, scales = [t.cpu() for t in moe.moe_quant_fp8(x.cuda())]
    clean = x.clone()
    clean[3, 5] = 0
    want, scale = _quant64(clean)
    for t in (0, 1, 2, 5):
        assert torch.equal(codes[t], want[t]) and torch.equal(scales[t], scale[t]), t
    assert codes[3, 5] % 128 == 127
    keep = torch.arange(256) != 5
    assert torch.equal(codes[3][keep], want[3][keep]) and torch.equal(scales[3], scale[3])
    assert torch.equal(codes[4, :128], want[4, :128]) and scales[4, 0] == scale[4, 0]
    assert scales[4, 1] == float("inf") and codes[4, 200] % 128 == 127
    assert (codes[4, 128:][torch.arange(128) != 72] % 128 == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, I", [(1, 16), (2, 128), (33, 1040), (9, 272), (257, 384)])
def test_silu_mul_quantisation(M, I, dtype):
    g = torch.Generator().manual_seed(M * I)
    gu = (4 * torch.randn(M, 2 * I, generator=g)).to(dtype)
    codes, scales = moe.moe_silu_mul_quant_fp8(gu.cuda())
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    v = gate * torch.sigmoid(gate) * up
    _, scale = _quant64(v)
    assert ((scales.cpu().double() - scale.double()).abs() <= 20 * U * scale.double()).all()
    wide = scales.cpu().double().repeat_interleave(128, 1)[:, :I]
    back = codes.cpu().view(F8).double() * wide
    assert ((back - v).abs() <= (E4M3 + 20 * U) * v.abs() + (2.0 ** -10 + 20 * U) * wide).all()


def test_silu_of_large_and_special_gates():
    """Gates where exp overflows either way, times an up value of 1."""
    gate = torch.tensor([0.0, -0.0, 1e-20, 30.0, 88.0, 104.0, 1e30, -1.0, -20.0, -88.0, -104.0,
                         -1e30, 3e38, -3e38, 2.0, -2.0])
    gu = torch.cat([gate, torch.ones(16)])[None].contiguous()
    for i in range(16):
        one = gu.clone()
        one[0, :16] = 0
        one[0, i] = gate[i]
        codes, scales = moe.moe_silu_mul_quant_fp8(one.cuda())
        v = float(gate[i].double() * torch.sigmoid(gate[i].double()))
        back = float(codes.cpu().view(F8).double()[0, i] * scales.cpu().double())
        top = max(abs(v), 1e-12)
        assert abs(float(scales) - top / 448) <= 20 * U * top / 448, i
        assert abs(back - v) <= (E4M3 + 20 * U) * abs(v) + 2.0 ** -10 * top / 448, i
        assert (codes.cpu()[0][torch.arange(16) != i] % 128 == 0).all()
    for bad in ((float("nan"), 1.0), (float("-inf"), 1.0), (1.0, float("nan"))):
        one = gu.clone()
        one[0, :16] = 1.0
        one[0, 3], one[0, 19] = bad
        codes, scales = moe.moe_silu_mul_quant_fp8(one.cuda())
        assert codes[0, 3] % 128 == 127 and torch.isfinite(scales).all()
        assert (codes[0][torch.arange(16) != 3] == 0x7E).all()


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantisation_of_strided_rows(silu, dtype):
    M, K = 37, 400
    g = torch.Generator().manual_seed(3)
    n = K * (2 if silu else 1)
    x = torch.full((M, n + 24), float("nan"), dtype=dtype)
    x[:, :n] = torch.randn(M, n, generator=g).to(dtype)
    x = x.cuda()[:, :n]
    fn = moe.moe_silu_mul_quant_fp8 if silu else moe.moe_quant_fp8
    want = fn(x.contiguous())
    codes = torch.full((M + 2, K + 32), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((M + 2, 4 + 5), 9.0, device="cuda")
    fn(x, codes=codes[1:M + 1, 16:K + 16], scales=scales[1:M + 1, 2:6])
    assert torch.equal(codes[1:M + 1, 16:K + 16], want[0])
    assert torch.equal(scales[1:M + 1, 2:6], want[1])
    codes[1:M + 1, 16:K + 16] = 9
    scales[1:M + 1, 2:6] = 9.0
    assert (codes == 9).all() and (scales == 9.0).all()


def test_refuses_misaligned_tensors():
    """First elements off 16 bytes: refused by the library, nothing written."""
    a = torch.zeros(4 * 128 + 8, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, 1, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_gemm_fp8(a[8:].view(4, 128), s, a[:-8].view(4, 128), s[:1])
    x = torch.zeros(4 * 128 + 4, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_quant_fp8(x[2:-2].view(4, 128))
    with pytest.raises(ValueError):
        moe.moe_quant_fp8(x[:512].view(4, 128), codes=torch.empty(4, 128, dtype=torch.uint8))


def _dense(seed, H, I):
    g = torch.Generator().manual_seed(seed)
    w13, w2 = _codes(g, 2 * I, H), _codes(g, H, I)
    s13 = (torch.rand(_blocks(2 * I), _blocks(H), generator=g) + 0.5) / (100 * math.sqrt(H))
    s2 = (torch.rand(_blocks(H), _blocks(I), generator=g) + 0.5) / (100 * math.sqrt(I))
    return (w13, w2, s13, s2), g


@pytest.mark.parametrize("T, H, I", [(1, 256, 128), (3, 400, 208), (16, 1024, 384),
                                     (130, 512, 656)])
def test_dense_layer(T, H, I):
    """The four operators in a row, and the layer's formula without any
    rounding.  Each quantisation rounds by at most 2^-4, uniformly: 2^-4 /
    sqrt(3) = 3.6 % of the root mean square; the first one enters SiLU(g) u
    through both g and u, in all sqrt((2 x 3.6)^2 + 3.6^2) = 8 %, and gu's bf16
    and the output's add 0.3 %."""
    weights, g = _dense(T + H, H, I)
    dense = moe.DenseFP8(*weights)
    x = torch.randn(T, H, generator=g).bfloat16()
    out = dense.forward(x.cuda())
    a, sa = moe.moe_quant_fp8(x.cuda())
    gu = moe.moe_gemm_fp8(a, sa, dense.w13, dense.s13)
    h, sh = moe.moe_silu_mul_quant_fp8(gu)
    assert torch.equal(out, moe.moe_gemm_fp8(h, sh, dense.w2, dense.s2))
    w13, w2, s13, s2 = weights
    wide = lambda w, s: w.view(F8).double() * s.double().repeat_interleave(128, 0)[:w.shape[0]] \
        .repeat_interleave(128, 1)[:, :w.shape[1]]  # noqa: E731
    p = x.double() @ wide(w13, s13).T
    ref = (p[:, :I] * torch.sigmoid(p[:, :I]) * p[:, I:]) @ wide(w2, s2).T
    rel = ((out.double().cpu() - ref).norm() / ref.norm()).item()
    assert rel <= 0.085, rel


def test_decoder_stack_in_a_graph():
    """A decoder's feed-forward parts together: a dense block, then an expert
    layer on the rows in hand, captured in one graph and replayed with new rows
    between eager calls on the same stream and another one."""
    H, I, E, k, T = 512, 384, 12, 3, 4
    weights, g = _dense(4, H, I)
    dense = moe.DenseFP8(*weights)
    router = torch.randn(E, H, generator=g).bfloat16() / math.sqrt(H)
    w13 = _codes(g, E, 256, H)
    w2 = _codes(g, E, H, 128)
    s13 = torch.rand(E, 2, H // 128, generator=g) / (100 * math.sqrt(H))
    s2 = torch.rand(E, H // 128, 1, generator=g) / (100 * math.sqrt(128))
    layer = moe.DeviceLayer(router, w13, w2, k, 0, s13, s2, packed=True)

    def step(x):
        y = x + dense.forward(x)
        return y + layer.forward_few(y)

    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    step(x)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out = step(x)
    other = torch.cuda.Stream()
    for _ in range(5):
        fresh = torch.randn(T, H, generator=g).bfloat16().cuda()
        x.copy_(fresh)
        graph.replay()
        eager = step(fresh)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            there = step(fresh)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(there, eager)


def test_calls_on_another_stream():
    """`stream` given, results allocated there."""
    a, sa, b, sb = [t.cuda() for t in _operands(8, 70, 256, 512)]
    want = moe.moe_gemm_fp8(a, sa, b, sb)
    x = torch.randn(70, 512, device="cuda")
    wq = moe.moe_quant_fp8(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        out = moe.moe_gemm_fp8(a, sa, b, sb, stream=s)
        q = moe.moe_quant_fp8(x, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(q[0], wq[0]) and torch.equal(q[1], wq[1])


@pytest.mark.parametrize("lo, hi", [(-40, -8), (-8, 0), (0, 8), (8, 40), (-1e-3, 1e-3)])
def test_silu_in_fp32(lo, hi):
    """A scale is its block's largest v / 448: one gate a block, an up value of
    2^40, and SiLU shows in it.  exp to one unit in the last place (2 u), 1 + exp,
    the quotient and the one by 448 (u each): 5 u, and products of them."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 1 << 22
    gate = lo + (hi - lo) * torch.rand(n, generator=g, device="cuda")
    gu = torch.zeros(n, 32, device="cuda")
    gu[:, 0], gu[:, 16] = gate, 2.0 ** 40
    _, scales = moe.moe_silu_mul_quant_fp8(gu)
    want = (gate.double() * torch.sigmoid(gate.double())).abs() * 2.0 ** 40 / 448
    off = (scales[:, 0].double() - want).abs() / want.clamp(min=1e-300)
    assert off.max().item() <= 5 * U * (1 + 10 * U)


@pytest.mark.parametrize("T, H, I", [(3, 400, 208), (130, 512, 656)])
def test_dense_layer_with_its_gate_up_product_in_fp32(T, H, I):
    weights, g = _dense(T * H, H, I)
    dense = moe.DenseFP8(*weights, gate_up=torch.float32)
    x = torch.randn(T, H, generator=g).cuda()
    a, sa = moe.moe_quant_fp8(x)
    gu = moe.moe_gemm_fp8(a, sa, dense.w13, dense.s13, out_dtype=torch.float32)
    _check_product(gu, a.cpu(), sa.cpu(), *[w.cpu() for w in (dense.w13, dense.s13)])
    h, sh = moe.moe_silu_mul_quant_fp8(gu)
    want = moe.moe_gemm_fp8(h, sh, dense.w2, dense.s2, out_dtype=torch.float32)
    assert torch.equal(dense.forward(x, out=torch.empty_like(x)), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", [(16, 48, 384), (200, 256, 640)])
@pytest.mark.parametrize("cancel", [False, True])
def test_product_of_few_large_codes_among_small_ones(M, N, K, cancel, dtype):
    """In every eight codes of K one of 256, the others' products near 2^-13 of
    its: bf16 results lose up to 2^-13 of each eight's largest product for each of
    the other seven (and the roundings of fp32, and half a step); fp32 results
    nothing of that.  CANCEL: the large ones cancel."""
    g = torch.Generator().manual_seed(M + K)
    small = lambda rows, e: (1 + torch.randint(0, 8, (rows, K), generator=g) / 8) * 2.0 ** e  # noqa: E731
    a, b = small(M, 1), small(N, 1)
    a[:, ::8] = b[:, ::8] = 256
    if cancel:
        b[:, 8::16] = -256
    a, b = [t.to(F8).view(torch.uint8) for t in (a, b)]
    sa, sb = torch.ones(M, _blocks(K)), torch.ones(_blocks(N), _blocks(K))
    out = moe.moe_gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
    ref, mag = _product(a, sa, b, sb)
    tol = (K + 2 * _blocks(K) + 8) * U * mag
    if dtype == torch.bfloat16:
        tol = tol + K // 8 * 7 * 2.0 ** -13 * 65536
        tol = BF16 * (ref.abs() + tol) + tol
    assert ((out.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("M, N", [
    (1, (1 << 27) + 3),     # blocks of 512 threads for 16 columns
    (1 << 30, 1),           # the most rows: 2^24 tiles of 64 rows
])
def test_product_of_more_blocks_than_a_grid_dimension_holds(M, N):
    """Operands that repeat every 1024 rows: so must the result."""
    K, P = 16, 1024
    a, sa, b, sb = _operands(6, min(M, P), min(N, P), K)
    repeat = lambda t, n, p: t.cuda().repeat((n + p - 1) // p, 1)[:n]  # noqa: E731
    blocks = sb[:, :1].repeat(8, 1)[:8]   # 128 columns each
    out = moe.moe_gemm_fp8(repeat(a, M, P), repeat(sa, M, P), repeat(b, N, P),
                           repeat(blocks, _blocks(N), 8))
    first = out[:P, :P].clone()
    _check_product(first, a, sa, b, blocks[:_blocks(min(N, P))])
    flat, first = out.view(-1), first.view(-1)
    whole = flat.numel() // P * P
    assert torch.equal(flat[:whole].view(-1, P), first.expand(whole // P, P))
    assert torch.equal(flat[whole:], first[:flat.numel() - whole])


def test_quantisation_of_the_longest_row():
    """One row of 2^31 - 16 values, which repeat every 2048."""
    n, P = (1 << 31) - 16, 2048
    base = torch.randn(1, P, generator=torch.Generator().manual_seed(9)).bfloat16()
    want, scale = _quant64(base)
    end, end_scale = _quant64(base[:, :n % P])   # its last block has 112 values
    codes, scales = moe.moe_quant_fp8(base.cuda().repeat(1, (n + P - 1) // P)[:, :n])
    want, scale = want.cuda(), scale.cuda()
    whole = n // P * P
    assert torch.equal(codes[0, :whole].view(-1, P), want.expand(whole // P, P))
    assert torch.equal(codes[0, whole:].cpu(), end[0])
    assert torch.equal(scales[0, :-16].view(-1, 16), scale.expand(n // P, 16))
    assert torch.equal(scales[0, -16:].cpu(), end_scale[0])


B, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kernel, M, N, K, dtypes", [
    # waves of 5 or 6, 8, 4 or 5 K blocks; weights that one block reads, or several
    ("rows 16", 3, 200, 5136, (B, F)), ("rows 16", 16, 4100, 8176, (B, F)),
    ("rows 16", 20, 100, 4240, (B, F)), ("rows 16", 37, 1001, 5136, (B, F)),
    ("rows 32", 24, 4096, 4368, (B, F)), ("rows 32", 17, 3000, 5008, (B, F)),
    ("rows 32", 64, 2000, 5136, (B, F)), ("rows 32", 65, 2000, 5008, (F,)),
    # 9, 16, 17 or 18 and 33 K blocks: two stages of scales and more, odd ends of
    # two-block stages, several turns of the ring; columns and K that end inside
    ("tile 64 x 32", 33, 3000, 1040, (B, F)), ("tile 64 x 32", 65, 3000, 1936, (B, F)),
    ("tile 64 x 32", 33, 3000, 2064, (B, F)), ("tile 64 x 32", 33, 4090, 4112, (B, F)),
    ("tile 64 x 64", 65, 6000, 1040, (B, F)), ("tile 64 x 64", 70, 6000, 1936, (B, F)),
    ("tile 64 x 64", 130, 3000, 2192, (B, F)), ("tile 64 x 64", 130, 3000, 4112, (B, F)),
    ("tile 64 x 128", 130, 6000, 1040, (B,)), ("tile 64 x 128", 130, 6000, 1936, (B,)),
    ("tile 64 x 128", 130, 6000, 2064, (B,)), ("tile 64 x 128", 150, 5900, 4112, (B,)),
    ("tile 128 x 128", 1000, 2050, 1040, (B, F)), ("tile 128 x 128", 1000, 2050, 1936, (B, F)),
    ("tile 128 x 128", 1000, 2050, 2064, (B, F)), ("tile 128 x 128", 520, 3900, 4112, (B, F)),
    ("tile 128 x 256", 2050, 2050, 1040, (B, F)), ("tile 128 x 256", 2050, 2050, 1936, (B, F)),
    ("tile 128 x 256", 2050, 2050, 2064, (B, F)), ("tile 128 x 256", 1000, 4100, 4112, (B, F)),
    ("tile 256 x 256", 2050, 4090, 1040, (B,)), ("tile 256 x 256", 2050, 4090, 1936, (B,)),
    ("tile 256 x 256", 2050, 4090, 2064, (B,)), ("tile 256 x 256", 4000, 2100, 4112, (B,)),
])
def test_product_by_every_kernel_over_long_k(kernel, M, N, K, dtypes):
    """Scales that differ by powers of two from block to block, and bounds of the
    formula: fp32 as in _check_product; bf16 half a step, and of each eight
    products seven times 2^-13 of the largest (at most the product of the largest
    codes), beside the fp32 roundings."""
    a, sa, b, sb = [t.cuda() for t in _operands(M + N + K, M, N, K)]
    sa *= torch.exp2(torch.arange(_blocks(K), device="cuda") % 5 - 2.0)
    sb *= torch.exp2(torch.arange(_blocks(K), device="cuda") % 3 - 1.0)
    nb = _blocks(K)
    a64 = a.view(F8).double() * sa.double().repeat_interleave(128, 1)[:, :K]
    b64 = b.view(F8).double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    eights = lambda t: t.abs().view(t.shape[0], K // 8, 8).amax(2)  # noqa: E731
    for dtype in dtypes:
        assert moe.moe_gemm_fp8_kernel(M, N, K, dtype) == kernel
        tol = (K + 2 * nb + 8) * U * mag
        if dtype == torch.bfloat16:
            tol = tol + 7 * 2.0 ** -13 * (eights(a64) @ eights(b64).T)
            tol = BF16 * (ref.abs() + tol) + tol
        out = moe.moe_gemm_fp8(a, sa, b, sb, out_dtype=dtype)
        off = (out.double() - ref).abs()
        assert (off <= tol).all(), float((off / tol).max())
        for _ in range(3):
            assert torch.equal(out, moe.moe_gemm_fp8(a, sa, b, sb, out_dtype=dtype))


def test_the_kernels_over_long_k_are_all_there_are():
    """Every kernel that some sizes take is among those above."""
    tested = {(case[0], d) for case in
              test_product_by_every_kernel_over_long_k.pytestmark[0].args[1] for d in case[4]}
    sizes = [int(2 ** (i / 3)) for i in range(43)]
    taken = {(moe.moe_gemm_fp8_kernel(M, N, K, d), d) for d in (B, F) for M in sizes for N in sizes
             for K in (16, 128, 1024, 2048, 8192, 65536)}
    assert taken == tested


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", [(40, 40, 272), (300, 260, 272)])
def test_product_of_the_widest_rows(M, N, K, dtype):
    """Strides at their limits, 2^23 bytes and 2^21 scales, and results 2^23
    values apart: every tile's last row lies 2 GB behind its first."""
    a, sa, b, sb = _operands(11, M, N, K)
    wide = lambda t, ld: torch.empty(t.shape[0], ld, dtype=t.dtype, device="cuda")[:, :t.shape[1]].copy_(t)  # noqa: E731
    out = torch.full((M, 1 << 23), 5.0, dtype=dtype, device="cuda")
    moe.moe_gemm_fp8(wide(a, 1 << 23), wide(sa, 1 << 21), wide(b, 1 << 23), sb.cuda(), out=out[:, 3:N + 3])
    _check_product(out[:, 3:N + 3].clone(), a, sa, b, sb)
    assert (out[:, :3] == 5).all() and (out[:, N + 3:] == 5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_more_results_than_32_bits_address(dtype):
    """Operands that repeat every 1024 rows: so must the result, both ways."""
    M, N, K, P = 66 * 1024, 33 * 1024, 16, 1024
    a, sa, b, sb = [t.cuda() for t in _operands(12, P, P, K)]
    out = moe.moe_gemm_fp8(a.repeat(66, 1), sa.repeat(66, 1), b.repeat(33, 1), sb.repeat(33, 1),
                           out_dtype=dtype)
    first = out[:P, :P].clone()
    _check_product(first, *[t.cpu() for t in (a, sa, b, sb)])
    for m in range(66):
        assert torch.equal(out[m * P:(m + 1) * P].view(P, 33, P), first[:, None].expand(P, 33, P)), m


@pytest.mark.parametrize("silu", [False, True])
def test_quantisation_of_rows_far_apart(silu):
    """Rows of the input 2^29 values apart, of the codes 2^30 and of the scales
    2^28: 4 GB between the first and the last."""
    M, K = 5, 272
    n = K * (2 if silu else 1)
    fn = moe.moe_silu_mul_quant_fp8 if silu else moe.moe_quant_fp8
    x = torch.empty(M, 1 << 29, dtype=torch.bfloat16, device="cuda")[:, :n]
    x.copy_(torch.randn(M, n, generator=torch.Generator().manual_seed(13)))
    want = fn(x.contiguous())
    codes = torch.empty(M, 1 << 30, dtype=torch.uint8, device="cuda")[:, :K]
    scales = torch.empty(M, 1 << 28, device="cuda")[:, :3]
    fn(x, codes=codes, scales=scales)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
