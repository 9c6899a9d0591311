"""GPU tests of the 4-bit microscaled operators (quantisation, SiLU*mul
quantisation, values of codes, product) against their formulas in 64 bits.

Bounds (u = 2^-24 for fp32, half a step of bf16 2^-8):
  codes    a function of the input, equal bit by bit.
  values   exact.
  SiLU     v to 16 u (the exponential, a sum, a quotient, a product), so that a
           code lies between those of v (1 - 16 u) and v (1 + 16 u).
  product  S = sum of |a b| under their scales.  128 products at a time are exact
           but for one rounding of accumulator and sum together; up to 8 partial
           sums meet: ceil(K / 128) + 9 roundings of u of at most S.  bf16
           results: half a step of the result more."""
import pytest
import torch

import expert_layer_moe_amd as moe

pytestmark = pytest.mark.gpu
U, BF16 = 2.0 ** -24, 2.0 ** -8
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
MIDDLES = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _pack(codes):
    return codes[..., ::2] | codes[..., 1::2] << 4


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _quant64(x):
    """(codes [M, K], one to a byte, scale codes) of rows of 64-bit values."""
    M, K = x.shape
    wide = x.view(M, K // 32, 32)
    bad = ~torch.isfinite(wide).all(2)
    top = torch.where(bad, 1.0, wide.abs().nan_to_num(0, 0, 0).amax(2))
    # frexp: top = m 2^e with m in [1/2, 1)
    e = torch.where(top > 0, torch.frexp(top).exponent.long() - 3, -127).clamp(min=-127)
    q = torch.where(bad[..., None], 0.0, wide) / torch.exp2(e.double())[..., None]
    below = torch.searchsorted(MIDDLES, q.abs().contiguous())
    upto = torch.searchsorted(MIDDLES, q.abs().contiguous(), right=True)
    code = torch.where(upto % 2 == 0, upto, below)   # of a tie the even one
    code += 8 * torch.signbit(q).long()
    code[bad] = 0
    return code.view(M, K).to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def _values64(codes, scales):
    """64-bit values of packed codes under scale codes."""
    c = _unpack(codes).long()
    v = VALUES[c & 7] * (1.0 - 2.0 * (c >> 3).double())
    s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return v * s.repeat_interleave(32, 1)


def _rows(seed, M, K, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-12, 12, (M, K // 32), generator=g)
                                                   .float()).repeat_interleave(32, 1)
    return x.to(dtype)


def _check_quant(got, x):
    codes, scales = got
    want, want_s = _quant64(x.double())
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), _pack(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, K", [(1, 32), (1, 64), (3, 96), (2, 1024), (7, 4128), (129, 544), (1000, 32),
                                  (64, 7168), (1, 65536)])
def test_quant(M, K, dtype):
    x = _rows(M + K, M, K, dtype)
    _check_quant(moe.moe_quant_mxfp4(x.cuda()), x)


def test_every_bf16_value():
    """Each of the 65536, beside 31 zeros and beside a value of each exponent."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    x = torch.zeros(65536, 32, dtype=torch.bfloat16)
    x[:, 5] = every
    y = x.clone()
    # the block's largest: of the same exponent or up to 5 more
    size = every.float().abs()
    up = torch.exp2(torch.frexp(size).exponent.float() + torch.arange(65536) % 6)
    y[:, 17] = torch.where(torch.isfinite(up), up, 1.0).bfloat16()
    for v in (x, y, -y):
        _check_quant(moe.moe_quant_mxfp4(v.cuda()), v)


def test_ties_and_borders_in_fp32():
    """Midpoints of codes and their fp32 neighbours at scales over the whole
    range, the smallest ones below the normal numbers."""
    mid = torch.cat([MIDDLES, torch.tensor([0.0, 6, 7, 7.5], dtype=torch.float64)]).float()
    near = torch.cat([mid, torch.nextafter(mid, torch.tensor(9.0)),
                      torch.nextafter(mid, torch.tensor(-9.0))])
    near = torch.cat([near, near.new_tensor([4.0])])[:32]
    near = torch.nn.functional.pad(near, (0, 32 - near.numel()))
    near[31] = 7.9999995   # exponent 2, so that the scale is 1
    rows = torch.stack([near.double() * 2.0 ** e for e in range(-148, 126)]).float()
    rows = torch.cat([rows, -rows])
    _check_quant(moe.moe_quant_mxfp4(rows.cuda()), rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_that_are_not_finite(dtype):
    """NaN and infinities take their own block and no other."""
    x = _rows(3, 9, 256, dtype)
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"), -float("nan"))):
        x[2 * i, 32 * i + 7 * i] = bad
    codes, scales = moe.moe_quant_mxfp4(x.cuda())
    _check_quant((codes, scales), x)
    back = moe.moe_dequant_mxfp4(codes, scales).cpu()
    assert torch.equal(torch.isnan(back).view(9, 8, 32).all(2), scales.cpu() == 255)
    assert int(torch.isnan(back).sum()) == 4 * 32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_of_strided_rows(dtype):
    """Strides of input and outputs; gaps stay as they were, scales lie at an odd
    address."""
    x = _rows(4, 21, 352, dtype)
    wide = torch.full((21, 400), float("nan"), dtype=dtype, device="cuda")
    wide[:, 16:368] = x.cuda()
    codes = torch.full((23, 208), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((23, 17), 0x5B, dtype=torch.uint8, device="cuda")
    moe.moe_quant_mxfp4(wide[:, 16:368], codes[1:22, 16:192], scales[1:22, 3:14])
    _check_quant((codes[1:22, 16:192], scales[1:22, 3:14]), x)
    codes[1:22, 16:192] = 0x5A
    scales[1:22, 3:14] = 0x5B
    assert (codes == 0x5A).all() and (scales == 0x5B).all()


def _between(got, lo, hi):
    return (got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, I", [(1, 32), (5, 96), (33, 1056), (200, 2048), (17, 4128)])
def test_silu_mul_quant(M, I, dtype):
    g = torch.Generator().manual_seed(M + I)
    gu = (2.5 * torch.randn(M, 2 * I, generator=g)).to(dtype)
    codes, scales = moe.moe_silu_mul_quant_mxfp4(gu.cuda())
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    v = gate * torch.sigmoid(gate) * up
    lo, hi = v * (1 - 16 * U), v * (1 + 16 * U)
    (clo, slo), (chi, shi) = _quant64(lo), _quant64(hi)
    scales = scales.cpu()
    assert (_between(scales.int(), slo.int(), shi.int())).all()
    same = (slo == shi).repeat_interleave(32, 1)
    assert same.double().mean() > 0.99
    back = _values64(codes.cpu(), scales)
    inside = _between(back, _values64(_pack(clo), slo), _values64(_pack(chi), shi))
    assert inside[same].all()


def test_silu_of_far_gates():
    """Gates whose exponential is 0 or infinite: SiLU is the gate, or 0."""
    gu = torch.zeros(4, 128)
    gu[0, :64], gu[0, 64:] = 200.0, 3.0
    gu[1, :64], gu[1, 64:] = -200.0, 3.0
    gu[2, :64], gu[2, 64:] = float("-inf"), 1.0     # 0 / infinity aside: -inf / inf
    gu[3, 5] = float("nan")
    codes, scales = [t.cpu() for t in moe.moe_silu_mul_quant_mxfp4(gu.cuda())]
    back = _values64(codes, scales)
    assert (back[0] == 512.0).all()    # 600 = 4.6875 x 2^7, to 4 x 2^7
    assert (back[1] == 0).all()
    assert (scales[2] == 255).all() and (scales[3] == torch.tensor([255, 0])).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequant_of_every_code_under_every_scale(dtype):
    codes = torch.randint(0, 256, (256, 16 * 24), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(1))
    codes[:, :16] = _pack(torch.arange(16).repeat(2).to(torch.uint8))
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 24)
    got = moe.moe_dequant_mxfp4(codes.cuda(), scales.cuda(), out_dtype=dtype).cpu()
    want = _values64(codes, scales).to(dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and int(nan.sum()) == 24 * 32
    assert torch.equal(got[~nan], want[~nan])
    assert torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))


@pytest.mark.parametrize("M, K", [(1, 32), (3, 96), (129, 544), (64, 7168)])
def test_dequant_of_strided_rows(M, K):
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 256, (M, K // 2 + 16), generator=g, dtype=torch.uint8).cuda()[:, 16:]
    scales = torch.randint(90, 160, (M, K // 32 + 5), generator=g, dtype=torch.uint8).cuda()[:, 5:]
    big = torch.full((M + 2, K + 24), 7.0, device="cuda")
    out = big[1:M + 1, 8:K + 8]
    assert moe.moe_dequant_mxfp4(codes, scales.view(torch.float8_e8m0fnu), out=out) is out
    assert torch.equal(out.double().cpu(), _values64(codes.cpu(), scales.cpu()))
    big[1:M + 1, 8:K + 8] = 7.0
    assert (big == 7.0).all()


# ---- product ---------------------------------------------------------------------
def _operands(seed, M, N, K, spread=6):
    g = torch.Generator().manual_seed(seed)
    u8 = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8)  # noqa: E731
    return (u8(0, 256, M, K // 2), u8(127 - spread, 128 + spread, M, K // 32),
            u8(0, 256, N, K // 2), u8(127 - spread, 128 + spread, N, K // 32))


def _check_product(out, a, sa, b, sb):
    K = 2 * a.shape[1]
    a64, b64 = _values64(a, sa), _values64(b, sb)
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    tol = (-(-K // 128) + 9) * U * mag
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + BF16) + BF16 * ref.abs()
    off = (out.double().cpu() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


SIZES = [(1, 1, 32), (1, 16, 128), (1, 130, 288), (2, 127, 1024), (15, 129, 800), (16, 128, 2048),
         (17, 1, 544), (31, 65, 256), (33, 1001, 1312), (64, 64, 224), (65, 257, 1152),
         (100, 384, 1056), (129, 640, 512), (257, 255, 1824), (300, 2048, 256), (1000, 520, 736),
         (2049, 130, 160), (520, 4100, 288), (16, 4096, 96), (1, 600, 7200), (40, 1000, 2080),
         (4096, 4090, 544), (3000, 4096, 1056), (16, 1040, 16384), (5, 33, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", SIZES)
def test_product(M, N, K, dtype):
    a, sa, b, sb = _operands(M * 7 + N * 3 + K, M, N, K)
    args = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    out = moe.moe_gemm_mxfp4(*args, out_dtype=dtype)
    _check_product(out, a, sa, b, sb)
    assert torch.equal(out, moe.moe_gemm_mxfp4(*args, out_dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, N, K", [(3, 50, 544), (70, 131, 800), (260, 300, 256), (300, 1000, 1120)])
def test_product_of_strided_rows(M, N, K, dtype):
    """Row strides of every operand (those of the scales odd); the gaps of the
    output and the rows around it stay as they were, also at an odd first column."""
    a, sa, b, sb = _operands(1, M, N, K)
    wide = lambda t, pad, value: torch.cat([t, t.new_full((t.shape[0], pad), value)], 1).cuda()[:, :t.shape[1]]  # noqa: E731
    big = torch.full((M + 2, N + 9), 5.0, dtype=dtype, device="cuda")
    out = big[1:M + 1, 3:N + 3]
    moe.moe_gemm_mxfp4(wide(a, 48, 0x77), wide(sa, 3 - sa.shape[1] % 2, 255), wide(b, 16, 0x77),
                       wide(sb, 5, 255).view(torch.float8_e8m0fnu), out=out)
    _check_product(out, a, sa, b, sb)
    big[1:M + 1, 3:N + 3] = 5.0
    assert (big == 5.0).all()


@pytest.mark.parametrize("M, N, K", [(1, 70, 160), (16, 130, 1056), (60, 300, 544), (200, 256, 512),
                                     (700, 4096, 288)])
def test_nan_scales_stay_in_their_rows(M, N, K):
    a, sa, b, sb = [t.cuda() for t in _operands(2, M, N, K)]
    want = moe.moe_gemm_mxfp4(a, sa, b, sb)
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[M // 2, K // 32 - 1] = 255
    sb2[7, 0] = 255
    got = moe.moe_gemm_mxfp4(a, sa2, b, sb2)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[M // 2], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("M", [4, 100, 600])
def test_product_of_largest_codes_and_far_scales(M):
    """6 x 6 in every place; scales 2^-100 to 2^100 whose products meet, and some
    that cancel all but small terms."""
    N, K = 300, 1024
    a, b = torch.full((M, K // 2), 0x77, dtype=torch.uint8), torch.full((N, K // 2), 0x77, dtype=torch.uint8)
    sa = torch.tensor([27, 227, 127, 140] * 8, dtype=torch.uint8).repeat(M, 1)
    sb = torch.tensor([227, 27, 130, 101] * 8, dtype=torch.uint8).repeat(N, 1)
    b[:, 300:] |= 0x88   # negative from there on
    for dtype in (torch.float32, torch.bfloat16):
        out = moe.moe_gemm_mxfp4(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
        _check_product(out, a, sa, b, sb)


def test_rows_behind_each_other_have_the_bits_of_a_smaller_call():
    """Rows of one call do not change with the others' values."""
    a, sa, b, sb = [t.cuda() for t in _operands(5, 300, 512, 1024)]
    want = moe.moe_gemm_mxfp4(a, sa, b, sb)
    a2 = torch.flip(a, [0]).clone()
    a2[100] = a[100]
    sa2 = torch.flip(sa, [0]).clone()
    sa2[100] = sa[100]
    assert torch.equal(moe.moe_gemm_mxfp4(a2, sa2, b, sb)[100], want[100])


@pytest.mark.parametrize("kernel, M, N, K", [
    # K ends inside a line of 256 values (of 1, 1, 3 and 7 blocks left), with odd and even
    # numbers of lines, up to several turns of the ring; rows and columns end inside a tile
    ("rows 16", 3, 200, 5152), ("rows 16", 37, 1001, 8160), ("rows 16", 17, 130, 16416),
    ("tile 16 x 32", 17, 8200, 1312), ("tile 16 x 32", 20, 6000, 2080), ("tile 16 x 32", 37, 3000, 16416),
    ("tile 16 x 32", 70, 3000, 864), ("tile 16 x 32", 16, 13000, 4320),
    ("tile 32 x 64", 100, 4090, 864), ("tile 32 x 64", 200, 2100, 2080), ("tile 32 x 64", 100, 4090, 16416),
    ("tile 64 x 64", 520, 4090, 800), ("tile 64 x 64", 65, 6000, 2080), ("tile 64 x 64", 130, 4090, 8224),
    ("tile 64 x 128", 260, 6000, 2080), ("tile 64 x 128", 130, 8200, 4320), ("tile 64 x 128", 260, 4090, 16416),
    ("tile 64 x 128", 700, 6000, 800),
    ("tile 128 x 128", 1000, 8200, 288), ("tile 128 x 128", 2050, 4090, 800), ("tile 128 x 128", 2050, 2100, 1504),
    ("tile 128 x 128", 2050, 4090, 8224),
    ("tile 128 x 128 of 8 waves", 1000, 4090, 96), ("tile 128 x 128 of 8 waves", 1300, 2050, 800),
    ("tile 128 x 128 of 8 waves", 520, 6000, 2272), ("tile 128 x 128 of 8 waves", 1000, 4090, 8416),
    ("tile 128 x 256", 520, 13000, 2080), ("tile 128 x 256", 1000, 6000, 4320), ("tile 128 x 256", 330, 20000, 16416),
    ("tile 256 x 256", 3900, 4090, 4128), ("tile 256 x 256", 8000, 8100, 2080), ("tile 256 x 256", 2000, 8190, 8416),
])
def test_product_by_every_kernel_over_long_k(kernel, M, N, K):
    assert moe.moe_gemm_mxfp4_kernel(M, N, K) == kernel
    a, sa, b, sb = [t.cuda() for t in _operands(M + N + K, M, N, K)]
    values = lambda codes, scales: moe.moe_dequant_mxfp4(codes, scales, out_dtype=torch.float32).double()  # noqa: E731
    a64, b64 = values(a, sa), values(b, sb)
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    for dtype in (torch.float32, torch.bfloat16):
        tol = (-(-K // 128) + 9) * U * mag
        if dtype == torch.bfloat16:
            tol = tol * (1 + BF16) + BF16 * ref.abs()
        out = moe.moe_gemm_mxfp4(a, sa, b, sb, out_dtype=dtype)
        off = (out.double() - ref).abs()
        assert (off <= tol).all(), float((off / tol).max())
        for _ in range(3):
            assert torch.equal(out, moe.moe_gemm_mxfp4(a, sa, b, sb, out_dtype=dtype))


def test_the_kernels_over_long_k_are_all_there_are():
    """Every kernel that some sizes take is among those above."""
    tested = {case[0] for case in test_product_by_every_kernel_over_long_k.pytestmark[0].args[1]}
    sizes = [int(2 ** (i / 3)) for i in range(43)]
    taken = {moe.moe_gemm_mxfp4_kernel(M, N, K) for M in sizes for N in sizes
             for K in (32, 256, 1024, 2080, 8192, 65536)}
    assert taken == tested


@pytest.mark.parametrize("M, N, K", [(40, 40, 544), (300, 260, 544)])
def test_product_of_the_widest_rows(M, N, K):
    """Code rows 2^23 bytes apart, scale rows and results as far: every tile's last row
    lies up to 2 GB behind its first."""
    a, sa, b, sb = _operands(11, M, N, K)
    wide = lambda t: torch.empty(t.shape[0], 1 << 23, dtype=t.dtype, device="cuda")[:, :t.shape[1]].copy_(t)  # noqa: E731
    out = torch.full((M, 1 << 23), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_gemm_mxfp4(wide(a), wide(sa), wide(b), wide(sb), out=out[:, 3:N + 3])
    _check_product(out[:, 3:N + 3], a, sa, b, sb)
    assert (out[:, :3] == 5.0).all() and (out[:, N + 3:N + 40] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_silu_of_zeros_keeps_their_signs(dtype):
    """SiLU(-0) = -0: the codes of zeros of either sign, by ups of either sign, beside a
    value and among themselves."""
    gu = torch.zeros(4, 128, dtype=dtype)
    gu[:, 0:64:3] = -0.0
    gu[:, 64:] = torch.where(torch.arange(64) % 2 == 0, 2.0, -2.0).to(dtype)
    gu[2:, 5] = 1.0
    want, want_s = _quant64((gu[:, :64] * gu[:, 64:]).double())
    want[2:, 5], want_s[2:, 0] = 7 + 8, 127 - 2   # -2 SiLU(1) = -1.46: -5.8 under 1/4, code -6
    codes, scales = moe.moe_silu_mul_quant_mxfp4(gu.cuda())
    assert torch.equal(scales.cpu(), want_s) and torch.equal(codes.cpu(), _pack(want))


def test_quant_and_values_of_rows_far_apart():
    """Rows 2^28 values, and codes and scales 2^28 bytes apart: the last one lies 2^31
    values and 2^32 bytes behind."""
    M, K = 17, 96
    x = _rows(3, M, K, torch.bfloat16)
    gu = torch.cat([x, x.flip(1)], 1)
    want, want_s = moe.moe_quant_mxfp4(x.cuda())
    silu, silu_s = moe.moe_silu_mul_quant_mxfp4(gu.cuda())
    big = torch.empty(M, 1 << 28, dtype=torch.bfloat16, device="cuda")
    bytes_ = torch.empty(M, 1 << 28, dtype=torch.uint8, device="cuda")
    vx, vg, vo = big[:, 8:8 + K], big[:, 1024:1024 + 2 * K], big[:, 2048:2048 + K]
    vx.copy_(x)
    vg.copy_(gu)
    vc, vs = bytes_[:, 16:16 + K // 2], bytes_[:, 1001:1001 + K // 32]
    moe.moe_quant_mxfp4(vx, codes=vc, scales=vs)
    assert torch.equal(vc, want) and torch.equal(vs, want_s)
    moe.moe_dequant_mxfp4(vc, vs, out=vo)
    assert torch.equal(vo.double().cpu(), _values64(want.cpu(), want_s.cpu()))
    moe.moe_silu_mul_quant_mxfp4(vg, codes=vc, scales=vs)
    assert torch.equal(vc, silu) and torch.equal(vs, silu_s)


def test_more_blocks_than_a_grid_takes_at_once():
    """2^31 + 2^20 values to codes and 2^32 + 2^20 back: the workgroups take a second turn."""
    K = 1 << 20
    x = _rows(4, 1, K, torch.bfloat16).cuda()
    want, want_s = moe.moe_quant_mxfp4(x)
    codes, scales = moe.moe_quant_mxfp4(x.expand(2049, K).contiguous())
    assert torch.equal(scales, want_s.expand(2049, -1)) and (codes == want).all()
    del codes, scales
    out = moe.moe_dequant_mxfp4(want.expand(4097, -1).contiguous(), want_s.expand(4097, -1).contiguous())
    one = moe.moe_dequant_mxfp4(want, want_s)
    assert all(torch.equal(part, one.expand_as(part)) for part in out.split(512))


@pytest.mark.parametrize("M, N, K", [(5, 40, 800), (70, 131, 800), (300, 300, 1120)])
def test_product_with_scales_at_odd_addresses(M, N, K):
    a, sa, b, sb = _operands(6, M, N, K)
    odd = lambda t: torch.cat([t.new_full((t.shape[0], 1), 255), t], 1).cuda()[:, 1:]  # noqa: E731
    out = moe.moe_gemm_mxfp4(a.cuda(), odd(sa), b.cuda(), odd(sb), out_dtype=torch.float32)
    _check_product(out, a, sa, b, sb)


def test_empty_matrices_are_refused():
    e = lambda *shape: torch.empty(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *shape: torch.empty(shape, device="cuda")  # noqa: E731
    for call in (lambda: moe.moe_quant_mxfp4(f(0, 64)), lambda: moe.moe_quant_mxfp4(f(3, 0)),
                 lambda: moe.moe_silu_mul_quant_mxfp4(f(0, 64)), lambda: moe.moe_dequant_mxfp4(e(0, 16), e(0, 1)),
                 lambda: moe.moe_gemm_mxfp4(e(0, 16), e(0, 1), e(4, 16), e(4, 1)),
                 lambda: moe.moe_gemm_mxfp4(e(4, 16), e(4, 1), e(0, 16), e(0, 1)),
                 lambda: moe.moe_gemm_mxfp4(e(4, 0), e(4, 0), e(4, 0), e(4, 0)),
                 lambda: moe.moe_add_rms_norm(f(0, 64), None, f(64)),
                 lambda: moe.moe_add_rms_norm_quant_fp8(f(2, 0), None, f(0))):
        with pytest.raises(moe.MoeError, match="INVALID_ARG"):
            call()
    # (and codes that are not 16-byte aligned)
    with pytest.raises(moe.MoeError, match="INVALID_ARG"):
        moe.moe_gemm_mxfp4(e(4, 32)[:, 8:24], e(4, 1), e(4, 16), e(4, 1))


@pytest.mark.parametrize("M, N", [((1 << 26) + 40, 3), (5, (1 << 26) + 40)])
def test_product_of_more_blocks_than_a_grid_is_wide(M, N):
    """Rows that repeat every 1000: so do their results."""
    a, sa, b, sb = [t.cuda() for t in _operands(8, min(M, 1000), min(N, 1000), 32)]
    want = moe.moe_gemm_mxfp4(a, sa, b, sb)
    # (torch's indexing fills 40 rows alone of 2^26 + 40)
    wide = lambda t, n: t.repeat(-(-n // t.shape[0]), 1)[:n] if n > 1000 else t  # noqa: E731
    args = wide(a, M), wide(sa, M), wide(b, N), wide(sb, N)
    at = max(M, N) // 1000 * 1000 - 1000
    assert torch.equal(args[0][at:at + 1000], a) if M > N else torch.equal(args[2][at:at + 1000], b)
    out = moe.moe_gemm_mxfp4(*args)
    for i in range(0, max(M, N) - 1000, 1000 * 1000):
        part = out[i:i + 1000] if M > N else out[:, i:i + 1000]
        assert torch.equal(part, want)
    last = max(M, N) // 1000 * 1000
    assert torch.equal(out[last:] if M > N else out[:, last:],
                       want[:M - last] if M > N else want[:, :N - last])


@pytest.mark.parametrize("M, N", [(2, 3), (100, 300)])
def test_product_over_a_million_values(M, N):
    K = 1 << 20
    a, sa, b, sb = [t.cuda() for t in _operands(9, M, N, K)]
    values = lambda codes, scales: moe.moe_dequant_mxfp4(codes, scales, out_dtype=torch.float32).double()  # noqa: E731
    a64, b64 = values(a, sa), values(b, sb)
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    out = moe.moe_gemm_mxfp4(a, sa, b, sb, out_dtype=torch.float32)
    assert ((out.double() - ref).abs() <= (-(-K // 128) + 9) * U * mag).all()


def test_given_results_of_every_type():
    """uint8 or the float8 types, the results of each other's bits."""
    x = _rows(2, 9, 192, torch.bfloat16).cuda()
    e8m0, e4m3 = torch.float8_e8m0fnu, torch.float8_e4m3fn
    codes, scales = moe.moe_quant_mxfp4(x)
    given = torch.empty(9, 6, dtype=torch.uint8, device="cuda").view(e8m0)
    got = moe.moe_quant_mxfp4(x, scales=given)
    assert got[1] is given and torch.equal(given.view(torch.uint8), scales) and torch.equal(got[0], codes)
    out = moe.moe_gemm_mxfp4(codes, scales.view(e8m0), codes, scales)
    assert torch.equal(out, moe.moe_gemm_mxfp4(codes, scales, codes, given))
    silu, silu_s = moe.moe_silu_mul_quant_mxfp4(x[:, :128])
    given = torch.empty(9, 2, dtype=torch.uint8, device="cuda").view(e8m0)
    assert moe.moe_silu_mul_quant_mxfp4(x[:, :128], codes=silu.clone(), scales=given)[1] is given
    assert torch.equal(given.view(torch.uint8), silu_s)
    w = torch.ones(192, dtype=torch.bfloat16, device="cuda")
    c8, s8, _ = moe.moe_add_rms_norm_quant_fp8(x, None, w)
    given = torch.empty(9, 192, dtype=torch.uint8, device="cuda").view(e4m3)
    got = moe.moe_add_rms_norm_quant_fp8(x, None, w, codes=given, scales=torch.empty_like(s8))
    assert got[0] is given and torch.equal(given.view(torch.uint8), c8) and torch.equal(got[1], s8)


def _near(seed, M, N, K, base_a, base_b, few):
    """Codes at random, or few and far apart ones, under scale codes of which no two products
    lie more than 2^12 apart."""
    g = torch.Generator().manual_seed(seed)
    u8 = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8)  # noqa: E731

    def codes(n):
        if not few:
            return u8(0, 256, n, K // 2)
        of = torch.tensor([1, 7, 9, 15], dtype=torch.uint8)[u8(0, 4, n, K).int()]   # 0.5, 6 and negative
        return _pack(torch.where(torch.rand(n, K, generator=g) < 0.3, of, 0))
    return codes(M), u8(base_a, base_a + 7, M, K // 32), codes(N), u8(base_b, base_b + 7, N, K // 32)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("base_a, base_b", [(123, 124), (0, 247), (247, 0), (1, 244), (0, 127), (0, 116), (248, 40)])
@pytest.mark.parametrize("kernel, M, N, K", [
    ("rows 16", 40, 60, 32), ("rows 16", 33, 520, 128), ("tile 16 x 32", 260, 520, 128),
    ("tile 64 x 64", 700, 1000, 96), ("tile 64 x 128", 2000, 2050, 128), ("tile 128 x 128", 2050, 2050, 128),
    ("tile 128 x 128 of 8 waves", 3900, 1000, 128), ("tile 256 x 256", 3900, 3000, 128)])
def test_four_blocks_of_near_scales_are_rounded_once(kernel, M, N, K, base_a, base_b, few):
    """Up to 128 products whose scales lie within 2^12: the nearest fp32 to the exact sum, bit
    by bit, also where scale codes are the smallest and largest and results below the normal
    numbers.  (Sums of 128 products of 4 bits over 2^12 have 28 bits: exact in 64.)"""
    assert moe.moe_gemm_mxfp4_kernel(M, N, K) == kernel
    a, sa, b, sb = _near(M + base_a, M, N, K, base_a, base_b, few)
    out = moe.moe_gemm_mxfp4(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=torch.float32)
    want = (_values64(a, sa) @ _values64(b, sb).T).float()
    assert torch.isfinite(want).all() and (want != 0).any()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("spread", [2, 7, 12, 20, 45])
@pytest.mark.parametrize("kernel, M, N, K", [("rows 16", 17, 130, 128), ("rows 16", 17, 130, 2080),
                                             ("tile 16 x 32", 260, 520, 128), ("tile 64 x 64", 520, 1000, 544)])
def test_products_of_far_scales(kernel, M, N, K, spread):
    """Scales of a row up to 2^(2 spread) apart, and pairs of blocks that cancel.  A step of four
    blocks: two roundings of u of at most S = sum of |a b|, and 8 u of the step's own part of S
    for what small blocks lose beside large ones: 8 u S in all; and the joining."""
    assert moe.moe_gemm_mxfp4_kernel(M, N, K) == kernel
    a, sa, b, sb = _operands(M + K + spread, M, N, K, spread)
    half = K // 64   # (of the blocks, the last `half` cancel the first, of every second row of b)
    a[:, 16 * half:32 * half], sa[:, half:2 * half] = a[:, :16 * half], sa[:, :half]
    b[::2, 16 * half:32 * half], sb[::2, half:2 * half] = b[::2, :16 * half] ^ 0x88, sb[::2, :half]
    a, sa, b, sb = [t.cuda() for t in (a, sa, b, sb)]
    values = lambda codes, scales: moe.moe_dequant_mxfp4(codes, scales, out_dtype=torch.float32).double()  # noqa: E731
    a64, b64 = values(a, sa), values(b, sb)
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    tol = (2 * -(-K // 128) + 8 + 9) * U * mag
    out = moe.moe_gemm_mxfp4(a, sa, b, sb, out_dtype=torch.float32)
    off = (out.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())


def _gates():
    """Every bf16 value from 2^-20 to 85 in size, of either sign, fp32 ones among them, and those
    from -85 to where the exponential ends, -88.7."""
    g = torch.Generator().manual_seed(12)
    every = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).float()
    every = every[(every.abs() >= 2.0 ** -20) & (every.abs() <= 85)]
    size = torch.exp2(26.4 * torch.rand(1 << 17, generator=g) - 20)
    far = -85 - 3.7 * torch.rand(1 << 13, generator=g)
    return torch.cat([every, size * (1 - 2 * torch.randint(0, 2, size.shape, generator=g)), far])


def test_silu_to_the_last_bit():
    """SiLU as the formula has it, g / (1 + exp(-g)), each rounded: ups that take it to middles
    between codes, so that one step of its last bit shows.  A gate's block: a value of 7, so
    that the scale is 1, and four middles at seven neighbouring ups."""
    g = _gates()
    dev = g.cuda()
    silu = (dev / (1 + torch.exp(-dev))).cpu()
    # (the 8-bit operator divides: its scale is the block's largest over 448)
    rows = torch.zeros(g.numel(), 256)
    rows[:, 0], rows[:, 128] = g, 1.0
    _, scale = moe.moe_silu_mul_quant_fp8(rows.cuda())
    assert torch.equal(scale.cpu()[:, 0], silu.abs().clamp(min=1e-12) / torch.full_like(silu, 448.0))

    gu = torch.zeros(g.numel(), 64)
    gu[:, :32], gu[:, 32:] = g[:, None], 0.0
    gu[:, 0], gu[:, 32] = 100.0, 0.07
    at = 33
    for middle in (0.25, 0.75, 1.25, 1.75):
        up = (middle / silu.double()).float()
        for step in range(-3, 4):
            gu[:, at] = (up.view(torch.int32) + step).view(torch.float32)
            at += 1

    def codes_of(s):
        v = s[:, None] * gu[:, 32:]
        v[:, 0] = torch.tensor(100.0) * gu[0, 32]
        return _quant64(v.double())
    want, want_s = codes_of(silu)
    assert (want_s == 127).all()
    for step in (-1, 1):   # a last bit off shows in nearly every block
        off, _ = codes_of((silu.view(torch.int32) + step).view(torch.float32))
        assert (off != want).any(1).double().mean() > 0.9
    codes, scales = moe.moe_silu_mul_quant_mxfp4(gu.cuda())
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), _pack(want))


TILES = [("tile 16 x 32", 260, 520, 544), ("tile 32 x 64", 520, 520, 2080), ("tile 64 x 64", 520, 1000, 544),
         ("tile 64 x 128", 1300, 1000, 2080), ("tile 128 x 128 of 8 waves", 1000, 2050, 1056),
         ("tile 128 x 128", 2000, 2050, 544), ("tile 128 x 256", 2000, 2050, 4128),
         ("tile 256 x 256", 3900, 3000, 544)]


def _check_on_gpu(out, a, sa, b, sb):
    K = 2 * a.shape[1]
    a64, b64 = [moe.moe_dequant_mxfp4(c.contiguous(), s.contiguous(), out_dtype=torch.float32).double()
                for c, s in ((a, sa), (b, sb))]
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    assert ((out.double() - ref).abs() <= (-(-K // 128) + 9) * U * mag).all()


@pytest.mark.parametrize("kernel, M, N, K", TILES)
def test_every_tile_of_the_widest_rows(kernel, M, N, K):
    """Code rows 2^23 bytes apart, the most there may be, with other codes between them: a
    tile of 256 rows spans 2^31 bytes.  The last tiles are not full."""
    assert moe.moe_gemm_mxfp4_kernel(M, N, K) == kernel
    a, sa, b, sb = [t.cuda() for t in _operands(M + N, M, N, K)]

    def wide(t):
        big = torch.full((t.shape[0], 1 << 23), 0x77, dtype=torch.uint8, device="cuda")
        big[:, :t.shape[1]].copy_(t)
        return big[:, :t.shape[1]]
    out = moe.moe_gemm_mxfp4(wide(a), sa, wide(b), sb, out_dtype=torch.float32)
    _check_on_gpu(out, a, sa, b, sb)


@pytest.mark.parametrize("kernel, M, N, K", TILES)
def test_every_tile_with_scales_at_odd_addresses(kernel, M, N, K):
    assert moe.moe_gemm_mxfp4_kernel(M, N, K) == kernel
    a, sa, b, sb = [t.cuda() for t in _operands(M + N + 1, M, N, K)]
    odd = lambda t, by: torch.cat([t.new_full((t.shape[0], by), 255), t], 1)[:, by:]  # noqa: E731
    wide = lambda t: torch.cat([t, t.new_full((t.shape[0], 48), 0x77)], 1)[:, :t.shape[1]]  # noqa: E731
    out = moe.moe_gemm_mxfp4(wide(a), odd(sa, 1), wide(b), odd(sb, 3 - sb.shape[1] % 2), out_dtype=torch.float32)
    _check_on_gpu(out, a, sa, b, sb)
