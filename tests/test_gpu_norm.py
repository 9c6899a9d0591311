"""GPU tests of the root-mean-square norm with the residual's addition, as
floats and as fp8 codes, against its formula in 64 bits.

Bounds (u = 2^-24 for fp32, half a step of bf16 2^-8, of e4m3 2^-4):
  r     a function of its two inputs, equal bit by bit.
  out   a row's sum of squares is made of at most 32 values in a lane, six steps
        across lanes and 16 across waves, all positive: 55 u, half of that in the
        root; mean, eps, root, quotient and two products: 6 u.  34 u of the value,
        and half a step of its type.
  scale 34 u and two roundings: 36 u.
  codes those of a value and a scale so far off: half a step of e4m3 and of its
        smallest values (2^-10 scale), plus that."""
import pytest
import torch

import expert_layer_moe_amd as moe

pytestmark = pytest.mark.gpu
U, BF16, E4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
F8 = torch.float8_e4m3fn
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _inputs(seed, M, H, x_type, res_type, w_type):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(M, H) * torch.exp2(torch.randint(-9, 9, (M, 1), generator=g).float())).to(x_type)
    res = None if res_type is None else (3 * n(M, H)).to(res_type)
    return x, res, (1 + 0.3 * n(H)).to(w_type)


def _norm64(x, res, w, eps):
    r = x.float() if res is None else (x.float() + res.float()).to(res.dtype)
    r64 = r.double()
    return r, r64 / torch.sqrt(r64.square().mean(1, keepdim=True) + eps) * w.double()


def _check_out(out, want):
    half = BF16 if out.dtype == B else U
    tol = want.abs() * (34 * U * (1 + half) + half)
    off = (out.double().cpu() - want).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


def _check_codes(codes, scales, want):
    M, H = want.shape
    nb = -(-H // 128)
    wide = torch.nn.functional.pad(want, (0, nb * 128 - H)).view(M, nb, 128)
    scale = wide.abs().amax(2).clamp(min=1e-12) / 448
    assert ((scales.double().cpu() - scale).abs() <= 36 * U * scale).all()
    wide_scale = scale.repeat_interleave(128, 1)[:, :H]
    got = codes.view(F8).double().cpu() * wide_scale
    tol = (E4M3 + 72 * U) * want.abs() * (1 + 36 * U) + 2.0 ** -10 * wide_scale
    off = (got - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


SIZES = [(1, 16), (1, 64), (3, 144), (2, 512), (5, 528), (33, 1040), (7, 2048), (4, 2064), (37, 5136),
         (9, 7168), (3, 8192), (2, 8208), (3, 16384), (2, 20000), (2, 32768), (700, 256)]
TYPES = [(B, B, B, B), (F, F, F, F), (B, None, B, B), (F, None, F, F), (B, F, F, B), (F, B, B, F),
         (B, F, B, F), (F, None, B, B)]


@pytest.mark.parametrize("M, H", SIZES)
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v).replace("torch.", "") for v in t))
def test_norm(M, H, types):
    xt, rt, wt, ot = types
    x, res, w = _inputs(M + H, M, H, xt, rt, wt)
    r, want = _norm64(x, res, w, 1e-6)
    dev = [None if t is None else t.cuda() for t in (x, res, w)]
    out, kept = moe.moe_add_rms_norm(*dev, eps=1e-6, out_dtype=ot)
    assert out.dtype == ot
    _check_out(out, want)
    assert (kept is None) == (rt is None)
    if kept is not None:
        assert kept.dtype == rt and torch.equal(kept.cpu(), r)
        assert torch.equal(dev[1].cpu(), res)
    codes, scales, kept2 = moe.moe_add_rms_norm_quant_fp8(*dev, eps=1e-6)
    _check_codes(codes, scales, want)
    if kept is not None:
        assert torch.equal(kept2, kept)
    # beside codes, the same floats; and the same codes
    out2 = torch.empty_like(out)
    again = moe.moe_add_rms_norm_quant_fp8(*dev, eps=1e-6, out=out2)
    assert torch.equal(out2, out) and torch.equal(again[0], codes) and torch.equal(again[1], scales)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("H", [48, 1296, 7168])
def test_codes_are_the_quantisation_of_the_fp32_norm(dtype, H):
    """Bit for bit what moe_quant_fp8 makes of the fp32 result."""
    x, res, w = [t.cuda() for t in _inputs(1, 40, H, dtype, dtype, dtype)]
    out, _ = moe.moe_add_rms_norm(x, res, w, out_dtype=F)
    codes, scales, _ = moe.moe_add_rms_norm_quant_fp8(x, res, w)
    want, want_s = moe.moe_quant_fp8(out)
    assert torch.equal(codes, want) and torch.equal(scales, want_s)


@pytest.mark.parametrize("dtype", [B, F])
def test_in_place(dtype):
    """residual_out may be residual and out may be x."""
    x, res, w = [t.cuda() for t in _inputs(2, 50, 1040, dtype, dtype, dtype)]
    want, kept = moe.moe_add_rms_norm(x, res, w, out_dtype=dtype)
    x2, res2 = x.clone(), res.clone()
    got = moe.moe_add_rms_norm(x2, res2, w, out=x2, residual_out=res2)
    assert got[0] is x2 and got[1] is res2
    assert torch.equal(x2, want) and torch.equal(res2, kept)


@pytest.mark.parametrize("xt, rt, ot", [(B, B, B), (F, F, F), (B, F, F)])
def test_strided_rows(xt, rt, ot):
    """Strides of all arrays; gaps and neighbouring rows stay as they were."""
    M, H = 19, 400
    x, res, w = _inputs(3, M, H, xt, rt, B)
    r, want = _norm64(x, res, w, 1e-5)

    def wide(t, dtype, fill):
        big = torch.full((M + 2, H + 48), fill, dtype=dtype, device="cuda")
        view = big[1:M + 1, 16:H + 16]
        if t is not None:
            view.copy_(t.cuda())
        return big, view
    bx, vx = wide(x, xt, float("nan"))
    br, vr = wide(res, rt, float("nan"))
    bk, vk = wide(None, rt, 3.0)
    bo, vo = wide(None, ot, 4.0)
    bc, vc = wide(None, torch.uint8, 9)
    bs = torch.full((M + 2, 7), 5.0, device="cuda")
    vs = bs[1:M + 1, 2:6]
    moe.moe_add_rms_norm_quant_fp8(vx, vr, w.cuda(), eps=1e-5, codes=vc, scales=vs, residual_out=vk, out=vo)
    assert torch.equal(vk.cpu(), r)
    _check_out(vo, want)
    _check_codes(vc, vs, want)
    for big, view, fill in ((bk, vk, 3.0), (bo, vo, 4.0), (bc, vc, 9), (bs, vs, 5.0)):
        view.fill_(fill)
        assert (big == fill).all()


def test_rows_that_are_not_finite_stay_alone():
    x, _, w = _inputs(4, 8, 640, F, None, F)
    want, _ = moe.moe_add_rms_norm(x.cuda(), None, w.cuda(), out_dtype=F)
    x[2, 100], x[5, 3] = float("nan"), float("inf")
    x[6] = 0.0
    x[7] = 2.0 ** 100
    got, _ = moe.moe_add_rms_norm(x.cuda(), None, w.cuda(), out_dtype=F)
    assert torch.isnan(got[2]).all()
    assert torch.isnan(got[5, 3]) and int(torch.isnan(got[5]).sum()) == 1 and int((got[5] == 0).sum()) == 639
    assert (got[6] == 0).all() and (got[7] == 0).all()
    keep = torch.tensor([0, 1, 3, 4])
    assert torch.equal(got[keep], want[keep])
    codes, scales, _ = moe.moe_add_rms_norm_quant_fp8(x.cuda(), None, w.cuda())
    assert torch.isnan(codes[2].view(F8).float()).all() and torch.isfinite(scales).all()
    assert (codes[6] == 0).all()


def test_a_row_of_zeros_without_eps_is_nan():
    x = torch.zeros(2, 32, device="cuda")
    x[1] = 1.0
    out, _ = moe.moe_add_rms_norm(x, None, torch.ones(32, device="cuda"), eps=0.0, out_dtype=F)
    assert torch.isnan(out[0]).all() and (out[1] == 1).all()


def test_rows_do_not_depend_on_how_many():
    x, res, w = [t.cuda() for t in _inputs(6, 600, 2064, B, B, B)]
    all_rows, _ = moe.moe_add_rms_norm(x, res, w)
    for i in (0, 7, 599):
        one, _ = moe.moe_add_rms_norm(x[i:i + 1], res[i:i + 1], w)
        assert torch.equal(one[0], all_rows[i])


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("H", [16, 528, 1296, 5136, 8208, 16400, 32752])
def test_in_place_where_rows_end_inside_a_wave(dtype, H):
    """Lanes behind a row's end read its last values, which others may have replaced."""
    x, res, w = [t.cuda() for t in _inputs(H, 300, H, dtype, dtype, dtype)]
    want, kept = moe.moe_add_rms_norm(x, res, w, out_dtype=dtype)
    codes, scales, _ = moe.moe_add_rms_norm_quant_fp8(x, res, w)
    for _ in range(3):
        x2, res2 = x.clone(), res.clone()
        got_c, got_s, got_r = moe.moe_add_rms_norm_quant_fp8(x2, res2, w, residual_out=res2, out=x2)
        assert got_r is res2 and torch.equal(x2, want) and torch.equal(res2, kept)
        assert torch.equal(got_c, codes) and torch.equal(got_s, scales)


def test_more_rows_than_blocks():
    M = (1 << 20) + 3
    x, res, w = [t.cuda() for t in _inputs(7, 1000, 16, B, B, B)]
    want, kept = moe.moe_add_rms_norm(x, res, w)
    at = torch.arange(M, device="cuda") % 1000
    out, r = moe.moe_add_rms_norm(x[at], res[at], w)
    assert torch.equal(out, want[at]) and torch.equal(r, kept[at])


def test_rows_far_apart():
    """Rows 2^28 values apart: the last one lies 2^31 values and 2^32 bytes behind."""
    M, H = 9, 400
    x, res, w = [t.cuda() for t in _inputs(8, M, H, B, B, F)]
    want = moe.moe_add_rms_norm_quant_fp8(x, res, w, out=(want_out := torch.empty_like(x)))
    big = torch.empty(M, 1 << 28, dtype=B, device="cuda")
    vx, vr, vk, vo = [big[:, 1024 * i:1024 * i + H] for i in range(4)]
    vx.copy_(x)
    vr.copy_(res)
    vc = torch.empty(M, 1 << 28, dtype=torch.uint8, device="cuda")[:, 16:16 + H]
    vs = torch.empty(M, 1 << 28, dtype=F, device="cuda")[:, 1:5]
    moe.moe_add_rms_norm_quant_fp8(vx, vr, w, codes=vc, scales=vs, residual_out=vk, out=vo)
    for got, wanted in zip((vc, vs, vk, vo), (*want, want_out)):
        assert torch.equal(got, wanted)


@pytest.mark.parametrize("M, H", [(1, 16), (40, 528), (30, 2064), (9, 7168), (3, 20000)])
@pytest.mark.parametrize("types", [(F, None, F, F), (F, F, F, F), (B, B, B, F), (B, F, B, F)],
                         ids=lambda t: "-".join(str(v).replace("torch.", "") for v in t))
def test_a_row_is_the_quotient_by_one_root_times_the_weights(M, H, types):
    """out = (r / root) * weight, each of the two rounded once: bit by bit, of one fp32 root a
    row.  The root lies 28 u (the sum's 55 in half) and 1.5 u (mean, eps and root: two halves
    and one) off at most, and a step is u or 2 u of the value: among 30 steps to either side."""
    xt, rt, wt, ot = types
    x, res, w = _inputs(M + H + 1, M, H, xt, rt, wt)
    r, _ = _norm64(x, res, w, 1e-6)
    r, w32 = r.float(), w.float()
    root = torch.sqrt(r.double().square().mean(1, keepdim=True) + 1e-6).float()
    out, _ = moe.moe_add_rms_norm(*[None if t is None else t.cuda() for t in (x, res, w)], eps=1e-6, out_dtype=ot)
    out = out.cpu()
    found = torch.zeros(M, dtype=torch.bool)
    for step in range(-30, 31):
        at = (root.view(torch.int32) + step).view(torch.float32)
        found |= (r / at * w32 == out).all(1)
    assert found.all(), int((~found).sum())


@pytest.mark.parametrize("dtype", [B, F])
def test_zeros_of_a_row_keep_their_signs(dtype):
    x, _, w = _inputs(9, 5, 144, dtype, None, dtype)
    w = w.abs()
    x[:, ::3], x[:, 1::3] = 0.0, -0.0
    out, _ = moe.moe_add_rms_norm(x.cuda(), None, w.cuda(), out_dtype=dtype)
    assert (out[:, ::3] == 0).all() and (out[:, 1::3] == 0).all()
    assert torch.equal(torch.signbit(out).cpu(), torch.signbit(x))


def test_rows_of_small_values_without_eps():
    """From 2^-60 on, beside zeros and values whose squares are lost; the same row times a power
    of two has the same result."""
    x, _, w = _inputs(11, 6, 528, F, None, F)
    x = torch.randn(6, 528, generator=torch.Generator().manual_seed(12)).clamp(-4, 4)
    x[:, ::5] *= 2.0 ** -30
    x[:, 1::5] = 0.0
    x[:, 2::5] = 1 + x[:, 2::5].abs()
    _, want = _norm64(x, None, w, 0.0)
    for scale in (1.0, 2.0 ** -60, 2.0 ** 55):
        out, _ = moe.moe_add_rms_norm((x * scale).cuda(), None, w.cuda(), eps=0.0, out_dtype=F)
        _check_out(out, want)
