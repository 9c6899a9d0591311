"""CPU-side checks of the 4-bit operators and the norm with the residual's addition:
arguments that the library or the binding refuses (no GPU needed: nothing below reaches
a launch)."""
import copy
import ctypes
import pickle

import pytest
import torch

import expert_layer_moe_amd as moe

INVALID, UNSUPPORTED = -1, -2
FAKE = 1 << 20   # never dereferenced: validation fails first
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


# ---- the library --------------------------------------------------------------------
def _g(M=4, N=8, K=128, dt=moe.MOE_BF16, lda=0, ldb=0, ld_as=0, ld_bs=0, ldo=0):
    return moe.moe_mx_gemm_desc(M, N, K, dt, lda, ldb, ld_as, ld_bs, ldo)


def _gemm(lib, d, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, out=FAKE):
    return lib.moe_gemm_mxfp4(None if d is None else ctypes.byref(d), a, sa, b, sb, out, None)


@pytest.mark.parametrize("kw, status", [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=-1), INVALID),
    (dict(K=112), UNSUPPORTED), (dict(K=16), UNSUPPORTED), (dict(K=1), UNSUPPORTED),
    (dict(dt=moe.MOE_FP8_E4M3), INVALID), (dict(dt=99), INVALID),
    (dict(lda=48), INVALID), (dict(ldb=48), INVALID), (dict(lda=72), UNSUPPORTED),
    (dict(ldb=72), UNSUPPORTED), (dict(ld_as=3), INVALID), (dict(ld_bs=3), INVALID),
    (dict(ldo=7), INVALID), (dict(lda=-64), INVALID), (dict(ldo=-8), INVALID), (dict(ld_bs=-4), INVALID),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(M=1 << 20, N=(1 << 18) + 1), UNSUPPORTED), (dict(M=1 << 30, N=1 << 9), UNSUPPORTED),
    (dict(lda=(1 << 23) + 16), UNSUPPORTED), (dict(ldb=(1 << 23) + 16), UNSUPPORTED),
    (dict(K=(1 << 24) + 32), UNSUPPORTED),
])
def test_gemm_refuses(lib, kw, status):
    assert _gemm(lib, _g(**kw)) == status
    assert lib.moe_gemm_mxfp4_kernel(ctypes.byref(_g(**kw))) is None


def test_gemm_refuses_pointers(lib):
    assert _gemm(lib, None) == INVALID
    for name in ("a", "sa", "b", "sb", "out"):
        assert _gemm(lib, _g(), **{name: None}) == INVALID, name
    for name in ("a", "b"):
        assert _gemm(lib, _g(), **{name: FAKE + 8}) == INVALID, name


def test_gemm_names_the_kernel_it_takes(lib):
    assert moe.moe_gemm_mxfp4_kernel(1, 4096, 7168) == "rows 16"
    assert moe.moe_gemm_mxfp4_kernel(16, 8192, 16384) == "tile 16 x 32"
    assert moe.moe_gemm_mxfp4_kernel(8192, 4096, 7168) == "tile 256 x 256"
    for sizes in ((0, 8, 128), (4, 8, 120), (1 << 30, 1 << 9, 128)):
        with pytest.raises(moe.MoeError):
            moe.moe_gemm_mxfp4_kernel(*sizes)
    with pytest.raises(ValueError):
        moe.moe_gemm_mxfp4_kernel(4, 8, 1 << 32)
    assert lib.moe_gemm_mxfp4_kernel(None) is None


@pytest.mark.parametrize("entry, per_col", [("moe_quant_mxfp4", 1), ("moe_silu_mul_quant_mxfp4", 2),
                                            ("moe_dequant_mxfp4", 1)])
@pytest.mark.parametrize("kw, status", [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(rows=-3), INVALID),
    (dict(cols=48), UNSUPPORTED), (dict(cols=16), UNSUPPORTED),
    (dict(dt=moe.MOE_FP8_E4M3), INVALID), (dict(dt=-1), INVALID),
    (dict(ld_in=64), INVALID), (dict(ld_in=516), UNSUPPORTED),
    (dict(ld_in=514, dt=moe.MOE_F32), UNSUPPORTED), (dict(ld_in=-512), INVALID),
    (dict(ld_codes=48), INVALID), (dict(ld_codes=72), UNSUPPORTED), (dict(ld_codes=-64), INVALID),
    (dict(ld_scales=3), INVALID), (dict(rows=(1 << 31) - 1, cols=64), UNSUPPORTED),
])
def test_quant_and_dequant_refuse(lib, entry, per_col, kw, status):
    v = dict(rows=4, cols=128, dt=moe.MOE_BF16, ld_in=0, ld_codes=0, ld_scales=0)
    v.update(kw)
    d = moe.moe_quant_desc(v["rows"], v["cols"], v["dt"], v["ld_in"], v["ld_codes"], v["ld_scales"])
    assert getattr(lib, entry)(ctypes.byref(d), FAKE, FAKE, FAKE, None) == status


def test_quant_and_dequant_refuse_pointers(lib):
    d = moe.moe_quant_desc(4, 128, moe.MOE_BF16, 0, 0, 0)
    for entry, first, second, third in (("moe_quant_mxfp4", 8, 8, 0), ("moe_silu_mul_quant_mxfp4", 8, 8, 0),
                                        ("moe_dequant_mxfp4", 8, 0, 8)):
        f = getattr(lib, entry)
        assert f(None, FAKE, FAKE, FAKE, None) == INVALID
        off = [(FAKE + first, FAKE, FAKE), (FAKE, FAKE + second, FAKE), (FAKE, FAKE, FAKE + third)]
        for args in [(None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)] + \
                [a for a in off if a != (FAKE, FAKE, FAKE)]:
            assert f(ctypes.byref(d), *args, None) == INVALID


def _norm(rows=4, cols=256, x=1, res=1, w=1, out=1, eps=1e-6, ld_x=0, ld_res=0, ld_res_out=0,
          ld_out=0, ld_codes=0, ld_scales=0):
    return moe.moe_norm_desc(rows, cols, x, res, w, out, eps, ld_x, ld_res, ld_res_out, ld_out,
                             ld_codes, ld_scales)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("kw, status", [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=24), UNSUPPORTED), (dict(cols=32768 + 16), UNSUPPORTED),
    (dict(x=2), INVALID), (dict(res=2), INVALID), (dict(w=9), INVALID), (dict(out=2), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(ld_x=128), INVALID), (dict(ld_x=260), UNSUPPORTED), (dict(x=0, ld_x=258), UNSUPPORTED),
    (dict(ld_res=128), INVALID), (dict(ld_res=260), UNSUPPORTED), (dict(ld_res_out=260), UNSUPPORTED),
    (dict(ld_res_out=-256), INVALID), (dict(ld_out=128), INVALID), (dict(ld_out=260), UNSUPPORTED),
])
def test_norm_refuses(lib, codes, kw, status):
    d = _norm(**kw)
    if codes:
        got = lib.moe_add_rms_norm_quant_fp8(ctypes.byref(d), *[FAKE] * 7, None)
    else:
        got = lib.moe_add_rms_norm(ctypes.byref(d), *[FAKE] * 5, None)
    assert got == status


@pytest.mark.parametrize("kw, status", [
    (dict(ld_codes=240), INVALID), (dict(ld_codes=264), UNSUPPORTED), (dict(ld_scales=1), INVALID),
    (dict(ld_scales=-2), INVALID),
])
def test_norm_refuses_strides_of_codes(lib, kw, status):
    assert lib.moe_add_rms_norm_quant_fp8(ctypes.byref(_norm(**kw)), *[FAKE] * 7, None) == status


def test_norm_refuses_pointers(lib):
    assert lib.moe_add_rms_norm(None, *[FAKE] * 5, None) == INVALID
    assert lib.moe_add_rms_norm_quant_fp8(None, *[FAKE] * 7, None) == INVALID
    d = ctypes.byref(_norm())
    # x, residual, weight, residual_out, out: a residual alone needs residual_out
    for at in (0, 2, 3, 4):
        args = [FAKE] * 5
        args[at] = None
        assert lib.moe_add_rms_norm(d, *args, None) == INVALID, at
    for at in range(5):
        args = [FAKE] * 5
        args[at] = FAKE + 8
        assert lib.moe_add_rms_norm(d, *args, None) == INVALID, at
    # ..., codes, scales (of 4-byte alignment alone)
    for at in (0, 2, 3, 5, 6):
        args = [FAKE] * 7
        args[at] = None
        assert lib.moe_add_rms_norm_quant_fp8(d, *args, None) == INVALID, at
    for at in range(6):
        args = [FAKE] * 7
        args[at] = FAKE + 8
        assert lib.moe_add_rms_norm_quant_fp8(d, *args, None) == INVALID, at


# ---- the binding --------------------------------------------------------------------
def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _refused(fn, *args, **kw):
    with pytest.raises((ValueError, TypeError)) as refusal:
        fn(*args, **kw)
    return str(refusal.value)


@pytest.mark.parametrize("change, named", [
    (dict(a=_codes(3, 4, 64)), "a: "), (dict(a=_codes(4, 64).short()), "a: "), (dict(a=7), "a: "),
    (dict(b=_codes(8, 48)), "b: "), (dict(b=_codes(8)), "b: "), (dict(a_scale=_codes(4, 5)), "a_scale: "),
    (dict(a_scale=torch.ones(4, 4)), "a_scale: "), (dict(b_scale=_codes(4, 8).t()), "b_scale"),
    (dict(b_scale=None), "b_scale: "), (dict(out=torch.empty(4, 9)), "out: "),
    (dict(out=torch.empty(4, 8).half()), "out: "), (dict(out=torch.empty(8, 4).t()), "out"),
    (dict(a=_codes(64, 4).t()), "a must"), (dict(a=_codes(1, 64).expand(4, 64)), "a has rows"),
    (dict(a_scale=_codes(1, 4).expand(4, 4)), "a_scale has rows"),
    (dict(out=torch.empty(1, 8).expand(4, 8)), "out has rows"),
    (dict(b=_codes(1, 64).expand(8, 64)), "b has rows"), (dict(out_dtype=torch.float16), "out_dtype"),
    (dict(), "on the GPU"),
])
def test_binding_refuses_products(change, named):
    """Wrong shapes, types and orders, broadcast rows (a stride of 0, which the
    descriptor reads as dense); right ones are refused for not being on a GPU."""
    args = dict(a=_codes(4, 64), a_scale=_codes(4, 4), b=_codes(8, 64), b_scale=_codes(8, 4))
    args.update(change)
    assert named in _refused(moe.moe_gemm_mxfp4, **args)


@pytest.mark.parametrize("fn, x, kw, named", [
    (moe.moe_quant_mxfp4, torch.zeros(128), {}, "input: "),
    (moe.moe_quant_mxfp4, torch.zeros(2, 128).half(), {}, "input: "),
    (moe.moe_quant_mxfp4, torch.zeros(128, 32).t(), {}, "contiguous rows"),
    (moe.moe_quant_mxfp4, torch.zeros(2, 48), {}, "32 n columns"),
    (moe.moe_quant_mxfp4, torch.zeros(1, 128).expand(4, 128), {}, "overlap"),
    (moe.moe_quant_mxfp4, torch.zeros(600).as_strided((4, 128), (64, 1)), {}, "overlap"),
    (moe.moe_quant_mxfp4, torch.zeros(2, 128), {}, "on the GPU"),
    (moe.moe_quant_mxfp4, [1, 2], {}, "a tensor expected"),
    (moe.moe_silu_mul_quant_mxfp4, torch.zeros(2, 96), {}, "64 n columns"),
    (moe.moe_silu_mul_quant_mxfp4, torch.zeros(2, 128), {}, "on the GPU"),
    (moe.moe_dequant_mxfp4, _codes(2, 24), dict(scales=_codes(2, 2)), "16 n columns"),
    (moe.moe_dequant_mxfp4, _codes(2, 32).short(), dict(scales=_codes(2, 2)), "codes: "),
    (moe.moe_dequant_mxfp4, _codes(2, 32), dict(scales=_codes(2, 2)), "on the GPU"),
])
def test_binding_refuses_quantisations(fn, x, kw, named):
    assert named in _refused(fn, x, **kw)


@pytest.mark.parametrize("fn", [moe.moe_add_rms_norm, moe.moe_add_rms_norm_quant_fp8])
@pytest.mark.parametrize("change, named", [
    (dict(x=torch.zeros(256)), "x: "), (dict(x=torch.zeros(4, 256).half()), "x: "),
    (dict(eps="1"), "real number"), (dict(), "on the GPU"),
    (dict(x=torch.zeros(1, 256).expand(4, 256)), "x has rows"),
    (dict(weight=torch.ones(255)), "weight: "), (dict(weight=torch.ones(256).double()), "weight: "),
    (dict(weight=torch.ones(512)[::2]), "weight: "), (dict(weight=torch.ones(1, 256)), "weight: "),
    (dict(residual=torch.zeros(4, 272)), "residual: "), (dict(residual=None, residual_out=torch.zeros(4, 256)),
                                                         "without a residual"),
    (dict(residual_out=torch.zeros(4, 256).bfloat16()), "residual_out: "),
    (dict(residual_out=torch.zeros(256, 4).t()), "residual_out must"),
])
def test_binding_refuses_norms(fn, change, named):
    args = dict(x=torch.zeros(4, 256), residual=torch.zeros(4, 256), weight=torch.ones(256))
    args.update(change)
    assert named in _refused(fn, **args)


def test_binding_refuses_sizes_beyond_the_descriptors():
    """More rows or columns than 32 bits hold."""
    big = (1 << 32) + 128
    meta = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    for M, N, K in ((big, 8, 128), (4, big, 128), (4, 8, big), (4, 8, 1 << 31)):
        assert "2^31" in _refused(moe.moe_gemm_mxfp4, meta(M, K // 2), meta(M, K // 32), meta(N, K // 2),
                                  meta(N, K // 32))
    for M, K in ((big, 128), (4, big), (1 << 31, 32)):
        for fn, per_col in ((moe.moe_quant_mxfp4, 1), (moe.moe_silu_mul_quant_mxfp4, 2)):
            assert "2^31" in _refused(fn, meta(M, per_col * K, dtype=F32))
        for fn in (moe.moe_add_rms_norm, moe.moe_add_rms_norm_quant_fp8):
            assert "2^31" in _refused(fn, meta(M, K, dtype=F32), None, meta(K, dtype=F32))
        assert "2^31" in _refused(moe.moe_dequant_mxfp4, meta(M, K // 2), meta(M, K // 32)) or K == big
    # (an overlong row of codes is refused as one, not by its own length alone)
    assert "2^31" in _refused(moe.moe_dequant_mxfp4, meta(4, 1 << 30), meta(4, 1 << 26))


# ---- the dense layer in 4 bits ------------------------------------------------------
def test_dense_layer_refuses_shapes_and_types():
    w13, w2, s13, s2 = _codes(128, 32), _codes(64, 32), _codes(128, 2), _codes(64, 2)
    layer = moe.DenseFP4(w13, w2, s13.view(torch.float8_e8m0fnu), s2, device="cpu")
    assert (layer.H, layer.I, layer.gate_up) == (64, 64, BF)
    assert torch.equal(pickle.loads(pickle.dumps(layer)).w13, copy.deepcopy(layer).w13)
    for args in ((w13, _codes(64, 48), s13, s2), (_codes(127, 32), w2, s13, s2),
                 (_codes(128, 24), w2, s13, s2), (w13, w2, _codes(128, 1), s2),
                 (w13, w2, s13, _codes(64, 3)), (w13.short(), w2, s13, s2),
                 (w13, w2, s13.float(), s2), (w13, w2.view(torch.float8_e8m0fnu), s13, s2)):
        with pytest.raises(ValueError):
            moe.DenseFP4(*args, device="cpu")
    with pytest.raises(ValueError, match="gate_up"):
        moe.DenseFP4(w13, w2, s13, s2, device="cpu", gate_up=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        layer.forward(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="on the GPU"):
        layer.forward_normed(torch.zeros(2, 64), None, torch.ones(64))


def test_dense_layer_refuses_the_type_of_its_normed_rows():
    w13, w2, s13, s2 = _codes(128, 32), _codes(64, 32), _codes(128, 2), _codes(64, 2)
    assert moe.DenseFP4(w13, w2, s13, s2, device="cpu").normed == BF
    layer = moe.DenseFP4(w13, w2, s13, s2, device="cpu", normed=F32)
    assert pickle.loads(pickle.dumps(layer)).normed == F32
    with pytest.raises(ValueError, match="normed"):
        moe.DenseFP4(w13, w2, s13, s2, device="cpu", normed=torch.float16)
