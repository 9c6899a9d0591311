"""CPU-side checks of the few-row layer, the fp8 block-scale product and the
token quantisations: arguments that the library or the binding refuses, and
workspace sizes (no GPU needed: nothing below reaches a launch)."""
import ctypes

import pytest
import torch

import expert_layer_moe_amd as moe
from expert_layer_moe_amd.binding import moe_desc

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 1 << 20   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def _layer(**kw):
    base = dict(T=4, H=256, E=8, n_shared=0, I=64, act_dtype=moe.MOE_BF16, w_dtype=moe.MOE_BF16,
                w13_scale=None, w2_scale=None, block_m=0, w_layout=0)
    base.update(kw)
    return moe_desc(**base)


def _few(lib, d, topk=2, workspace_bytes=1 << 30, **ptr):
    p = dict(x=FAKE, valid=None, router=FAKE, w13=FAKE, w2=FAKE, out=FAKE, ws=FAKE)
    p.update(ptr)
    return lib.moe_forward_few(None if d is None else ctypes.byref(d), p["x"], p["valid"],
                               p["router"], p["w13"], p["w2"], topk, p["out"], p["ws"],
                               workspace_bytes, None)


SCALED = dict(w_dtype=moe.MOE_FP8_E4M3, w13_scale=FAKE, w2_scale=FAKE, I=128)


@pytest.mark.parametrize("kw, topk, status", [
    (dict(T=0), 2, INVALID),
    (dict(T=-1), 2, INVALID),
    (dict(T=moe.FEW_MAX_ROWS + 1), 2, UNSUPPORTED),
    (dict(H=0), 2, INVALID),
    (dict(H=192), 2, UNSUPPORTED),
    (dict(H=200), 2, UNSUPPORTED),
    (dict(I=48), 2, UNSUPPORTED),
    (dict(H=32768, I=32768), 2, UNSUPPORTED),
    (dict(act_dtype=moe.MOE_F32, w_dtype=moe.MOE_F32), 2, UNSUPPORTED),
    (dict(), 0, INVALID),
    (dict(), 9, INVALID),
    (dict(SCALED, w13_scale=None), 2, INVALID),
    (dict(SCALED, I=64), 2, UNSUPPORTED),
])
def test_few_refuses_layers(lib, kw, topk, status):
    d = _layer(**kw)
    assert _few(lib, d, topk) == status
    assert lib.moe_few_workspace_size(ctypes.byref(d), topk) == 0
    with pytest.raises(moe.MoeError):
        moe.alloc_few_workspace(d, topk, "cpu")


def test_few_refuses_pointers_and_small_workspaces(lib):
    d = _layer()
    assert _few(lib, None) == INVALID
    for name in ("x", "router", "w13", "w2", "out", "ws"):
        assert _few(lib, d, **{name: None}) == INVALID, name
    for name in ("x", "router", "w13", "w2", "ws"):
        assert _few(lib, d, **{name: FAKE + 8}) == INVALID, name
    n = moe.moe_few_workspace_size(d, 2)
    assert n > 0
    assert _few(lib, d, workspace_bytes=n - 1) == WORKSPACE
    assert _few(lib, d, workspace_bytes=0) == WORKSPACE


def test_few_workspace_sizes():
    """The logits take 8 parts of T rows of 4 E bytes.  Beside small tables:
    where the rows fit on chip 5 parts of 2 I sums of 4 bytes for each of the T
    (k + n_shared) assignments, otherwise 4 bytes of h' for each, and a row
    more."""
    for kw, k, on_chip in ((dict(), 1, True), (dict(T=2, H=1024, E=48, I=96), 3, True),
                           (dict(T=16, E=256, n_shared=1, H=7168, I=256), 8, False),
                           (dict(SCALED, T=6, E=48), 3, True),
                           (dict(SCALED, T=6, E=48, H=7168), 3, False)):
        d = _layer(**kw)
        rows = d.T * (k + d.n_shared)
        need = (40 * rows * d.I if on_chip else 4 * (rows + 1) * d.I) + 32 * d.T * d.E
        size = moe.moe_few_workspace_size(d, k)
        assert need <= size <= need + 32 * d.T * 64 + (20 << 10)


def _gemm(lib, d, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, out=FAKE):
    return lib.moe_gemm_fp8(None if d is None else ctypes.byref(d), a, sa, b, sb, out, None)


def _g(M=4, N=8, K=128, dt=moe.MOE_BF16, lda=0, ldb=0, ld_as=0, ldo=0):
    return moe.moe_gemm_desc(M, N, K, dt, lda, ldb, ld_as, ldo)


@pytest.mark.parametrize("kw, status", [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=-1), INVALID),
    (dict(K=120), UNSUPPORTED), (dict(K=8), UNSUPPORTED),
    (dict(dt=moe.MOE_FP8_E4M3), INVALID), (dict(dt=99), INVALID),
    (dict(lda=112), INVALID), (dict(ldb=112), INVALID), (dict(lda=136), UNSUPPORTED),
    (dict(ldb=136), UNSUPPORTED), (dict(K=256, ld_as=1), INVALID), (dict(ldo=7), INVALID),
    (dict(lda=-128), INVALID), (dict(ldo=-8), INVALID),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(lda=(1 << 23) + 16), UNSUPPORTED), (dict(ldb=(1 << 23) + 16), UNSUPPORTED),
    (dict(K=(1 << 23) + 16), UNSUPPORTED), (dict(ld_as=(1 << 21) + 1), UNSUPPORTED),
])
def test_gemm_refuses(lib, kw, status):
    assert _gemm(lib, _g(**kw)) == status


def test_gemm_refuses_pointers(lib):
    assert _gemm(lib, None) == INVALID
    for name in ("a", "sa", "b", "sb", "out"):
        assert _gemm(lib, _g(), **{name: None}) == INVALID, name
    for name in ("a", "b"):
        assert _gemm(lib, _g(), **{name: FAKE + 8}) == INVALID, name


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("kw, status", [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(rows=-3), INVALID),
    (dict(cols=24), UNSUPPORTED), (dict(cols=8), UNSUPPORTED),
    (dict(dt=moe.MOE_FP8_E4M3), INVALID),
    (dict(ld_in=16), INVALID), (dict(ld_in=516), UNSUPPORTED),
    (dict(ld_in=514, dt=moe.MOE_F32), UNSUPPORTED),
    (dict(ld_codes=112), INVALID), (dict(ld_codes=136), UNSUPPORTED),
    (dict(cols=256, ld_scales=1), INVALID), (dict(ld_in=-512), INVALID),
    (dict(rows=(1 << 31) - 1, cols=256), UNSUPPORTED),
])
def test_quant_refuses(lib, silu, kw, status):
    v = dict(rows=4, cols=128, dt=moe.MOE_BF16, ld_in=0, ld_codes=0, ld_scales=0)
    v.update(kw)
    d = moe.moe_quant_desc(v["rows"], v["cols"], v["dt"], v["ld_in"], v["ld_codes"],
                           v["ld_scales"])
    entry = lib.moe_silu_mul_quant_fp8 if silu else lib.moe_quant_fp8
    assert entry(ctypes.byref(d), FAKE, FAKE, FAKE, None) == status


@pytest.mark.parametrize("silu", [False, True])
def test_quant_refuses_pointers(lib, silu):
    entry = lib.moe_silu_mul_quant_fp8 if silu else lib.moe_quant_fp8
    d = moe.moe_quant_desc(4, 128, moe.MOE_BF16, 0, 0, 0)
    assert entry(None, FAKE, FAKE, FAKE, None) == INVALID
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None),
                 (FAKE + 8, FAKE, FAKE), (FAKE, FAKE + 8, FAKE)):
        assert entry(ctypes.byref(d), *args, None) == INVALID


def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("change", [
    dict(a=_codes(3, 4, 128)), dict(a=_codes(4, 128).short()), dict(b=_codes(8, 112)),
    dict(a_scale=torch.ones(4, 2)), dict(a_scale=torch.ones(4, 1).double()),
    dict(b_scale=torch.ones(2, 1)), dict(out=torch.empty(4, 9)),
    dict(out=torch.empty(4, 8).half()), dict(out=torch.empty(8, 4).t()),
    dict(a=_codes(128, 4).t()), dict(a=_codes(1, 128).expand(4, 128)),
    dict(a_scale=torch.ones(1, 1).expand(4, 1)), dict(out=torch.empty(1, 8).expand(4, 8)),
    dict(b=_codes(1, 128).expand(8, 128)), dict(),
])
def test_binding_refuses_products(change):
    """Wrong shapes, types and orders, broadcast rows (a stride of 0, which the
    descriptor reads as dense); right ones (the last) are refused for
    not being on a GPU."""
    args = dict(a=_codes(4, 128), a_scale=torch.ones(4, 1), b=_codes(8, 128),
                b_scale=torch.ones(1, 1))
    args.update(change)
    with pytest.raises(ValueError) as refusal:
        moe.moe_gemm_fp8(**args)
    assert ("on the GPU" in str(refusal.value)) == (not change)


@pytest.mark.parametrize("fn, x, kw", [
    (moe.moe_quant_fp8, torch.zeros(128), {}),
    (moe.moe_quant_fp8, torch.zeros(2, 128).half(), {}),
    (moe.moe_quant_fp8, torch.zeros(128, 2).t(), {}),
    (moe.moe_quant_fp8, torch.zeros(2, 128), dict(codes=_codes(2, 64))),
    (moe.moe_quant_fp8, torch.zeros(2, 128), dict(scales=torch.zeros(2, 2))),
    (moe.moe_quant_fp8, torch.zeros(2, 128), {}),
    (moe.moe_quant_fp8, torch.zeros(1, 128).expand(4, 128), {}),
    (moe.moe_quant_fp8, torch.zeros(600).as_strided((4, 128), (64, 1)), {}),
    (moe.moe_quant_fp8, torch.zeros(4, 128), dict(codes=_codes(1, 128).expand(4, 128))),
    (moe.moe_silu_mul_quant_fp8, torch.zeros(1, 256).expand(4, 256), {}),
    (moe.moe_silu_mul_quant_fp8, torch.zeros(2, 33), {}),
    (moe.moe_silu_mul_quant_fp8, torch.zeros(2, 256), {}),
])
def test_binding_refuses_quantisations(fn, x, kw):
    good = not kw and x.is_contiguous() and x.dim() == 2 and x.dtype == torch.float32 \
        and x.shape[1] % 2 == 0
    with pytest.raises(ValueError) as refusal:
        fn(x, **kw)
    assert ("on the GPU" in str(refusal.value)) == good


def test_binding_refuses_layers():
    bf = torch.bfloat16
    d = _layer(T=2, E=4, H=128, I=32)
    good = dict(x=torch.zeros(2, 128, dtype=bf), valid_rows=None,
                router_w=torch.zeros(4, 128, dtype=bf), w13=torch.zeros(4, 64, 128, dtype=bf),
                w2=torch.zeros(4, 128, 32, dtype=bf), topk=2, out=torch.zeros(2, 128, dtype=bf),
                workspace=_codes(1 << 16))
    for change in (dict(x=torch.zeros(3, 128, dtype=bf)), dict(x=torch.zeros(2, 128)),
                   dict(out=torch.zeros(2, 256, dtype=bf)[:, ::2]),
                   dict(valid_rows=torch.ones(2)), dict(valid_rows=_codes(3)),
                   dict(workspace=torch.zeros(1 << 16)), {}):
        with pytest.raises(ValueError):
            moe.moe_forward_few(d, **dict(good, **change))


def test_dense_layer_refuses_shapes():
    w13, w2 = _codes(64, 128), _codes(128, 32)
    s13, s2 = torch.ones(1, 1), torch.ones(1, 1)
    moe.DenseFP8(w13, w2, s13, s2, device="cpu")
    for args in ((w13, _codes(128, 48), s13, s2), (_codes(63, 128), w2, s13, s2),
                 (w13, w2, torch.ones(2, 1), s2), (w13, w2, s13, torch.ones(1, 2))):
        with pytest.raises(ValueError):
            moe.DenseFP8(*args, device="cpu")


def _bf16_layer(E=4, H=128, I=32, n_shared=0, experts=None):
    n = E + n_shared if experts is None else experts
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    return moe.DeviceLayer(zeros(E, H), zeros(n, 2 * I, H), zeros(n, H, I), 2, n_shared, device="cpu")


def _forward_few(layer, T=2):
    x = torch.zeros(T, layer.H, dtype=torch.bfloat16)
    return layer.forward_few(x, out=torch.empty_like(x), workspace=_codes(1 << 20))


@pytest.mark.parametrize("make, named", [
    # a shared expert whose weights are not there
    (lambda: _bf16_layer(n_shared=1, experts=4), "w13: "),
    (lambda: _with(_bf16_layer(), w13=torch.zeros(4, 64, 256, dtype=torch.bfloat16)), "w13: "),
    (lambda: _with(_bf16_layer(), w2=torch.zeros(4, 128, 16, dtype=torch.bfloat16)), "w2: "),
    (lambda: _with(_bf16_layer(), w2=torch.zeros(4, 64, 32, dtype=torch.bfloat16)), "w2: "),
    (lambda: _with(_bf16_layer(), w2=torch.zeros(4, 128, 32, dtype=torch.uint8)), "w2: "),
    (lambda: _with(_bf16_layer(), w2=torch.zeros(4, 32, 128, dtype=torch.bfloat16).mT), "w2: "),
    (lambda: _with(_bf16_layer(), router=torch.zeros(3, 128, dtype=torch.bfloat16)), "router_w: "),
    (_bf16_layer, "on the GPU"),
])
def test_layer_of_few_rows_checks_its_weights(make, named):
    """Weights of other shapes, types or orders than the layer's are refused on
    every call; right ones (the last) for not being on a GPU."""
    with pytest.raises(ValueError, match=named):
        _forward_few(make())


def _with(layer, **arrays):
    for name, t in arrays.items():
        setattr(layer, name, t)
    return layer


def test_layer_of_few_rows_takes_its_arrays_as_they_are(monkeypatch):
    """Weights, scales and router put in the layer's place after a call are
    those of the next one."""
    from expert_layer_moe_amd import binding
    E, H, I = 4, 128, 128
    scales = lambda: (torch.ones(E, 2, 1), torch.ones(E, 1, 1))  # noqa: E731
    layer = moe.DeviceLayer(torch.zeros(E, H, dtype=torch.bfloat16), _codes(E, 2 * I, H),
                            _codes(E, H, I), 2, 0, *scales(), device="cpu")
    calls = []

    def enqueue(entry, device, stream, desc, x, valid, router, w13, w2, *rest):
        d = desc._obj
        calls.append((d.T, d.w13_scale, d.w2_scale, router, w13, w2))

    monkeypatch.setattr(binding, "_device_of", lambda *tensors: 0)
    monkeypatch.setattr(binding, "_enqueue", enqueue)
    held = []
    for _ in range(3):
        _forward_few(layer)
        assert calls[-1] == (2, *(t.data_ptr() for t in (layer.s13, layer.s2, layer.router,
                                                         layer.w13, layer.w2)))
        held.append((layer.s13, layer.s2, layer.w13, layer.w2, layer.router))
        layer.s13, layer.s2 = scales()
        layer.w13, layer.w2, layer.router = layer.w13.clone(), layer.w2.clone(), layer.router.clone()
    assert len(set(calls)) == 3


@pytest.mark.parametrize("arrays, named", [
    (dict(s13=torch.ones(4, 1, 1)), "s13"), (dict(s13=None), "s13"),
    (dict(s2=torch.ones(4, 2, 1)), "s2"), (dict(s2=torch.ones(4, 1, 1).double()), "s2"),
    (dict(s13=torch.ones(1, 2, 1).expand(4, 2, 1)), "s13"),
    (dict(s2=torch.ones(4, 1, 1, device="meta")), "s2"),
])
def test_layer_checks_scales_put_in_place_later(arrays, named):
    """The descriptor holds addresses only, so the layer checks what is behind
    them whenever it makes one."""
    layer = moe.DeviceLayer(torch.zeros(4, 128, dtype=torch.bfloat16), _codes(4, 256, 128),
                            _codes(4, 128, 128), 2, 0, torch.ones(4, 2, 1), torch.ones(4, 1, 1),
                            device="cpu")
    layer.desc(1)
    _with(layer, **arrays)
    with pytest.raises(ValueError, match=named):
        layer.desc(1)
    with pytest.raises(ValueError, match=named):
        _forward_few(layer)


def test_layers_are_copied_and_pickled():
    import copy
    import io
    import pickle
    layer = _bf16_layer()
    layer.w2.normal_()
    layer._few_ws[2, 0] = _codes(16)
    file = io.BytesIO()
    torch.save(layer, file)
    file.seek(0)
    for other in (copy.copy(layer), copy.deepcopy(layer), pickle.loads(pickle.dumps(layer)),
                  torch.load(file, weights_only=False)):
        assert torch.equal(other.w2, layer.w2) and other.topk == 2
        # what calls share is each layer's own
        assert other._few_ws == {} and other._few_lock is not layer._few_lock
        with pytest.raises(ValueError, match="on the GPU"):
            _forward_few(other)
    dense = moe.DenseFP8(_codes(64, 128), _codes(128, 32), torch.ones(1, 1), torch.ones(1, 1),
                         device="cpu")
    assert torch.equal(pickle.loads(pickle.dumps(dense)).w13, copy.deepcopy(dense).w13)


def test_dense_layer_takes_the_type_of_its_gate_up_product():
    arrays = _codes(64, 128), _codes(128, 32), torch.ones(1, 1), torch.ones(1, 1)
    assert moe.DenseFP8(*arrays, device="cpu").gate_up == torch.bfloat16
    assert moe.DenseFP8(*arrays, device="cpu", gate_up=torch.float32).gate_up == torch.float32
    with pytest.raises(ValueError, match="gate_up"):
        moe.DenseFP8(*arrays, device="cpu", gate_up=torch.float16)


@pytest.mark.parametrize("M, N", [(1 << 20, (1 << 18) + 1), (1 << 30, 1 << 9), (1 << 9, 1 << 30)])
def test_gemm_refuses_more_results_than_it_has_blocks_for(lib, M, N):
    assert _gemm(lib, _g(M=M, N=N)) == UNSUPPORTED


def test_binding_refuses_sizes_beyond_the_descriptors():
    """More rows or columns than 32 bits hold: their low bits are small sizes that
    the library would take."""
    big = (1 << 32) + 128
    meta = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    f32 = dict(dtype=torch.float32)
    for M, N, K in ((big, 8, 128), (4, big, 128), (4, 8, big)):
        nb = (K + 127) // 128
        with pytest.raises(ValueError, match="2\\^31"):
            moe.moe_gemm_fp8(meta(M, K), meta(M, nb, **f32), meta(N, K),
                             meta((N + 127) // 128, nb, **f32))
    for M, K in ((big, 128), (4, big), (1 << 31, 16)):
        for fn, per_col in ((moe.moe_quant_fp8, 1), (moe.moe_silu_mul_quant_fp8, 2)):
            with pytest.raises(ValueError, match="2\\^31"):
                fn(meta(M, per_col * K, **f32))


@pytest.mark.parametrize("change, named", [
    (dict(x=torch.zeros(3, 128, dtype=torch.bfloat16)), "x: "), (dict(x=torch.zeros(2, 128)), "x: "),
    (dict(x=torch.zeros(2, 256, dtype=torch.bfloat16)[:, ::2]), "x: "),
    (dict(x=torch.zeros(256, dtype=torch.bfloat16)), "x: "),
    (dict(out=torch.zeros(2, 256, dtype=torch.bfloat16)[:, ::2]), "out: "),
    (dict(out=torch.zeros(2, 128)), "out: "), (dict(out=torch.zeros(2, 64).bfloat16()), "out: "),
    (dict(valid_rows=torch.ones(2)), "valid_rows: "), (dict(valid_rows=_codes(3)), "valid_rows: "),
    (dict(valid_rows=_codes(4)[::2]), "valid_rows: "),
    (dict(workspace=torch.zeros(1 << 16)), "workspace: "),
    (dict(workspace=_codes(1 << 17)[::2]), "workspace: "),
    (dict(router_w=torch.zeros(3, 128, dtype=torch.bfloat16)), "router_w: "),
    (dict(w13=torch.zeros(4, 32, 128, dtype=torch.bfloat16)), "w13: "),
    (dict(w2=torch.zeros(4, 128, 32)), "w2: "),
    ({}, "on the GPU"),
])
def test_binding_names_what_it_refuses_of_a_layer(change, named):
    """Each argument's own check (nothing here is on a GPU, which is all that is
    wrong with the last)."""
    bf = torch.bfloat16
    good = dict(x=torch.zeros(2, 128, dtype=bf), valid_rows=None,
                router_w=torch.zeros(4, 128, dtype=bf), w13=torch.zeros(4, 64, 128, dtype=bf),
                w2=torch.zeros(4, 128, 32, dtype=bf), topk=2, out=torch.zeros(2, 128, dtype=bf),
                workspace=_codes(1 << 16))
    with pytest.raises(ValueError, match="^" + named if change else named):
        moe.moe_forward_few(_layer(T=2, E=4, H=128, I=32), **dict(good, **change))


def test_workspace_of_a_capture_on_the_layer_s_device(monkeypatch):
    """A layer on device 1, whose current stream is being captured, while device 0
    is the current one: the capture gets workspaces of its own."""
    import contextlib
    from types import SimpleNamespace
    current = [0]

    @contextlib.contextmanager
    def on(device):
        current.append(device)
        yield
        current.pop()

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device)
    monkeypatch.setattr(torch.cuda, "device", on)
    capturing = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[-1] in capturing)
    layer = _bf16_layer()
    layer.router = SimpleNamespace(get_device=lambda: 1, device="cpu")
    eager = layer.few_workspace(2)
    assert layer.few_workspace(2) is eager
    capturing.append(1)
    graphs = [layer.few_workspace(2) for _ in range(2)]
    assert len({t.data_ptr() for t in (eager, *graphs)}) == 3
    capturing.clear()
    assert layer.few_workspace(2) is eager and current == [0]


def test_gemm_names_the_kernel_it_takes(lib):
    assert moe.moe_gemm_fp8_kernel(1, 4096, 7168) == "rows 16"
    assert moe.moe_gemm_fp8_kernel(8192, 4096, 7168) == "tile 256 x 256"
    assert moe.moe_gemm_fp8_kernel(8192, 4096, 7168, torch.float32) == "tile 128 x 256"
    for sizes in ((0, 8, 128), (4, 8, 120), (1 << 30, 1 << 9, 128)):
        with pytest.raises(moe.MoeError):
            moe.moe_gemm_fp8_kernel(*sizes)
    with pytest.raises(ValueError):
        moe.moe_gemm_fp8_kernel(4, 8, 128, torch.float16)
    with pytest.raises(ValueError):
        moe.moe_gemm_fp8_kernel(4, 8, 1 << 32)
    assert lib.moe_gemm_fp8_kernel(None) is None
    assert lib.moe_gemm_fp8_kernel(ctypes.byref(_g(lda=112))) is None
