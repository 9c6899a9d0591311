"""GPU tests of the operators of a decoder's feed-forward rows as they are used
together: norm with the residual's addition, then an expert layer or a dense layer in
8 or 4 bits; eager, on other streams, from two threads, captured and replayed."""
import math
import threading

import pytest
import torch

import expert_layer_moe_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _weights(seed, H, I):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(2 * I, H, generator=g) / math.sqrt(H),
            torch.randn(H, I, generator=g) / math.sqrt(I), g)


def _fp8(w):
    """128 x 128 blocks in e4m3 codes."""
    N, K = w.shape
    pad = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    tiles = pad.view(pad.shape[0] // 128, 128, pad.shape[1] // 128, 128)
    s = tiles.abs().amax((1, 3)).clamp(min=1e-12) / 448
    codes = (tiles / s[:, None, :, None]).reshape(pad.shape)[:N, :K].to(torch.float8_e4m3fn)
    return codes.contiguous().view(torch.uint8), s


def _layers(seed, H, I):
    w13, w2, g = _weights(seed, H, I)
    (c13, s13), (c2, s2) = _fp8(w13), _fp8(w2)
    norm = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    return moe.DenseFP8(c13, c2, s13, s2), moe.DenseFP4.quantised(w13.bfloat16(), w2), norm, g


@pytest.mark.parametrize("gate_up", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T, H, I", [(1, 256, 128), (3, 416, 224), (16, 1024, 384), (130, 512, 672)])
def test_dense_fp4_is_its_operators_in_a_row(T, H, I, gate_up):
    w13, w2, g = _weights(T + H, H, I)
    dense = moe.DenseFP4.quantised(w13.bfloat16(), w2, gate_up=gate_up)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    a, sa = moe.moe_quant_mxfp4(x)
    c13, s13 = moe.moe_quant_mxfp4(w13.bfloat16().cuda())
    c2, s2 = moe.moe_quant_mxfp4(w2.cuda())
    gu = moe.moe_gemm_mxfp4(a, sa, c13, s13, out_dtype=gate_up)
    h, sh = moe.moe_silu_mul_quant_mxfp4(gu)
    want = moe.moe_gemm_mxfp4(h, sh, c2, s2)
    assert torch.equal(dense.forward(x), want)
    same = moe.DenseFP4(c13, c2, s13.view(torch.float8_e8m0fnu), s2, gate_up=gate_up)
    assert torch.equal(same.forward(x), want)
    out = torch.empty(T, H, dtype=torch.float32, device="cuda")
    assert dense.forward(x, out=out) is out
    assert torch.equal(out, moe.moe_gemm_mxfp4(h, sh, c2, s2, out_dtype=torch.float32))


def test_dense_fp4_of_exact_values():
    """Weights and rows that are codes already, of which each row of w2 picks one h: the
    layer's formula, with the roundings of gu (bf16, 2^-8), SiLU (2^-20) and of the code
    of h alone, which lies 1/4 of h away at most where h is its block's largest."""
    H, I, T = 64, 32, 5
    g = torch.Generator().manual_seed(0)
    grid = torch.tensor([0.5, 1, 1.5, 2, 3, 4, 6])
    pick = lambda *shape: grid[torch.randint(0, 7, shape, generator=g)] * \
        (1 - 2 * torch.randint(0, 2, shape, generator=g))  # noqa: E731
    w13, x = pick(2 * I, H) / 64, pick(T, H)
    x[:, ::32] = 6   # (so that a block's power of two is 1, and w13's 2^-6)
    w13[:, ::32] = 6 / 64
    w2 = torch.zeros(H, I)
    w2[:I] = torch.eye(I)
    dense = moe.DenseFP4.quantised(w13, w2, gate_up=torch.float32)
    out = dense.forward(x.cuda(), out=torch.empty(T, H, device="cuda")).double().cpu()
    p = x.double() @ w13.double().T
    h = p[:, :I] * torch.sigmoid(p[:, :I]) * p[:, I:]
    assert (out[:, I:] == 0).all()
    at = h.abs().argmax(1, keepdim=True)
    got, want = out.gather(1, at), h.gather(1, at)
    assert ((got - want).abs() <= want.abs() * (0.25 + 2 ** -10)).all()


@pytest.mark.parametrize("T, H, I, residual", [(1, 256, 128, True), (7, 416, 224, True),
                                               (40, 1056, 160, False), (200, 512, 672, True)])
def test_normed_forward(T, H, I, residual):
    fp8, fp4, norm, g = _layers(T, H, I)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    res = torch.randn(T, H, generator=g).cuda() if residual else None
    normed, kept = moe.moe_add_rms_norm(x, res, norm, out_dtype=torch.float32)
    out, r = fp8.forward_normed(x, res, norm)
    assert torch.equal(out, fp8.forward(normed))
    assert (r is None and kept is None) or torch.equal(r, kept)
    out, r = fp4.forward_normed(x, res, norm)
    assert torch.equal(out, fp4.forward(moe.moe_add_rms_norm(x, res, norm)[0]))
    assert (r is None and kept is None) or torch.equal(r, kept)
    if residual:   # in place, into a given result
        into = torch.empty(T, H, dtype=torch.float32, device="cuda")
        mine = res.clone()
        got, r = fp8.forward_normed(x, mine, norm, out=into, residual_out=mine)
        assert got is into and r is mine and torch.equal(mine, kept)


def _step(layers, layer, x, residual):
    """norm, dense in 8 bits, norm, experts, norm, dense in 4 bits"""
    fp8, fp4, norm = layers
    y, residual = fp8.forward_normed(x, residual, norm)
    y, residual = moe.moe_add_rms_norm(y, residual, norm)
    y = layer.forward_few(y)
    return fp4.forward_normed(y, residual, norm)


def _stack(seed, T):
    H, I, E = 512, 384, 12
    fp8, fp4, norm, g = _layers(seed, H, I)
    router = torch.randn(E, H, generator=g).bfloat16() / math.sqrt(H)
    w13 = (torch.randn(E, 256, H, generator=g) / math.sqrt(H)).bfloat16()
    w2 = (torch.randn(E, H, 128, generator=g) / math.sqrt(128)).bfloat16()
    layer = moe.DeviceLayer(router, w13, w2, 3, packed=True)
    rows = lambda: (torch.randn(T, H, generator=g).bfloat16().cuda(),
                    torch.randn(T, H, generator=g).bfloat16().cuda())  # noqa: E731
    return (fp8, fp4, norm), layer, rows


def test_decoder_rows_in_a_graph():
    """Replayed with new rows between eager calls on the same stream and another one."""
    layers, layer, rows = _stack(1, 4)
    x, res = rows()
    _step(layers, layer, x, res)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out, kept = _step(layers, layer, x, res)
    other = torch.cuda.Stream()
    for _ in range(5):
        fresh = rows()
        x.copy_(fresh[0])
        res.copy_(fresh[1])
        graph.replay()
        want, want_kept = _step(layers, layer, *fresh)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kept, want_kept)
        with torch.cuda.stream(other):
            again, _ = _step(layers, layer, *fresh)
        torch.cuda.synchronize()
        assert torch.equal(again, want)


def test_calls_on_a_given_stream():
    """stream=: the results are there for that stream's work, and the current one is
    another."""
    fp8, fp4, norm, g = _layers(3, 512, 384)
    x = torch.randn(33, 512, generator=g).bfloat16().cuda()
    res = torch.randn(33, 512, generator=g).bfloat16().cuda()
    want = fp4.forward_normed(x, res, norm), fp8.forward_normed(x, res, norm)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            y, r = x * 1, res * 1   # (written on that stream alone)
        a = fp4.forward_normed(y, r, norm, stream=side)
        b = fp8.forward_normed(y, r, norm, stream=side)
        side.synchronize()
        for got, w in zip((*a, *b), (*want[0], *want[1])):
            assert torch.equal(got, w)


def test_two_threads_at_once():
    """Calls from two threads, each on a stream of its own."""
    fp8, fp4, norm, g = _layers(4, 512, 384)
    xs = [torch.randn(64, 512, generator=g).bfloat16().cuda() for _ in range(2)]
    res = [torch.randn(64, 512, generator=g).bfloat16().cuda() for _ in range(2)]
    want = [fp4.forward_normed(x, r, norm) for x, r in zip(xs, res)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                out, kept = fp4.forward_normed(xs[i], res[i], norm)
                stream.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(kept, want[i][1])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_each_operator_captured_and_replayed():
    g = torch.Generator().manual_seed(9)
    K, N = 544, 304   # (rows of 300 bf16 values would end inside 16 bytes, which SiLU refuses)
    w = torch.randn(N, K, generator=g).bfloat16().cuda()
    norm = torch.rand(K, generator=g).cuda()
    b, sb = moe.moe_quant_mxfp4(w)
    x, res = torch.zeros(200, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(200, K, device="cuda")

    def run(x, res):
        out, kept = moe.moe_add_rms_norm(x, res, norm)
        codes, scales, kept8 = moe.moe_add_rms_norm_quant_fp8(x, kept, norm, out=torch.empty_like(out))
        a, sa = moe.moe_quant_mxfp4(out)
        h, sh = moe.moe_silu_mul_quant_mxfp4(moe.moe_gemm_mxfp4(a, sa, b, sb)[:, :256])
        return (out, kept, codes, scales, kept8, a, sa, h, sh, moe.moe_dequant_mxfp4(h, sh),
                moe.moe_gemm_mxfp4(a[:16], sa[:16], b, sb, out_dtype=torch.float32))

    run(x, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(x, res)
    for _ in range(4):
        x.copy_(torch.randn(200, K, generator=g).bfloat16())
        res.copy_(torch.randn(200, K, generator=g))
        graph.replay()
        want = run(x, res)
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)


@pytest.mark.parametrize("inference", [False, True])
@pytest.mark.parametrize("M", [3, 3000])
def test_results_of_one_call_do_not_touch(M, inference):
    """Small results of a call lie in one allocation: apart, aligned, and each a tensor of
    its own to torch (in place, copied, resized, on the host); large ones in their own."""
    import copy
    with torch.inference_mode(inference):
        x = torch.randn(M, 416, device="cuda").bfloat16()
        w = torch.ones(416, device="cuda")
        calls = [lambda: moe.moe_quant_mxfp4(x), lambda: moe.moe_silu_mul_quant_mxfp4(x[:, :384]),
                 lambda: moe.moe_add_rms_norm(x, x, w, out_dtype=torch.float32),
                 lambda: moe.moe_add_rms_norm_quant_fp8(x, x.float(), w),
                 lambda: moe.moe_add_rms_norm_quant_fp8(x, None, w)[:2]]
        for call in calls:
            want = [t.cpu() for t in call()]
            assert all(t.is_contiguous() and t.data_ptr() % 256 == 0 for t in call())
            for i in range(len(want)):
                got = call()
                shared = len({t.untyped_storage().data_ptr() for t in got}) < len(got)
                assert shared == (sum(-(-t.nbytes // 256) * 256 for t in got) <= 1 << 20)
                got[i].zero_()
                assert torch.equal(copy.deepcopy(got[i]).cpu(), torch.zeros_like(want[i]))
                for j in range(len(want)):
                    assert torch.equal(got[j].cpu(), torch.zeros_like(want[j]) if i == j else want[j])
                got[i].resize_(M + 1000, 416)
                got[i].fill_(1)
                del got
                assert all(torch.equal(t.cpu(), v) for t, v in zip(call(), want))


@pytest.mark.parametrize("inference", [False, True])
@pytest.mark.parametrize("more", [1, 5, 1000])
def test_a_result_that_grows_leaves_the_others(more, inference):
    """Each result of a call resized to more rows and written, others of the call looked at
    behind that, and the call's memory used anew."""
    with torch.inference_mode(inference):
        x = torch.randn(3, 416, device="cuda").bfloat16()
        w = torch.ones(416, device="cuda")
        calls = [lambda: moe.moe_quant_mxfp4(x), lambda: moe.moe_silu_mul_quant_mxfp4(x[:, :384]),
                 lambda: moe.moe_add_rms_norm(x, x, w, out_dtype=torch.float32),
                 lambda: moe.moe_add_rms_norm_quant_fp8(x, x.float(), w),
                 lambda: moe.moe_add_rms_norm_quant_fp8(x, None, w)[:2]]
        for call in calls:
            want = [t.cpu() for t in call()]
            for i in range(len(want)):
                got = call()
                got[i].resize_(3 + more, want[i].shape[1])
                assert torch.equal(got[i][:3].cpu(), want[i])
                got[i].fill_(1)
                for j in range(len(want)):
                    assert i == j or torch.equal(got[j].cpu(), want[j])
                # (what the grown one lay in is not free while others lie beside it)
                later = [call() for _ in range(4)]
                for j in range(len(want)):
                    assert torch.equal(got[j].cpu(), torch.ones(got[j].shape, dtype=got[j].dtype) if i == j else want[j])
                    assert all(torch.equal(t[j].cpu(), want[j]) for t in later)


def test_a_result_whose_memory_is_given_back_leaves_the_others():
    x = torch.randn(3, 416, device="cuda").bfloat16()
    want = [t.cpu() for t in moe.moe_quant_mxfp4(x)]
    for i in range(2):
        got = moe.moe_quant_mxfp4(x)
        got[i].untyped_storage().resize_(0)
        assert torch.equal(got[1 - i].cpu(), want[1 - i])


@pytest.mark.parametrize("i", [0, 1, 2])
def test_results_in_use_on_another_stream_keep_their_memory(i):
    """record_stream of one result of a call: the memory of all is not given out again while
    that stream has work, and is afterwards."""
    x = torch.randn(3, 416, device="cuda").bfloat16()
    w = torch.ones(416, device="cuda")
    call = lambda: moe.moe_add_rms_norm_quant_fp8(x, x.float(), w)  # noqa: E731
    call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call()
    place = {t.untyped_storage().data_ptr() for t in got}
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got[i].record_stream(side)
    del got
    during = [call() for _ in range(3)]
    assert not side.query(), "the side stream was done too early to tell"
    assert not place & {t.untyped_storage().data_ptr() for r in during for t in r}
    side.synchronize()
    del during
    torch.cuda.empty_cache()


def test_results_handed_to_another_process_keep_their_memory():
    """torch counts the readers of a storage that it shares; as long as there may be some, its
    memory is not given out again, though the tensors here are gone."""
    x = torch.randn(3, 416, device="cuda").bfloat16()
    for i in range(2):
        got = moe.moe_quant_mxfp4(x)
        place = got[0].untyped_storage().data_ptr()
        got[i].untyped_storage()._share_cuda_()
        del got
        later = [moe.moe_quant_mxfp4(x) for _ in range(4)]
        assert place not in {t.untyped_storage().data_ptr() for r in later for t in r}


def test_the_storage_of_a_result_ends_with_it():
    """So that what torch does to a storage as a whole (copies, files) does not reach behind."""
    x = torch.randn(5, 416, device="cuda").bfloat16()
    w = torch.ones(416, device="cuda")
    for got in (moe.moe_quant_mxfp4(x), moe.moe_add_rms_norm(x, x, w), moe.moe_add_rms_norm_quant_fp8(x, x, w)):
        for t in got:
            assert t.untyped_storage().nbytes() == t.storage_offset() * t.element_size() + t.nbytes


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("rows", [torch.bfloat16, torch.float32])
def test_dense_fp4_takes_its_codes_of_the_norm_in_either_type(T, rows):
    """normed=fp32: no rounding to bf16 between the norm and the codes, whose scales and codes
    it changes."""
    H, I = 1056, 96
    w13, w2, g = _weights(T, H, I)
    dense = moe.DenseFP4.quantised(w13.bfloat16(), w2, normed=torch.float32)
    half = moe.DenseFP4.quantised(w13.bfloat16(), w2)
    norm = (1 + 0.1 * torch.randn(H, generator=g)).to(rows).cuda()
    x, res = torch.randn(T, H, generator=g).to(rows).cuda(), torch.randn(T, H, generator=g).to(rows).cuda()
    normed, kept = moe.moe_add_rms_norm(x, res, norm, out_dtype=torch.float32)
    into = lambda: torch.empty(T, H, device="cuda")  # noqa: E731
    out, r = dense.forward_normed(x, res, norm, out=into())
    assert torch.equal(out, dense.forward(normed, out=into())) and torch.equal(r, kept)
    rounded, _ = half.forward_normed(x, res, norm, out=into())
    assert torch.equal(rounded, dense.forward(normed.bfloat16(), out=into())) and not torch.equal(rounded, out)
