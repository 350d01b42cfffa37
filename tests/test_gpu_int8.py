"""8-bit products and the row quantiser on the GPU against 64-bit restatements: one token to
many, odd sizes, rows that start on any byte, extreme values, scales that are not finite,
streams, graphs and the norm -> 8 bits -> product chain."""
import numpy as np
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, seed, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(lo, hi + 1, (M, K), generator=g, dtype=torch.int32).to(torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8)
    xs = torch.rand(M, generator=g) * 0.02 + 0.001
    ws = torch.rand(N, generator=g) * 0.02 + 0.001
    return x, xs, w, ws, torch.randn(N, generator=g)


def _np(t):
    return t.detach().double().cpu().numpy()


SIZES = [
    # M, N, K
    (1, 1, 1), (1, 17, 5), (3, 1, 64), (1, 512, 256), (1, 4096, 1024), (2, 300, 4096), (5, 64, 48), (8, 128, 1000),
    (7, 33, 129), (9, 40, 16), (16, 512, 512), (31, 77, 333), (64, 256, 96), (127, 128, 64), (128, 128, 128),
    (129, 257, 127), (200, 320, 320), (301, 777, 1000), (513, 512, 256), (1000, 96, 2048), (256, 1024, 4096),
    (3136, 512, 256), (40000, 64, 72),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_product(size, out):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, xs, w, ws, bias = _inputs(M, N, K, M + 3 * N + K)
    y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), out=out)
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "none")
    ref.check(_np(y), want, tol, out == "bf16", "y")
    assert cg.device_status() == 0


# The kernel between few rows and many: each count of 16-row tiles, K shorter than its eight warps
# share and longer than they hold, rows of either operand off 16 bytes.
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(5, 16, 16), (6, 33, 520), (8, 1000, 2064), (16, 15, 4112), (17, 48, 64), (32, 257, 2048), (33, 100, 530),
                                  (48, 130, 1000), (49, 64, 96), (64, 129, 515), (64, 512, 512), (50, 2048, 2048)])
def test_rows_between_few_and_many(size, out):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, xs, w, ws, bias = _inputs(M, N, K, 3 * M + N + 7 * K)
    y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), act="silu", out=out)
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "silu")
    ref.check(_np(y), want, tol, out == "bf16", "y")
    xf = torch.randn(M, K, generator=torch.Generator().manual_seed(M + K)).to(torch.bfloat16)
    y = cg.int8_linear(xf.cuda(), w.cuda(), ws.cuda(), bias.cuda(), out="f32")
    q, s = ref.quantize_rows(xf.float().numpy())
    want, tol = ref.int8_product(q, s, w.numpy(), ws.numpy(), bias.numpy(), "none")
    ref.check(_np(y), want, tol, False, "y")


# Rows of y that start on 2, 4, 8 bytes in every tile shape; rows of x of every length class whose
# vectors straddle 16 bytes.
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(5000, 1002, 144), (5000, 1004, 64), (5001, 1003, 80), (2000, 90, 112), (2000, 92, 96), (333, 42, 64),
                                  (40, 31, 48)])
def test_rows_of_y_off_16_bytes(size, out):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, xs, w, ws, bias = _inputs(M, N, K, 5 * M + N + K)
    canvas = torch.full((M * N + 64,), 7.0, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    y = canvas[:M * N].view(M, N)
    plan = cg.Int8MatmulPlan(M, N, K, out=out, act="silu")
    plan.forward(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), y=y)
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "silu")
    ref.check(_np(y), want, tol, out == "bf16", "y")
    assert torch.all(canvas[M * N:] == 7.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(9, 250), (50, 257), (33, 500), (21, 1022), (17, 2047), (5, 4090), (3, 5001), (700, 36)])
def test_quantize_rows_that_straddle_vectors(M, K, dtype):
    import cnn_convolution_implicit_gb300 as cg
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(M + K)) * 3).to(dtype)
    q, s = cg.quantize_rows(x.cuda())
    wq, ws = ref.quantize_rows(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    _, _, w, wsc, bias = _inputs(M, 48, K, 8)
    y = cg.int8_linear(x.cuda(), w.cuda(), wsc.cuda(), bias.cuda(), out="f32")
    want, tol = ref.int8_product(wq, ws, w.numpy(), wsc.numpy(), bias.numpy(), "none")
    ref.check(_np(y), want, tol, False, "y")


# Every tile shape and split of K: pairs of SMs over several rounds, 128, 64 and 32 columns, two, four
# and eight CTAs to a tile, a K that the split does not divide, and each with rows off 16 bytes.
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(5000, 1000, 528), (5000, 1001, 520), (9000, 512, 256), (16, 4096, 4096), (300, 2048, 1040),
                                  (128, 100, 2000), (40, 33, 1999), (1000, 704, 304), (2000, 96, 3000), (20, 5000, 70)])
def test_tile_shapes(size, out):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, xs, w, ws, bias = _inputs(M, N, K, M + N + 5 * K)
    y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), act="relu", out=out)
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "relu")
    ref.check(_np(y), want, tol, out == "bf16", "y")
    assert cg.device_status() == 0


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("bias_on", [True, False])
@pytest.mark.parametrize("size", [(1, 96, 160), (5, 96, 100), (140, 200, 130)])
def test_activation_and_bias(size, act, bias_on):
    import cnn_convolution_implicit_gb300 as cg
    x, xs, w, ws, bias = _inputs(*size, 5)
    y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda() if bias_on else None, act=act, out="f32")
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy() if bias_on else None, act)
    ref.check(_np(y), want, 2 * tol + 16 * ref.U32 * np.abs(want), False, "y")


@pytest.mark.parametrize("size", [(1, 64, 1024), (6, 64, 1024), (130, 128, 1024), (130, 64, 4096), (2, 64, 131071),
                                  (130, 40, 20000)])
def test_extreme_values(size):
    """Every product at its largest: -128 * -128 summed over K, past 2^24 where K > 1024."""
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((N, K), -128, dtype=torch.int8)
    w[1::2] = 127
    one_m, one_n = torch.ones(M), torch.ones(N)
    y = cg.int8_matmul(x.cuda(), one_m.cuda(), w.cuda(), one_n.cuda(), out="f32")
    want, tol = ref.int8_product(x.numpy(), one_m.numpy(), w.numpy(), one_n.numpy(), None, "none")
    ref.check(_np(y), want, tol, False, "y")
    if K <= 1024:
        assert np.array_equal(_np(y), want)


@pytest.mark.parametrize("size", [(4, 64, 200), (300, 130, 1024)])
def test_sum_is_exact(size):
    """Unit scales: the FP32 result is the integer sum itself."""
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, _, w, _, _ = _inputs(M, N, K, 77)
    y = cg.int8_matmul(x.cuda(), torch.ones(M).cuda(), w.cuda(), torch.ones(N).cuda(), out="f32")
    assert np.array_equal(_np(y), x.double().numpy() @ w.double().numpy().T)


@pytest.mark.parametrize("M", [1, 4, 150])
def test_scales_that_are_not_finite_stay_in_their_row_and_column(M):
    import cnn_convolution_implicit_gb300 as cg
    x, xs, w, ws, bias = _inputs(M, 70, 96, 4)
    clean = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda())
    ws[3] = float("nan")
    xs[M - 1] = float("nan")
    y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda())
    assert torch.isnan(y[M - 1]).all() and torch.isnan(y[:, 3]).all()
    keep = [c for c in range(70) if c != 3]
    assert torch.equal(y[:M - 1][:, keep], clean[:M - 1][:, keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 7), (5, 24), (64, 256), (77, 1001), (1000, 130), (2, 131071)])
def test_quantize_rows_bit_for_bit(M, K, dtype):
    import cnn_convolution_implicit_gb300 as cg
    g = torch.Generator().manual_seed(M * 7 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g) * 3)).to(dtype)
    q, s = cg.quantize_rows(x.cuda())
    wq, ws = ref.quantize_rows(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("K", [40, 33])
def test_quantize_rows_odd_rows(K):
    """Zero rows, rows too small to scale, NaN and Inf rows; their neighbours untouched."""
    import cnn_convolution_implicit_gb300 as cg
    x = torch.randn(8, K, generator=torch.Generator().manual_seed(3))
    x[1] = 0
    x[2] = 0
    x[2, 5] = 1e-38
    x[3, 7] = float("nan")
    x[4, 0] = float("-inf")
    x[5] *= 1e-28
    x[6] *= 1e36
    q, s = cg.quantize_rows(x.cuda())
    wq, ws = ref.quantize_rows(x.numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert s[1] == 0 and s[2] == 0 and torch.isnan(s[3:5]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [(1, 512, 1024), (1, 33, 77), (4, 96, 260), (8, 300, 4096), (37, 128, 200),
                                  (700, 512, 256), (260, 96, 1030)])
def test_linear_is_quantize_then_product(size, dtype):
    """The call that quantises gives the values of the two calls apart."""
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    _, _, w, ws, bias = _inputs(M, N, K, 8)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(dtype)
    y = cg.int8_linear(x.cuda(), w.cuda(), ws.cuda(), bias.cuda(), out="f32")
    q, s = ref.quantize_rows(x.float().numpy())
    want, tol = ref.int8_product(q, s, w.numpy(), ws.numpy(), bias.numpy(), "none")
    ref.check(_np(y), want, tol, False, "y")


@pytest.mark.parametrize("M", [1, 5, 150])
def test_linear_rows_that_are_not_finite(M):
    import cnn_convolution_implicit_gb300 as cg
    _, _, w, ws, bias = _inputs(M, 64, 96, 8)
    x = torch.randn(M, 96, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[M - 1, 4] = float("nan")
    y = cg.int8_linear(x.cuda(), w.cuda(), ws.cuda(), bias.cuda())
    assert torch.isnan(y[M - 1]).all() and torch.isfinite(y[:M - 1]).all()
    x[M - 1] = 0
    y = cg.int8_linear(x.cuda(), w.cuda(), ws.cuda(), bias.cuda(), out="f32")
    assert torch.equal(y[M - 1].cpu(), bias)


def test_pixels_keep_their_shape():
    import cnn_convolution_implicit_gb300 as cg
    x = torch.randn(2, 5, 7, 64, device="cuda").to(torch.bfloat16)
    _, _, w, ws, bias = (t.cuda() for t in _inputs(1, 48, 64, 2))
    assert tuple(cg.int8_linear(x, w, ws, bias).shape) == (2, 5, 7, 48)
    q, s = cg.quantize_rows(x)
    assert tuple(q.shape) == (2, 5, 7, 64)
    y = cg.int8_matmul(q, s, w, ws, bias)
    assert tuple(y.shape) == (2, 5, 7, 48) and torch.equal(y, cg.int8_linear(x, w, ws, bias))


def test_norm_to_product_chain():
    """Norm, activation, 8-bit pixels and their product, against 64 bits from the same 8-bit pixels."""
    import cnn_convolution_implicit_gb300 as cg
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 12, 10, 128, generator=g).to(torch.bfloat16).cuda()
    _, _, w, ws, bias = _inputs(1, 96, 128, 3)
    q, s = cg.group_norm_int8(x, 16, act="silu")
    y = cg.int8_matmul(q, s, w.cuda(), ws.cuda(), bias.cuda(), out="f32")
    want, tol = ref.int8_product(q.view(-1, 128).cpu().numpy(), s.cpu().numpy(), w.numpy(), ws.numpy(), bias.numpy(), "none")
    ref.check(_np(y).reshape(-1, 96), want, tol, False, "y")


@pytest.mark.parametrize("size", [(1, 512, 512), (6, 200, 300), (300, 256, 512)])
def test_side_stream_graph_and_repeat(size):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, xs, w, ws, bias = (t.cuda() for t in _inputs(M, N, K, 6))
    xb = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    plan = cg.Int8MatmulPlan(M, N, K, act="silu")
    want, want_q = plan.forward(x, xs, w, ws, bias), plan.forward_quantize(xb, w, ws, bias)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = plan.forward(x, xs, w, ws, bias, stream=side), plan.forward_quantize(xb, w, ws, bias, stream=side)
    assert plan.device_status(side) == 0
    assert torch.equal(a, want) and torch.equal(b, want_q)
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, xs, w, ws, bias, y=y)
        yq = plan.forward_quantize(xb, w, ws, bias)
    x.neg_()
    xb.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, plan.forward(x, xs, w, ws, bias)) and torch.equal(yq, plan.forward_quantize(xb, w, ws, bias))


def test_output_past_2_31_elements():
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = (1 << 20) + 77, 2112, 64
    x = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int32).to(torch.int8)
    w = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int32).to(torch.int8)
    xs, ws = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    y = cg.int8_matmul(x, xs, w, ws)
    at = torch.cat([torch.arange(100), torch.arange(M - 300, M)])
    want, tol = ref.int8_product(x[at].cpu().numpy(), xs[at].cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(), None, "none")
    ref.check(_np(y[at]), want, tol, True, "y")


def test_binding_refusals():
    import cnn_convolution_implicit_gb300 as cg
    x, xs, w, ws, bias = (t.cuda() for t in _inputs(4, 32, 48, 1))
    plan = cg.Int8MatmulPlan(4, 32, 48)
    with pytest.raises(ValueError):
        plan.forward(x.float(), xs, w, ws)
    with pytest.raises(ValueError):
        plan.forward(x, xs[:3], w, ws)
    with pytest.raises(ValueError):
        plan.forward(x, xs, w.t(), ws)
    with pytest.raises(ValueError):
        plan.forward(x, xs, w, ws, bias.cpu())
    with pytest.raises(ValueError):
        plan.forward(x, xs, w, ws, y=torch.empty(4, 32, device="cuda"))   # BF16 plan
    with pytest.raises(ValueError):
        plan.forward_quantize(x, w, ws)                                    # int8 rows need no quantiser
    with pytest.raises(ValueError):
        cg.int8_matmul(x[:, :40].contiguous(), xs, w, ws)                  # K
    with pytest.raises(ValueError):
        cg.int8_matmul(x, xs, w, ws, out="f16")
    with pytest.raises(ValueError):
        cg.quantize_rows(torch.zeros(0, 5, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [(5, 4096, 4096), (16, 512, 8192), (32, 700, 8200), (48, 96, 1000), (300, 512, 256),
                                  (65, 256, 16384), (2000, 600, 72), (129, 77, 515)])
def test_linear_reads_what_its_quantiser_wrote(size, dtype):
    """The product starts while its rows are still being quantised, into memory that holds those of
    the call before: every call gives the bits of the two calls one after the other."""
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    _, _, w, ws, bias = (t.cuda() for t in _inputs(1, N, K, 12))
    plan = cg.Int8MatmulPlan(M, N, K, out="f32")
    g = torch.Generator(device="cuda").manual_seed(M)
    rows = [(torch.randn(M, K, device="cuda", generator=g) * 2.0 ** i).to(dtype) for i in range(8)]
    want = [plan.forward(*cg.quantize_rows(x), w, ws, bias) for x in rows]
    for _ in range(4):
        got = [plan.forward_quantize(x, w, ws, bias) for x in rows]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert plan.device_status() == 0


def test_plans_of_few_rows_take_no_status_word():
    """The kernels of few rows have no waits: however many such plans are alive, a convolution's plan
    made after them has a word of its own, and theirs read 0 without touching the library's."""
    import ctypes
    import gc
    import cnn_convolution_implicit_gb300 as cg
    from cnn_convolution_implicit_gb300 import binding, operators
    binding._plan_cache.clear()  # plans other tests left alive hold words
    operators._int8_plans.clear()
    gc.collect()
    assert cg.device_status() == 0
    few = [cg.Int8MatmulPlan(m, 8, 16) for m in (1, 4, 5, 32) for _ in range(300)]
    own, many = cg.ConvPlan(1, 8, 8, 8, 8, 3, 3, 1, 1, 1, 1, "bf16"), cg.Int8MatmulPlan(400, 8, 16)
    elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream()
    assert cg.lib().conv_check_wait_timeout(1_000_000, ctypes.c_void_p(elapsed.data_ptr()),
                                            ctypes.c_void_p(stream.cuda_stream)) == 0
    assert own.device_status() == 0 and many.device_status() == 0
    assert all(few[i].device_status() == 0 for i in range(0, len(few), 100))
    assert cg.device_status() == 2 | 4  # the library's word, untouched by the reads above
    assert cg.device_status() == 0


def test_many_row_counts_leave_status_words():
    """Row counts that vary, as token counts do: the functional forms' plans stay few, a convolution's
    plan made after them has a status word of its own, and a shape that fell out comes back."""
    import ctypes
    import cnn_convolution_implicit_gb300 as cg
    from cnn_convolution_implicit_gb300 import binding, operators
    assert cg.device_status() == 0
    x, xs, w, ws, bias = (t.cuda() for t in _inputs(1400, 8, 16, 3))
    first = cg.int8_matmul(x[:100], xs[:100], w, ws, bias)
    for m in range(100, 1400):
        cg.int8_matmul(x[:m], xs[:m], w, ws, bias)
    assert len(operators._int8_plans) <= operators._int8_plans.limit
    own = cg.ConvPlan(1, 8, 8, 8, 8, 3, 3, 1, 1, 1, 1, "bf16")
    elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
    assert cg.lib().conv_check_wait_timeout(1_000_000, ctypes.c_void_p(elapsed.data_ptr()),
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert own.device_status() == 0 and cg.device_status() == 2 | 4 and cg.device_status() == 0
    assert torch.equal(cg.int8_matmul(x[:100], xs[:100], w, ws, bias), first)
    assert len(binding._plan_cache) <= binding._plan_cache.limit
