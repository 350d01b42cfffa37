"""The many-row 8-bit product in every tile shape and split of K that its rule chooses on 152 SMs,
each with rows of y on and off 16 bytes and rows of x and w on and off 16 bytes.  The sizes are
checked against the rule without a GPU, so a change of it cannot leave a kernel untested unseen."""
import pytest
import torch

import operator_refs as ref
from test_gpu_int8 import _inputs, _np

import cnn_convolution_implicit_gb300 as cg

# tile rows, columns, CTAs that share its K: M, N, K, output; y off 16 bytes and K % 16, y off, K % 16, neither
TILES = {
    (128, 32, 1): [(100, 17, 70, "bf16"), (100, 17, 128, "bf16"), (65, 16, 70, "f32"), (100, 16, 64, "bf16")],
    (128, 32, 2): [(5001, 17, 2005, "f32"), (5001, 17, 2000, "bf16"), (5001, 16, 2005, "bf16"), (5001, 16, 2000, "f32")],
    (128, 32, 4): [(65, 17, 520, "bf16"), (65, 513, 1024, "f32"), (65, 16, 520, "bf16"), (65, 512, 1024, "bf16")],
    (128, 32, 8): [(65, 17, 1030, "f32"), (100, 17, 1024, "bf16"), (65, 16, 1030, "f32"), (100, 16, 1024, "bf16")],
    (128, 64, 1): [(5001, 97, 70, "f32"), (257, 2049, 64, "bf16"), (129, 4096, 70, "bf16"), (513, 1024, 64, "f32")],
    (128, 64, 2): [(5001, 41, 1030, "f32"), (2000, 130, 1024, "bf16"), (50, 4096, 1030, "f32"), (257, 1024, 1024, "f32")],
    (128, 64, 4): [(50, 2049, 1030, "bf16"), (50, 2049, 1024, "bf16"), (50, 2048, 1030, "f32"), (3000, 40, 1024, "f32")],
    (128, 64, 8): [(385, 97, 2005, "f32"), (65, 513, 2000, "bf16"), (1000, 40, 2005, "f32"), (65, 512, 2000, "f32")],
    (128, 128, 1): [(257, 4101, 70, "f32"), (257, 4101, 64, "f32"), (129, 8192, 70, "bf16"), (513, 2048, 64, "f32")],
    (128, 128, 2): [(2000, 257, 2005, "f32"), (5001, 97, 2000, "f32"), (50, 8192, 2005, "f32"), (513, 1024, 2000, "f32"),
                    (256, 4096, 4096, "bf16"), (65, 8192, 4096, "bf16")],
    (128, 128, 4): [(257, 1031, 2005, "bf16"), (50, 4101, 2000, "f32"), (257, 1024, 2005, "bf16"), (50, 4096, 2000, "f32"),
                    (65, 4096, 4096, "bf16")],
    (128, 128, 8): [(513, 257, 4100, "bf16"), (50, 1031, 8192, "f32"), (200, 700, 4100, "f32"), (50, 1024, 8192, "bf16")],
    (256, 256, 1): [(1000, 4101, 130, "bf16"), (5001, 513, 256, "bf16"), (257, 8192, 130, "bf16"), (513, 4096, 256, "bf16")],
}
SIZES = [(tile, size) for tile, sizes in TILES.items() for size in sizes]


def _alignment(N, K, out):
    return N % (8 if out == "bf16" else 4) == 0, K % 16 == 0


def test_sizes_cover_the_rule():
    reached = {}
    for M in (33, 50, 65, 100, 129, 200, 257, 385, 513, 800, 1000, 2000, 5000, 20000, 200704):
        for N in (1, 16, 40, 64, 97, 128, 256, 513, 700, 1024, 2048, 4096, 8192, 16384):
            for K in (16, 64, 70, 130, 256, 520, 1024, 2000, 4096, 8192, 16384):
                plan = cg.Int8MatmulPlan(M, N, K)
                if plan.kernel == "tiles":
                    reached.setdefault(plan.tile, (M, N, K))
    assert set(reached) == set(TILES), "tiles without a test: %s" % {t: s for t, s in reached.items() if t not in TILES}
    for tile, sizes in TILES.items():
        assert {_alignment(N, K, out) for _, N, K, out in sizes} == {(a, b) for a in (True, False) for b in (True, False)}
        for M, N, K, out in sizes:
            plan = cg.Int8MatmulPlan(M, N, K, out)
            assert (plan.kernel, plan.tile) == ("tiles", tile), (M, N, K, out, plan.kernel, plan.tile)


def test_few_and_middling_rows_have_no_tile():
    for M, kernel in ((1, "few_rows"), (4, "few_rows"), (5, "mid_rows"), (32, "mid_rows"), (64, "mid_rows")):
        plan = cg.Int8MatmulPlan(M, 512, 512)
        assert (plan.kernel, plan.tile) == (kernel, (0, 0, 0))
    assert cg.Int8MatmulPlan(65, 512, 512).kernel == "tiles"
    assert cg.lib().conv_int8_plan_info(None, None, None, None, None) == 1
    assert cg.lib().conv_int8_plan_info(plan._plan, None, None, None, None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tile,size", SIZES)
def test_tile(tile, size):
    M, N, K, out = size
    x, xs, w, ws, bias = _inputs(M, N, K, M + 5 * N + K)
    plan = cg.Int8MatmulPlan(M, N, K, out, act="relu")
    assert plan.tile == tile
    canvas = torch.full((M * N + 64,), 7.0, device="cuda", dtype=plan.torch_dtype)
    plan.forward(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), y=canvas[:M * N].view(M, N))
    want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "relu")
    ref.check(_np(canvas[:M * N].view(M, N)), want, tol, out == "bf16", "y")
    assert torch.all(canvas[M * N:] == 7.0) and plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(1, 33, 4112), (1, 64, 16384), (2, 50, 12000), (3, 40, 5000), (4, 70, 8191), (3, 17, 12289)])
def test_few_rows_past_one_chunk_of_k(size):
    """Up to 4 rows, w in several chunks of K: exact sums, rows on and off 16 bytes."""
    M, N, K = size
    x, xs, w, ws, bias = _inputs(M, N, K, K)
    for out in ("f32", "bf16"):
        y = cg.int8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), bias.cuda(), act="relu", out=out)
        want, tol = ref.int8_product(x.numpy(), xs.numpy(), w.numpy(), ws.numpy(), bias.numpy(), "relu")
        ref.check(_np(y), want, tol, out == "bf16", "y")
    assert torch.equal(cg.int8_matmul(x.cuda(), torch.ones(M).cuda(), w.cuda(), torch.ones(N).cuda(), out="f32").cpu().double(),
                       (x.double() @ w.double().t()).float().double())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 3), (8, 1)])
def test_channels_past_2_30(M, K):
    N = (1 << 30) + 7
    x = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int32).to(torch.int8)
    w = torch.empty(N, K, dtype=torch.int8, device="cuda").random_(-127, 128)
    xs, ws = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda")
    y = cg.int8_matmul(x, xs, w, ws)
    for at in (slice(0, 200), slice(N // 2, N // 2 + 200), slice(N - 200, N)):
        want, tol = ref.int8_product(x.cpu().numpy(), xs.cpu().numpy(), w[at].cpu().numpy(), ws[at].cpu().numpy(), None, "none")
        ref.check(_np(y[:, at]), want, tol, True, "y")
