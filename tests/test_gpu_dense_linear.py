"""The linear layer in 16 bits with its epilogue (svdq_dense_linear_forward) against its definition in 64 bits."""
import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def make(seed, M, K, N, dtype, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = lambda *shape, s=1.0: (torch.randn(*shape, generator=g) * s).to(dtype).cuda()
    return t(M, K), t(K, N, s=0.05), t(N) if bias else None, t(M, N) if residual else None


def check(seed, M, K, N, dtype, activation=None, bias=True, residual=True):
    import rank_gemm_quantize_b200 as rq
    X, W, b, r = make(seed, M, K, N, dtype, bias, residual)
    Y = rq.linear(X, W, b, activation, r)
    torch.cuda.synchronize()
    assert rq.operator_status() == rq.Status.OK
    ops.check(Y, *ops.linear(X, W, b, activation, r))


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 255, 257])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows(M, dtype):
    check(1, M, 264, 136, dtype)


@pytest.mark.parametrize("K", [8, 16, 56, 64, 72, 512, 1032, 4104])
@pytest.mark.parametrize("M", [3, 200])
def test_inner_sizes(K, M):
    check(2, M, K, 144, BF16)


@pytest.mark.parametrize("N", [8, 64, 72, 128, 136, 1000, 2056])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_outer_sizes(N, M):
    check(3, M, 328, N, F16)


@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N", [(5, 640, 256), (700, 256, 512), (2100, 192, 1032)])
@pytest.mark.parametrize("bias,residual", [(True, True), (False, False)])
def test_epilogue(activation, M, K, N, bias, residual):
    check(4, M, K, N, BF16, activation, bias, residual)


@pytest.mark.parametrize("activation", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activation_over_its_range(activation):
    """One input times weight 1: every bf16 value from -30 to 30 goes through the activation alone."""
    import rank_gemm_quantize_b200 as rq
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    values = bits[bits.float().abs() <= 30]
    X = torch.zeros(values.numel(), 8, dtype=BF16)
    X[:, 0] = values
    W = torch.zeros(8, 8, dtype=BF16)
    W[0] = 1
    Y = rq.linear(X.cuda(), W.cuda(), activation=activation)
    ops.check(Y, *ops.linear(X, W, None, activation, None))
    assert torch.equal(Y, Y[:, :1].expand(-1, 8))


@pytest.mark.parametrize("M,K,N", [(1, 2048, 9216), (37, 2056, 1000), (300, 1536, 640), (1500, 512, 1536)])
def test_larger(M, K, N):
    check(5, M, K, N, BF16, "silu")


@pytest.mark.parametrize("M,K,N", [(9000, 64, 8), (8500, 8, 72), (300, 40, 8200), (257, 1000, 8192), (4097, 520, 1000)])
def test_many_tiles(M, K, N):
    """Two SMs a tile: one column block or row block, a ragged last one, little to sum."""
    check(11, M, K, N, BF16, "gelu_tanh")
    check(12, M, K, N, F16, None, bias=False)


def test_two_calls_at_once():
    """On two streams, large and small, each right."""
    import rank_gemm_quantize_b200 as rq
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    cases = [make(13, 2000, 1024, 1032, BF16), make(14, 3, 4096, 2048, BF16)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [rq.linear(X, W, b, "relu", r, stream=s) for (X, W, b, r), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for y, (X, W, b, r) in zip(got, cases):
        ops.check(y, *ops.linear(X, W, b, "relu", r))


def test_in_place_on_the_residual():
    import rank_gemm_quantize_b200 as rq
    for M in (4, 150, 1200):
        X, W, b, r = make(6, M, 256, 392, BF16)
        want = ops.linear(X, W, b, None, r)
        assert rq.linear(X, W, b, residual=r, out=r) is r
        ops.check(r, *want)


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    import rank_gemm_quantize_b200 as rq
    for M in (20, 400):
        X, W, b, r = make(7, M, 136, 264, BF16)
        X[3, 5] = float("inf")
        X[M - 1, 0] = float("nan")
        r[7, 9] = float("-inf")
        Y = rq.linear(X, W, b, None, r)
        ops.check(Y, *ops.linear(X, W, b, None, r))


@pytest.mark.parametrize("M", [6, 900])
def test_graph_stream_and_repetition(M):
    import rank_gemm_quantize_b200 as rq
    X, W, b, r = make(8, M, 1024, 520, BF16)
    first = rq.linear(X, W, b, "gelu", r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = rq.linear(X, W, b, "gelu", r, stream=side)
    c = rq.linear(X, W, b, "gelu", r)
    torch.cuda.synchronize()
    assert torch.equal(first, a) and torch.equal(first, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = rq.linear(X, W, b, "gelu", r)
    X.copy_(X.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    ops.check(captured, *ops.linear(X, W, b, "gelu", r))


def test_what_lies_around_the_output_stays():
    import rank_gemm_quantize_b200 as rq
    for M in (3, 131, 1030):
        X, W, b, _ = make(9, M, 72, 136, BF16)
        big = torch.full((M + 64, 136), 5.0, dtype=BF16, device="cuda")
        rq.linear(X, W, b, out=big[32:32 + M])
        assert (big[:32] == 5).all() and (big[32 + M:] == 5).all()
        ops.check(big[32:32 + M], *ops.linear(X, W, b, None, None))


def test_nothing_to_do():
    import rank_gemm_quantize_b200 as rq
    X, W, b, r = make(10, 0, 64, 64, BF16)
    assert rq.linear(X, W, b, "relu", r).shape == (0, 64)


# More than 37 tiles of 256 x 128 go to pairs of SMs, more than 74 in tiles of 256 columns.
PAIRS = [(1030, 264, 1000), (10000, 72, 8), (300, 136, 2600), (20000, 64, 8), (2600, 200, 1032)]


@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N", PAIRS)
@pytest.mark.parametrize("dtype,bias,residual", [(BF16, True, True), (F16, False, False), (BF16, True, False), (F16, False, True)])
def test_pairs(M, K, N, dtype, activation, bias, residual):
    check(21, M, K, N, dtype, activation, bias, residual)


@pytest.mark.parametrize("M,K,N", PAIRS)
def test_pairs_in_place_in_a_graph_with_infinities(M, K, N):
    import rank_gemm_quantize_b200 as rq
    X, W, b, r = make(22, M, K, N, BF16)
    X[3, 5] = float("inf")
    X[M - 1, 0] = float("nan")
    r[7, 5] = float("-inf")
    start, want = r.clone(), ops.linear(X, W, b, "relu", r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.linear(X, W, b, "relu", r, out=r)
    for _ in range(2):
        r.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        ops.check(r, *want)


@pytest.mark.parametrize("M,K,N", PAIRS)
def test_what_lies_around_the_output_of_pairs_stays(M, K, N):
    import rank_gemm_quantize_b200 as rq
    X, W, b, _ = make(23, M, K, N, BF16)
    around = torch.full((M + 300, N), 3.0, dtype=BF16, device="cuda")
    rq.linear(X, W, b, out=around[:M])
    torch.cuda.synchronize()
    ops.check(around[:M], *ops.linear(X, W, b, None, None))
    assert (around[M:] == 3).all()
