"""The status words of attention and the 16-bit linear layer: a wait that gives up is reported once, and the next
calls are right."""
import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def calls():
    """One call of each kernel whose waits the words record: few and many queries, few and many tiles."""
    import rank_gemm_quantize_b200 as rq
    g = torch.Generator().manual_seed(1)
    t = lambda *shape: torch.randn(*shape, generator=g).to(BF16).cuda()
    for n, m in ((1, 9000), (300, 300)):
        q, k, v = t(n, 4, 64), t(m, 2, 64), t(m, 2, 64)
        ops.check(rq.attention(q, k, v, causal=True), *ops.attention(q, k, v, [n], [m], True))
    for M, N in ((5, 136), (1030, 1000)):
        X, W = t(M, 264), t(264, N)
        ops.check(rq.linear(X, W), *ops.linear(X, W, None, None, None))


@pytest.mark.parametrize("kernels", [0, 1, 2])
def test_a_wait_that_gives_up_is_reported_once(kernels):
    import rank_gemm_quantize_b200 as rq
    calls()
    assert rq.operator_status() == rq.Status.OK
    rq.selftest_operator_wait(kernels)
    assert rq.operator_status() == rq.Status.DEVICE_TIMEOUT
    assert rq.operator_status() == rq.Status.OK
    calls()
    assert rq.operator_status() == rq.Status.OK


def test_several_words_are_one_status():
    import rank_gemm_quantize_b200 as rq
    for kernels in (2, 0):
        rq.selftest_operator_wait(kernels)
    assert rq.operator_status() == rq.Status.DEVICE_TIMEOUT
    assert rq.operator_status() == rq.Status.OK
