"""What the calls around the quantized layers refuse, without a GPU: every bad call
returns SVDQ_ERR_INVALID_ARG or SVDQ_ERR_UNSUPPORTED before any device work (the
pointers are never dereferenced), and the binding raises ValueError."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # a 16-byte-aligned address that is never touched
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def rq():
    import rank_gemm_quantize_b200 as rq
    from rank_gemm_quantize_b200 import build
    build.build()
    return rq


def refused(rq, status, want, message):
    assert status == want, (status, rq.lib().svdq_last_error())
    assert message in rq.lib().svdq_last_error()


def attention_args(rq, **change):
    c = rq._Attention(dtype=0, batch=1, q_rows=4, k_rows=9, q_heads=4, kv_heads=2, head_dim=64, causal=1, scale=0.125,
                      q_row_stride=256, q_head_stride=64, k_row_stride=128, k_head_stride=64, v_row_stride=128,
                      v_head_stride=64, q=FAKE, k=FAKE, v=FAKE, q_offsets=FAKE, k_offsets=FAKE, out=FAKE, workspace=FAKE,
                      workspace_bytes=1 << 30)
    for name, value in change.items():
        setattr(c, name, value)
    return c


@pytest.mark.parametrize("change,status,message", [
    (dict(dtype=2), INVALID, b"dtype"), (dict(dtype=-1), INVALID, b"dtype"), (dict(batch=0), INVALID, b"batch"),
    (dict(batch=65536), UNSUPPORTED, b"batch"), (dict(q_rows=-1), INVALID, b"q_rows"), (dict(k_rows=-1), INVALID, b"k_rows"),
    (dict(kv_heads=3), INVALID, b"kv_heads"), (dict(kv_heads=0), INVALID, b"kv_heads"),
    (dict(q_heads=258, kv_heads=2), INVALID, b"128 times"), (dict(head_dim=0), INVALID, b"head_dim"),
    (dict(head_dim=60), INVALID, b"head_dim"), (dict(head_dim=136), INVALID, b"head_dim"), (dict(causal=2), INVALID, b"causal"),
    (dict(scale=0.0), INVALID, b"scale"), (dict(scale=-1.0), INVALID, b"scale"), (dict(scale=float("nan")), INVALID, b"scale"),
    (dict(scale=float("inf")), INVALID, b"scale"), (dict(scale=1e31), INVALID, b"scale"), (dict(q_rows=1 << 29), UNSUPPORTED, b"2^30"),
    (dict(q_row_stride=100), INVALID, b"strides"), (dict(k_row_stride=0), INVALID, b"strides"),
    (dict(v_head_stride=-64), INVALID, b"strides"), (dict(k_head_stride=1 << 38), INVALID, b"strides"),
])
def test_attention_refuses_bad_configurations(rq, change, status, message):
    c, n = attention_args(rq, **change), ctypes.c_size_t()
    refused(rq, rq.lib().svdq_attention_workspace_size(ctypes.byref(c), ctypes.byref(n)), status, message)
    refused(rq, rq.lib().svdq_attention_forward(ctypes.byref(c), None), status, message)


@pytest.mark.parametrize("q,k,v,qo,ko,out,batch,message", [
    (None, FAKE, FAKE, FAKE, FAKE, FAKE, 1, b"NULL"), (FAKE, None, FAKE, FAKE, FAKE, FAKE, 1, b"NULL"),
    (FAKE, FAKE, None, FAKE, FAKE, FAKE, 1, b"NULL"), (FAKE, FAKE, FAKE, FAKE, FAKE, None, 1, b"NULL"),
    (FAKE + 8, FAKE, FAKE, FAKE, FAKE, FAKE, 1, b"aligned"), (FAKE, FAKE + 2, FAKE, FAKE, FAKE, FAKE, 1, b"aligned"),
    (FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 4, 1, b"aligned"), (FAKE, FAKE, FAKE, FAKE + 2, FAKE, FAKE, 1, b"offsets"),
    (FAKE, FAKE, FAKE, None, FAKE, FAKE, 2, b"offsets"), (FAKE, FAKE, FAKE, FAKE, None, FAKE, 2, b"offsets"),
])
def test_attention_refuses_bad_pointers(rq, q, k, v, qo, ko, out, batch, message):
    c = attention_args(rq, batch=batch, q=q, k=k, v=v, q_offsets=qo, k_offsets=ko, out=out)
    refused(rq, rq.lib().svdq_attention_forward(ctypes.byref(c), None), INVALID, message)
    assert rq.lib().svdq_attention_forward(None, None) == INVALID
    assert rq.lib().svdq_attention_workspace_size(ctypes.byref(c), None) == INVALID


@pytest.mark.parametrize("change,status,message", [
    (dict(dtype=2), INVALID, b"dtype"), (dict(activation=5), INVALID, b"activation"), (dict(activation=-1), INVALID, b"activation"),
    (dict(M=-1), INVALID, b"M must"), (dict(K=0), INVALID, b"multiples of 8"), (dict(K=12), INVALID, b"multiples of 8"),
    (dict(N=100), INVALID, b"multiples of 8"), (dict(M=1 << 23), UNSUPPORTED, b"exceeds"), (dict(X=None), INVALID, b"NULL"),
    (dict(W=None), INVALID, b"NULL"), (dict(Y=None), INVALID, b"NULL"), (dict(X=FAKE + 2), INVALID, b"aligned"),
    (dict(W=FAKE + 8), INVALID, b"aligned"), (dict(bias=FAKE + 4), INVALID, b"aligned"),
    (dict(residual=FAKE + 2), INVALID, b"aligned"), (dict(Y=FAKE + 8), INVALID, b"aligned"),
])
def test_linear_refuses_bad_arguments(rq, change, status, message):
    a = rq._DenseLinear(dtype=0, activation=0, M=4, K=64, N=64, X=FAKE, W=FAKE, Y=FAKE)
    for name, value in change.items():
        setattr(a, name, value)
    refused(rq, rq.lib().svdq_dense_linear_forward(ctypes.byref(a), None), status, message)
    assert rq.lib().svdq_dense_linear_forward(None, None) == INVALID


def norm_args(rq, **change):
    a = rq._ResidualNorm(dtype=0, x_dtype=0, rows=4, dim=64, seqs=1, post_norm=0, norm=2, residual_scale=1.0, eps=1e-6,
                         x=FAKE, y=FAKE, x_out=FAKE, h_out=FAKE)
    for name, value in change.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("change,status,message", [
    (dict(dtype=2), INVALID, b"dtype"), (dict(x_dtype=1), INVALID, b"x_dtype"), (dict(rows=-1), INVALID, b"rows"),
    (dict(dim=0), INVALID, b"dim"), (dict(dim=16385), UNSUPPORTED, b"dim"), (dict(seqs=0), INVALID, b"seqs"),
    (dict(norm=3), INVALID, b"norm"), (dict(post_norm=-1), INVALID, b"norm"), (dict(eps=-1.0), INVALID, b"eps"),
    (dict(eps=float("nan")), INVALID, b"eps"), (dict(residual_scale=float("inf")), INVALID, b"residual_scale"),
    (dict(seqs=2), INVALID, b"offsets"), (dict(y=None), INVALID, b"without y"), (dict(y=None, x_out=None, gate=FAKE), INVALID, b"without y"),
    (dict(y=None, x_out=None, residual_scale=2.0), INVALID, b"without y"), (dict(post_weight=FAKE), INVALID, b"post norm"),
    (dict(norm=0), INVALID, b"without a norm"), (dict(norm=0, h_out=None, shift=FAKE), INVALID, b"without a norm"),
    (dict(y=None, x_out=None, norm=0, h_out=None), INVALID, b"nothing to do"), (dict(x=None), INVALID, b"NULL"),
    (dict(x_out=None), INVALID, b"NULL"), (dict(h_out=None), INVALID, b"NULL"), (dict(x=FAKE + 8), INVALID, b"aligned"),
    (dict(scale=FAKE + 2), INVALID, b"aligned"), (dict(offsets=FAKE + 2), INVALID, b"offsets"),
])
def test_norm_refuses_bad_arguments(rq, change, status, message):
    a = norm_args(rq, **change)
    refused(rq, rq.lib().svdq_residual_norm(ctypes.byref(a), None), status, message)
    assert rq.lib().svdq_residual_norm(None, None) == INVALID


def test_nothing_to_do_is_no_error(rq):
    c = attention_args(rq, q_rows=0, q=None, out=None)
    assert rq.lib().svdq_attention_forward(ctypes.byref(c), None) == 0
    assert rq.lib().svdq_dense_linear_forward(ctypes.byref(rq._DenseLinear(M=0, K=64, N=64)), None) == 0
    assert rq.lib().svdq_residual_norm(ctypes.byref(norm_args(rq, rows=0, x=None, y=None, x_out=None, h_out=None)), None) == 0


def test_binding_refuses_tensors_off_the_gpu(rq):
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: rq.attention(t, t, t), lambda: rq.linear(t[0], t[0].T.contiguous()), lambda: rq.residual_norm(t[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_unknown_names(rq):
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation"):
        rq.linear(t, t.T.contiguous(), activation="swish")
    with pytest.raises(ValueError, match="norm"):
        rq.residual_norm(t, norm="batch")
    with pytest.raises(ValueError, match="float32"):
        rq.residual_norm(t.double())
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        rq.linear(t.float(), t.float())


@pytest.mark.parametrize("kernels", [-1, 3])
def test_selftest_refuses_unknown_kernels(rq, kernels):
    refused(rq, rq.lib().svdq_selftest_operator_wait(kernels, None), INVALID, b"kernels")


def test_attention_refuses_work_that_passes_64_bits(rq):
    """Overlapping offsets can give each of 65535 sequences 2^16 row tiles and 2^24 key tiles."""
    c = attention_args(rq, batch=65535, q_rows=65535, q_heads=16, kv_heads=1, q_row_stride=1024, k_row_stride=64, v_row_stride=64,
                       k_rows=1 << 30)
    n = ctypes.c_size_t()
    refused(rq, rq.lib().svdq_attention_workspace_size(ctypes.byref(c), ctypes.byref(n)), UNSUPPORTED, b"too large")
    refused(rq, rq.lib().svdq_attention_forward(ctypes.byref(c), None), UNSUPPORTED, b"too large")
