"""The norms around a block with its gate and residual (svdq_residual_norm) against the definition in 64 bits."""
import itertools

import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(seed, rows, dim, seqs, dtype, x_dtype, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    t = lambda *shape, s=1.0, o=0.0, d=dtype: (torch.randn(*shape, generator=g) * s + o).to(d).cuda()
    vectors = {"gate": t(seqs, dim), "scale": t(seqs, dim, s=0.5), "shift": t(seqs, dim),
               "post_weight": t(dim, o=1.0), "post_bias": t(dim), "weight": t(dim, o=1.0), "bias": t(dim)}
    return t(rows, dim, s=2.0, o=offset, d=x_dtype), t(rows, dim, o=0.2), vectors


def offsets(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).cuda()


def check(seed, lengths, dim, dtype, x_dtype, names, **how):
    import rank_gemm_quantize_b200 as rq
    x, y, vectors = make(seed, sum(lengths), dim, len(lengths), dtype, x_dtype)
    how.update({n: vectors[n] for n in names})
    got = rq.residual_norm(x, y, offsets=offsets(lengths), **how)
    sequence = torch.repeat_interleave(torch.tensor(lengths))
    for g, w, what in zip(got, ops.residual_norm(x, y, sequence, **how), ("x", "h")):
        if w is None:
            assert g is None
        else:
            ops.check(g, *w, what=what)


@pytest.mark.parametrize("dim", [1, 7, 8, 31, 64, 130, 256, 257, 512, 513, 520, 1030, 2048, 2056, 4095, 4104, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("dtype,x_dtype", [(BF16, BF16), (F16, F32)])
def test_dims(dim, dtype, x_dtype):
    check(1, [3, 0, 2], dim, dtype, x_dtype, ["gate", "scale", "shift", "weight", "post_weight"], norm="layer",
          post_norm="rms", residual_scale=0.7)


@pytest.mark.parametrize("norm,post_norm", list(itertools.product([None, "layer", "rms"], repeat=2)))
@pytest.mark.parametrize("dtype,x_dtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_norms_and_types(norm, post_norm, dtype, x_dtype):
    names = ["gate"] + ["weight", "bias", "scale", "shift"] * (norm is not None) + ["post_weight", "post_bias"] * (post_norm is not None)
    for dim in (384, 99):
        check(2, [1, 9, 4], dim, dtype, x_dtype, names, norm=norm, post_norm=post_norm)
        check(3, [1, 9, 4], dim, dtype, x_dtype, [], norm=norm, post_norm=post_norm, residual_scale=-0.3, eps=1e-3)


def test_first_norm_without_a_block():
    import rank_gemm_quantize_b200 as rq
    for x_dtype in (BF16, F32):
        x, _, v = make(4, 11, 640, 1, BF16, x_dtype)
        x2, h = rq.residual_norm(x, norm="layer", scale=v["scale"][0], shift=v["shift"], weight=v["weight"], dtype=BF16)
        assert x2 is x and h.dtype == BF16
        want = ops.residual_norm(x, None, torch.zeros(11, dtype=torch.long), norm="layer", scale=v["scale"], shift=v["shift"],
                                 weight=v["weight"])
        ops.check(h, *want[1])


def test_large_mean_and_constant_rows():
    """Rows whose mean is a thousand times their deviation, constant ones and zeros."""
    import rank_gemm_quantize_b200 as rq
    x, y, _ = make(5, 6, 1024, 1, F16, F32, offset=3000.0)
    x[1] = 17.0
    y[1] = 0
    x[2] = 0
    y[2] = 0
    for norm in ("layer", "rms"):
        got = rq.residual_norm(x, y, norm=norm)
        for g, w in zip(got, ops.residual_norm(x, y, torch.zeros(6, dtype=torch.long), norm=norm)):
            ops.check(g, *w, what=norm)


def test_infinities_and_nan_stay_in_their_rows():
    import rank_gemm_quantize_b200 as rq
    x, y, _ = make(6, 9, 300, 1, BF16, BF16)
    clean = rq.residual_norm(x, y, norm="layer", post_norm="rms")
    x[4, 7], y[6, 0] = float("inf"), float("nan")
    got = rq.residual_norm(x, y, norm="layer", post_norm="rms")
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert all(torch.equal(g[keep], c[keep]) for g, c in zip(got, clean))
    assert got[1][4].isnan().all() and got[0][6].isnan().all() and got[0][4, 7] == float("inf")


@pytest.mark.parametrize("dim", [256, 2050])
def test_rows_of_no_sequence_stay(dim):
    import rank_gemm_quantize_b200 as rq
    x, y, v = make(7, 20, dim, 2, BF16, BF16)
    out_x, out_h = torch.full_like(x, 7.0), torch.full_like(x, 9.0)
    o = torch.tensor([3, 8, 15], dtype=torch.int32).cuda()
    rq.residual_norm(x, y, offsets=o, gate=v["gate"], out_x=out_x, out_h=out_h)
    for rows in (slice(0, 3), slice(15, 20)):
        assert (out_x[rows] == 7).all() and (out_h[rows] == 9).all()
    sequence = torch.tensor([0] * 5 + [1] * 7)
    want = ops.residual_norm(x[3:15], y[3:15], sequence, gate=v["gate"])
    ops.check(out_x[3:15], *want[0])
    ops.check(out_h[3:15], *want[1])


@pytest.mark.parametrize("bad", [[-9, 4, 2], [0, 1 << 30, 5], [30, 20, 10], [-(1 << 31), (1 << 31) - 1, 0]])
def test_bad_offsets_stay_inside_the_tensors(bad):
    import rank_gemm_quantize_b200 as rq
    x, y, v = make(8, 20, 136, 2, BF16, BF16)
    rq.residual_norm(x, y, offsets=torch.tensor(bad, dtype=torch.int32).cuda(), gate=v["gate"])
    torch.cuda.synchronize()
    ops.check(rq.residual_norm(x, y)[0], *ops.residual_norm(x, y, torch.zeros(20, dtype=torch.long))[0])


def test_in_place():
    import rank_gemm_quantize_b200 as rq
    for dim in (64, 1000, 5000):
        x, y, v = make(9, 13, dim, 1, BF16, BF16)
        want = rq.residual_norm(x, y, norm="layer", post_norm="layer", gate=v["gate"])
        got = rq.residual_norm(x, y, norm="layer", post_norm="layer", gate=v["gate"], out_x=x, out_h=y)
        assert got[0] is x and got[1] is y
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_many_sequences_and_a_graph():
    import rank_gemm_quantize_b200 as rq
    g = torch.Generator().manual_seed(10)
    lengths = torch.randint(0, 4, (300,), generator=g).tolist()
    rows, o = sum(lengths), offsets(lengths)
    x, y, v = make(11, rows, 72, 300, BF16, F32)
    how = {n: v[n] for n in ("gate", "scale", "shift")}
    rq.residual_norm(x, y, offsets=o, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rq.residual_norm(x, y, offsets=o, **how)
    x.mul_(0.5)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = rq.residual_norm(x, y, offsets=o, **how, stream=side)
    torch.cuda.synchronize()
    want = ops.residual_norm(x, y, torch.repeat_interleave(torch.tensor(lengths)), **how)
    for a, b, w in zip(got, other, want):
        assert torch.equal(a, b)
        ops.check(a, *w)


def test_nothing_to_do():
    import rank_gemm_quantize_b200 as rq
    x, y, v = make(12, 0, 64, 1, BF16, BF16)
    x1, h = rq.residual_norm(x, y, gate=v["gate"])
    assert x1.shape == h.shape == (0, 64)
