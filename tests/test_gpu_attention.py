"""Attention of packed sequences (svdq_attention_forward) against its definition in 64 bits."""
import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def make(seed, q_lengths, k_lengths, heads, kv_heads, dim, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    t = lambda n, h, s=1.0: (torch.randn(n, h, dim, generator=g) * s).to(dtype).cuda()
    return t(sum(q_lengths), heads, spread), t(sum(k_lengths), kv_heads), t(sum(k_lengths), kv_heads)


def offsets(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).cuda()


def run(q, k, v, q_lengths, k_lengths, causal, **how):
    import rank_gemm_quantize_b200 as rq
    o = rq.attention(q, k, v, offsets(q_lengths), offsets(k_lengths), causal=causal, **how)
    torch.cuda.synchronize()
    assert rq.operator_status() == rq.Status.OK
    return o


def check(seed, q_lengths, k_lengths, heads, kv_heads, dim, dtype, causal, scale=None):
    q, k, v = make(seed, q_lengths, k_lengths, heads, kv_heads, dim, dtype)
    o = run(q, k, v, q_lengths, k_lengths, causal, scale=scale)
    ops.check(o, *ops.attention(q, k, v, q_lengths, k_lengths, causal, scale))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127, 1, 129], [300, 0, 5, 257]])
def test_prompts(lengths, causal):
    check(1, lengths, lengths, 4, 2, 64, BF16, causal)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (6, 2), (5, 5), (40, 1), (128, 1)])
@pytest.mark.parametrize("lengths", [[70, 9], [1, 1, 1]])
def test_groups(heads, kv_heads, lengths):
    check(2, lengths, [n + 61 for n in lengths], heads, kv_heads, 64, BF16, True)


@pytest.mark.parametrize("dim", [8, 24, 64, 72, 96, 120, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_lengths", [[140], [1, 3]])
def test_head_dims(dim, dtype, q_lengths):
    check(3, q_lengths, [n + 90 for n in q_lengths], 4, 2, dim, dtype, True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("k_lengths", [[1], [64], [777], [5000, 1, 63, 2047], [0, 20, 0, 9000], [30000], [40000, 3, 900],
                                       [500] * 19 + [0, 1, 3000, 64, 65] * 3])
def test_single_tokens(k_lengths, dtype):
    check(4, [1] * len(k_lengths), k_lengths, 8, 2, 128, dtype, True)


@pytest.mark.parametrize("q_lengths,k_lengths", [([2, 8, 17], [4000, 100, 2500]), ([33], [9001]), ([70, 1], [3000, 8000]),
                                                ([3, 11, 1], [30000, 20000, 50]), ([2] * 30, [100, 1200, 7] * 10)])
@pytest.mark.parametrize("causal", [False, True])
def test_pieces_of_long_sequences(q_lengths, k_lengths, causal):
    check(5, q_lengths, k_lengths, 8, 2, 128, BF16, causal)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_long_prompts(dtype, dim, causal):
    check(6, [1100, 513, 256], [1100, 700, 256], 4, 2, dim, dtype, causal)


@pytest.mark.parametrize("q_lengths,k_lengths", [([5, 200], [2, 60]), ([3], [0]), ([300, 2], [1, 1])])
def test_queries_that_see_no_key_give_zero(q_lengths, k_lengths):
    q, k, v = make(7, q_lengths, k_lengths, 4, 2, 64, BF16)
    o = run(q, k, v, q_lengths, k_lengths, True)
    ops.check(o, *ops.attention(q, k, v, q_lengths, k_lengths, True))
    at = 0
    for n, m in zip(q_lengths, k_lengths):
        assert not o[at:at + max(0, n - m)].count_nonzero()
        at += n


@pytest.mark.parametrize("before", [30, 2500, 20000])
@pytest.mark.parametrize("q_lengths", [[1, 1, 1], [150, 300, 70], [20, 20, 20], [3, 40, 3]])
def test_what_a_query_does_not_see_does_not_reach_it(q_lengths, before):
    """Infinities and NaN in the keys and values behind a query and in other sequences; a
    sequence's own last key is seen by its last query, which gets what the definition gives."""
    k_lengths = [n + before for n in q_lengths]
    q, k, v = make(8, q_lengths, k_lengths, 4, 2, 64, BF16)
    starts = [0, k_lengths[0], k_lengths[0] + k_lengths[1]]
    k[starts[1]:starts[2]] = float("nan")  # the whole middle sequence
    v[starts[1]:starts[2]] = float("inf")
    v[starts[1] - 1, 0, 3] = float("inf")  # last value of the first one
    v[starts[1] - 1, 1, 5] = float("nan")
    v[-2, 1, 1] = float("-inf")
    v[-1, 1, 2] = float("nan")
    o = run(q, k, v, q_lengths, k_lengths, True)
    a, b = q_lengths[0], q_lengths[0] + q_lengths[1]
    assert o[a:b].isnan().all()
    for rows, keys, n, m in ((slice(0, a), slice(0, starts[1]), q_lengths[0], k_lengths[0]),
                             (slice(b, None), slice(starts[2], None), q_lengths[2], k_lengths[2])):
        ops.check(o[rows], *ops.attention(q[rows], k[keys], v[keys], [n], [m], True))


def test_large_scores_and_scales():
    """Scores of hundreds: one key takes all; and a scale that makes all keys alike."""
    q, k, v = make(9, [40, 1], [200, 900], 4, 2, 64, BF16, spread=40.0)
    for scale in (None, 1e-6, 2.0):
        o = run(q, k, v, [40, 1], [200, 900], True, scale=scale)
        ops.check(o, *ops.attention(q, k, v, [40, 1], [200, 900], True, scale), what=f"scale {scale}")


@pytest.mark.parametrize("lengths", [[300, 77], [1, 1, 1, 1]])
def test_views_of_a_joint_projection(lengths):
    """q, k and v as views of one [rows, (heads + 2 kv heads) dim] matrix, and a transposed layout."""
    import rank_gemm_quantize_b200 as rq
    heads, kv, dim, rows = 6, 2, 64, sum(lengths)
    g = torch.Generator().manual_seed(10)
    y = torch.randn(rows, (heads + 2 * kv) * dim, generator=g).to(BF16).cuda()
    q, k, v = y.view(rows, heads + 2 * kv, dim).split([heads, kv, kv], 1)
    want = ops.attention(q, k, v, lengths, lengths, True)
    o = rq.attention(q, k, v, offsets(lengths), causal=True)
    ops.check(o, *want)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]  # [heads, rows, dim] in memory
    assert torch.equal(rq.attention(*turned, offsets(lengths), causal=True), o)


def test_one_sequence_needs_no_offsets():
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(11, [200], [200], 4, 2, 64, BF16)
    assert torch.equal(rq.attention(q, k, v, causal=True), run(q, k, v, [200], [200], True))
    assert torch.equal(rq.attention(q[:1], k, v), run(q[:1], k, v, [1], [200], False))


@pytest.mark.parametrize("n,more", [(1, 0), (130, 0), (1, 30000), (130, 3000)])
def test_rows_behind_the_last_sequence_stay(n, more):
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(12, [n, n, n], [500 + more, 20, 80], 4, 2, 64, BF16)
    out = torch.full_like(q, 7.0)
    o = rq.attention(q, k, v, offsets([n, n]), offsets([500 + more, 20]), causal=True, out=out)
    assert o is out and (out[2 * n:] == 7).all()
    ops.check(out[:2 * n], *ops.attention(q[:2 * n], k[:520 + more], v[:520 + more], [n, n], [500 + more, 20], True))


@pytest.mark.parametrize("bad", [[0, 900, 300], [-5, 20, 1 << 30], [300, 200, 100], [-(1 << 31), (1 << 31) - 1, 7]])
def test_bad_offsets_stay_inside_the_tensors(bad):
    """Offsets that leave the tensors or run backwards give some result, and the next call is right."""
    import rank_gemm_quantize_b200 as rq
    for n, m in ((2, 600), (2, 40000), (300, 600), (300, 9000)):
        q, k, v = make(13, [n], [m], 4, 2, 64, BF16)
        o = torch.tensor(bad, dtype=torch.int32).cuda()
        rq.attention(q, k, v, o, o, causal=True)
        torch.cuda.synchronize()
        assert rq.operator_status() == rq.Status.OK
        ops.check(run(q, k, v, [n], [m], True), *ops.attention(q, k, v, [n], [m], True))


@pytest.mark.parametrize("q_lengths,k_lengths", [([1] * 5, [700, 3000, 1, 64, 200]), ([1, 1], [40000, 900]), ([400, 130], [400, 900]),
                                                ([300], [6000])])
def test_graph_stream_and_repetition(q_lengths, k_lengths):
    """Captured and replayed on new inputs, on another stream, twice at once, and bit for bit alike."""
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(14, q_lengths, k_lengths, 8, 2, 128, BF16)
    qo, ko = offsets(q_lengths), offsets(k_lengths)
    first = rq.attention(q, k, v, qo, ko, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = rq.attention(q, k, v, qo, ko, causal=True, stream=side)
    b = rq.attention(q, k, v, qo, ko, causal=True)
    torch.cuda.synchronize()
    assert torch.equal(first, a) and torch.equal(first, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = rq.attention(q, k, v, qo, ko, causal=True)
    q2, k2, v2 = make(15, q_lengths, k_lengths, 8, 2, 128, BF16)
    for t, n in ((q, q2), (k, k2), (v, v2)):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    ops.check(captured, *ops.attention(q2, k2, v2, q_lengths, k_lengths, True))


def test_given_workspace_and_its_check():
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(16, [1, 1], [30000, 900], 4, 2, 64, BF16)
    need = rq.attention_workspace_size(q, k, v, batch=2)
    assert need > 0
    qo, ko = offsets([1, 1]), offsets([30000, 900])
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    o = rq.attention(q, k, v, qo, ko, workspace=ws)
    assert torch.equal(o, rq.attention(q, k, v, qo, ko))
    assert (ws[need:] == 0xFF).all()
    with pytest.raises(rq.SvdqError, match="workspace"):
        rq.attention(q, k, v, qo, ko, workspace=ws[:256])


def test_many_sequences():
    """More sequences than threads of a CTA, most of them short or empty."""
    g = torch.Generator().manual_seed(17)
    k_lengths = torch.randint(0, 40, (700,), generator=g).tolist()
    q_lengths = [min(1, n) for n in k_lengths]
    k_lengths[13] = 2500
    check(18, q_lengths, k_lengths, 2, 1, 64, BF16, True)


def test_many_prompts():
    """More sequences than lanes of a warp, through the kernel for many queries."""
    g = torch.Generator().manual_seed(22)
    lengths = torch.randint(30, 200, (45,), generator=g).tolist()
    lengths[7] = 0
    check(23, lengths, [n + 3 for n in lengths], 4, 2, 64, BF16, True)


def test_scores_that_keep_growing():
    """Keys in the order of their scores: the running maximum grows all along, far past any threshold."""
    for n, m, dtype in ((1, 3000, F16), (200, 1500, BF16), (150, 1200, F16)):
        q, k, v = make(24, [n], [m], 2, 1, 64, dtype)
        direction = torch.zeros(64)
        direction[0] = 1
        k[:, 0] = (torch.linspace(-20, 20, m)[:, None] * direction).to(dtype).cuda() + 0.1 * k[:, 0]
        q[:] = (30 * direction).to(dtype).cuda()
        for causal in (False, True):
            ops.check(run(q, k, v, [n], [m], causal), *ops.attention(q, k, v, [n], [m], causal))


@pytest.mark.parametrize("q_lengths,k_lengths", [([1, 1], [900, 30]), ([1, 1], [30000, 500]), ([200], [200]), ([300, 20], [5000, 900])])
def test_two_calls_at_once(q_lengths, k_lengths):
    """The same call on two streams, with workspaces of their own."""
    import rank_gemm_quantize_b200 as rq
    inputs = [make(s, q_lengths, k_lengths, 4, 2, 128, BF16) for s in (25, 26)]
    qo, ko = offsets(q_lengths), offsets(k_lengths)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [rq.attention(q, k, v, qo, ko, causal=True, stream=s) for (q, k, v), s in zip(inputs, streams)]
    torch.cuda.synchronize()
    for o, (q, k, v) in zip(got, inputs):
        ops.check(o, *ops.attention(q, k, v, q_lengths, k_lengths, True))


def test_keys_and_queries_of_one_tensor_and_one_row():
    """q, k and v the same tensor; a single row whose strides mean nothing."""
    import rank_gemm_quantize_b200 as rq
    q, _, _ = make(27, [90], [90], 2, 2, 64, BF16)
    ops.check(rq.attention(q, q, q, causal=True), *ops.attention(q, q, q, [90], [90], True))
    row = torch.randn(3, 2, 64).to(BF16).cuda().as_strided((1, 2, 64), (7, 64, 1))
    ops.check(rq.attention(row, row, row), *ops.attention(row, row, row, [1], [1], False))


def test_refused_views():
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(28, [8], [8], 2, 2, 64, BF16)
    with pytest.raises(ValueError, match="contiguous"):
        rq.attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)
    with pytest.raises(rq.SvdqError, match="strides"):
        rq.attention(q, k[:1].expand(8, 2, 64), v)
    with pytest.raises(rq.SvdqError, match="aligned"):
        flat = torch.zeros(8 * 128 + 4, dtype=BF16, device="cuda")
        rq.attention(flat[4:].view(8, 2, 64), k, v)
    with pytest.raises(ValueError, match="k_offsets"):
        rq.attention(q[:3], k, v, offsets([3]))
    with pytest.raises(ValueError, match="int32"):
        rq.attention(q, k, v, offsets([8]).long())
    with pytest.raises(ValueError, match="all float16"):
        rq.attention(q, k, v.half())


def test_nothing_to_do():
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(19, [0], [5], 4, 2, 64, BF16)
    assert rq.attention(q, k, v).shape == (0, 4, 64)
    q, k, v = make(20, [5], [0], 4, 2, 64, BF16)
    assert not rq.attention(q, k, v).count_nonzero()


def test_long_cache_passes_31_bits_of_offset():
    """Keys whose byte offset passes 2^31 (values 2^32): a batch of two sequences, the second far out."""
    import rank_gemm_quantize_b200 as rq
    rows, kv, dim = 2_200_000, 8, 128
    k = torch.zeros(rows, kv, dim, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    q, kk, vv = make(21, [1, 1], [500, 700], 16, kv, dim, BF16)
    k[:500], k[-700:], v[:500], v[-700:] = kk[:500], kk[500:], vv[:500], vv[500:]
    # three sequences, the middle one without queries
    o = rq.attention(q, k, v, torch.tensor([0, 1, 1, 2], dtype=torch.int32).cuda(),
                     torch.tensor([0, 500, rows - 700, rows], dtype=torch.int32).cuda(), causal=True)
    ops.check(o, *ops.attention(q, kk, vv, [1, 1], [500, 700], True))


# Twenty key heads are too many for one cluster an item: small sizes in the kernels that larger calls take.
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (72, F16), (128, BF16)])
@pytest.mark.parametrize("q_lengths,k_lengths", [([1, 1], [1, 64]), ([1, 8, 3], [0, 65, 700]), ([17], [17]), ([8], [9]),
                                                 ([130, 0, 255], [131, 5, 255]), ([256, 257], [256, 400]),
                                                 ([40, 3, 129], [640, 1200, 129]), ([1] * 6, [3000, 5, 900, 64, 0, 513])])
def test_many_key_heads(q_lengths, k_lengths, dim, dtype, causal):
    check(30, q_lengths, k_lengths, 40, 20, dim, dtype, causal)


@pytest.mark.parametrize("before", [30, 900])
@pytest.mark.parametrize("q_lengths", [[1, 1, 1], [150, 300, 70], [3, 40, 3]])
def test_what_a_query_does_not_see_with_many_key_heads(q_lengths, before):
    k_lengths = [n + before for n in q_lengths]
    q, k, v = make(31, q_lengths, k_lengths, 40, 20, 64, BF16)
    a, b = k_lengths[0], k_lengths[0] + k_lengths[1]
    k[a:b] = float("nan")
    v[a:b] = float("inf")
    v[a - 1, 0, 3] = float("inf")
    v[a - 1, 19, 5] = float("nan")
    v[-2, 1, 1] = float("-inf")
    v[-1, 1, 2] = float("nan")
    o = run(q, k, v, q_lengths, k_lengths, True)
    n, m = q_lengths[0], q_lengths[0] + q_lengths[1]
    assert o[n:m].isnan().all()
    ops.check(o[:n], *ops.attention(q[:n], k[:a], v[:a], [n], [a], True))
    ops.check(o[m:], *ops.attention(q[m:], k[b:], v[b:], [q_lengths[2]], [k_lengths[2]], True))


@pytest.mark.parametrize("q_lengths,k_lengths", [([5, 200], [2, 60]), ([3, 1], [0, 9]), ([300, 2], [1, 1])])
def test_queries_that_see_no_key_with_many_key_heads(q_lengths, k_lengths):
    q, k, v = make(32, q_lengths, k_lengths, 40, 20, 64, BF16)
    o = run(q, k, v, q_lengths, k_lengths, True)
    ops.check(o, *ops.attention(q, k, v, q_lengths, k_lengths, True))
    at = 0
    for n, m in zip(q_lengths, k_lengths):
        assert not o[at:at + max(0, n - m)].count_nonzero()
        at += n


@pytest.mark.parametrize("q_lengths,k_lengths", [([300], [3000]), ([1, 1, 1], [9000, 2, 700]), ([1] * 5, [20000, 1, 700, 64, 3])])
def test_shares_and_join_in_a_graph(q_lengths, k_lengths):
    """Replayed on new inputs and on new lengths of the same totals."""
    import rank_gemm_quantize_b200 as rq
    q, k, v = make(33, q_lengths, k_lengths, 16, 8, 128, BF16)
    qo, ko = offsets(q_lengths), offsets(k_lengths)
    rq.attention(q, k, v, qo, ko, causal=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = rq.attention(q, k, v, qo, ko, causal=True)
    for seed, turned in ((34, False), (35, True), (36, True)):
        k2 = k_lengths[::-1] if turned else k_lengths
        for t, n in zip((q, k, v), make(seed, q_lengths, k_lengths, 16, 8, 128, BF16)):
            t.copy_(n)
        ko.copy_(offsets(k2))
        graph.replay()
        torch.cuda.synchronize()
        ops.check(o, *ops.attention(q, k, v, q_lengths, k2, True))
    assert rq.operator_status() == rq.Status.OK


# One odd key, at another of the 32 places of a block of scores for each of 32 heads: prompts, shares of the
# keys and their join, single tokens by stretches and by clusters.
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_lengths,k_lengths,first,causal", [
    ([40, 40], [200, 90], 32, False), ([200], [200], 0, True), ([200], [200], 96, True), ([40], [3000], 1056, False),
    ([40], [3000], 2944, True), ([1, 1, 1], [700, 30, 5], 640, True), ([1], [777], 64, True)])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16)])
def test_one_odd_key_at_every_place(q_lengths, k_lengths, first, causal, dim, dtype, value):
    """A NaN or an infinity among the scores that a row sees makes the row NaN."""
    q, k, v = make(41, q_lengths, k_lengths, 32, 32, dim, dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    for h in range(32):
        k[first + h, h, 0] = value
    o = run(q, k, v, q_lengths, k_lengths, causal)
    ops.check(o, *ops.attention(q, k, v, q_lengths, k_lengths, causal))


@pytest.mark.parametrize("every", [False, True])
@pytest.mark.parametrize("q_lengths,k_lengths,kv_heads", [
    ([40, 3], [200, 90], 32), ([200], [150], 32), ([40], [3000], 32), ([1500], [1300], 2), ([1, 1, 1], [700, 30, 5], 32),
    ([12, 1], [9, 3000], 32), ([1], [777], 32), ([9], [5], 2)])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16)])
def test_scores_of_minus_infinity(q_lengths, k_lengths, kv_heads, dim, dtype, every):
    """Minus infinity leaves a key out; a row that sees only such keys is NaN, one that sees no key at all is 0."""
    q, k, v = make(42, q_lengths, k_lengths, kv_heads, kv_heads, dim, dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    if every:
        k[:k_lengths[0], :, 0] = float("-inf")
    else:
        for h in range(kv_heads):
            k[h % k_lengths[0], h, 0] = float("-inf")
    o = run(q, k, v, q_lengths, k_lengths, True)
    want, bound = ops.attention(q, k, v, q_lengths, k_lengths, True)
    assert want.isnan().any() or not every
    ops.check(o, want, bound)


@pytest.mark.parametrize("batch", [31, 32, 33, 34])
def test_more_sequences_than_lanes_in_clusters(batch):
    """Lone tokens of few keys with one key head: eight CTAs a sequence, however many sequences find place."""
    k_lengths = [(97 * i) % 500 for i in range(batch)]
    check(43, [1] * batch, k_lengths, 1, 1, 128, BF16, True)
    check(44, [0 if i % 3 == 1 else 1 for i in range(batch)], k_lengths, 4, 1, 64, F16, True)


@pytest.mark.parametrize("q_lengths,k_lengths", [([40], [8200]), ([40], [15900]), ([33, 20], [16384, 40]), ([64], [40000])])
def test_more_shares_of_one_sequence(q_lengths, k_lengths):
    """One key head, so that the keys of a row tile go to as many CTAs as a share of 512 keys, or a warp, allows."""
    check(45, q_lengths, k_lengths, 1, 1, 64, BF16, True)
    check(46, [n // 4 for n in q_lengths], k_lengths, 8, 1, 128, F16, False)


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 3), (8, 4), (20, 1)])
@pytest.mark.parametrize("batch", [5, 40, 300])
def test_units_in_parts(batch, kv_heads, group):
    """Ragged tokens and pieces of few rows, some without queries or keys: stretches begin anywhere in their keys."""
    g = torch.Generator().manual_seed(batch + kv_heads)
    k_lengths = torch.randint(0, 20000 // batch, (batch,), generator=g).tolist()
    k_lengths[batch // 2], k_lengths[-1] = 4000, 0
    q_lengths = torch.randint(0, 3, (batch,), generator=g).tolist()
    q_lengths[batch // 2] = 1 + 20 // group
    for dim, dtype, causal in ((64, F16, True), (128, BF16, False)):
        check(47, q_lengths, k_lengths, kv_heads * group, kv_heads, dim, dtype, causal)


@pytest.mark.parametrize("keys", [6143, 6144, 6145, 8300])
def test_lone_tokens_on_both_sides_of_the_clusters(keys):
    """A cluster takes a lone sequence up to eight times 768 keys, stretches and a join longer ones."""
    check(48, [1], [keys], 8, 2, 128, BF16, True)
    check(49, [2, 1], [keys, keys], 4, 4, 64, F16, True)
