"""The operators around the quantized layers on a stream other than the current one: what a call makes must not
lie where work of another stream is still under way."""
import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
LONG = 400_000_000  # cycles that the work before a call waits: a fifth of a second


def attention_call(g):
    import rank_gemm_quantize_b200 as rq
    q, k, v = (torch.randn(n, h, 128, generator=g).to(BF16) for n, h in ((1, 32), (30000, 8), (30000, 8)))
    need = rq.attention_workspace_size(q.cuda(), k.cuda(), v.cuda())
    return lambda t, s: [rq.attention(*t, causal=True, stream=s)], [q, k, v], [ops.attention(q, k, v, [1], [30000], True)], need


def prompt_call(g):
    import rank_gemm_quantize_b200 as rq
    q, k, v = (torch.randn(700, h, 128, generator=g).to(BF16) for h in (4, 2, 2))
    return lambda t, s: [rq.attention(*t, causal=True, stream=s)], [q, k, v], [ops.attention(q, k, v, [700], [700], True)], q.nbytes


def linear_call(g):
    import rank_gemm_quantize_b200 as rq
    X, W = (torch.randn(*s, generator=g).to(BF16) for s in ((600, 256), (256, 1024)))
    return lambda t, s: [rq.linear(*t, stream=s)], [X, W], [ops.linear(X, W, None, None, None)], 600 * 1024 * 2


def norm_call(g):
    import rank_gemm_quantize_b200 as rq
    x, y = (torch.randn(700, 1024, generator=g).to(BF16) for _ in range(2))
    want = ops.residual_norm(x, y, torch.zeros(700, dtype=torch.long))
    return lambda t, s: list(rq.residual_norm(*t, stream=s)), [x, y], list(want), x.nbytes


CALLS = [attention_call, prompt_call, linear_call, norm_call]


def right(got, want):
    for o, w in zip(got, want):
        ops.check(o, *w)


@pytest.fixture(params=CALLS)
def case(request):
    """(the call on tensors and a stream, its inputs, its results, bytes of what it makes), run once."""
    call, inputs, want, nbytes = request.param(torch.Generator().manual_seed(1))
    inputs = [t.cuda() for t in inputs]
    call(inputs, None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return call, inputs, want, nbytes


def filled(nbytes):
    """Tensors of this size, in the places that the allocator would give next."""
    return [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]


def test_memory_that_the_current_stream_still_reads(case):
    """Work under way on the current stream reads a temporary that is freed before the call on another stream."""
    call, inputs, want, nbytes = case
    side = torch.cuda.Stream()
    temporary = filled(nbytes)
    read = [torch.empty_like(t) for t in temporary]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(LONG)
    for r, t in zip(read, temporary):
        r.copy_(t)
    del temporary, r, t
    got = call(inputs, side)
    torch.cuda.synchronize()
    assert all((r == 7).all() for r in read)
    right(got, want)


@pytest.mark.parametrize("handle", [False, True])
def test_the_default_stream_under_another_current_one(case, handle):
    """What a call on the default stream makes and drops is not handed to the current stream while the call waits."""
    call, inputs, want, nbytes = case
    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    with torch.cuda.stream(side):
        with torch.cuda.stream(default):
            torch.cuda._sleep(LONG)
        got = call(inputs, default.cuda_stream if handle else default)
        later = filled(nbytes)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in later)
    right(got, want)


def test_results_used_on_the_current_stream_and_dropped(case):
    """The next tensors of the call's stream do not lie where the current stream still reads a result."""
    call, inputs, want, nbytes = case
    side = torch.cuda.Stream()
    got = call(inputs, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full_like(t, 7.0) for t in read]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in over)
    right(read, want)


def test_inputs_dropped_after_the_call(case):
    """The next tensors of the current stream do not lie where the call still reads its inputs."""
    call, inputs, want, _ = case
    side = torch.cuda.Stream()
    sizes = [t.nbytes for t in inputs]
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    got = call([t.clone() for t in inputs], side)  # the clones come long before the call runs
    over = [torch.full((n,), 0, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    del over
    right(got, want)


@pytest.mark.parametrize("raw", [False, True])
def test_captured_on_a_joined_stream(case, raw):
    """A call on a second stream of a capture, replayed."""
    call, inputs, want, _ = case
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(inputs, side.cuda_stream if raw else side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        right(got, want)
