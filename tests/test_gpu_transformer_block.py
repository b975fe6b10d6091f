"""A transformer block out of the quantized layers and the operators around them, as a user runs
it: modulation from a 16-bit linear layer, norms with gates, W4A4 QKV projection, attention over
packed sequences on views of its output, 16-bit output projection, fused W4A4 MLP block.

Every operator's result is compared with its 64-bit definition on the inputs it had in the
run, so no stage's rounding enters the next one's bound. The quantized layers have tests of
their own."""
import pytest
import torch

import operators as ops

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LENGTHS, DIM, HEADS, KV, HEAD = [70, 1, 130], 512, 8, 4, 64


class Block:
    def __init__(self, seed):
        import rank_gemm_quantize_b200 as rq
        g = torch.Generator().manual_seed(seed)
        t = lambda *shape, s=1.0: (torch.randn(*shape, generator=g) * s).to(BF16).cuda()
        rows = sum(LENGTHS)
        self.rq = rq
        self.offsets = torch.tensor([0] + LENGTHS).cumsum(0).to(torch.int32).cuda()
        self.sequence = torch.repeat_interleave(torch.tensor(LENGTHS))
        self.x = (torch.randn(rows, DIM, generator=g) * 2 + 0.3).cuda()
        self.cond = t(len(LENGTHS), DIM)
        self.w_mod, self.b_mod = t(DIM, 6 * DIM, s=0.02), t(6 * DIM, s=0.1)
        self.w_out, self.b_out = t(HEADS * HEAD, DIM, s=0.04), t(DIM, s=0.1)
        absmax = lambda n: torch.full((n,), 4.0, device="cuda")
        layer = lambda k, n: rq.Layer.prepare(t(k, n, s=0.04), t(n, s=0.05), absmax(k), rq.NVFP4_G16, 32)
        self.qkv = layer(DIM, (HEADS + 2 * KV) * HEAD)
        self.mlp = rq.MlpBlock(layer(DIM, 2048), layer(2048, DIM))

    def run(self):
        """Everything the block computes, by name."""
        rq, s = self.rq, {}
        s["mod"] = rq.linear(self.cond, self.w_mod, self.b_mod, "silu")
        gate1, scale1, shift1, gate2, scale2, shift2 = (m.contiguous() for m in s["mod"].chunk(6, 1))
        s["vectors"] = gate1, scale1, shift1, gate2, scale2, shift2
        _, s["h1"] = rq.residual_norm(self.x, offsets=self.offsets, norm="layer", scale=scale1, shift=shift1, dtype=BF16)
        s["qkv"] = self.qkv.forward(s["h1"])
        s["heads"] = s["qkv"].view(-1, HEADS + 2 * KV, HEAD).split([HEADS, KV, KV], 1)
        s["o"] = rq.attention(*s["heads"], self.offsets, causal=True)
        s["y1"] = rq.linear(s["o"].view(-1, HEADS * HEAD), self.w_out, self.b_out)
        s["x1"], s["h2"] = rq.residual_norm(self.x, s["y1"], offsets=self.offsets, gate=gate1, norm="layer", scale=scale2,
                                            shift=shift2)
        s["y2"] = self.mlp.forward(s["h2"])
        s["x2"], none = rq.residual_norm(s["x1"], s["y2"], offsets=self.offsets, gate=gate2, post_norm="rms", norm=None)
        assert none is None
        return s

    def close(self):
        for layer in (self.qkv, self.mlp.up, self.mlp.down):
            assert layer.device_status() == self.rq.Status.OK
            layer.close()


def test_each_stage_of_a_block():
    b = Block(1)
    s = b.run()
    torch.cuda.synchronize()
    assert b.rq.operator_status() == b.rq.Status.OK
    gate1, scale1, shift1, gate2, scale2, shift2 = s["vectors"]
    ops.check(s["mod"], *ops.linear(b.cond, b.w_mod, b.b_mod, "silu", None), what="modulation")
    want = ops.residual_norm(b.x, None, b.sequence, norm="layer", scale=scale1, shift=shift1)
    ops.check(s["h1"], *want[1], what="first norm")
    ops.check(s["o"], *ops.attention(*s["heads"], LENGTHS, LENGTHS, True), what="attention")
    ops.check(s["y1"], *ops.linear(s["o"].view(-1, HEADS * HEAD), b.w_out, b.b_out, None, None), what="output projection")
    want = ops.residual_norm(b.x, s["y1"], b.sequence, gate=gate1, norm="layer", scale=scale2, shift=shift2)
    ops.check(s["x1"], *want[0], what="residual")
    ops.check(s["h2"], *want[1], what="second norm")
    want = ops.residual_norm(s["x1"], s["y2"], b.sequence, gate=gate2, post_norm="rms", norm=None)
    ops.check(s["x2"], *want[0], what="last residual")
    b.close()


def test_block_in_a_graph():
    """Captured once, replayed on another stream content: bit for bit the eager block."""
    b = Block(2)
    b.run()  # workspaces and attributes are set up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = b.run()
    b.x.mul_(0.7)
    b.cond.add_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    got = {n: captured[n].clone() for n in ("o", "x1", "h2", "x2")}
    want = b.run()
    for n, t in got.items():
        assert torch.equal(t, want[n]), n
    b.close()


def test_decoding_steps_continue_a_prompt():
    """Queries one at a time against the keys so far give what the whole prompt's pass gives, within the
    bounds of both."""
    import rank_gemm_quantize_b200 as rq
    g = torch.Generator().manual_seed(3)
    n = 300
    q, k, v = (torch.randn(n, h, HEAD, generator=g).to(BF16).cuda() for h in (HEADS, KV, KV))
    whole = rq.attention(q, k, v, causal=True)
    want, bound = ops.attention(q, k, v, [n], [n], True)
    ops.check(whole, want, bound)
    for i in (0, 1, 63, 64, 127, 128, 200, 299):
        ops.check(rq.attention(q[i:i + 1], k[:i + 1], v[:i + 1], causal=True), want[i:i + 1], bound[i:i + 1])
