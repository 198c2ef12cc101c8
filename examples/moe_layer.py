"""A feed-forward layer of a mixture-of-experts model, and the output head.

    python examples/moe_layer.py [--tokens 1,16,64] [--hidden 2048] ...

The routed experts are packed in 4 bits (moe), the shared expert, which every
token passes, and the head in 8 (ffn_f8, linear_f8): few weights are read by
all tokens, so they keep the wider format.  Weights are random.  The result is
compared with the same layer in plain PyTorch on the dequantized weights, and
the step is captured into a graph, replayed and timed as a decoder would run
it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_block_quant_amd as qblk  # noqa: E402


class Layer:
    def __init__(self, hidden, inter, shared, experts, top_k, vocab, fmt=qblk.SB4, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def draw(rows, k):
            return torch.randn(rows, k, device="cuda", generator=gen) * k ** -0.5

        self.fmt, self.inter, self.experts, self.top_k = fmt, inter, experts, top_k
        self.router = draw(experts, hidden)
        self.gate_up = qblk.quantize(draw(experts * 2 * inter, hidden), fmt)
        self.down = qblk.quantize(draw(experts * hidden, inter), fmt)
        self.w13, self.s13 = qblk.quantize_f8(draw(2 * shared, hidden))
        self.w2, self.s2 = qblk.quantize_f8(draw(hidden, shared))
        self.head, self.head_scale = qblk.quantize_f8(draw(vocab, hidden))

    def __call__(self, x):
        """x (n, hidden) bf16 -> (layer output (n, hidden), logits (n, vocab)), both bf16."""
        scores = x.float() @ self.router.T
        y, _, _ = qblk.moe(self.fmt, x, scores, self.gate_up, self.down, self.inter, self.top_k)
        y = x + y + qblk.ffn_f8(x, self.w13, self.s13, self.w2, self.s2)
        return y, qblk.linear_f8(y, self.head, self.head_scale)

    def plain(self, x):
        """The same in PyTorch: dequantized weights, fp32, activations not quantized."""
        n, hidden = x.shape
        f, xf = torch.nn.functional, x.float()

        def wide(codes, scale):
            s = scale.view(-1, codes.shape[1] // 128).repeat_interleave(128, 0)[:codes.shape[0]]
            return codes.float() * s.repeat_interleave(128, 1)

        gu = qblk.dequant(self.gate_up, self.fmt, self.experts * 2 * self.inter, hidden, torch.float32)
        dn = qblk.dequant(self.down, self.fmt, self.experts * hidden, self.inter, torch.float32)
        gu, dn = gu.view(self.experts, 2 * self.inter, hidden), dn.view(self.experts, hidden, self.inter)
        scores, ids = torch.topk(xf @ self.router.T, self.top_k)
        weights = torch.softmax(scores, 1)  # over the chosen ones: renormalized
        y = xf.clone()
        for t in range(n):
            for j in range(self.top_k):
                g, u = (gu[ids[t, j]] @ xf[t]).split(self.inter)
                y[t] += weights[t, j] * (dn[ids[t, j]] @ (f.silu(g) * u))
        g, u = (xf @ wide(self.w13, self.s13).T).split(self.w2.shape[1], 1)
        y += (f.silu(g) * u) @ wide(self.w2, self.s2).T
        return y, y @ wide(self.head, self.head_scale).T


def run(tokens, hidden=2048, inter=1024, shared=2048, experts=32, top_k=4, vocab=16384, replays=50):
    """Yields (tokens, relative error of the output, of the logits, us per step)."""
    layer = Layer(hidden, inter, shared, experts, top_k, vocab)
    for n in tokens:
        x = torch.randn(n, hidden, device="cuda").bfloat16()
        want = layer.plain(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # libraries set themselves up outside the capture
            layer(x)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = layer(x)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        graph.replay()
        start.record()
        for _ in range(replays):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        err = [((a.float() - b).norm() / b.norm()).item() for a, b in zip(got, want)]
        yield n, err[0], err[1], start.elapsed_time(end) / replays * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", default="1,16,64", help="batch sizes, separated by commas")
    for name, value in (("hidden", 2048), ("inter", 1024), ("shared", 2048), ("experts", 32), ("top-k", 4),
                        ("vocab", 16384)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    for n, ey, el, us in run([int(t) for t in a.tokens.split(",")], a.hidden, a.inter, a.shared, a.experts, a.top_k,
                             a.vocab):
        print(f"{n:4d} tokens: {us:8.1f} us   relative error: output {ey:.2e}, logits {el:.2e}", flush=True)


if __name__ == "__main__":
    main()
