"""One layer's attention block on the library, as a training step and as a decoding loop.

    python examples/attention_block.py [--tokens 4096] [--sequences 4] [--steps 8]

Training: the FP8 QKV projection, norms and rotation, attention, the FP8 O projection, and back
through all of them (16 query and 8 key/value heads of 128, hidden 2048).  Decoding: the same weights over
a cache, the first half of a sequence as a prompt and the rest token by token; what comes out is the
training pass's output for those tokens, up to rounding.  Prints the errors of both against plain torch in
32 bits and the time of each part.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blockwise_fp8_gemm_act_amd as puro  # noqa: E402

HIDDEN, QH, KH, HD = 2048, 16, 8, 128
EPS, BASE = 1e-6, 1e6


class Block:
    """Weights of the block: bf16 masters, and their FP8 codes for both directions."""

    def __init__(self, seed=0, window=0, sinks=0, positions=4096):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, std: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
        self.wqkv, self.wo = new((QH + 2 * KH) * HD, HIDDEN, std=0.02), new(HIDDEN, QH * HD, std=0.02)
        self.wq, self.wk = 1 + new(HD, std=0.1), 1 + new(HD, std=0.1)
        self.qkv_codes, self.o_codes = puro.quant_weights([self.wqkv, self.wo])
        self.table = puro.rope_table(positions, HD, base=BASE)
        self.mask = dict(window=window, sinks=sinks)

    def project(self, x):
        q, s = puro.quant_act_1x128(x)
        return puro.gemm_fp8_blockwise(puro.FPROP, q, s, *self.qkv_codes[:2])

    def out(self, o):
        q, s = puro.quant_act_1x128(o.flatten(1))
        return puro.gemm_fp8_blockwise(puro.FPROP, q, s, *self.o_codes[:2])

    def forward(self, x, pos, starts):
        """x [T][HIDDEN] of packed sequences -> (y, what the backward step needs)."""
        qkv = self.project(x)
        q, k = puro.qk_norm_rope(qkv, self.wq, self.wk, self.table, pos, q_heads=QH, k_heads=KH, eps=EPS)
        v = qkv.view(len(x), -1, HD)[:, QH + KH:]                      # read where the projection left it
        o, lse = puro.attention(q, k, v, starts, starts, **self.mask)
        return self.out(o), (x, qkv, q, k, v, o, lse, pos, starts)

    def backward(self, dy, saved):
        """-> (dx, gradients of wqkv, wo (fp32), wq, wk)."""
        x, qkv, q, k, v, o, lse, pos, starts = saved
        act = lambda t: puro.quant_act_128x1(t, dual=True)             # token-major 128x1 and 1x128 codes  # noqa: E731
        dyt, dyts, dyq, dys = act(dy)
        oc, ocs = puro.quant_act_128x1(o.flatten(1))
        dwo = puro.gemm_fp8_blockwise(puro.WGRAD_TM, dyt, dyts, oc, ocs, out_dtype=torch.float32)
        do = puro.gemm_fp8_blockwise(puro.DGRAD, dyq, dys, *self.o_codes[2:]).view(o.shape)
        dqkv = torch.empty_like(qkv)
        heads = dqkv.view(len(x), -1, HD)
        dq, dk, _ = puro.attention_backward(do, q, k, v, o, lse, starts, starts, dv=heads[:, QH + KH:], **self.mask)
        _, dwq, dwk = puro.qk_norm_rope_backward(dq, dk, qkv, self.wq, self.wk, self.table, pos, eps=EPS, dx=heads[:, :QH + KH])
        gt, gts, gq, gs = act(dqkv)
        xc, xcs = puro.quant_act_128x1(x)
        dwqkv = puro.gemm_fp8_blockwise(puro.WGRAD_TM, gt, gts, xc, xcs, out_dtype=torch.float32)
        return puro.gemm_fp8_blockwise(puro.DGRAD, gq, gs, *self.qkv_codes[2:]), dwqkv, dwo, dwq, dwk


class Decoder:
    """The block over a cache with room for `room` tokens of each of `n` sequences."""

    def __init__(self, block, n, room):
        self.block, self.room = block, room
        self.k = torch.empty(n * room, KH, HD, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.first = torch.arange(n, dtype=torch.int32, device="cuda") * room
        self.length = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.starts = torch.arange(n + 1, dtype=torch.int32, device="cuda") * room

    def step(self, x, each):
        """`each` new tokens of every sequence, x [n * each][HIDDEN] -> y."""
        b, n = self.block, len(self.length)
        pos = (self.length[:, None] + torch.arange(each, dtype=torch.int32, device="cuda")).flatten()
        rows = pos + self.first.repeat_interleave(each)
        self.length += each
        q = puro.qk_norm_rope_append(b.project(x), b.wq, b.wk, b.table, pos, self.k, self.v, rows, q_heads=QH, eps=EPS)
        q_start = torch.arange(n + 1, dtype=torch.int32, device="cuda") * each
        o, _ = puro.attention(q, self.k, self.v, q_start, self.starts, self.length, max_k=self.room, **b.mask)
        return b.out(o)


def plain(block, qkv, pos, n, do):
    """Norms, rotation and attention in 32 bits, one sequence at a time: o, and the gradient of qkv under do."""
    length = len(qkv) // n
    outs, grads = [], []
    for s in range(n):
        rows = slice(s * length, (s + 1) * length)
        x = qkv[rows].float().view(length, -1, HD).requires_grad_(True)
        cos, sin = block.table[pos[rows].long()].unbind(1)
        turn = lambda t: torch.cat((t[..., :64] * cos[:, None] - t[..., 64:] * sin[:, None],  # noqa: E731
                                    t[..., 64:] * cos[:, None] + t[..., :64] * sin[:, None]), -1)
        norm = lambda t, w: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w.float()  # noqa: E731
        q = turn(norm(x[:, :QH], block.wq)).transpose(0, 1)
        k = turn(norm(x[:, QH:QH + KH], block.wk)).transpose(0, 1).repeat_interleave(QH // KH, 0)
        v = x[:, QH + KH:].transpose(0, 1).repeat_interleave(QH // KH, 0)
        i, j = torch.arange(length, device="cuda")[:, None], torch.arange(length, device="cuda")
        seen = j <= i
        if block.mask["window"]:
            seen &= (j > i - block.mask["window"]) | (j < block.mask["sinks"])
        a = torch.matmul(q, k.transpose(1, 2).contiguous()) * HD ** -0.5
        o = torch.matmul(a.masked_fill(~seen, float("-inf")).softmax(-1), v).transpose(0, 1)
        o.backward(do[rows].float())
        outs.append(o.detach())
        grads.append(x.grad.flatten(1))
    return torch.cat(outs), torch.cat(grads)


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def train(block, tokens, sequences, seed=1):
    """One forward and backward step -> (errors against plain torch, the step's y, x and positions)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    length = tokens // sequences
    x = torch.randn(sequences * length, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    dy = (torch.randn(x.shape, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    pos = torch.arange(len(x), dtype=torch.int32, device="cuda") % length
    starts = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * length
    y, saved = block.forward(x, pos, starts)
    grads = block.backward(dy, saved)
    qkv, o = saved[1], saved[5]
    # the operators' own part, from the same projection output and the same gradient of o
    dyq, dys = puro.quant_act_1x128(dy)
    do = puro.gemm_fp8_blockwise(puro.DGRAD, dyq, dys, *block.o_codes[2:]).view(o.shape)
    want_o, want_g = plain(block, qkv, pos, sequences, do)
    gq, gs = puro.quant_act_1x128(want_g.to(torch.bfloat16))
    want_dx = puro.gemm_fp8_blockwise(puro.DGRAD, gq, gs, *block.qkv_codes[2:])
    return dict(o=rel(o, want_o), dx=rel(grads[0], want_dx)), x, y, pos, starts, dy


def decode(block, x, y, sequences):
    """The first half of every sequence as a prompt, then token by token -> error against the training pass."""
    length = len(x) // sequences
    xs, ys = x.view(sequences, length, -1), y.view(sequences, length, -1)
    d = Decoder(block, sequences, length)
    half = length // 2
    out = [d.step(xs[:, :half].reshape(-1, HIDDEN), half).view(sequences, half, -1)]
    for t in range(half, length):
        out.append(d.step(xs[:, t].contiguous(), 1)[:, None])
    return rel(torch.cat(out, 1), ys)


def timed(f, n):
    f()
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    e[0].record()
    for _ in range(n):
        f()
    e[1].record()
    torch.cuda.synchronize()
    return e[0].elapsed_time(e[1]) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = Block(window=a.window, sinks=a.sinks, positions=max(4096, a.tokens // a.sequences))
    errors, x, y, pos, starts, dy = train(block, a.tokens, a.sequences)
    print("against plain torch in 32 bits: " + ", ".join("%s %.2e" % e for e in errors.items()))
    print("prompt and single tokens against the whole sequence: %.2e" % decode(block, x, y, a.sequences))
    _, saved = block.forward(x, pos, starts)
    print("forward %.3f ms, backward %.3f ms for %d tokens" % (
        timed(lambda: block.forward(x, pos, starts), a.steps), timed(lambda: block.backward(dy, saved), a.steps), len(x)))


if __name__ == "__main__":
    main()
