"""The attention half of a decoder layer on this library: FP8 projections and a 4-bit paged
key/value cache, for a batch of sequences that are first prompted and then decoded.

    lengths -> kv4_plan -> slots, positions, page tables
    x, residual -> rms_norm_group_quant -> qkv GEMM -> rotation -> kv4_write -> kv4_attention
                -> group_quant -> output GEMM -> (x for the next half, residual)

Run it on an MI355X:  python examples/decoder_layer.py
It decodes some tokens and prints how far the outputs are from the same layer in fp32 without
quantized activations and cache, and the time of a decode step as a replayed HIP graph.
"""
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_group_quant_amd as fq  # noqa: E402


def quantize_weight(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(e4m3 bytes [N, K], fp32 scales [N/128, K/128]) of w [N, K]: one scale per 128 x 128 block."""
    blocks = w.float().unflatten(0, (-1, 128)).unflatten(2, (-1, 128))
    s = blocks.abs().amax((1, 3)).clamp_min(1e-10) / 448
    q = (blocks / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(2, 3).flatten(0, 1).view(torch.uint8), s


def dequantize_weight(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def rotate(x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """Rotary embedding of x [T, heads, D]: pairs (i, i + D/2) turned by position * 10000^(-2i/D)."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = (positions.float()[:, None] * freq)[:, None]
    cos, sin = angle.cos(), angle.sin()
    a, b = x.float().split(half, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(x.dtype)


class AttentionLayer:
    """Weights, cache and page tables of one layer. hidden and heads * dim: multiples of 128."""

    def __init__(self, hidden, heads, kv_heads, dim, seqs, max_tokens, page=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim

        def weight(n, k):
            return quantize_weight(torch.randn(n, k, device=device, generator=g) / math.sqrt(k))

        self.norm = (1 + 0.1 * torch.randn(hidden, device=device, generator=g)).to(torch.bfloat16)
        self.w_qkv = weight((heads + 2 * kv_heads) * dim, hidden)
        self.w_out = weight(hidden, heads * dim)
        # pages enough for every sequence, taken in a scattered order
        per_seq = -(-max_tokens // page)
        self.cache = fq.alloc_kv4_cache(seqs * per_seq, page, kv_heads, dim, device=device)
        self.order = torch.randperm(seqs * per_seq, device=device, generator=g).to(torch.int32)
        self.table = torch.full((seqs, per_seq), -1, dtype=torch.int32, device=device)
        self.clear()

    def clear(self):
        """No tokens are cached, all pages are free."""
        self.lens = torch.zeros(self.table.shape[0], dtype=torch.int32, device=self.table.device)
        self.free = self.order

    def plan(self, q_lens, tokens):
        """The step in which sequence b gets q_lens[b] new tokens, `tokens` in all: the table's new entries, and what
        forward() takes. The step can be planned again until it is done()."""
        return fq.kv4_plan(self.cache, self.lens, q_lens, self.free, self.table, tokens)

    def done(self, plan):
        """The planned tokens are cached, their pages no longer free (without a copy to the host: the taken pages move
        to the list's end, behind as many as are ever needed)."""
        self.lens = plan.kv_lens
        n = self.free.numel()
        self.free = self.free[(torch.arange(n, device=self.free.device) + plan.pages_taken) % n]

    def forward(self, x, residual, plan, single=False):
        """Rows x [T, hidden] (bf16) of a planned step's tokens, one sequence after the other; single: one of each.
        Returns the layer's output and the new residual."""
        T, h, hk, d = x.shape[0], self.heads, self.kv_heads, self.dim
        q8, s8, residual = fq.rms_norm_group_quant(x, self.norm, residual=residual)
        qkv = torch.empty(T, (h + 2 * hk) * d, dtype=torch.bfloat16, device=x.device)
        fq.fp8q_gemm_blockscaled(q8, s8, *self.w_qkv, qkv)
        q, k, v = qkv.view(T, h + 2 * hk, d).split((h, hk, hk), 1)
        q, k = rotate(q, plan.positions), rotate(k, plan.positions)
        fq.fp8q_kv4_write(k, v, plan.slots, self.cache)
        o = fq.kv4_attention(q, self.cache, self.table, plan.kv_lens, 1 / math.sqrt(d),
                             q_indptr=None if single else plan.q_indptr)
        q8, s8 = fq.group_quant(o.view(T, h * d))
        y = torch.empty_like(x)
        fq.fp8q_gemm_blockscaled(q8, s8, *self.w_out, y)
        return y, residual

    def reference(self, x, residual, lens):
        """The same layer in fp32 over whole sequences of the given lengths, rows of x one sequence after
        the other, without quantized activations or cache."""
        h, hk, d = self.heads, self.kv_heads, self.dim
        res = x.float() + residual.float()
        y = res * torch.rsqrt(res.square().mean(-1, keepdim=True) + 1e-6) * self.norm.float()
        qkv = (y @ dequantize_weight(*self.w_qkv).t()).view(-1, h + 2 * hk, d)
        out = []
        for rows in qkv.split(lens):
            q, k, v = rows.split((h, hk, hk), 1)
            pos = torch.arange(rows.shape[0], device=x.device)
            q, k = rotate(q, pos), rotate(k, pos)
            k, v = (t.repeat_interleave(h // hk, 1).transpose(0, 1) for t in (k, v))
            a = q.transpose(0, 1) @ k.transpose(1, 2).contiguous() / math.sqrt(d)
            a = a.masked_fill(pos[None, :] > pos[:, None], -math.inf).softmax(-1)
            out.append((a @ v).transpose(0, 1).reshape(-1, h * d))
        return torch.cat(out) @ dequantize_weight(*self.w_out).t()


def decode_batch(layer, x, residual, prompt_lens, steps):
    """Prompts of the given lengths, then `steps` tokens for every sequence, one at a time. x, residual:
    one [prompt + steps, hidden] tensor per sequence. Returns the outputs in the same layout."""
    dev, seqs = x[0].device, len(prompt_lens)
    layer.clear()
    plan = layer.plan(torch.tensor(prompt_lens, dtype=torch.int32, device=dev), sum(prompt_lens))
    y, _ = layer.forward(*(torch.cat([t[:n] for t, n in zip(s, prompt_lens)]) for s in (x, residual)), plan)
    layer.done(plan)
    out = [list(part) for part in y.split(prompt_lens)]
    one = torch.ones(seqs, dtype=torch.int32, device=dev)
    for i in range(steps):
        plan = layer.plan(one, seqs)
        y, _ = layer.forward(*(torch.stack([t[n + i] for t, n in zip(s, prompt_lens)]) for s in (x, residual)), plan, True)
        layer.done(plan)
        for o, row in zip(out, y):
            o.append(row)
    return [torch.stack(o) for o in out]


def main():
    hidden, heads, kv_heads, dim, prompts, steps = 4096, 32, 8, 128, [700, 64, 1999, 1], 32
    layer = AttentionLayer(hidden, heads, kv_heads, dim, len(prompts), max(prompts) + steps)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = ([torch.randn(n + steps, hidden, device="cuda", generator=g).to(torch.bfloat16) for n in prompts]
                   for _ in range(2))
    out = torch.cat(decode_batch(layer, x, residual, prompts, steps))
    ref = layer.reference(torch.cat(x), torch.cat(residual), [n + steps for n in prompts])
    print(f"{len(prompts)} sequences, {sum(prompts)} prompt tokens, {steps} decoded tokens each: "
          f"relative difference to the fp32 layer {float((out.float() - ref).norm() / ref.norm()):.3f}")

    # a decode step as a graph: the rows and lengths are read from the captured tensors at each replay
    one = torch.ones(len(prompts), dtype=torch.int32, device="cuda")
    layer.lens = layer.lens - one  # the last token again, whose page is held
    row, res = torch.stack([t[-1] for t in x]), torch.stack([t[-1] for t in residual])

    def step():
        return layer.forward(row, res, layer.plan(one, len(prompts)), True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(200):
        graph.replay()
    torch.cuda.synchronize()
    print(f"a decode step of the layer: {(time.perf_counter() - t0) / 200 * 1e6:.0f} us")


if __name__ == "__main__":
    main()
