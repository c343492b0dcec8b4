"""One decoder layer over a 4-bit key/value cache: a prompt, then decode steps.

Attention (query, key and value projections, the cache, the output projection) runs
beside the MoE layer: moe_kv_append puts the new tokens' keys and values into the
cache, moe_kv_attend attends over it, moe_forward_prompt / moe_forward run the experts. Weights and
tokens are random, from a seed; the projections are plain matrix products.

    python examples/decode_layer.py [--prompt 300] [--steps 16] [--sequences 2]

Prints the time of the prompt and of a step, and how far the attention is from
plain fp32 attention over the cache's values read back (moe_kv_read).
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import expert_streaming_ffn_gb300 as moe  # noqa: E402
import synth  # noqa: E402

PAGE = 64


class Attention:
    """The attention block of one layer: heads of 64, four query heads a kv head, causal."""

    def __init__(self, ctx, d_model, sequences, max_tokens, seed, head_dim=64, group=4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.dim = ctx, head_dim
        self.heads = d_model // head_dim
        self.kv_heads = max(1, self.heads // group)
        rows = (self.heads + 2 * self.kv_heads) * head_dim
        self.w_in = (torch.randn((d_model, rows), generator=g, device="cuda") * d_model ** -0.5).bfloat16()
        self.w_out = (torch.randn((self.heads * head_dim, d_model), generator=g, device="cuda") * d_model ** -0.5).bfloat16()
        per = -(-max_tokens // PAGE)
        self.cache = moe.moe_kv_new_cache(sequences * per, self.kv_heads, head_dim, PAGE)
        # pages as an allocator might deal them out
        self.table = torch.randperm(sequences * per, generator=g, device="cuda").to(torch.int32).view(sequences, per)
        self.length = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.worst = 0.0

    def __call__(self, x, check=False):
        """x [sequences][new tokens][d_model] bf16: the block's output, added to nothing."""
        B, T, _ = x.shape
        qkv = (x.flatten(0, 1) @ self.w_in).unflatten(1, (-1, self.dim))
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        pos = (self.length[:, None] + torch.arange(T, device="cuda")).long()
        slots = torch.gather(self.table, 1, pos // PAGE) * PAGE + pos % PAGE
        moe.moe_kv_append(self.ctx, self.cache, k, v, slots.flatten().to(torch.int32))
        self.length += T
        out = moe.moe_kv_attend(self.ctx, self.cache, q, self.table, self.length)
        if check:
            self.worst = max(self.worst, self.difference(q.unflatten(0, (B, T)), out.unflatten(0, (B, T))))
        return (out.flatten(1) @ self.w_out).view(B, T, -1)

    def difference(self, q, out):
        """Largest difference from fp32 attention over the values read back."""
        worst, T = 0.0, q.shape[1]
        for b, n in enumerate(self.length.tolist()):
            t = torch.arange(n, device="cuda")
            slots = (self.table[b, t // PAGE] * PAGE + t % PAGE).to(torch.int32)
            k, v = moe.moe_kv_read(self.ctx, self.cache, slots, dtype=torch.float32)
            k, v = (z.repeat_interleave(self.heads // self.kv_heads, 1) for z in (k, v))
            s = torch.einsum("ihd,jhd->hij", q[b].float(), k) * self.dim ** -0.5
            s.masked_fill_(t > n - T + torch.arange(T, device="cuda")[:, None], float("-inf"))
            want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v)
            worst = max(worst, (out[b].float() - want).abs().max().item())
        return worst


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True))).bfloat16()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--sequences", type=int, default=2)
    a = ap.parse_args(argv)
    s = synth.SHAPES_TINY
    ctx = moe.moe_ctx_create(0)
    layer = moe.moe_layer_create(ctx, s, 4, moe.LFU)
    try:
        moe.moe_layer_set_weights(layer, synth.layer_weights(s, 0))

        def run(prompt, steps, check):
            attention = Attention(ctx, s.d_model, a.sequences, prompt + steps, seed=0)
            g = torch.Generator(device="cuda").manual_seed(1)
            x = torch.randn((a.sequences, prompt, s.d_model), generator=g, device="cuda").bfloat16()
            times = []
            for step in range(steps + 1):
                torch.cuda.synchronize()
                t = time.perf_counter()
                x = x + attention(norm(x), check and step in (0, steps))
                y = norm(x).flatten(0, 1).contiguous()
                ffn = moe.moe_forward_prompt if y.shape[0] > 64 else moe.moe_forward
                x = x + ffn(layer, y).view(x.shape).bfloat16()
                torch.cuda.synchronize()
                times.append(time.perf_counter() - t)
                x = x[:, -1:]  # the next token: what the last one became
            return attention, x, times

        run(a.prompt, min(2, a.steps), False)  # libraries load, workspaces grow
        _, _, times = run(a.prompt, a.steps, False)
        attention, x, _ = run(a.prompt, a.steps, True)
        moe.moe_kv_check(ctx)
        steps = sorted(times[1:] or times)
        print(f"{a.sequences} x {a.prompt} tokens, then {a.steps} steps: prompt {times[0] * 1e3:.2f} ms, step "
              f"{steps[len(steps) // 2] * 1e6:.0f} us; attention within {attention.worst:.1e} of fp32 over the cache's values")
        return attention.worst, x
    finally:
        moe.moe_layer_destroy(layer)
        moe.moe_ctx_destroy(ctx)


if __name__ == "__main__":
    main()
