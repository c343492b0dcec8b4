"""One decoder layer over a 4-bit key/value cache: a prompt, then decode steps.

Attention (query, key and value projections, the cache, the output projection) runs
beside the MoE layer: moe_rms_norm adds what came before to the residual and norms the sum, into
8 bits for the projections (moe_f8_matmul) or bf16 for the experts; moe_kv_append puts the new tokens' keys and
values into the cache, moe_kv_attend attends over it, moe_f8_quant_rows takes its output to the output projection, and
moe_forward_prompt / moe_forward run the experts. Weights and tokens are random, from a seed.

    python examples/decode_layer.py [--prompt 300] [--steps 16] [--sequences 2] [--projections f8|bf16]

Prints the time of the prompt and of a step, how far the attention is from
plain fp32 attention over the cache's values read back (moe_kv_read), and how far the projections
are from products in fp64 of the same operands. --projections bf16 keeps the projections' weights and rows in bf16 and
multiplies them with torch.
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


def values(codes, scales, weight):
    """What 8-bit rows or weights stand for, in fp64."""
    n, k = codes.shape
    scales = scales.double().repeat_interleave(128, 0)
    scales = scales[:n].repeat_interleave(128, 1)[:, :k] if weight else scales[:k].t()
    return codes.double() * scales


class Projection:
    """Rows times weights [n][k], both in 8 bits or both in bf16."""

    def __init__(self, ctx, w, kind):
        self.ctx, self.f8 = ctx, kind == "f8"
        self.w = moe.moe_f8_quant_weight(ctx, w) if self.f8 else w.bfloat16()
        self.worst = 0.0

    def __call__(self, x, dtype, check=False):
        """x: bf16 rows, or with 8 bits (codes, scales) as the norm gives them."""
        if self.f8:
            y = moe.moe_f8_matmul(self.ctx, *x, *self.w, dtype=dtype)
        else:
            y = (x @ self.w.t()).to(dtype)
        if check:
            self.worst = max(self.worst, self.difference(x, y))
        return y

    def difference(self, x, y):
        """Largest difference from the product in fp64, of an output's sum of magnitudes."""
        x, w = (values(*x, False), values(*self.w, True)) if self.f8 else (x.double(), self.w.double())
        return ((y.double() - x @ w.t()).abs() / (x.abs() @ w.abs().t())).max().item()


class Attention:
    """The attention block of one layer: heads of 64, four query heads a kv head, causal."""

    def __init__(self, ctx, d_model, sequences, max_tokens, seed, head_dim=64, group=4, projections="f8"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.dim = ctx, head_dim
        self.heads = d_model // head_dim
        self.kv_heads = max(1, self.heads // group)
        rows = (self.heads + 2 * self.kv_heads) * head_dim
        self.w_in, self.w_out = (Projection(ctx, torch.randn(shape, generator=g, device="cuda") * d_model ** -0.5, projections)
                                 for shape in ((rows, d_model), (d_model, self.heads * head_dim)))
        per = -(-max_tokens // PAGE)
        self.cache = moe.moe_kv_new_cache(sequences * per, self.kv_heads, head_dim, PAGE)
        # pages as an allocator might deal them out
        self.table = torch.randperm(sequences * per, generator=g, device="cuda").to(torch.int32).view(sequences, per)
        self.length = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.worst = 0.0

    def __call__(self, x, check=False):
        """The normed rows [sequences * new tokens][d_model], as the projection takes them: the block's output, fp32, added to nothing."""
        B = self.table.shape[0]
        qkv = self.w_in(x, torch.bfloat16, check).unflatten(1, (-1, self.dim))
        T = qkv.shape[0] // B
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        pos = (self.length[:, None] + torch.arange(T, device="cuda")).long()
        slots = torch.gather(self.table, 1, pos // PAGE) * PAGE + pos % PAGE
        moe.moe_kv_append(self.ctx, self.cache, k, v, slots.flatten().to(torch.int32))
        self.length += T
        out = moe.moe_kv_attend(self.ctx, self.cache, q, self.table, self.length)
        if check:
            self.worst = max(self.worst, self.difference(q.unflatten(0, (B, T)), out.unflatten(0, (B, T))))
        out = out.flatten(1)
        return self.w_out(moe.moe_f8_quant_rows(self.ctx, out) if self.w_out.f8 else out, torch.float32, check)

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


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--sequences", type=int, default=2)
    ap.add_argument("--projections", choices=["f8", "bf16"], default="f8")
    a = ap.parse_args(argv)
    s = synth.SHAPES_TINY
    ctx = moe.moe_ctx_create(0)
    layer = moe.moe_layer_create(ctx, s, 4, moe.LFU)
    try:
        moe.moe_layer_set_weights(layer, synth.layer_weights(s, 0))

        def run(prompt, steps, check):
            attention = Attention(ctx, s.d_model, a.sequences, prompt + steps, seed=0, projections=a.projections)
            g = torch.Generator(device="cuda").manual_seed(1)
            x = torch.randn((a.sequences * prompt, s.d_model), generator=g, device="cuda").bfloat16()
            weights = [1 + 0.1 * torch.randn((s.d_model,), generator=g, device="cuda") for _ in range(2)]

            def normed(h, residual=None):
                """The norm in front of the attention block: (its rows for the projection, the residual's sum)."""
                if a.projections == "f8":
                    _, total, codes, scales = moe.moe_rms_norm(ctx, h, weights[0], residual=residual, dtype=None, f8=True)
                    return (codes, scales), total
                out, total, _, _ = moe.moe_rms_norm(ctx, h, weights[0], residual=residual, dtype=torch.bfloat16)
                return out, total

            rows, _ = normed(x)
            times = []
            for step in range(steps + 1):
                torch.cuda.synchronize()
                t = time.perf_counter()
                o = attention(rows, check and step in (0, steps))
                y, x, _, _ = moe.moe_rms_norm(ctx, o, weights[1], residual=x, dtype=torch.bfloat16)
                ffn = (moe.moe_forward_prompt if y.shape[0] > 64 else moe.moe_forward)(layer, y)
                # the next tokens: what the last ones became
                last = slice(x.shape[0] // a.sequences - 1, None, x.shape[0] // a.sequences)
                rows, x = normed(ffn[last], x[last])
                torch.cuda.synchronize()
                times.append(time.perf_counter() - t)
            return attention, x, times

        run(a.prompt, min(2, a.steps), False)  # libraries load, workspaces grow
        _, _, times = run(a.prompt, a.steps, False)
        attention, x, _ = run(a.prompt, a.steps, True)
        moe.moe_kv_check(ctx)
        moe.moe_f8_check(ctx)
        steps = sorted(times[1:] or times)
        print(f"{a.sequences} x {a.prompt} tokens, then {a.steps} steps: prompt {times[0] * 1e3:.2f} ms, step "
              f"{steps[len(steps) // 2] * 1e6:.0f} us; attention within {attention.worst:.1e} of fp32 over the cache's values, "
              f"projections within {max(attention.w_in.worst, attention.w_out.worst):.1e} of their sums of magnitudes")
        return attention.worst, x
    finally:
        moe.moe_layer_destroy(layer)
        moe.moe_ctx_destroy(ctx)


if __name__ == "__main__":
    main()
