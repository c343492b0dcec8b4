"""How exact attention over the 4-bit cache is, by checks that do not weaken with length.

Every block counts: the values of the tokens of block b (16 tokens) are 1 in dimension b mod head_dim and 0
elsewhere, so an output element is the weight of the blocks of its dimension: a sum of positive terms, which a
block left out, counted twice or misplaced changes by a known share. The bound is relative. Queries are small, so
logits are off by delta = 3 U dot at most (test_gpu_kv.py) with a small dot, all weights matter, none is below fp16's range, and
  |out - exact| <= (2 delta e^(2 delta) + 3 U + u) exact + 6 r |w|,  |lse - exact| <= delta + 2^-20.
The last term, |w| being the root of the sum of the squared weights: the decode kernel rounds a weight together with its
scale, so the error is relative to what the codes span (1 here) for an element of 0 too; the roundings, each r as below, are
independent as all weights differ, and six deviations are allowed.
The mistakes are planted in the exact result, and the bound has to reject each.

Error of a call as a whole: the relative L2 error of normally distributed rows against what the roundings give. One
rounding to fp16 has a relative error of r = 2^-10 / sqrt(12) * sqrt(3 / (8 ln 2)) = 2.07e-4, root mean square over mantissas
spread as 1/x; to bf16 8 r. With independent values of mean zero each of these adds its own square:
  output: r or 8 r;  prompt kernel: V r, P r, and K r times the logits' deviation (1 here); queries are exact;
  decode kernel: weights times scale r times the size of what they multiply, relative to that of the values: codes from 8
  for fp16 outputs, values less the middle of their group, 1; codes from 0 for bf16 outputs, values less their group's least, which
  for 64 normal values lies 2.4 deviations below: sqrt(1 + 2.4^2) = 2.6.
Allowed is 1.25 times that: the sums are over thousands of outputs, and mantissas are not spread quite so.
"""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402

U = 2.0 ** -11
R = 2.0 ** -10 / np.sqrt(12) * np.sqrt(3 / (8 * np.log(2)))


@pytest.fixture(scope="module")
def ctx():
    moe.load()
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def within(got, lse, out, rl, delta, u, norm):
    rel = 2 * delta * np.exp(2 * delta) + 3 * U + u
    return bool((np.abs(got - out) <= rel * out + 6 * R * norm).all() and abs(lse - rl) <= delta + 2.0 ** -20)


# head_dim, page, lengths, new tokens, query heads, kv heads, dtype, max_q, window, rows looked at
BLOCKS = [
    (128, 64, [70000, 3, 1000], 1, 8, 2, "f16", 1, 0, 3),  # a segment over many CTAs
    (64, 16, [30000], 1, 8, 2, "f16", 1, 0, 1),
    (256, 32, [20011, 9000], 1, 8, 2, "bf16", 1, 0, 2),
    (128, 16, [9000] * 40, 1, 16, 2, "bf16", 1, 0, 6),  # ranges that cut segments anywhere
    (64, 64, [100, 7000, 0, 2500] * 10, 1, 8, 4, "f16", 1, 0, 8),
    (256, 16, [3000] * 12, 2, 32, 2, "f16", 2, 1000, 6),
    (128, 64, [50000], 3, 32, 2, "bf16", 3, 20000, 3),
    (128, 64, [30000], 64, 8, 1, "f16", 64, 0, 4),  # row tiles whose keys are split over CTAs
    (64, 32, [20000], 100, 16, 2, "bf16", 100, 0, 4),
    (256, 64, [9000, 400], 64, 8, 1, "f16", 64, 0, 6),
    (128, 64, [4000], 1100, 32, 16, "f16", 1100, 0, 4),  # the last wave's split
    (64, 16, [9000], 700, 16, 2, "f16", 700, 3000, 4),
]


@pytest.mark.parametrize("i", range(len(BLOCKS)))
def test_every_block_counts(ctx, i):
    D, P, lens, T, Hq, H, dtype, hint, window, look = BLOCKS[i]
    rng = np.random.default_rng(1000 + i)
    g = torch.Generator(device="cuda").manual_seed(i)
    u = U if dtype == "f16" else 2.0 ** -8
    B, need = len(lens), [-(-n // P) for n in lens]
    cache = moe.moe_kv_new_cache(sum(need) + 1, H, D, P)
    cache.tensor.random_(0, 256, generator=g)
    order = torch.randperm(sum(need) + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            t = torch.arange(n, device="cuda")
            k = torch.randn((n, H, D), generator=g, device="cuda")
            v = torch.zeros((n, D), device="cuda")
            v[t, t // 16 % D] = 1
            moe.moe_kv_append(ctx, cache, k, v[:, None].expand(n, H, D), table[b, t // P] * P + (t % P).to(torch.int32))
    new = [min(T, n) if n else 1 for n in lens]
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = (0.05 * torch.randn((int(q_start[-1]), Hq, D), generator=g, device="cuda")).to(torch.float16 if dtype == "f16" else torch.bfloat16)
    lse = torch.empty((q.shape[0], Hq), device="cuda")
    got = moe.moe_kv_attend(ctx, cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            q_start=torch.from_numpy(q_start.astype(np.int32)).cuda(), max_q=hint, window=window, lse=lse)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    got, lse, q64 = got.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    rows = np.unique(np.r_[0, q.shape[0] - 1, rng.integers(0, q.shape[0], look)])
    mistakes = 0
    for r in rows:
        b = int(np.searchsorted(q_start, r, side="right") - 1)
        n, pos = lens[b], lens[b] - (q_start[b + 1] - r)
        if n == 0:
            assert (got[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        t = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
        pages = cache.tensor[table[b, :need[b]].long()].cpu().numpy().reshape(need[b], H, P // 16, 18 * D)
        K, V = kv.read(pages, P, t)
        for h in rng.choice(Hq, 2, replace=False):
            kh = h // (Hq // H)
            z = D ** -0.5 * (K[:, kh] @ q64[r, h])
            p = np.exp(z)
            tol = 3 * U * D ** -0.5 * (np.abs(K[:, kh]) @ np.abs(q64[r, h])).max(), u, np.sqrt((p * p).sum()) / p.sum()

            def answer(p):
                return p @ V[:, kh] / p.sum(), np.log(p.sum())

            out, rl = answer(p)
            assert within(got[r, h], lse[r, h], out, rl, *tol), (r, h, np.abs(got[r, h] / np.maximum(out, 1e-9) - 1).max(), lse[r, h] - rl)
            # nothing, the opposite, and one block (of some) left out or counted twice are not taken for the answer
            assert not within(0 * out, rl, out, rl, *tol) and not within(-out, rl, out, rl, *tol)
            if len(t) > 32:
                one = t // 16 == rng.integers(t[0] // 16 + 1, t[-1] // 16)
                for factor in (0.0, 2.0):
                    wrong, wl = answer(np.where(one, factor * p, p))
                    assert not within(wrong, wl, out, rl, *tol)
                    mistakes += 1
    assert mistakes or max(lens) < 48


def reference(cache, ctx, q, n, causal):
    """Outputs in 64 bits, from the values read back (which the oracle checks elsewhere)."""
    k, v = (x.double() for x in moe.moe_kv_read(ctx, cache, torch.arange(n, dtype=torch.int32, device="cuda"), dtype=torch.float32))
    T, Hq, D = q.shape
    k, v = (x.repeat_interleave(Hq // cache.heads, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) * D ** -0.5
    if causal:
        s.masked_fill_(torch.arange(n, device="cuda") > n - T + torch.arange(T, device="cuda")[:, None], float("-inf"))
    return torch.einsum("hij,jhd->ihd", s.softmax(-1), v)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kernel,T,n", [("decode", 2, 4000), ("decode", 1, 700), ("decode", 1, 30000), ("prompt", 300, 1000), ("prompt", 64, 4000)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_error_is_what_the_roundings_give(ctx, D, dtype, kernel, T, n, causal):
    g = torch.Generator(device="cuda").manual_seed(D + n)
    H, Hq = 4, 16
    cache = moe.moe_kv_new_cache(-(-n // 64), H, D, 64)
    k, v = (torch.randn((n, H, D), generator=g, device="cuda") for _ in range(2))
    moe.moe_kv_append(ctx, cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    q = torch.randn((T, Hq, D), generator=g, device="cuda").to(dtype)
    table = torch.arange(-(-n // 64), dtype=torch.int32, device="cuda")[None]
    got = moe.moe_kv_attend(ctx, cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), causal=causal,
                            max_q=1 if kernel == "decode" else 4096)
    want = reference(cache, ctx, q, n, causal)
    rms = R * np.sqrt((64 if dtype == torch.bfloat16 else 1) +
                      (3 if kernel == "prompt" else 1 if dtype == torch.float16 else 2.6 ** 2))
    err = ((got.double() - want).norm() / want.norm()).item()
    assert err <= 1.25 * rms, (err, rms)
