"""Attention over the 4-bit cache where its work is cut up: many sequences,
many short segments to a CTA, segments cut between CTAs, row tiles split in the last
wave, and NaN in values that only some rows see.

Large calls are checked on sampled rows: row i of a causal sequence is the one
new token of the same cache cut off behind it, so the oracle computes just
that. Bounds as in test_gpu_kv.py (the same check).
"""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402
from tests.test_gpu_kv import U, check, make_cache  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    moe.load()
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def filled(ctx, seed, kv_len, H, D, P):
    """A cache of these sequences, filled by moe_kv_append (checked elsewhere), and its table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // P) for n in kv_len]
    cache = moe.moe_kv_new_cache(sum(need) + 1, H, D, P)
    cache.tensor.random_(0, 256, generator=g)
    order = torch.randperm(sum(need) + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(kv_len), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    lens = torch.tensor(kv_len, device="cuda")
    b, pos = torch.nonzero(torch.arange(max(max(kv_len), 1), device="cuda") < lens[:, None], as_tuple=True)
    slots = table[b, pos // P] * P + (pos % P).to(torch.int32)
    k = torch.randn((len(b), H, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((len(b), H, D), generator=g, device="cuda").bfloat16()
    if len(b):
        moe.moe_kv_append(ctx, cache, k, v, slots)
    return cache, table, g


def expect(cache, table, kv_len, q_start, q, rows, scale, window=0):
    """The oracle on the given rows of a causal call."""
    D, P = cache.dim, cache.page_tokens
    b = [int(np.searchsorted(q_start, r, side="right") - 1) for r in rows]
    cut = [int(kv_len[i] - (q_start[i + 1] - r) + 1) for i, r in zip(b, rows)]
    tb = table.cpu().numpy()[b]
    used = np.unique(np.concatenate([t[:-(-n // P)] for t, n in zip(tb, cut) if n > 0] or [np.zeros(1, int)]))
    pages = cache.tensor[torch.from_numpy(used).cuda().long()].cpu().numpy().reshape(len(used), -1, P // 16, 18 * D)
    tb = np.searchsorted(used, tb).clip(max=len(used) - 1)
    return kv.attend(pages, P, q[rows].double().cpu().numpy(), tb, [max(n, 0) for n in cut], np.arange(len(rows) + 1), scale, True, window)


def run(ctx, seed, kv_len, n_new, Hq, H, D, P, dtype, hint, sample, window=0):
    cache, table, g = filled(ctx, seed, kv_len, H, D, P)
    q_start = np.concatenate([[0], np.cumsum(n_new)])
    n = int(q_start[-1])
    q = torch.randn((n, Hq, D), generator=g, device="cuda").to(dtype)
    lse = torch.zeros((n, Hq), device="cuda")
    args = (table, torch.tensor(kv_len, dtype=torch.int32, device="cuda"))
    qs = torch.from_numpy(q_start.astype(np.int32)).cuda()
    got = moe.moe_kv_attend(ctx, cache, q, *args, q_start=qs, max_q=hint, window=window, lse=lse)
    again = moe.moe_kv_attend(ctx, cache, q, *args, q_start=qs, max_q=hint, window=window)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    assert torch.equal(got, again)
    rows = np.unique(np.concatenate([np.random.default_rng(seed).integers(0, n, sample), [0, n - 1]]))
    ref = expect(cache, table, kv_len, q_start, q, rows, D ** -0.5, window)
    t = torch.from_numpy(rows).cuda()
    with np.errstate(invalid="ignore"):
        check(got[t].double().cpu().numpy(), lse[t].double().cpu().numpy(), q[t], ref, 2.0 ** -8 if dtype == torch.bfloat16 else U)
    return got, cache, q, args, qs


@pytest.mark.parametrize("B,H,top", [(33, 2, 40), (300, 1, 60), (300, 8, 9), (1300, 8, 5), (700, 16, 33)])
def test_many_sequences(ctx, B, H, top):
    lens = np.random.default_rng(B).integers(0, top + 1, B).tolist()
    run(ctx, B, lens, [1] * B, 2 * H, H, 64, 16, torch.bfloat16, 1, 60)


@pytest.mark.parametrize("D,P,lens", [(128, 64, [70000, 3, 1000]), (64, 16, [30000]), (256, 32, [20011, 9000])])
def test_segments_cut_between_ctas(ctx, D, P, lens):
    run(ctx, D, lens, [1] * len(lens), 8, 2, D, P, torch.float16, 1, 3)


@pytest.mark.parametrize("D,T,n,window", [(64, 2600, 5000, 0), (128, 1100, 4000, 0), (256, 1300, 2500, 0), (128, 1100, 9000, 2500)])
def test_row_tiles_split_in_the_last_wave(ctx, D, T, n, window):
    got, cache, q, args, qs = run(ctx, D + 1, [n], [T], 32, 16, D, 64, torch.float16, T, 4, window)
    # and all rows against the decode kernel, whose arithmetic is another
    other = moe.moe_kv_attend(ctx, cache, q, *args, q_start=qs, max_q=1, window=window)
    # each is within 3 U dot + 3 U mag + u of the exact row by the bound of test_gpu_kv.py;
    # dot <= 64 and mag <= 1.2 for these standard normal rows
    tol = 2 * (2 * 3 * U * 64 / np.sqrt(D) * 2 + 3 * U + U) * 1.2
    assert (got.float() - other.float()).abs().max().item() <= tol


@pytest.mark.parametrize("hint", [1, 4096])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_values_reach_only_the_rows_that_see_them(ctx, D, hint):
    """A NaN in token j's value group makes that group of the rows from j on NaN, and nothing else; a NaN key
    every group of them."""
    H, P, n, T = 2, 16, 200, 150
    cache, table, g = filled(ctx, D, [n], H, D, P)
    q = torch.randn((T, 2 * H, D), generator=g, device="cuda").half()
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    clean = moe.moe_kv_attend(ctx, cache, q, table, ln, max_q=hint)
    slot = lambda j: (table[0, j // P] * P + j % P).reshape(1)  # noqa: E731
    group = D // 64 - 1
    for j, where in ((120, "v"), (60, "k")):  # positions; new token i is at n - T + i
        saved = cache.tensor.clone()
        k, v = moe.moe_kv_read(ctx, cache, slot(j), dtype=torch.float32)
        (v if where == "v" else k)[0, 1, 64 * group + 3] = float("nan")  # kv head 1
        moe.moe_kv_append(ctx, cache, k, v, slot(j))
        got = moe.moe_kv_attend(ctx, cache, q, table, ln, max_q=hint)
        nan = got.isnan()
        want = torch.zeros_like(nan)
        first = max(0, j - (n - T))
        want[first:, 2:, 64 * group if where == "v" else 0:64 * group + 64 if where == "v" else D] = True
        assert torch.equal(nan, want), where
        keep = ~want
        keep[first:] = False  # later rows read a requantised token
        assert torch.equal(got[keep], clean[keep])
        cache.tensor.copy_(saved)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_segments_about_the_shortest_that_is_cut(ctx, D, dtype):
    for i, n in enumerate([1, 383, 384, 385, 511, 513, 767, 769, 1023, 1024, 1041]):
        run(ctx, 7 * D + i, [n], [1], 16, 8, D, 16, dtype, 1, 1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hint", [1, 17, 300, 5000, 100000])
def test_no_result_depends_on_max_len(ctx, D, hint):
    """Any value for the longest length, too small ones included."""
    lens = [5000, 77, 1300]
    cache, table, g = filled(ctx, D + hint, lens, 4, D, 32)
    q = torch.randn((3, 8, D), generator=g, device="cuda").bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = moe.moe_kv_attend(ctx, cache, q, table, ln, max_q=1, max_len=hint)
    ref = expect(cache, table, lens, np.arange(4), q, np.arange(3), D ** -0.5)
    lse = torch.zeros((3, 8), device="cuda")
    again = moe.moe_kv_attend(ctx, cache, q, table, ln, max_q=1, max_len=hint, lse=lse)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    assert torch.equal(got, again)
    check(got.double().cpu().numpy(), lse.double().cpu().numpy(), q, ref, 2.0 ** -8)


@pytest.mark.parametrize("D,window,lens", [(256, 100, [5000, 300, 90]), (256, 600, [7000] * 5), (128, 512, [9000, 1]), (64, 900, [20000] * 3)])
def test_windows_of_a_few_keys_behind_a_long_history(ctx, D, window, lens):
    run(ctx, D + window, lens, [min(3, n) for n in lens], 8, 4, D, 16, torch.float16, 3, 5, window)
