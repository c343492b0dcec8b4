"""Attention over the 4-bit cache at the edges of its arguments and of what its records hold.

Bounds are those of test_gpu_kv.py (U = 2^-11 a rounding to fp16, u the output's own) with two terms written
out. Weights are rounded together with their scale where codes are multiplied, so the error is one U of what the
group's codes span, at most twice its largest value, whatever the element: 2 U times the largest mag of the group. And a weight below
fp16's range is off by 2^-25 of the largest scale, whose codes span at most twice the largest value: seen * 2^-24 * top.
"""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402

U = 2.0 ** -11
HINTS = [1, 4096]  # max_q, which chooses the kernel: decode, prompt


@pytest.fixture(scope="module")
def ctx():
    moe.load()
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def unit(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def bound(e, dtype, more=0):
    """Of an output, from what the oracle says of it; `more` roundings of keys and values besides."""
    delta = (3 + more) * U * e["dot"][..., None]
    mag = e["mag"]
    group = np.repeat(mag.reshape(mag.shape[:-1] + (-1, 64)).max(-1), 64, -1)
    return (2 * delta * np.exp(2 * delta) + (3 + more) * U + unit(dtype)) * mag + 2 * U * group + e["seen"][..., None] * 2.0 ** -24 * e["top"][..., None]


def in_order(pages, P):
    """A cache of one sequence whose pages lie in order, and its table."""
    n_pages, H, _, per = pages.shape
    cache = moe.moe_kv_make_cache(torch.from_numpy(pages).cuda(), H, per // 18, P)
    return cache, torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]


def attend(ctx, cache, table, n, q, hint, **kw):
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = moe.moe_kv_attend(ctx, cache, q, table, ln, max_q=hint, **kw)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    return got


def exact(pages, P, q, n, **kw):
    table = np.arange(pages.shape[0])[None]
    scale = kw.pop("scale", q.shape[2] ** -0.5)
    return kv.attend(pages, P, q.double().cpu().numpy(), table, [n], [0, q.shape[0]], scale, **kw)


@pytest.mark.parametrize("B,H,hint", [(2, 64, 1), (2, 64, 4096), (16, 8, 1), (40, 4, 1)])
def test_page_tables_near_the_widest(ctx, B, H, hint):
    """A table far wider than the sequences are long (2^31 - 1,280 places) changes nothing: the answer is, to the bit, that of
    a narrow one. A wider one still is refused."""
    D, P, n, per = 64, 256, 300, ((1 << 31) - 1280) // 256
    g = torch.Generator(device="cuda").manual_seed(B)
    cache = moe.moe_kv_new_cache(3, H, D, P)
    k, v = (torch.randn((n, H, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    moe.moe_kv_append(ctx, cache, k, v, torch.arange(256, 256 + n, dtype=torch.int32, device="cuda"))
    wide = torch.zeros(per + 1, dtype=torch.int32, device="cuda")
    wide[:2] = torch.tensor([1, 2])
    q = torch.randn((B, 2 * H, D), generator=g, device="cuda").bfloat16()
    ln = torch.full((B,), n, dtype=torch.int32, device="cuda")
    want = moe.moe_kv_attend(ctx, cache, q, wide[:2].expand(B, 2), ln, max_q=hint, max_len=n)
    got = moe.moe_kv_attend(ctx, cache, q, wide[:per].expand(B, per), ln, max_q=hint, max_len=n)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    assert torch.equal(got, want) and want.abs().max() > 0
    with pytest.raises(moe.MoeError, match="max_pages") as e:
        moe.moe_kv_attend(ctx, cache, q, wide.expand(B, per + 1), ln, max_q=hint, max_len=n)
    assert e.value.status == moe.MOE_EINVAL


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("bits", [12.3, 20.6, 24.6])
@pytest.mark.parametrize("D,dtype,n", [(64, torch.bfloat16, 333), (128, torch.float16, 333), (128, torch.bfloat16, 2000), (256, torch.float16, 200)])
def test_small_weights_beside_a_key_that_takes_nearly_all(ctx, D, dtype, n, bits, hint):
    """One key takes nearly all of the softmax and its value is zero, so the output is made of weights `bits` binary
    orders below it. Keys, values and queries are exact in fp16 (codes times a power of two) and the values positive, so
    what is left is: the weights' rounding, U of normal ones and, below fp16's normal range, half its step, 2^-30 of the
    largest weight as that is stored as at least 2^5; the output's u, or 2^-25 where fp16 has no normal number;
    logits of up to 30 off by 30 * 2^-22; and fp32 sums, n 2^-24 of what the codes span, one for these values."""
    H, P, T = 1, 32, 2
    rng = np.random.default_rng(n + D)
    code = lambda lo, hi: rng.integers(lo, hi, (n, H, D)).astype(np.float32)  # noqa: E731
    k, v = code(0, 3), code(8, 16)
    sink = n // 2
    k[sink, :, :16] = 15
    v[sink] = 0
    for x in (k, v):  # every group spans 0 to 15, so that its scale is a power of two
        live = np.arange(n) != sink if x is v else np.arange(n) >= 0
        x[live, :, 62::64], x[live, :, 63::64] = 0, 15
    pages = kv.empty_pages(-(-n // P), H, D, P)
    kv.append(pages, P, k / 8, v / 16, np.arange(n))
    K, V = kv.read(pages, P, np.arange(n))
    assert (K == k / 8).all() and (V == v / 16).all()
    q = torch.zeros((T, 4, D), dtype=dtype, device="cuda")
    q[:, :, :16] = 1
    scale = bits * np.log(2) / 28
    cache, table = in_order(pages, P)
    lse = torch.zeros((T, 4), device="cuda")
    got = attend(ctx, cache, table, n, q, hint, scale=scale, causal=False, lse=lse).double().cpu().numpy()
    out, rl, _ = exact(pages, P, q, n, scale=float(np.float32(scale)), causal=False)
    z = scale * K[:, 0, :16].sum(-1)
    p = np.exp(z - z.max())
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # of an output below fp16's normal range
    live = np.arange(n) != sink
    low = ((p < 2.0 ** -14)[:, None] * V[:, 0]).sum(0) * 2.0 ** -30 / p.sum()
    tol = (U + unit(dtype) + 2 * 30 * 2.0 ** -22) * out + n * 2.0 ** -24 * p[live].sum() / p.sum() + low + tiny
    assert (np.abs(got - out) <= tol).all(), (np.abs(got - out) / tol).max()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= 1e-4).all()


# (least, largest) element of a group, the others small: held as up to 65,520, 65,540, 65,536 and 65,592
PAST = [(0.0, 65472.0), (-100.0, 1e30), (-np.inf, np.inf), (-57400.0, 65504.0)]


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.float16)])
def test_values_past_the_largest_fp16(ctx, D, dtype, side, hint):
    """A group's largest value lies above its largest element by up to 15 roundings of its scale, past fp16's
    65,504. Rows that do not see it are as they were (in the prompt kernel to the bit; in the decode
    kernel the power of two that weights are scaled by may be another, and the bound below holds). The others are within
    the bound, to which the prompt kernel adds 65,624 taken as 65,504, less than 4 U of the value. Queries are
    small where a key is that large, so that its logits are of ordinary size."""
    H, P, n, T = 2, 32, 200, 150
    rng = np.random.default_rng(D)
    k, v = (rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((T, 2 * H, D))
    at = D - 64 + 5  # the element that is large, in the last group
    q[:, :, D - 64:] *= 2.0 ** -14
    q = torch.from_numpy(q.astype(np.float32)).to(dtype).cuda()
    pages = kv.empty_pages(-(-n // P), H, D, P)
    kv.append(pages, P, k, v, np.arange(n))
    cache, table = in_order(pages, P)
    clean = attend(ctx, cache, table, n, q, hint)
    for j, (lo, hi) in zip((60, 90, 120, 170), PAST):
        x = (k if side == "k" else v)[j:j + 1].copy()
        x[0, 1, D - 64:] *= 0.01
        x[0, 1, at], x[0, 1, at + 1] = hi, lo
        changed = pages.copy()
        kv.append(changed, P, x if side == "k" else k[j:j + 1], v[j:j + 1] if side == "k" else x, [j])
        held = kv.read(changed, P, [j])[side == "v"]
        assert held.max() > 65504
        cache, table = in_order(changed, P)
        got = attend(ctx, cache, table, n, q, hint)
        first = j - (n - T)
        assert hint == 1 or torch.equal(got[:first], clean[:first])
        out, _, e = exact(changed, P, q, n)
        diff = np.abs(got.double().cpu().numpy() - out)
        assert (diff <= bound(e, dtype, 4)).all(), (lo, hi, np.argwhere(~(diff <= bound(e, dtype, 4)))[:4])


def affine(pages):
    """Writable views of the records' K and V affine words: fp16 [pages][H][blocks][16][NG][scale, bias] each."""
    d = pages.shape[-1] // 18
    return [pages[..., (16 + side) * d:(17 + side) * d].view(np.float16).reshape(pages.shape[:-1] + (16, d // 64, 2)) for side in (0, 1)]


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_nan_values(ctx, D, window, hint):
    """Ninety tokens whose values are NaN in one group, at two places: NaN is that group of the rows that see
    one of them, and nothing else; a windowed row between the places sees none."""
    H, P, n, T = 2, 32, 420, 400
    rng = np.random.default_rng(D)
    pages = kv.empty_pages(-(-n // P), H, D, P)
    kv.append(pages, P, *(rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2)), np.arange(n))
    q = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).half().cuda()
    cache, table = in_order(pages, P)
    clean = attend(ctx, cache, table, n, q, hint, window=window)
    bad = np.r_[150:195, 225:270]
    group = D // 64 - 1
    affine(pages)[1][bad // P, 1, bad % P // 16, bad % 16, group, 0] = np.nan  # kv head 1
    cache, table = in_order(pages, P)
    got = attend(ctx, cache, table, n, q, hint, window=window)
    pos = n - T + np.arange(T)[:, None]
    see = (bad <= pos) & ((bad > pos - window) if window else True)
    want = np.zeros((T, H, D), bool)
    want[see.any(1), 1, 64 * group:64 * group + 64] = True
    nan = got.isnan().cpu().numpy()
    assert (nan == want).all(), np.argwhere(nan != want)[:4]
    # the rest is what it was, but for other powers of two that the weights are scaled by: both within 3 U + u of
    # mag, at most the largest value, which is below 5
    diff = np.abs(got.double().cpu().numpy() - clean.double().cpu().numpy())[~want]
    assert diff.max() <= 2 * 4 * U * 5


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("share", [1.0, 0.5])
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (64, torch.bfloat16), (128, torch.float16), (128, torch.bfloat16),
                                     (256, torch.float16), (256, torch.bfloat16)])
def test_negative_scales(ctx, D, dtype, share, hint):
    """Records of the caller's own whose scales are negative, all of them or half: value = scale * code + bias
    all the same. A group's values are mirrored (code c for 15 - c), so they are of ordinary size."""
    H, P, n, T = 2, 32, 333, 3
    rng = np.random.default_rng(D + int(10 * share))
    pages = kv.empty_pages(-(-n // P), H, D, P)
    kv.append(pages, P, *(rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2)), np.arange(n))
    for a in affine(pages):
        turn = rng.random(a.shape[:-1]) < share
        a[..., 1] = np.where(turn, a[..., 1] + 15 * a[..., 0], a[..., 1])
        a[..., 0] = np.where(turn, -a[..., 0], a[..., 0])
    q = torch.from_numpy(rng.standard_normal((T, 4 * H, D)).astype(np.float32)).to(dtype).cuda()
    cache, table = in_order(pages, P)
    got = attend(ctx, cache, table, n, q, hint).double().cpu().numpy()
    out, _, e = exact(pages, P, q, n)
    assert (np.abs(got - out) <= bound(e, dtype)).all(), np.abs(got - out).max()


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("bits", [1e3, 1e5, 4e6])
@pytest.mark.parametrize("D,dtype,n", [(64, torch.float16, 333), (128, torch.bfloat16, 2000), (256, torch.float16, 200)])
def test_large_scores(ctx, D, dtype, n, bits, hint):
    """Scores far apart, to four million binary orders: two keys tie for the largest and all others vanish, so the output
    is the mean of the two values, exact (codes times a power of two) but for its own rounding and one U of the codes' span for
    the weights'. lse has the relative precision of fp32: a few roundings of 2^-24, 2^-21 in all."""
    H, P, T = 1, 32, 3
    rng = np.random.default_rng(n + D)
    k, v = (rng.integers(0, 9, (n, H, D)).astype(np.float32) for _ in range(2))
    pair = [n // 3, n - 2]
    k[pair, :, :16] = 15
    for x in (k, v):
        x[:, :, 62::64], x[:, :, 63::64] = 0, 15
    pages = kv.empty_pages(-(-n // P), H, D, P)
    kv.append(pages, P, k / 8, v / 16, np.arange(n))
    q = torch.zeros((T, 4, D), dtype=dtype, device="cuda")
    q[:, :, :16] = 1
    scale = float(np.float32(bits * np.log(2) / 30))
    cache, table = in_order(pages, P)
    lse = torch.zeros((T, 4), device="cuda")
    got = attend(ctx, cache, table, n, q, hint, scale=scale, causal=False, lse=lse).double().cpu().numpy()
    want = (v[pair] / 16).astype(np.float64).mean((0, 1))
    assert (np.abs(got - want) <= unit(dtype) * want + U).all()
    assert (np.abs(lse.double().cpu().numpy() - (30 * scale + np.log(2))) <= 30 * scale * 2.0 ** -21).all()


def test_read_refuses_a_type_that_its_outputs_do_not_have(ctx):
    cache = moe.moe_kv_new_cache(1, 2, 64, 16)
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.empty((1, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for given in (dict(k=k, v=v), dict(k=k), dict(v=v)):
        with pytest.raises(ValueError, match="float32"):
            moe.moe_kv_read(ctx, cache, s, dtype=torch.float32, **given)
        assert moe.moe_kv_read(ctx, cache, s, dtype=torch.bfloat16, **given)[0].dtype == torch.bfloat16
