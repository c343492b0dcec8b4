"""The 4-bit key/value cache on the GPU against the oracle (oracle/kv.py):
records byte for byte, rows read back exactly, attention in fp64 within the
bound below.

Bound of an attention output. Queries, keys, values and probabilities may enter
the tensor cores as fp16 (relative rounding U = 2^-11 each, fp32 sums), the output is
rounded to its type (u). A row's logits are then off by at most
delta = 3 U dot (dot = scale * max_j sum_d |q_d K_jd|: one U each for q and K, one for
everything in fp32), its weights by a factor within exp(+-2 delta), and the sum by a
further 3 U mag, mag = sum_j w_j |V_j| (P, V, and fp32 sums). A probability below
fp16's normal range, 2^-14 of the row's largest, is off by 2^-25 instead, and the largest
one a kernel scales by may be 2^8 off it: seen * 2^-17 * max|V| (the weights' sum is at least 1).
So |out - exact| <= (2 delta e^{2 delta} + 3 U + u) mag + seen 2^-17 top.
"""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402

U = 2.0 ** -11
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ctx():
    moe.load()
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def f32(t):
    return t.float().cpu().numpy()


def make_cache(pages, H, D, P):
    return moe.moe_kv_make_cache(torch.from_numpy(pages).cuda(), H, D, P)


def rows(rng, n, H, D, dtype):
    x = rng.standard_normal((n, H, D)) * np.exp(rng.uniform(-1, 1, (n, H, 1))) + rng.uniform(-1, 1, (1, H, D))
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).cuda()


def as_type(x64, dtype):
    """fp64 values rounded as the read does: to fp32, then to the type."""
    return torch.from_numpy(x64.astype(np.float32)).to(TYPES[dtype])


@pytest.mark.parametrize("D,P,H,n,dtype", [(64, 16, 1, 1, "bf16"), (64, 32, 3, 77, "f16"), (128, 64, 8, 130, "bf16"),
                                           (128, 128, 2, 33, "f32"), (256, 16, 5, 40, "f16"), (256, 256, 1, 19, "bf16"),
                                           (64, 64, 7, 500, "f32")])
def test_append_and_read_match_the_oracle(ctx, D, P, H, n, dtype):
    rng = np.random.default_rng(D + P + n)
    n_pages = -(-n // P) + 2
    pages = rng.integers(0, 256, (n_pages, H, P // 16, 18 * D), dtype=np.uint8)
    cache = make_cache(pages, H, D, P)
    k, v = rows(rng, n, H, D, dtype), rows(rng, n, H, D, dtype)
    slots = rng.permutation(n_pages * P)[:n].astype(np.int32)
    slots[3::7] = -1
    s = torch.from_numpy(slots).cuda()
    moe.moe_kv_append(ctx, cache, k, v, s)
    kv.append(pages, P, f32(k), f32(v), slots)
    got = cache.tensor.cpu().numpy()
    assert (got == pages).all()
    K, V = kv.read(pages, P, slots)
    for t in TYPES:
        gk, gv = moe.moe_kv_read(ctx, cache, s, dtype=TYPES[t])
        assert torch.equal(gk.cpu(), as_type(K, t)) and torch.equal(gv.cpu(), as_type(V, t))
    moe.moe_kv_check(ctx)


def test_append_extreme_values(ctx):
    D, P = 64, 16
    x = np.zeros((12, 1, D), np.float32)
    x[0] = 1e30
    x[1, 0, ::2], x[1, 0, 1::2] = np.inf, -np.inf
    x[2, 0, 5] = 1e-9
    x[3] = -1e-9
    x[4] = np.linspace(100, 100.001, D)
    x[5] = np.linspace(-6e4, 6e4, D)
    x[6] = np.arange(D) % 2  # ties at half a step
    x[6, 0, 7] = 0.5
    x[7, 0, 0] = 65504
    x[8] = 2.0 ** -24 * np.arange(D)
    x[9] = -0.0
    x[10, 0, 0], x[10, 0, 1] = 3e38, 1e-38
    pages = kv.empty_pages(1, 1, D, P)
    cache = make_cache(pages, 1, D, P)
    t = torch.from_numpy(x).cuda()
    slots = np.arange(12, dtype=np.int32)
    moe.moe_kv_append(ctx, cache, t, -t, torch.from_numpy(slots).cuda())
    kv.append(pages, P, x, -x, slots)
    K, V = kv.read(pages, P, slots)
    gk, gv = moe.moe_kv_read(ctx, cache, torch.from_numpy(slots).cuda(), dtype=torch.float32)
    np.testing.assert_array_equal(gk.cpu().numpy().astype(np.float64), K.astype(np.float32))
    np.testing.assert_array_equal(gv.cpu().numpy().astype(np.float64), V.astype(np.float32))
    # a NaN makes its own group NaN and no other
    y = torch.ones((1, 1, 128), device="cuda")
    y[0, 0, 70] = float("nan")
    c2 = make_cache(kv.empty_pages(1, 1, 128, P), 1, 128, P)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append(ctx, c2, y, y, z)
    gk, gv = moe.moe_kv_read(ctx, c2, z, dtype=torch.float32)
    assert (gk[..., :64] == 1).all() and gk[..., 64:].isnan().all() and gv[..., 64:].isnan().all()


def test_rows_with_strides_and_offsets(ctx):
    D, P, H, n = 128, 32, 4, 50
    rng = np.random.default_rng(5)
    pages = kv.empty_pages(3, H, D, P)
    cache = make_cache(pages, H, D, P)
    packed = rows(rng, n, 3 * H, D, "bf16")  # q | k | v of one projection
    k, v = packed[:, H:2 * H], packed[:, 2 * H:]
    slots = np.arange(n, dtype=np.int32) + 13
    s = torch.from_numpy(slots).cuda()
    moe.moe_kv_append(ctx, cache, k, v, s)
    kv.append(pages, P, f32(k), f32(v), slots)
    assert (cache.tensor.cpu().numpy() == pages).all()
    # heads outermost, and one row for every head (stride 0)
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    ve = v[:, :1].expand(n, H, D)
    moe.moe_kv_append(ctx, cache, kt, ve, s)
    kv.append(pages, P, f32(kt), f32(ve), slots)
    assert (cache.tensor.cpu().numpy() == pages).all()
    out = torch.zeros((2, H, n, D), dtype=torch.float16, device="cuda")
    moe.moe_kv_read(ctx, cache, s, k=out[0].transpose(0, 1), v=out[1].transpose(0, 1))
    K, V = kv.read(pages, P, slots)
    assert torch.equal(out[0].transpose(0, 1).cpu(), as_type(K, "f16"))
    assert torch.equal(out[1].transpose(0, 1).cpu(), as_type(V, "f16"))


# ---------------------------------------------------------------------------
# attention


def build(rng, kv_len, H, D, P, garbage=None):
    """Pages with garbage outside the sequences, and a table with garbage past their pages."""
    need = [-(-n // P) for n in kv_len]
    n_pages = sum(need) + 2
    pages = rng.integers(0, 256, (n_pages, H, P // 16, 18 * D), dtype=np.uint8)
    if garbage is not None:
        pages[:] = garbage
    order = rng.permutation(n_pages)
    table = np.full((len(kv_len), max(need + [1]) + 1), -7, np.int32)
    at = 0
    for b, n in enumerate(kv_len):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            t = np.arange(n)
            sl = table[b][t // P] * P + t % P
            K = rng.standard_normal((n, H, D)) * np.exp(rng.uniform(-1, 1, (1, H, D)))
            kv.append(pages, P, K.astype(np.float32), rng.standard_normal((n, H, D)).astype(np.float32), sl)
    return pages, table


def check(got, lse, q, ref, u):
    out, rl, e = ref
    delta = 3 * U * e["dot"][..., None]
    tol = (2 * delta * np.exp(2 * delta) + 3 * U + u) * e["mag"] + e["seen"][..., None] * 2.0 ** -17 * e["top"][..., None]
    bad = np.abs(got - out) > tol + 1e-30
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], np.abs(got - out).max())
    if lse is not None:
        fin = np.isfinite(rl)
        assert (np.isneginf(lse) == ~fin).all()
        assert (np.abs(lse - rl)[fin] <= (3 * U * e["dot"] + e["seen"] * 2.0 ** -24 + 1e-5 + 2.0 ** -22 * np.abs(rl))[fin]).all()


def attend_case(ctx, rng, kv_len, n_new, Hq, H, D, P, dtype, causal=True, window=0, scale=None, qmag=1.0, garbage=None, with_start=True,
                max_q=None):
    pages, table = build(rng, kv_len, H, D, P, garbage)
    cache = make_cache(pages, H, D, P)
    q_start = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    q = torch.from_numpy((qmag * rng.standard_normal((q_start[-1], Hq, D))).astype(np.float32)).to(TYPES[dtype]).cuda()
    tb, ln = torch.from_numpy(table).cuda(), torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    qs = torch.from_numpy(q_start).cuda() if with_start else None
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    mq = max(n_new) if max_q is None else max_q
    got = moe.moe_kv_attend(ctx, cache, q, tb, ln, q_start=qs, max_q=mq, scale=scale, causal=causal, window=window, lse=lse)
    torch.cuda.synchronize()
    moe.moe_kv_check(ctx)
    ref = kv.attend(pages, P, q.double().cpu().numpy(), table, kv_len, q_start, D ** -0.5 if scale is None else scale, causal, window)
    check(got.double().cpu().numpy(), lse.double().cpu().numpy(), q, ref, 2.0 ** -8 if dtype == "bf16" else U)
    return cache, q, tb, ln, qs, mq, got


# (kv lengths, new tokens, Hq, H, D, P, dtype, kwargs)
DECODE = [
    ([1], [1], 1, 1, 64, 16, "bf16", {}),
    ([1], [1], 8, 8, 128, 64, "f16", {}),
    ([15], [1], 4, 1, 256, 16, "bf16", {}),
    ([16, 17, 31, 33], [1] * 4, 16, 2, 128, 16, "bf16", {}),
    ([333], [1], 16, 8, 128, 64, "bf16", {}),
    ([2000], [1], 32, 8, 128, 64, "bf16", {}),
    ([5000], [1], 5, 5, 64, 256, "f16", {}),
    ([700, 0, 1, 64, 1025, 300], [1] * 6, 12, 4, 64, 32, "f16", {}),
    ([40, 0, 900], [1] * 3, 14, 2, 256, 128, "bf16", {}),
    ([600, 1300], [3, 3], 16, 8, 256, 16, "f16", {"window": 100}),
    ([600, 1300], [2, 5], 6, 2, 128, 32, "bf16", {"window": 1}),
    ([50, 2], [4, 4], 8, 2, 128, 32, "bf16", {}),  # two of the second's tokens see nothing
    ([777], [3], 22, 2, 128, 64, "f16", {"causal": False}),
    ([500] * 3, [2] * 3, 40, 1, 64, 64, "bf16", {"with_start": False}),
    ([300], [1], 8, 2, 128, 64, "bf16", {"scale": 0.0}),
    ([300], [1], 8, 2, 128, 64, "f16", {"scale": -0.05}),
    ([300, 299], [1, 1], 8, 2, 64, 64, "bf16", {"qmag": 40.0}),  # one key takes nearly all
    ([300, 200], [1, 0], 8, 2, 128, 16, "bf16", {"qmag": 1e-6}),
    ([300, 41], [1, 1], 8, 2, 128, 16, "f16", {"garbage": 0x7F}),  # NaN in every unused place
    ([300, 41], [1, 1], 8, 2, 256, 64, "f16", {"garbage": 0x7C}),  # huge values there
    ([20] * 70, [1] * 70, 4, 2, 64, 16, "bf16", {}),
]
PROMPT = [
    ([128], [128], 8, 2, 128, 64, "bf16", {}),
    ([129], [129], 4, 4, 64, 16, "f16", {}),
    ([1000], [77], 16, 2, 128, 32, "bf16", {}),
    ([300, 0, 64, 500], [300, 0, 1, 200], 6, 2, 128, 64, "bf16", {}),
    ([600], [600], 2, 1, 256, 64, "f16", {}),
    ([450], [321], 3, 1, 256, 16, "bf16", {"window": 70}),
    ([900], [400], 10, 2, 64, 128, "f16", {"window": 33}),
    ([333], [200], 7, 1, 128, 64, "bf16", {"causal": False}),
    ([100, 30], [150, 40], 8, 2, 128, 16, "bf16", {}),  # rows at positions below 0
    ([40], [40], 8, 1, 128, 32, "f16", {"garbage": 0x7F}),
    ([700], [130], 8, 1, 64, 32, "f16", {"garbage": 0x7C, "window": 600}),
    ([520], [260], 8, 2, 128, 32, "bf16", {"qmag": 40.0}),
    ([257, 257], [257, 257], 5, 5, 64, 32, "bf16", {"with_start": False}),
    ([3000], [64], 32, 4, 128, 64, "bf16", {}),
    ([2100], [33], 4, 1, 256, 64, "f16", {}),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_attention(ctx, i):
    *a, kw = DECODE[i]
    attend_case(ctx, np.random.default_rng(100 + i), *a, **kw)


@pytest.mark.parametrize("i", range(len(PROMPT)))
def test_prompt_attention(ctx, i):
    *a, kw = PROMPT[i]
    attend_case(ctx, np.random.default_rng(200 + i), *a, **kw)


@pytest.mark.parametrize("i", [3, 7, 9, 10, 12, 18])
def test_the_hint_changes_no_result_but_its_rounding(ctx, i):
    """max_q only chooses a kernel: a wrong one still gives the right answer."""
    *a, kw = DECODE[i]
    attend_case(ctx, np.random.default_rng(300 + i), *a, **kw, max_q=4096)


@pytest.mark.parametrize("i", [0, 3, 6, 8, 9])
def test_a_small_hint_on_a_prompt(ctx, i):
    *a, kw = PROMPT[i]
    attend_case(ctx, np.random.default_rng(400 + i), *a, **kw, max_q=1)


def test_strides_streams_and_repeats(ctx):
    rng = np.random.default_rng(9)
    D, P, H, Hq = 128, 64, 2, 8
    for kv_len, new in (([3000, 1000], [1, 1]), ([700, 900], [300, 257])):
        pages, table = build(rng, kv_len, H, D, P)
        cache = make_cache(pages, H, D, P)
        n = sum(new)
        packed = torch.from_numpy(rng.standard_normal((n, Hq + 2 * H, D)).astype(np.float32)).bfloat16().cuda()
        q = packed[:, :Hq]
        wide = torch.from_numpy(np.concatenate([table, table], 1)).cuda()
        tb, ln = wide[:, :table.shape[1]], torch.tensor(kv_len, dtype=torch.int32, device="cuda")
        qs = torch.tensor([0, new[0], n], dtype=torch.int32, device="cuda")
        first = moe.moe_kv_attend(ctx, cache, q.contiguous(), tb.contiguous(), ln, q_start=qs, max_q=max(new))
        out = torch.zeros((Hq, n, D), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = []
        for s in streams:  # the same call on several streams at once
            with torch.cuda.stream(s):
                for _ in range(4):
                    outs.append(moe.moe_kv_attend(ctx, cache, q, tb, ln, q_start=qs, max_q=max(new)))
        moe.moe_kv_attend(ctx, cache, q, tb, ln, q_start=qs, max_q=max(new), out=out.transpose(0, 1), stream=streams[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
        assert torch.equal(out.transpose(0, 1), first)


def test_captured_in_a_graph(ctx):
    rng = np.random.default_rng(10)
    D, P, H, Hq = 128, 64, 2, 8
    pages, table = build(rng, [2500], H, D, P)
    cache = make_cache(pages, H, D, P)
    q = torch.from_numpy(rng.standard_normal((1, Hq, D)).astype(np.float32)).bfloat16().cuda()
    k = torch.from_numpy(rng.standard_normal((1, H, D)).astype(np.float32)).bfloat16().cuda()
    tb, ln = torch.from_numpy(table).cuda(), torch.tensor([2500], dtype=torch.int32, device="cuda")
    slot = torch.tensor([int(table[0, 2499 // P]) * P + 2499 % P], dtype=torch.int32, device="cuda")

    def step():
        moe.moe_kv_append(ctx, cache, k, k, slot)
        return moe.moe_kv_attend(ctx, cache, q, tb, ln)

    want = step().clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    k.normal_()  # a new token through the same graph
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, step())


def test_far_pages_pass_32_bits(ctx):
    """A cache over 4 GiB: the last pages' byte offsets do not fit 32 bits."""
    D, P, H = 128, 256, 16
    per = moe.moe_kv_cache_bytes(H, D, P, 1)
    n_pages = (5 << 30) // per
    cache = moe.moe_kv_new_cache(n_pages, H, D, P)
    rng = np.random.default_rng(11)
    n = 300
    k, v = rows(rng, n, H, D, "bf16"), rows(rng, n, H, D, "bf16")
    t = np.arange(n)
    ids = np.array([n_pages - 1, n_pages - 2])
    slots = torch.from_numpy((ids[t // P] * P + t % P).astype(np.int32)).cuda()
    moe.moe_kv_append(ctx, cache, k, v, slots)
    small = kv.empty_pages(2, H, D, P)
    kv.append(small, P, f32(k), f32(v), t)
    K, V = kv.read(small, P, t)
    gk, gv = moe.moe_kv_read(ctx, cache, slots, dtype=torch.float32)
    assert torch.equal(gk.cpu(), as_type(K, "f32")) and torch.equal(gv.cpu(), as_type(V, "f32"))
    tb = torch.from_numpy(ids[None].astype(np.int32)).cuda()
    for new in (1, 200):
        q = rows(rng, new, H, D, "bf16")
        ln = torch.tensor([n], dtype=torch.int32, device="cuda")
        got = moe.moe_kv_attend(ctx, cache, q, tb, ln, max_q=new)
        ref = kv.attend(small, P, q.double().cpu().numpy(), np.array([[0, 1]]), [n], [0, new], D ** -0.5)
        check(got.double().cpu().numpy(), None, q, ref, 2.0 ** -8)


def test_bad_ids_are_skipped_and_noted(ctx):
    D, P, H = 64, 16, 1
    rng = np.random.default_rng(12)
    pages = kv.empty_pages(3, H, D, P)
    cache = make_cache(pages, H, D, P)
    k = rows(rng, 4, H, D, "bf16")
    slots = np.array([0, 48, 1, 2 ** 31 - 1], np.int32)  # 48 slots in all
    s = torch.from_numpy(slots).cuda()
    moe.moe_kv_append(ctx, cache, k, k, s)
    torch.cuda.synchronize()
    with pytest.raises(moe.MoeError, match="outside its cache"):
        moe.moe_kv_check(ctx)
    moe.moe_kv_check(ctx)
    kv.append(pages, P, f32(k)[[0, 2]], f32(k)[[0, 2]], [0, 1])
    assert (cache.tensor.cpu().numpy() == pages).all()
    gk, _ = moe.moe_kv_read(ctx, cache, s, dtype=torch.float32)
    torch.cuda.synchronize()
    with pytest.raises(moe.MoeError):
        moe.moe_kv_check(ctx)
    assert (gk[1] == 0).all() and (gk[3] == 0).all() and (gk[0] != 0).any()
    # a page id outside the cache hides its keys: the answer is that of the others
    t = np.arange(48)
    kk = rows(rng, 48, H, D, "bf16")
    moe.moe_kv_append(ctx, cache, kk, kk, torch.from_numpy(t.astype(np.int32)).cuda())
    for new, bad in ((1, 3), (1, -1), (20, 1 << 30)):
        q = rows(rng, new, H, D, "bf16")
        ln = torch.tensor([48], dtype=torch.int32, device="cuda")
        tb = torch.tensor([[0, bad, 2]], dtype=torch.int32, device="cuda")
        got = moe.moe_kv_attend(ctx, cache, q, tb, ln, max_q=new, causal=False)
        torch.cuda.synchronize()
        with pytest.raises(moe.MoeError, match="outside its cache"):
            moe.moe_kv_check(ctx)
        want = moe.moe_kv_attend(ctx, cache, q, torch.tensor([[0, 2]], dtype=torch.int32, device="cuda"),
                                 torch.tensor([32], dtype=torch.int32, device="cuda"), max_q=new, causal=False)
        np.testing.assert_allclose(f32(got), f32(want), atol=2 * 2.0 ** -8 * np.abs(f32(want)).max())
    # a length past the table counts as the table's
    q = rows(rng, 1, H, D, "bf16")
    tb = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    a = moe.moe_kv_attend(ctx, cache, q, tb, torch.tensor([1000], dtype=torch.int32, device="cuda"), causal=False)
    b = moe.moe_kv_attend(ctx, cache, q, tb, torch.tensor([32], dtype=torch.int32, device="cuda"), causal=False)
    assert torch.equal(a, b)
    moe.moe_kv_check(ctx)


def test_empty_calls(ctx):
    cache = moe.moe_kv_new_cache(1, 2, 64, 16)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    moe.moe_kv_append(ctx, cache, e, e, z)
    k, v = moe.moe_kv_read(ctx, cache, z)
    assert k.shape == v.shape == (0, 2, 64)
    assert moe.moe_kv_attend(ctx, cache, e, torch.empty((0, 3), dtype=torch.int32, device="cuda"), z).shape == (0, 2, 64)
    # sequences without pages at all
    q = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = moe.moe_kv_attend(ctx, cache, q, torch.empty((2, 0), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert (out == 0).all()


def test_refusals(ctx):
    cache = moe.moe_kv_new_cache(2, 2, 64, 16)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, dtype=torch.int32, device="cuda")
    tb, ln = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    before = cache.tensor.clone()
    pad = torch.zeros(3 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    off = pad[1:1 + 3 * 2 * 64].view(3, 2, 64)  # rows off the 16-byte boundary
    odd = torch.zeros((3, 2, 68), dtype=torch.bfloat16, device="cuda")[..., :64]
    for bad in (lambda: moe.moe_kv_append(ctx, cache, off, k, s), lambda: moe.moe_kv_append(ctx, cache, k, odd, s),
                lambda: moe.moe_kv_read(ctx, cache, s, k=off, v=k), lambda: moe.moe_kv_attend(ctx, cache, odd, tb, ln),
                lambda: moe.moe_kv_attend(ctx, cache, q[:, :3], tb, ln),  # 3 heads over 2 kv heads
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, window=-1),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, scale=float("nan")),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, causal=2),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb[:0], ln[:0]),  # rows of no sequence
                lambda: moe.moe_kv_attend(ctx, cache, q.float(), tb, ln)):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.status == moe.MOE_EINVAL
    for bad in (lambda: moe.moe_kv_append(ctx, cache, k.double(), k.double(), s), lambda: moe.moe_kv_append(ctx, cache, k, k[:2], s),
                lambda: moe.moe_kv_append(ctx, cache, k, k, s.long()), lambda: moe.moe_kv_append(ctx, cache, k[..., :32], k[..., :32], s),
                lambda: moe.moe_kv_append(ctx, cache, k.cpu(), k.cpu(), s), lambda: moe.moe_kv_append(ctx, cache, k, k, s[:2]),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln.long()), lambda: moe.moe_kv_attend(ctx, cache, q, tb.t(), ln),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, q_start=s[:1]), lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, out=q[:1]),
                lambda: moe.moe_kv_attend(ctx, cache, q, tb, ln, lse=torch.zeros(3, device="cuda")),
                lambda: moe.moe_kv_make_cache(cache.tensor, 2, 128, 16), lambda: moe.moe_kv_make_cache(cache.tensor.cpu(), 2, 64, 16)):
        with pytest.raises(ValueError):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(cache.tensor, before)
    moe.moe_kv_check(ctx)


def test_launches_are_counted_and_timed(ctx):
    cache = moe.moe_kv_new_cache(8, 2, 64, 16)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, dtype=torch.int32, device="cuda")
    moe.moe_ctx_set_profiling(ctx, True)
    moe.moe_ctx_reset_kernel_times(ctx)
    n0 = moe.moe_ctx_launches(ctx)
    moe.moe_kv_append(ctx, cache, k, k, s)
    moe.moe_kv_read(ctx, cache, s)
    moe.moe_kv_attend(ctx, cache, k, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), s[2:] + 1)
    t = moe.moe_ctx_kernel_times(ctx)
    moe.moe_ctx_set_profiling(ctx, False)
    assert moe.moe_ctx_launches(ctx) == n0 + 3
    for kind in ("kv_append", "kv_read", "kv_attend"):
        assert t[kind][0] == 1 and t[kind][1] > 0
