"""Norm, 8-bit quantisation and 8-bit matrix products against plain 64-bit forms.

Bounds (u = 2^-24, half a step of fp32):
* norm: h = x + r is off by u of itself; the sum of dim squares is in order within a thread (at most 32 of them) and in a
  tree across threads (at most 10 steps), so off by 43 u of itself, its root by 22 u; rsqrtf by 4 u (2 ulp), the factor
  1 / dim, its product and the addition of eps by u each under the root, and two products: 32 u of |y| in all, and half
  a step of the output's type.
* quantised y: half a step of e4m3, 2^-4 of the value or, among subnormal codes, 2^-10 of the scale, besides the error of y.
* matrix product: a K-block's 128 products are exact and summed in fp32 in any order, whichever way a step rounds (2 u each):
  256 u of the sum of their magnitudes; its two scales' product and the addition to the K-blocks before, u each.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import expert_streaming_ffn_gb300 as moe  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
LEAST = 448 * 2.0 ** -126
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ctx():
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def half_step(y, dtype):
    """Half a step of `dtype` around y (subnormals among them)."""
    f = torch.finfo(dtype)
    return torch.maximum(y.abs() * (f.eps / 2), torch.full_like(y, f.smallest_normal * f.eps / 2))


def wide(t, dim, n):
    return t.repeat_interleave(128, dim).narrow(dim, 0, n)


def value(codes, scales, weight=False):
    """Codes [n][k] and their scales as fp64 values."""
    n, k = codes.shape
    s = wide(wide(scales.double(), 0, n), 1, k) if weight else wide(scales.double(), 0, k).t()
    return codes.double() * s, s


def block_top(y):
    """Largest magnitude of each block of 128 of a row, [n][blocks]."""
    n, d = y.shape
    return torch.nn.functional.pad(y, (0, -d % 128)).abs().view(n, -1, 128).amax(-1)


# ---- norm --------------------------------------------------------------------------


def norm_ref(x, weight, eps, residual):
    h = x.double() + (residual.double() if residual is not None else 0.0)
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, y * weight.double() if weight is not None else y


def check_norm(x, weight, eps, residual, got):
    out, total, codes, scales = got
    h, y = norm_ref(x, weight, eps, residual)
    if residual is not None:
        assert ((total.double() - h).abs() <= U * h.abs() + half_step(h, total.dtype) * (1 + 2 * U)).all()
    else:
        assert total is None
    if out is not None:
        assert ((out.double() - y).abs() <= 32 * U * y.abs() + half_step(y, out.dtype) * (1 + 32 * U)).all()
    if codes is not None:
        y = y.flatten(1) if y.dim() == 3 else y
        want = block_top(y).clamp(min=LEAST) / 448
        assert ((scales.t().double() - want).abs() <= 33 * U * want).all()
        v, s = value(codes, scales)
        assert ((v - y).abs() <= y.abs() * (2.0 ** -4 + 64 * U) + s * (2.0 ** -10 + 64 * U)).all()


@pytest.mark.parametrize("n,heads,dim", [(1, 1, 2816), (3, 1, 16), (5, 1, 48), (77, 1, 2048), (9, 1, 272), (2, 1, 4096), (3, 1, 4112),
                                         (2, 1, 8192), (2, 1, 16400), (1, 1, 32768), (33, 5, 64), (7, 32, 128), (6, 3, 256), (4, 2, 320)])
@pytest.mark.parametrize("xt,rt,wt,ot", [("f32", "bf16", "bf16", "bf16"), ("bf16", None, None, "f32"), ("f16", "f32", "f32", "f16"),
                                         ("f32", "f32", "f16", "f32"), ("bf16", "f16", "bf16", None)])
def test_norm(ctx, n, heads, dim, xt, rt, wt, ot):
    g = rng(n * dim + heads)
    x = (randn(g, n, heads, dim) * torch.exp(randn(g, dim))).to(T[xt])
    r = (2 * randn(g, n, heads, dim)).to(T[rt]) if rt else None
    w = (1 + 0.3 * randn(g, dim)).to(T[wt]) if wt else None
    got = moe.moe_rms_norm(ctx, x, w, 1e-5, residual=r, dtype=T.get(ot), f8=heads == 1)
    if ot is None and heads > 1:
        assert got[0] is None
    check_norm(x, w, 1e-5, r, got)


@pytest.mark.parametrize("n,heads,dim", [(81000, 1, 64), (2601, 16, 128), (20001, 1, 256), (19000, 1, 272), (10007, 1, 512), (5003, 1, 1008),
                                         (5000, 1, 1024), (3001, 1, 2816), (1301, 1, 4096), (1000, 1, 5008), (700, 1, 8192), (400, 1, 16400)])
@pytest.mark.parametrize("xt,rt,wt,ot", [("f32", "bf16", "bf16", "bf16"), ("f16", None, "f32", "f32"), ("bf16", "f32", None, None)])
def test_norm_of_many_rows(ctx, n, heads, dim, xt, rt, wt, ot):
    """Rows enough that each thread takes several vectors, or rows, at a time."""
    g = rng(n)
    x = (randn(g, n, heads, dim) * torch.exp(randn(g, dim))).to(T[xt])
    r = randn(g, n, heads, dim).to(T[rt]) if rt else None
    w = (1 + 0.3 * randn(g, dim)).to(T[wt]) if wt else None
    if ot is None and heads > 1:
        ot = "f16"
    check_norm(x, w, 1e-5, r, moe.moe_rms_norm(ctx, x, w, 1e-5, residual=r, dtype=T.get(ot), f8=heads == 1))


def test_norm_rows_of_wider_tensors_in_place(ctx):
    """Heads of a fused projection, normed where they lie; the residual's sum over the residual; what lies beside stays."""
    g = rng(1)
    qkv = randn(g, 37, 12, 128).bfloat16()
    before = qkv.clone()
    w = randn(g, 128)
    part = qkv[:, 2:7]
    got = moe.moe_rms_norm(ctx, part, w, out=part)
    assert got[0] is part
    check_norm(before[:, 2:7], w, 1e-6, None, got)
    assert (qkv[:, :2] == before[:, :2]).all() and (qkv[:, 7:] == before[:, 7:]).all()
    x, res = randn(g, 5, 2816), randn(g, 9, 2816 + 64).bfloat16()
    old = res.clone()
    view = res[2:7, 32:-32]
    got = moe.moe_rms_norm(ctx, x, residual=view, sum=view, dtype=torch.bfloat16, f8=True)
    check_norm(x, None, 1e-6, old[2:7, 32:-32], got)
    old[2:7, 32:-32] = view
    assert (res == old).all()


def test_norm_strided_codes_and_scales(ctx):
    g = rng(2)
    x = randn(g, 6, 400).half()
    codes = torch.zeros((8, 512), dtype=torch.uint8, device="cuda").view(F8)
    scales = torch.full((6, 11), -3.0, device="cuda")
    c, s = codes[1:7, 16:416], scales[1:5, 2:8]
    got = moe.moe_rms_norm(ctx, x, dtype=None, codes=c, scales=s)
    check_norm(x, None, 1e-6, None, got)
    keep = torch.ones_like(scales, dtype=torch.bool)
    keep[1:5, 2:8] = False
    assert (scales[keep] == -3).all()
    raw = codes.view(torch.uint8).clone()
    raw[1:7, 16:416] = 0
    assert (raw == 0).all()


def test_norm_special_values(ctx):
    """Rows of zeros; tiny and huge rows; a NaN stays in its row; an infinity makes its row NaN or zero as the formula says."""
    g = rng(3)
    x = randn(g, 8, 512)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 100] = math.nan
    x[6] = 1e-42  # subnormal
    out, _, codes, scales = moe.moe_rms_norm(ctx, x, eps=1e-12, f8=True)
    ok = [0, 1, 2, 3, 5, 7]
    check_norm(x[ok], None, 1e-12, None, (out[ok], None, codes[ok], scales[:, ok]))
    assert (out[1] == 0).all() and (codes[1].float() == 0).all() and torch.isfinite(out[6]).all()
    assert torch.isnan(out[4]).all() and torch.isnan(scales[:, 4]).all() and torch.isnan(codes[4].float()).all()


def test_norm_of_nothing(ctx):
    out, total, codes, scales = moe.moe_rms_norm(ctx, torch.empty((0, 256), device="cuda"), f8=True)
    assert out.shape == (0, 256) and codes.shape == (0, 256) and scales.shape == (2, 0)


# ---- quantisation ------------------------------------------------------------------


def quant_ref(x, weight):
    """As IEEE arithmetic gives it, on the CPU."""
    x = x.float().cpu()
    n, k = x.shape
    if weight:
        b = torch.nn.functional.pad(x, (0, -k % 128, 0, -n % 128)).view(-(-n // 128), 128, -(-k // 128), 128)
        s = b.abs().amax((1, 3)).clamp(min=LEAST) / 448
        q = x / wide(wide(s, 0, n), 1, k)
    else:
        s = (block_top(x).clamp(min=LEAST) / 448).t()
        q = x / wide(s, 0, k).t()
    return q.clamp(-448, 448).to(F8), s


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,k", [(1, 16), (1, 128), (3, 4096), (129, 144), (64, 2816), (257, 704), (1000, 272), (2501, 4096), (5003, 2064)])
def test_quant_is_exact(ctx, n, k, dtype, weight):
    g = rng(n + k)
    x = (randn(g, n, k) * torch.exp(2 * randn(g, 1, k))).to(T[dtype])
    if k >= 256:
        x[0, :128] = 0
        x[0, 128:256] = (torch.arange(128, device="cuda") % 57 * 8 + 4).to(T[dtype])  # ties, and the largest not a nice number
    codes, scales = (moe.moe_f8_quant_weight if weight else moe.moe_f8_quant_rows)(ctx, x)
    want, s = quant_ref(x, weight)
    assert (scales.cpu() == s).all()
    assert (codes.cpu().float() == want.float()).all()


@pytest.mark.parametrize("weight", [False, True])
def test_quant_special_values(ctx, weight):
    """An infinity or a NaN makes its block NaN and no other; zeros stay zeros; magnitudes below 2^-117 keep a normal scale."""
    x = randn(rng(4), 260, 512)
    x[0, 3] = math.nan
    x[1, 200] = math.inf
    x[2, 300] = -math.inf
    x[128:256, 128:256] = 0
    x[128:256, 256:384] = 1e-40
    codes, scales = (moe.moe_f8_quant_weight if weight else moe.moe_f8_quant_rows)(ctx, x)
    v, _ = value(codes, scales, weight)
    bad = torch.zeros((260, 4), dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    if weight:
        bad[:128, :3] = True
    assert (torch.isnan(v) == wide(bad, 1, 512)).all()
    assert (v[128:256, 128:256] == 0).all() and (v[128:256, 256:384].abs() <= 2e-40).all()
    y = torch.where(torch.isfinite(x), x, 0.0).double()
    _, s = value(codes, scales, weight)
    good = ~torch.isnan(v)
    assert ((v - y).abs() <= y.abs() * (2.0 ** -4 + 4 * U) + s * (2.0 ** -10 + 4 * U))[good].all()


def test_quant_strided(ctx):
    x = randn(rng(5), 50, 600).bfloat16()[3:40, 8:-16]
    assert x.shape == (37, 576)
    codes = torch.zeros((40, 640), dtype=torch.uint8, device="cuda").view(F8)
    scales = torch.full((5, 64), 7.0, device="cuda")
    moe.moe_f8_quant_rows(ctx, x, codes[:37, :576], scales[:, :37])
    want, s = quant_ref(x, False)
    assert (codes[:37, :576].cpu().float() == want.float()).all() and (scales[:, :37].cpu() == s).all()
    assert (codes.view(torch.uint8)[37:] == 0).all() and (codes.view(torch.uint8)[:, 576:] == 0).all() and (scales[:, 37:] == 7).all()


# ---- matrix product ------------------------------------------------------------------


def operands(g, m, n, k):
    """Codes and scales of all signs and sizes (what a quantiser never writes among them: any code, scales below zero)."""
    a = (randn(g, m, k) * 40).clamp(-448, 448).to(F8)
    w = (randn(g, n, k) * 40).clamp(-448, 448).to(F8)
    kb, nb = -(-k // 128), -(-n // 128)
    return a, randn(g, kb, m) * 0.02, w, randn(g, nb, kb) * 0.02


def check_matmul(a, sa, w, sw, out):
    m, k = a.shape
    A, _ = value(a, sa)
    W, _ = value(w, sw, True)
    want = A @ W.t()
    size = A.abs() @ W.abs().t()
    err = (256 + 2 + -(-k // 128)) * U * size + half_step(want, out.dtype) * (1 + 1e-3)
    assert ((out.double() - want).abs() <= err).all()


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 6144, 2816), (1, 128, 128), (2, 2816, 4096), (5, 999, 2048), (16, 130, 144), (17, 257, 2832),
                                   (32, 704, 2816), (33, 64, 512), (64, 8192, 640), (65, 100, 2048), (77, 2816, 4096), (128, 6144, 256),
                                   (129, 385, 1040), (143, 1000, 2816), (200, 128, 16384), (257, 300, 704), (300, 2816, 2048), (1000, 515, 1296),
                                   (2049, 1030, 400), (40, 40000, 272), (513, 6144, 2816),
                                   (1052, 1154, 7536), (2200, 631, 4096), (600, 330, 16384), (700, 2047, 2064)])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
def test_matmul(ctx, m, n, k, dtype):
    ops = operands(rng(m + n + k), m, n, k)
    check_matmul(*ops, moe.moe_f8_matmul(ctx, *ops, dtype=T[dtype]))


@pytest.mark.parametrize("m,n,k", [(1, 2000, 2816), (13, 2000, 4096), (40, 2000, 4096), (300, 2000, 4096), (1000, 1000, 4096)])
def test_matmul_keeps_fp32(ctx, m, n, k):
    """Sums are held in fp32 throughout. Of 32 K-blocks each addition rounds by u of the sum so far at most, whose rms is at most
    the result's: sqrt(33) u if they are independent, and 2 u for the scales: 8 u of the result's norm."""
    g = rng(m)
    a, sa = moe.moe_f8_quant_rows(ctx, randn(g, m, k))
    w, sw = moe.moe_f8_quant_weight(ctx, randn(g, n, k) * k ** -0.5)
    out = moe.moe_f8_matmul(ctx, a, sa, w, sw, dtype=torch.float32).double()
    want = value(a, sa)[0] @ value(w, sw, True)[0].t()
    assert (out - want).norm() <= 8 * U * want.norm()


@pytest.mark.parametrize("m,n,k", [(3, 200, 400), (40, 333, 1024), (100, 300, 272), (700, 777, 528)])
@pytest.mark.parametrize("pad", [1, 8])
def test_matmul_strided(ctx, m, n, k, pad):
    """Operands and output inside larger ones; bytes behind a row's end are never used, those behind out's rows stay."""
    g = rng(m)
    a, sa, w, sw = operands(g, m, n, k)

    def inside(t, rows, cols):
        big = torch.full((t.shape[0] + 3, t.shape[1] + cols), 0x7F, dtype=torch.uint8, device="cuda").view(F8)  # NaN around
        big.view(torch.uint8)[rows:rows + t.shape[0], 16:16 + t.shape[1]] = t.view(torch.uint8)
        return big[rows:rows + t.shape[0], 16:16 + t.shape[1]]

    def around(t):
        big = torch.full((t.shape[0] + 2, t.shape[1] + 5), math.nan, device="cuda")
        big[1:-1, 3:-2] = t
        return big[1:-1, 3:-2]

    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((m + 2, n + 2 * pad), 5.0, dtype=dtype, device="cuda")
        ops = inside(a, 1, 48), around(sa), inside(w, 2, 32), around(sw)
        moe.moe_f8_matmul(ctx, *ops, out=out[1:-1, pad:-pad])
        check_matmul(a, sa, w, sw, out[1:-1, pad:-pad])
        out[1:-1, pad:-pad] = 5
        assert (out == 5).all()


@pytest.mark.parametrize("m", [2, 30, 50, 100, 400])
def test_matmul_nan_and_infinity_stay_in_place(ctx, m):
    """A NaN row, a NaN weight and an infinite scale reach the outputs that they are part of and no others; zeros give zeros."""
    g = rng(m)
    n, k = 300, 640
    a, sa, w, sw = operands(g, m, n, k)
    a.view(torch.uint8)[1, 130] = 0x7F
    w.view(torch.uint8)[200, 7] = 0xFF
    sa[2, 0] = math.inf
    clean = operands(rng(m), m, n, k)
    out = moe.moe_f8_matmul(ctx, a, sa, w, sw, dtype=torch.float32)
    base = moe.moe_f8_matmul(ctx, *clean, dtype=torch.float32)
    assert torch.isnan(out[1]).all() and torch.isnan(out[:, 200]).all()
    assert not torch.isfinite(out[0]).any()
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[:2] = False
    rest[:, 200] = False
    assert (out[rest] == base[rest]).all()
    z = torch.zeros_like(a.view(torch.uint8)).view(F8)
    assert (moe.moe_f8_matmul(ctx, z, clean[1], w[:190], sw[:2], dtype=torch.float16) == 0).all()


def test_matmul_of_no_rows(ctx):
    a, sa, w, sw = operands(rng(0), 0, 50, 256)
    assert moe.moe_f8_matmul(ctx, a, sa, w, sw).shape == (0, 50)


def test_matmul_of_zero_accumulates_nothing_left_over(ctx):
    """Repeated calls of several shapes give the same bits, whatever ran before on the SMs' tensor memory."""
    shapes = [(1, 500, 512), (20, 1000, 2816), (60, 300, 1024), (100, 2816, 704), (600, 900, 1024), (1052, 1154, 7536), (2000, 400, 8192)]
    ops = [operands(rng(i), *s) for i, s in enumerate(shapes)]
    first = [moe.moe_f8_matmul(ctx, *o, dtype=torch.float32) for o in ops]
    for _ in range(5):
        again = [moe.moe_f8_matmul(ctx, *o, dtype=torch.float32) for o in reversed(ops)][::-1]
        assert all((x == y).all() for x, y in zip(first, again))


# ---- together ----------------------------------------------------------------------


def layer(ctx, p, x, res):
    """The dense parts of a decoder layer: norm, projection, heads' norm, quantisation, output projection, norm."""
    _, _, c, s = moe.moe_rms_norm(ctx, x, p["n1"], residual=res, sum=res, dtype=None, f8=True)
    qkv = moe.moe_f8_matmul(ctx, c, s, *p["w_in"])
    q = qkv.unflatten(1, (-1, 64))
    moe.moe_rms_norm(ctx, q, p["nh"], out=q)
    c2, s2 = moe.moe_f8_quant_rows(ctx, qkv)
    o = moe.moe_f8_matmul(ctx, c2, s2, *p["w_out"], dtype=torch.float32)
    y, _, _, _ = moe.moe_rms_norm(ctx, o, p["n2"], residual=res, sum=res, dtype=torch.bfloat16)
    return c, s, qkv, c2, s2, o, y


def params(ctx, d, h, seed):
    g = rng(seed)
    return dict(n1=(1 + 0.1 * randn(g, d)).bfloat16(), nh=(1 + 0.1 * randn(g, 64)).bfloat16(), n2=1 + 0.1 * randn(g, d),
                w_in=moe.moe_f8_quant_weight(ctx, (randn(g, h, d) * d ** -0.5).bfloat16()),
                w_out=moe.moe_f8_quant_weight(ctx, (randn(g, d, h) * h ** -0.5).bfloat16()))


@pytest.mark.parametrize("n", [1, 29, 300])
def test_together(ctx, n):
    """Each step against 64 bits from the step before's outputs; the same on another stream; and captured and replayed with new inputs."""
    d, h = 512, 768
    p = params(ctx, d, h, n)
    g = rng(n + 1)
    x, res0 = randn(g, n, d), (3 * randn(g, n, d)).bfloat16()
    res = res0.clone()
    got = layer(ctx, p, x, res)
    c, s, qkv, c2, s2, o, y = got
    mid = (x + res0.float()).bfloat16()
    check_norm(x, p["n1"], 1e-6, res0, (None, mid, c, s))
    check_matmul(c2, s2, *p["w_out"], o)
    want, sc = quant_ref(qkv, False)
    assert (c2.cpu().float() == want.float()).all() and (s2.cpu() == sc).all()
    check_norm(o, p["n2"], 1e-6, mid, (y, res, None, None))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        res1 = res0.clone()
        other = layer(ctx, p, x, res1)
    side.synchronize()
    assert all((a.float() == b.float()).all() for a, b in zip(got, other)) and (res1 == res).all()
    graph = torch.cuda.CUDAGraph()
    x2, res2 = torch.zeros_like(x), torch.zeros_like(res)
    with torch.cuda.graph(graph):
        kept = layer(ctx, p, x2, res2)
    for _ in range(2):
        x2.copy_(x)
        res2.copy_(res0)
        graph.replay()
        torch.cuda.synchronize()
        assert all((a.float() == b.float()).all() for a, b in zip(got, kept)) and (res2 == res).all()


def test_two_streams_at_once(ctx):
    """Calls of two streams that run at the same time share nothing."""
    p = [params(ctx, 1024, 2048, i) for i in range(2)]
    x = [randn(rng(i), 40, 1024) for i in range(2)]
    res = [randn(rng(9 + i), 40, 1024).bfloat16() for i in range(2)]
    want = []
    for i in range(2):
        r = res[i].clone()
        want.append(layer(ctx, p[i], x[i], r)[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                r = res[i].clone()
                got[i].append(layer(ctx, p[i], x[i], r)[-1])
    torch.cuda.synchronize()
    assert all((y == want[i]).all() for i in range(2) for y in got[i])


def test_profiling_counts_the_calls(ctx):
    moe.moe_ctx_set_profiling(ctx, True)
    try:
        moe.moe_ctx_reset_kernel_times(ctx)
        n0 = moe.moe_ctx_launches(ctx)
        x = randn(rng(0), 4, 256)
        _, _, c, s = moe.moe_rms_norm(ctx, x, f8=True)
        w = moe.moe_f8_quant_weight(ctx, x)
        moe.moe_f8_quant_rows(ctx, x)
        moe.moe_f8_matmul(ctx, c, s, *w)
        torch.cuda.synchronize()
        t = moe.moe_ctx_kernel_times(ctx)
        assert [t[k][0] for k in ("rms_norm", "f8_quant", "f8_matmul")] == [1, 2, 1]
        assert moe.moe_ctx_launches(ctx) - n0 == 4
        assert t["f8_matmul"][3] == 2 * 4 * 4 * 256
    finally:
        moe.moe_ctx_set_profiling(ctx, False)


@pytest.mark.parametrize("tokens", [1, 3, 100])
@pytest.mark.parametrize("source", ["out", "sum", "product"])
def test_rows_go_straight_into_the_experts(ctx, tokens, source):
    """moe_forward right behind the call that writes its x, nothing in between: it reads these rows, not the ones before."""
    import synth

    s = synth.SHAPES_TINY
    layer = moe.moe_layer_create(ctx, s, 4, moe.LFU)
    try:
        moe.moe_layer_set_weights(layer, synth.layer_weights(s, 0))
        moe.moe_layer_set_deterministic(layer, True)
        g = rng(tokens)
        x = torch.zeros((tokens, s.d_model), dtype=torch.bfloat16, device="cuda")
        k = 65536  # a product that takes its time
        w = moe.moe_f8_quant_weight(ctx, randn(g, s.d_model, k) * k ** -0.5)
        rows = [randn(g, tokens, s.d_model) for _ in range(24)]
        zero = torch.zeros_like(x)
        wide_rows = [moe.moe_f8_quant_rows(ctx, randn(g, tokens, k)) for _ in range(24)]
        noise = torch.empty((1 << 22,), device="cuda")

        def write(i):
            if source == "out":
                moe.moe_rms_norm(ctx, rows[i], out=x)
            elif source == "sum":
                moe.moe_rms_norm(ctx, rows[i], residual=zero, sum=x, dtype=None, f8=True)
            else:
                moe.moe_f8_matmul(ctx, *wide_rows[i], *w, out=x)

        want, got = [], []
        for i in range(24):
            write(i)
            torch.cuda.synchronize()
            want.append(moe.moe_forward(layer, x).clone())
            torch.cuda.synchronize()
        for i in range(24):
            noise.normal_()  # the device is behind the host, so that the calls queue up
            write(i)
            got.append(moe.moe_forward(layer, x))
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(want, got))
    finally:
        moe.moe_layer_destroy(layer)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import expert_streaming_ffn_gb300 as moe
ctx = moe.moe_ctx_create(0)
a = torch.randn(({m}, 1024), device="cuda")
w = torch.randn((700, 1024), device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    _, _, c, s = moe.moe_rms_norm(ctx, a, dtype=None, f8=True)
    q = moe.moe_f8_quant_weight(ctx, w)
    out = moe.moe_f8_matmul(ctx, c, s, *q, dtype=torch.float32)
graph.replay()
torch.cuda.synchronize()
n = torch.nn.functional.rms_norm(a, (1024,), eps=1e-6) @ w.t()
print(((out - n).norm() / n.norm()).item())
"""


@pytest.mark.parametrize("m", [4, 24, 700])
def test_first_calls_of_a_process_can_be_captured(m):
    """The first call of each kind looks a few things up and allocates nothing, so it may be part of a graph. 8 bits a side: each
    operand within 2^-4 of itself, so the product's relative error in the 2-norm is below 2 * 2^-4."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, m=m)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert float(r.stdout.split()[-1]) < 2 * 2.0 ** -4


def test_calls_from_several_threads(ctx):
    """Host threads with a stream each, the same context: the same bits as one after the other."""
    import threading

    p = params(ctx, 512, 1024, 3)
    shapes = [1, 20, 50, 90, 300]
    x = [randn(rng(i), n, 512) for i, n in enumerate(shapes)]
    res = [randn(rng(30 + i), n, 512).bfloat16() for i, n in enumerate(shapes)]
    want = []
    for i in range(len(shapes)):
        r = res[i].clone()
        want.append(layer(ctx, p, x[i], r)[-1])
    torch.cuda.synchronize()
    got, errors = [[] for _ in shapes], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    r = res[i].clone()
                    got[i].append(layer(ctx, p, x[i], r)[-1])
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all((y == want[i]).all() for i in range(len(shapes)) for y in got[i])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_offsets_past_32_bits(ctx, dtype):
    """Rows whose elements lie beyond 2^31 of each other: norm, quantisation and product by strides."""
    stride = (1 << 31) // 2 + 4096 if dtype == "f32" else (1 << 31) + 4096
    n, d = 3, 256
    if (n - 1) * stride * (4 if dtype == "f32" else 2) > 40 << 30:
        pytest.skip("no room")
    x = torch.empty(((n - 1) * stride + d,), dtype=T[dtype], device="cuda").as_strided((n, d), (stride, 1))
    x.copy_(randn(rng(8), n, d))
    small = x.contiguous()
    out, _, c, s = moe.moe_rms_norm(ctx, x, out=x, f8=True)
    want, _, cw, sw = moe.moe_rms_norm(ctx, small, f8=True)
    assert (x == want).all() and (c.float() == cw.float()).all() and (s == sw).all()
    c1, s1 = moe.moe_f8_quant_rows(ctx, x)
    c2, s2 = moe.moe_f8_quant_rows(ctx, want)
    assert (c1.float() == c2.float()).all() and (s1 == s2).all()
    w = moe.moe_f8_quant_weight(ctx, randn(rng(9), 500, d))
    y = torch.empty(((n - 1) * stride + 500,), dtype=T[dtype], device="cuda").as_strided((n, 500), (stride, 1))
    moe.moe_f8_matmul(ctx, c1, s1, *w, out=y)
    assert (y == moe.moe_f8_matmul(ctx, c1, s1, *w, dtype=T[dtype])).all()


def test_tensors_on_another_device_than_the_context(ctx, monkeypatch):
    """A context of another device is refused in the binding, before anything is launched."""
    x = randn(rng(10), 4, 256)
    a, w = moe.moe_f8_quant_rows(ctx, x), moe.moe_f8_quant_weight(ctx, x)
    monkeypatch.setitem(moe._ctx_devices, ctx, 1)
    for call in (lambda: moe.moe_rms_norm(ctx, x), lambda: moe.moe_f8_quant_rows(ctx, x),
                 lambda: moe.moe_f8_quant_weight(ctx, x), lambda: moe.moe_f8_matmul(ctx, *a, *w)):
        with pytest.raises(ValueError, match="context"):
            call()
