"""The forms of the 8-bit product at the ends of their ranges. Bounds and helpers are those of test_gpu_dense.py."""
import pytest

torch = pytest.importorskip("torch")
import expert_streaming_ffn_gb300 as moe  # noqa: E402
import test_gpu_dense as dense  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def ctx():
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


def check(ctx, m, n, k, dtype):
    ops = dense.operands(dense.rng(m + n + k), m, n, k)
    dense.check_matmul(*ops, moe.moe_f8_matmul(ctx, *ops, dtype=dense.T[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("n,k", [(1, 16), (15, 128), (17, 144), (33, 1024), (129, 1040), (4864, 2048), (4865, 2048), (2000, 2064), (1000, 4096),
                                 (1001, 4112), (4864, 4096), (4865, 4080), (7296, 2448), (7297, 2448), (7296, 4096)])
def test_up_to_16_rows(ctx, m, n, k, dtype):
    """A K-block a warp and fewer, up to as many as it holds, and one more; a round of CTAs of 16 weights, three or two
    an SM, and one more."""
    check(ctx, m, n, k, dtype)


def test_an_expired_wait_is_reported_until_it_is_asked_for(ctx):
    """By every product, to whatever thread, and by the check, which takes it back; the cache's check does not; also behind the last
    call, as with a replayed graph. (The note is made on the host.)"""
    import threading

    ops = dense.operands(dense.rng(0), 3, 100, 256)
    want = moe.moe_f8_matmul(ctx, *ops, dtype=torch.float32)
    torch.cuda.synchronize()
    moe.moe_f8_check(ctx)
    moe.moe_ctx_inject_f8_timeout(ctx)
    errors = []

    def other():
        try:
            moe.moe_f8_matmul(ctx, *ops)
        except moe.MoeError as e:
            errors.append(e.status)

    for _ in range(2):
        t = threading.Thread(target=other)
        t.start()
        t.join()
    moe.moe_kv_check(ctx)
    n = moe.moe_ctx_launches(ctx)
    other()
    assert errors == [moe.MOE_ETIMEOUT] * 3 and moe.moe_ctx_launches(ctx) == n
    with pytest.raises(moe.MoeError) as e:
        moe.moe_f8_check(ctx)
    assert e.value.status == moe.MOE_ETIMEOUT
    moe.moe_f8_check(ctx)
    assert torch.equal(moe.moe_f8_matmul(ctx, *ops, dtype=torch.float32), want)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant_is_exact_near_the_least_scale(ctx, dtype, weight):
    """Blocks whose scale is 2^-126 to 2^-60, of values at ties between codes and one step of the type beside them. The reference
    divides on the CPU, by IEEE arithmetic with subnormals, and rounds the quotient."""
    g = torch.Generator().manual_seed(7)
    per = 128 if weight else 1  # rows that share a scale
    exps = [-126, -125, -124, -122, -120, -117, -112, -104, -97, -94, -93, -92, -91, -90, -89, -88, -60]
    reps = 4 if weight else 400
    bits = 13 if dtype == "f32" else 3  # of the scale: 448 times it is exact
    s = torch.cat([torch.ldexp(1.0 + torch.randint(0, 1 << bits, (reps,), generator=g) / (1 << bits), torch.tensor(float(e))) for e in exps])
    s = s.double().repeat_interleave(per)
    n = s.numel()
    small = (2 * torch.randint(0, 8, (n, 128), generator=g) + 1) * 2.0 ** -10  # between subnormal codes
    large = (17 + 2 * torch.randint(0, 8, (n, 128), generator=g)) * torch.ldexp(torch.tensor(1.0), torch.randint(-10, 4, (n, 128), generator=g).float())
    tie = torch.where(torch.rand((n, 128), generator=g) < 0.6, small, large).double()
    x = (tie * s[:, None]).to(dense.T[dtype])
    step = torch.randint(-1, 2, (n, 128), generator=g)
    as_int = x.view(torch.int32 if dtype == "f32" else torch.int16)
    x = (as_int + step.to(as_int.dtype)).clamp(min=0).view(x.dtype)
    x = torch.where(torch.rand((n, 128), generator=g) < 0.5, -x, x)
    x[:, 0] = (448 * s).to(x.dtype)
    codes, scales = (moe.moe_f8_quant_weight if weight else moe.moe_f8_quant_rows)(ctx, x.cuda())
    want, ws = dense.quant_ref(x, weight)
    assert (ws.double().flatten().repeat_interleave(per)[:n] == s).all()
    assert (scales.cpu() == ws).all()
    assert (codes.cpu().float() == want.float()).all()


@pytest.mark.parametrize("m,n,k,dtype", [(4099, 2304, 2064, "bf16"), (4099, 2304, 2064, "f32"), (3000, 5001, 4096, "f16"), (5000, 2560, 4096, "bf16"),
                                         (2560, 8200, 2832, "f32")])
def test_more_tiles_than_pairs_of_sms(ctx, m, n, k, dtype):
    """The rows form with two and more tiles of 256 x 256 a pair of CTAs, full and ragged ones: 17 x 9, 12 x 20, 20 x 10, 10 x 33."""
    check(ctx, m, n, k, dtype)


@pytest.mark.parametrize("m,n,k,dtype", [(5, 100003, 272, "f32"), (16, 50001, 1040, "bf16"), (13, 78000, 528, "f16"), (30, 45001, 400, "f32"),
                                         (32, 90000, 272, "bf16"), (64, 41000, 784, "f16"), (100, 30011, 272, "f32")])
def test_more_tiles_of_weights_than_ctas(ctx, m, n, k, dtype):
    """The weights form of 16, 32 and 64 rows with two and more tiles a CTA (304 of them)."""
    check(ctx, m, n, k, dtype)


@pytest.mark.parametrize("m", [1, 9, 16, 30, 60, 128, 2000])
def test_outputs_past_fp16(ctx, m):
    """Sums past fp16's largest number, 65,504, become infinities of their sign: from 65,520 on, halfway to the next step."""
    n, k = (2000, 4096) if m == 2000 else (300, 512)
    a = torch.ones((m, k), device="cuda").to(dense.F8)
    w = torch.ones((n, k), device="cuda").to(dense.F8)
    sums = torch.tensor([65504.0, 65519.0, 65520.0, 65536.0, 1e6, -65504.0, -65520.0, -1e9, 3.0], device="cuda")
    want = sums[torch.arange(m, device="cuda") % 9]
    sa = torch.zeros((k // 128, m), device="cuda")
    sa[0] = want / 128  # all exact
    sw = torch.ones((-(-n // 128), k // 128), device="cuda")
    out = moe.moe_f8_matmul(ctx, a, sa, w, sw, dtype=torch.float16)
    assert torch.equal(out, want.half()[:, None].expand(m, n))
    assert torch.isinf(out).any() == (m > 2)


def test_norm_of_infinities(ctx):
    """h / sqrt(inf) is NaN where h is infinite and 0 elsewhere: so are the outputs; a block with a NaN is NaN, others of the row
    are zeros; other rows are as without."""
    for n, d in ((6, 512), (6, 2816), (3000, 640), (2, 8208)):
        x = torch.randn((n, d), generator=dense.rng(d), device="cuda")
        r = torch.randn((n, d), generator=dense.rng(d + 1), device="cuda")
        clean = moe.moe_rms_norm(ctx, x, residual=r, f8=True)
        bad = x.clone()
        bad[0, 130] = float("inf")
        bad[1, d - 1] = float("-inf")
        out, total, codes, scales = moe.moe_rms_norm(ctx, bad, residual=r, f8=True)
        assert torch.equal(total, bad + r)
        want = torch.zeros((2, d), device="cuda")
        want[0, 130] = want[1, d - 1] = float("nan")
        assert torch.equal(torch.isnan(out[:2]), torch.isnan(want)) and (out[:2][~torch.isnan(want)] == 0).all()
        blocks = torch.zeros((2, -(-d // 128)), dtype=torch.bool, device="cuda")
        blocks[0, 1] = blocks[1, -1] = True
        assert torch.equal(torch.isnan(scales[:, :2].t()), blocks)
        value = codes[:2].float() * scales[:, :2].t().repeat_interleave(128, 1)[:, :d]
        nan = blocks.repeat_interleave(128, 1)[:, :d]
        assert torch.isnan(value[nan]).all() and (value[~nan] == 0).all()
        for a, b in zip((out, total, codes.float(), scales.t()), (clean[0], clean[1], clean[2].float(), clean[3].t())):
            assert torch.equal(a[2:], b[2:])
