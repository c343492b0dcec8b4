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
