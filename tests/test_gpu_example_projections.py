"""The decoder-layer example's projections, in 8 bits and in bf16. A product of K = 512 in fp32, in any order and whichever way
steps round, is off by (512 + 8) 2^-23 of the sum of its magnitudes, and its output by half a step of bf16, 2^-8 of itself."""
import pytest

torch = pytest.importorskip("torch")
import expert_streaming_ffn_gb300 as moe  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BOUND = 520 * 2.0 ** -23 + 2.0 ** -8


@pytest.mark.parametrize("projections", ["f8", "bf16"])
@pytest.mark.parametrize("sequences,new", [(1, 1), (2, 150)])
def test_projections(projections, sequences, new):
    from examples import decode_layer

    ctx = moe.moe_ctx_create(0)
    try:
        made = {kind: decode_layer.Attention(ctx, 512, sequences, 200, seed=3, projections=kind) for kind in ("f8", "bf16")}
        x = torch.randn((sequences * new, 512), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        out, _, codes, scales = moe.moe_rms_norm(ctx, x, dtype=torch.bfloat16, f8=True)
        rows = {"f8": (codes, scales), "bf16": out}
        attention = made[projections]
        y = attention(rows[projections], check=True)
        assert y.shape == (sequences * new, 512) and y.dtype == torch.float32
        assert attention.w_in.worst <= BOUND and attention.w_out.worst <= BOUND and attention.worst < 0.1
        # the two kinds take the same rows and weights: apart by what 8 bits a side round, 2^-4 of each value at most
        q = {kind: made[kind].w_in(rows[kind], torch.float32) for kind in made}
        assert (q["f8"] - q["bf16"]).norm() <= 2 * 2.0 ** -4 * q["bf16"].norm()
    finally:
        moe.moe_ctx_destroy(ctx)


@pytest.mark.parametrize("projections", ["f8", "bf16"])
def test_example_runs(projections):
    from examples import decode_layer

    worst, x = decode_layer.main(["--prompt", "70", "--steps", "3", "--projections", projections])
    assert torch.isfinite(x).all() and worst < 0.1
