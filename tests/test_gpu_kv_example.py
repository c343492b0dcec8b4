"""The decoder-layer example: cache, attention and experts together, prompt then
decode steps. Its attention is checked against fp32 attention over the cache's own values: the
bound is that of test_gpu_kv.py for these sizes (rows of unit variance: dot <= 40,
values up to 5, bf16 outputs)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

U = 2.0 ** -11


@pytest.mark.parametrize("argv", [["--prompt", "300", "--steps", "5"], ["--prompt", "1", "--steps", "3", "--sequences", "3"]])
def test_decoder_layer(argv):
    from examples import decode_layer

    worst, x = decode_layer.main(argv)
    delta = 3 * U * 40 / 8
    assert worst <= (2 * delta + 3 * U + 2.0 ** -8) * 5
    assert torch.isfinite(x).all()
