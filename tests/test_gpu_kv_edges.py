"""Attention over the 4-bit cache at the edges of its arguments and of what its records hold."""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402

HINTS = [1, 4096]  # max_q, which chooses the kernel: decode, prompt


@pytest.fixture(scope="module")
def ctx():
    moe.load()
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


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
