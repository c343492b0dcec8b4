"""Outputs that a call makes itself, on a stream other than the current one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402
import synth  # noqa: E402


@pytest.fixture(scope="module")
def calls():
    """Calls by name, each of a stream, with their inputs; and how many outputs each makes."""
    moe.load()
    ctx = moe.moe_ctx_create(0)
    s = synth.SHAPES_TINY
    layer = moe.moe_layer_create(ctx, s, 4, moe.LFU)
    moe.moe_layer_set_weights(layer, synth.layer_weights(s, 0))
    moe.moe_layer_set_deterministic(layer)
    x = torch.from_numpy(synth.tokens(s, 0, 0, 4, False).view(np.int16)).view(torch.bfloat16).cuda()
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = moe.moe_kv_new_cache(8, 2, 128, 16)
    slots = torch.arange(100, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((100, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    moe.moe_kv_append(ctx, cache, k, v, slots)
    q = torch.randn((3, 4, 128), generator=g, device="cuda").bfloat16()
    table, ln = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.tensor([100], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    yield {
        "attend": lambda st: (moe.moe_kv_attend(ctx, cache, q, table, ln, stream=st),),
        "read": lambda st: moe.moe_kv_read(ctx, cache, slots, stream=st),
        "read v": lambda st: moe.moe_kv_read(ctx, cache, slots, k=k, stream=st)[1:],
        "route": lambda st: moe.moe_route(layer, x, s.top_k, stream=st),
        "forward": lambda st: (moe.moe_forward(layer, x, stream=st),),
        "forward_prompt": lambda st: (moe.moe_forward_prompt(layer, x, stream=st),),
    }
    torch.cuda.synchronize()
    moe.moe_layer_destroy(layer)
    moe.moe_ctx_destroy(ctx)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["attend", "read", "read v", "route", "forward", "forward_prompt"])
def test_new_outputs_are_of_the_calls_stream(calls, name, raw):
    """Memory that a kernel pending on the current stream still writes is not handed to a call on another stream, although
    torch counts it as free for the current one."""
    want = [o.clone() for o in calls[name](None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pending = [torch.empty_like(o) for o in want for _ in range(2)]
    taken = {p.data_ptr() for p in pending}
    torch.cuda._sleep(40_000_000)  # cycles: about 20 ms
    for p in pending:
        p.fill_(3)
    del p, pending
    got = calls[name](side.cuda_stream if raw else side)
    assert not taken & {o.data_ptr() for o in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_default_streams(calls):
    """0 and 1 are the legacy default stream; the per-thread one takes outputs that are given, and no others."""
    want = calls["attend"](None)[0]
    torch.cuda.synchronize()
    for handle in (0, 1):
        assert torch.equal(calls["attend"](handle)[0], want)
    for name in ("attend", "read", "route"):
        with pytest.raises(ValueError, match="per-thread"):
            calls[name](2)
