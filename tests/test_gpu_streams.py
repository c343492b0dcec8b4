"""Outputs that a call makes itself, on a stream other than the current one; and first calls under stream capture."""
import os
import subprocess
import sys

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


FIRST_CALLS = """
import torch
import expert_streaming_ffn_gb300 as moe
ctx = moe.moe_ctx_create(0)
cache = moe.moe_kv_new_cache(4, 2, 64, 16)
k = torch.randn((40, 2, 64), device="cuda").bfloat16()
v = torch.randn_like(k)
slots = torch.arange(40, dtype=torch.int32, device="cuda")
q, out = torch.randn((1, 4, 64), device="cuda").bfloat16(), torch.empty((1, 4, 64), dtype=torch.bfloat16, device="cuda")
table, ln = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([40], dtype=torch.int32, device="cuda")
rows = [torch.empty_like(k), torch.empty_like(v)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.moe_kv_append(ctx, cache, k, v, slots)
    moe.moe_kv_read(ctx, cache, slots, k=rows[0], v=rows[1])
    try:
        moe.moe_kv_attend(ctx, cache, q, table, ln, out=out)
        raise SystemExit("the first attention call was captured")
    except moe.MoeError as e:
        assert e.status == moe.MOE_ESTATE, e
graph.replay()
got = moe.moe_kv_read(ctx, cache, slots)
torch.cuda.synchronize()
assert torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1])
assert (rows[0] - k).abs().max() < 0.5 and (rows[1] - v).abs().max() < 0.5  # steps of a fifteenth of a span of 6 or so
want = moe.moe_kv_attend(ctx, cache, q, table, ln)
with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
    moe.moe_kv_attend(ctx, cache, q, table, ln, out=out)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, want)
moe.moe_ctx_destroy(ctx)
print("first calls ok")
"""


def test_first_calls_of_a_context_under_capture():
    """Append and read allocate nothing, so they can be a context's first calls and captured ones; the first attention call
    says that it cannot, and the capture goes on. In a process of its own, where no kernel has run before."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls ok" in r.stdout, r.stdout + r.stderr


def test_a_context_destroyed_with_calls_pending():
    """Destroying waits for them: a call that cuts segments uses the context's workspace, one with a bad slot its error words."""
    moe.load()
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 30000
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    k = torch.randn((n, 2, 128), generator=g, device="cuda").bfloat16()
    q = torch.randn((1, 8, 128), generator=g, device="cuda").bfloat16()
    table, ln = torch.arange(-(-n // 64), dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(3):
        ctx = moe.moe_ctx_create(0)
        cache = moe.moe_kv_new_cache(table.shape[1], 2, 128, 64)
        moe.moe_kv_append(ctx, cache, k, k, slots)
        outs.append(moe.moe_kv_attend(ctx, cache, q, table, ln))
        moe.moe_kv_append(ctx, cache, k[:2], k[:2], slots[:2] + 2 ** 30)  # past the end
        moe.moe_ctx_destroy(ctx)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and outs[0].abs().max() > 0
