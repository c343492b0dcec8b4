"""Cache calls, layer calls and readings of the kernel times of one context from several host threads."""
import ctypes
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import expert_streaming_ffn_gb300 as moe  # noqa: E402
import synth  # noqa: E402

ROUNDS = 300


def together(*bodies):
    """Runs them in a thread each; the first error of any is raised here."""
    errors = []

    def guarded(f):
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(f,)) for f in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


def attention(ctx, seed, n):
    """A cache of its own, filled: the attention call on it (of an output and a stream), its result, the cache, its slots and
    the rows in them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D, P = 2, 128, 32
    cache = moe.moe_kv_new_cache(-(-n // P), H, D, P)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n, H, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    moe.moe_kv_append(ctx, cache, k, v, slots)
    q = torch.randn((1, 8, D), generator=g, device="cuda").bfloat16()
    table, ln = torch.arange(-(-n // P), dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")

    def call(out, stream):
        moe.moe_kv_attend(ctx, cache, q, table, ln, out=out, stream=stream)

    return call, moe.moe_kv_attend(ctx, cache, q, table, ln), cache, slots, k, v


def cache_calls(ctx, seed, n, stream):
    """Calls on a cache: append, read and attention, whose results are compared with the first ones'."""
    call, want, cache, slots, k, v = attention(ctx, seed, n)
    rows = moe.moe_kv_read(ctx, cache, slots)
    outs = [torch.zeros_like(want) for _ in range(8)]
    back = [torch.empty_like(k), torch.empty_like(v)]
    torch.cuda.synchronize()

    def body():
        for i in range(ROUNDS):
            moe.moe_kv_append(ctx, cache, k, v, slots, stream=stream)
            call(outs[i % 8], stream)
            if i % 8 == 7:
                moe.moe_kv_read(ctx, cache, slots, k=back[0], v=back[1], stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])

    return body


def test_cache_and_layer_calls_and_kernel_times():
    moe.load()
    ctx = moe.moe_ctx_create(0)
    s = synth.SHAPES_TINY
    layer = moe.moe_layer_create(ctx, s, 4, moe.LFU)
    moe.moe_layer_set_weights(layer, synth.layer_weights(s, 0))
    moe.moe_layer_set_deterministic(layer)
    x = torch.from_numpy(synth.tokens(s, 0, 0, 1, False).view(np.int16)).view(torch.bfloat16).cuda()
    y = moe.moe_forward(layer, x)
    again = torch.empty_like(y)
    side = [torch.cuda.Stream() for _ in range(3)]
    a, b = cache_calls(ctx, 1, 300, side[0]), cache_calls(ctx, 2, 5000, side[1])  # the second cuts segments
    moe.moe_ctx_reset_kernel_times(ctx)
    moe.moe_ctx_set_profiling(ctx, True)
    n0 = moe.moe_ctx_launches(ctx)
    done = threading.Event()

    def layers():
        for _ in range(ROUNDS):
            moe.moe_forward(layer, x, y=again, stream=side[2])
        side[2].synchronize()
        assert torch.equal(again, y)

    def times():
        while not done.is_set():
            moe.moe_ctx_kernel_times(ctx)
            moe.moe_ctx_launches(ctx)
            moe.moe_kv_check(ctx)

    def others():
        try:
            together(a, b, layers)
        finally:
            done.set()

    together(others, times)
    torch.cuda.synchronize()
    t = moe.moe_ctx_kernel_times(ctx)
    moe.moe_ctx_set_profiling(ctx, False)
    assert t["kv_append"][0] == t["kv_attend"][0] == 2 * ROUNDS and t["kv_read"][0] == 2 * (ROUNDS // 8)
    assert t["router"][0] == ROUNDS
    # every launch counted once; attention that cuts segments has a second, joining one, and times both together
    timed = sum(v[0] for v in t.values())
    assert moe.moe_ctx_launches(ctx) - n0 == timed + ROUNDS
    moe.moe_layer_destroy(layer)
    moe.moe_ctx_destroy(ctx)


def test_the_per_thread_default_stream_is_a_stream_of_each_thread():
    """Its handle (2) is the same in every thread, the streams behind it are not: calls that share the context's workspace
    are ordered after one another all the same."""
    moe.load()
    ctx = moe.moe_ctx_create(0)
    together(*(cache_calls(ctx, seed, n, 2) for seed, n in ((1, 5000), (2, 7000), (3, 20000))))
    moe.moe_ctx_destroy(ctx)


def test_streams_that_are_made_anew():
    """A new stream may get the handle of one that was destroyed with work pending on it."""
    moe.load()
    ctx = moe.moe_ctx_create(0)
    rt = torch.cuda.cudart()
    calls = [attention(ctx, i, n)[:2] for i, n in enumerate((20000, 31000))]
    outs = [torch.zeros_like(calls[i % 2][1]) for i in range(40)]
    torch.cuda.synchronize()
    handles = []
    for i, out in enumerate(outs):
        h = ctypes.c_void_p()
        rt.cudaStreamCreate(ctypes.addressof(h))
        handles.append(h.value)
        calls[i % 2][0](out, h.value)
        rt.cudaStreamDestroy(h.value)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, calls[i % 2][1]), (i, len(set(handles)))
    moe.moe_ctx_destroy(ctx)
