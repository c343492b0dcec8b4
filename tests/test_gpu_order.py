"""moe_forward straight behind a call of this library that writes its rows x, on the same stream and with nothing between: it
reads these rows and not the ones before, whichever call it is."""
import pytest

torch = pytest.importorskip("torch")
import expert_streaming_ffn_gb300 as moe  # noqa: E402
import synth  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

S = synth.SHAPES_TINY
HEADS, DIM, PAGE = 4, 128, 64  # rows of HEADS * DIM = d_model
ROUNDS = 24


@pytest.fixture(scope="module")
def ctx():
    c = moe.moe_ctx_create(0)
    yield c
    moe.moe_ctx_destroy(c)


@pytest.fixture(scope="module")
def layer(ctx):
    h = moe.moe_layer_create(ctx, S, 4, moe.LFU)
    moe.moe_layer_set_weights(h, synth.layer_weights(S, 0))
    moe.moe_layer_set_deterministic(h, True)
    yield h
    moe.moe_layer_destroy(h)


def check(layer, x, write):
    """write(i) fills x with the i-th rows."""
    want, got = [], []
    for i in range(ROUNDS):
        write(i)
        torch.cuda.synchronize()
        want.append(moe.moe_forward(layer, x).clone())
        torch.cuda.synchronize()
    noise = torch.empty((1 << 22,), device="cuda")
    for i in range(ROUNDS):
        noise.normal_()  # the device is behind the host, so that the calls queue up
        write(i)
        got.append(moe.moe_forward(layer, x))
    torch.cuda.synchronize()
    assert len({w.sum().item() for w in want}) == ROUNDS
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def filled(ctx, tokens, sequences, g):
    """A cache of `sequences` sequences of `tokens` tokens, and their page table."""
    per = -(-tokens // PAGE)
    cache = moe.moe_kv_new_cache(sequences * per, HEADS, DIM, PAGE)
    kv = torch.randn((2, sequences * per * PAGE, HEADS, DIM), generator=g, device="cuda").bfloat16()
    moe.moe_kv_append(ctx, cache, kv[0], kv[1], torch.arange(kv.shape[1], dtype=torch.int32, device="cuda"))
    return cache, torch.arange(sequences * per, dtype=torch.int32, device="cuda").view(sequences, per)


@pytest.mark.parametrize("sequences,new,keys", [(1, 1, 200), (1, 1, 60000), (3, 1, 20000), (2, 50, 4000), (1, 100, 30000)])
def test_attention(ctx, layer, sequences, new, keys):
    """Decode steps of one and several sequences, whole and cut between CTAs, and prompts."""
    g = torch.Generator(device="cuda").manual_seed(keys)
    cache, table = filled(ctx, keys, sequences, g)
    length = torch.full((sequences,), keys, dtype=torch.int32, device="cuda")
    q = torch.randn((ROUNDS, sequences * new, HEADS, DIM), generator=g, device="cuda").mul_(3).bfloat16()
    x = torch.zeros((sequences * new, S.d_model), dtype=torch.bfloat16, device="cuda")
    out = x.view(-1, HEADS, DIM)
    check(layer, x, lambda i: moe.moe_kv_attend(ctx, cache, q[i], table, length, out=out))


@pytest.mark.parametrize("n", [1, 3, 100])
@pytest.mark.parametrize("which", ["k", "v"])
def test_rows_of_the_cache(ctx, layer, n, which):
    g = torch.Generator(device="cuda").manual_seed(n)
    cache, _ = filled(ctx, 4096, 1, g)
    extra = 40000  # rows behind x's that the call reads too, so that it takes its time
    slots = torch.randint(0, 4096, (ROUNDS, n + extra), generator=g, device="cuda").int()
    big = torch.zeros((n + extra, S.d_model), dtype=torch.bfloat16, device="cuda")
    other = torch.empty_like(big).view(-1, HEADS, DIM)
    rows = big.view(-1, HEADS, DIM)
    at = slice(extra, None)  # the last rows written
    check(layer, big[at], lambda i: moe.moe_kv_read(ctx, cache, slots[i], **({"k": rows, "v": other} if which == "k" else {"k": other, "v": rows})))


@pytest.mark.parametrize("tokens", [1, 3, 100])
def test_rows_behind_a_call_that_reads_them(ctx, layer, tokens):
    """The norm writes x, the quantiser reads it, then the experts do: the kernel between has been waited for, and so has the norm."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rows = torch.randn((ROUNDS, tokens, S.d_model), generator=g, device="cuda")
    x = torch.zeros((tokens, S.d_model), dtype=torch.bfloat16, device="cuda")

    def write(i):
        moe.moe_rms_norm(ctx, rows[i], out=x)
        moe.moe_f8_quant_rows(ctx, x)

    check(layer, x, write)
