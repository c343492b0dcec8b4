"""Cases of the operators between attention and the experts: root-mean-square norm of rows (with the residual's addition, and an
output in 8 bits for the products that follow), quantisation to 8 bits, and the matrix product of 8-bit rows and weights.

8 bits are e4m3 codes with an fp32 scale for each block: of rows, 128 elements of one row, scales held [block][row]; of weights
[n][k], 128 x 128 elements, scales held [n block][k block]. A value is scale * code; the scale is the block's largest magnitude
(at least 448 * 2^-126) over 448, the code the nearest to value / scale, ties to even. Blocks at the ends may be smaller.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0
LEAST = TOP * 2.0 ** -126
EPS = 1e-6


def listed():
    return [
        # decode: one token's expert output (fp32) into the residual, normed for the router (bf16) and for the next projection (8 bits)
        dict(name="norm_one_token", op="norm", tokens=1, heads=1, dim=2816, x="f32", residual="bf16", weight="bf16", out="bf16", f8=True, packed=False),
        # a decode batch behind attention: the output projection's rows into the residual
        dict(name="norm_batch", op="norm", tokens=77, heads=1, dim=2048, x="f16", residual="f32", weight="f32", out="f16", f8=False, packed=False),
        # query heads of a prompt normed one by one, as a part of the fused projection's output
        dict(name="norm_heads", op="norm", tokens=4099, heads=32, dim=128, x="bf16", residual="none", weight="bf16", out="bf16", f8=False, packed=True),
        # a long prompt's expert outputs into the residual, normed into 8 bits for the next layer's projections
        dict(name="norm_prompt", op="norm", tokens=32768, heads=1, dim=2816, x="f32", residual="bf16", weight="bf16", out="none", f8=True, packed=False),
        # a decode batch's attention output, before the output projection
        dict(name="quant_batch", op="quant", tokens=64, dim=4096, x="bf16", weight=False),
        # a prompt's attention output
        dict(name="quant_prompt", op="quant", tokens=16385, dim=4096, x="f16", weight=False),
        # a projection's weights, laid out when a model is loaded; its sides no multiples of 128
        dict(name="quant_weight", op="quant", tokens=10000, dim=2864, x="f32", weight=True),
        # decode of one token: the fused query, key and value projection
        dict(name="matmul_one_token", op="matmul", tokens=1, n=6144, k=2816, out="bf16"),
        # the logits of a few sequences over a large vocabulary of odd size, in fp32
        dict(name="matmul_logits", op="matmul", tokens=5, n=100003, k=2048, out="f32"),
        # a decode batch through the output projection
        dict(name="matmul_batch", op="matmul", tokens=77, n=2816, k=4096, out="f16"),
        # a 128-token prefill chunk and a little more, through the fused projection
        dict(name="matmul_chunk", op="matmul", tokens=143, n=6144, k=2816, out="bf16"),
        # a long prompt through a wide dense layer
        dict(name="matmul_prompt", op="matmul", tokens=8192, n=8192, k=8192, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "matmul", "matmul", "matmul"])
    if op == "norm":
        heads = rng.choice([1, 1, 1, rng.randint(2, 40)])
        dim = rng.choice([64, 128, 256]) if heads > 1 else 16 * _log(rng, 4, 1024)
        return dict(op="norm", tokens=_log(rng, 1, min(32768, 32768 * 2816 // (heads * dim))), heads=heads, dim=dim, x=rng.choice(["bf16", "f16", "f32"]),
                    residual=rng.choice(["none", "bf16", "f16", "f32"]), weight=rng.choice(["none", "bf16", "f32"]),
                    **rng.choice([dict(out="bf16", f8=False), dict(out="f16", f8=False), dict(out="f32", f8=False)] if heads > 1 else
                                 [dict(out="bf16", f8=False), dict(out="f16", f8=True), dict(out="bf16", f8=True), dict(out="none", f8=True)]),
                    packed=rng.random() < 0.3)
    if op == "quant":
        dim = 16 * _log(rng, 4, 1024)
        return dict(op="quant", tokens=_log(rng, 1, min(32768, 16384 * 4096 // dim)), dim=dim, x=rng.choice(["bf16", "f16", "f32"]), weight=rng.random() < 0.3)
    while True:
        m, n, k = _log(rng, 1, 8192), _log(rng, 32, 100003), 16 * _log(rng, 8, 1024)
        if rng.random() < 0.7:
            n = max(1, n // 64) * 64
        if m * n * k <= 8192 ** 3 and n * k <= 100003 * 2048 and m * n <= 8192 * 8192 and m * k <= 8192 * 8192:
            return dict(op="matmul", tokens=m, n=n, k=k, out=rng.choice(["bf16", "bf16", "f16", "f32"]))


def _size(t):
    return {"none": 0, "bf16": 2, "f16": 2, "f32": 4}[t]


def _blocks(n):
    return -(-n // 128)


def work(case):
    n = case["tokens"]
    if case["op"] == "norm":
        rows, d = n * case["heads"], case["dim"]
        codes = n * (d + 4 * _blocks(d)) if case["f8"] else 0
        return {"bytes": rows * d * (_size(case["x"]) + 2 * _size(case["residual"]) + _size(case["out"])) + d * _size(case["weight"]) + codes,
                "flops": rows * d * (5.0 + (3.0 if case["f8"] else 0.0))}
    if case["op"] == "quant":
        d = case["dim"]
        return {"bytes": n * d * (_size(case["x"]) + 1) + 4 * (_blocks(n) if case["weight"] else n) * _blocks(d), "flops": 3.0 * n * d}
    w, k = case["n"], case["k"]
    return {"bytes": n * k + w * k + 4 * _blocks(k) * (n + _blocks(w)) + n * w * _size(case["out"]), "flops": 2.0 * n * w * k}


# ---- the plain forms -----------------------------------------------------------


def _codes(x, largest):
    """fp32 values and their block's largest magnitude, of the same number of dimensions, to codes and scales."""
    scale = largest.clamp(min=LEAST) / TOP
    return (x / scale).clamp(-TOP, TOP).to(E4M3), scale


def _quant_rows(x):
    """Rows [n][d] in fp32 to codes [n][d] and scales [blocks][n]."""
    n, d = x.shape
    b = torch.nn.functional.pad(x, (0, -d % 128)).view(n, -1, 128)
    codes, scale = _codes(b, b.abs().amax(-1, keepdim=True))
    return codes.view(n, -1)[:, :d].contiguous(), scale[..., 0].t().contiguous()


def _quant_weight(w):
    """Weights [n][k] in fp32 to codes [n][k] and scales [n blocks][k blocks]."""
    n, k = w.shape
    b = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128))
    b = b.view(_blocks(n), 128, _blocks(k), 128)
    codes, scale = _codes(b, b.abs().amax((1, 3), keepdim=True))
    return codes.view(128 * _blocks(n), -1)[:n, :k].contiguous(), scale[:, 0, :, 0].contiguous()


def _norm(st):
    case, x = st["case"], st["x"]
    h = x.float()
    got = {}
    if case["residual"] != "none":
        h = h + st["residual"].float()
        got["sum"] = h.to(st["residual"].dtype)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    if case["weight"] != "none":
        y = y * st["weight"].float()
    if case["out"] != "none":
        got["out"] = y.to(DTYPES[case["out"]])
    if case["f8"]:
        got["codes"], got["scales"] = _quant_rows(y[:, 0])
    return got


def _quant(st):
    return dict(zip(("codes", "scales"), (_quant_weight if st["case"]["weight"] else _quant_rows)(st["x"].float())))


def _wide(scale, n):
    return scale.repeat_interleave(128, 0)[:n]


def _matmul(st):
    a = st["a"].float() * _wide(st["a_scales"], st["a"].shape[1]).t()
    w = st["w"].float() * _wide(_wide(st["w_scales"], st["w"].shape[0]).t(), st["w"].shape[1]).t()
    return torch.matmul(a, w.t()).to(DTYPES[st["case"]["out"]])


# ---- inputs ----------------------------------------------------------------------


def _rows(n, d, g):
    """Activations: a few channels much stronger than the rest, as residual streams have them."""
    chan = torch.exp(0.5 * torch.randn((d,), generator=g, device="cuda"))
    chan[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 12.0
    return torch.randn((n, d), generator=g, device="cuda") * chan


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = case["tokens"]
    if case["op"] == "norm":
        h, d = case["heads"], case["dim"]
        extra = h + 3 if case["packed"] else h  # packed: the rows are a part of wider ones
        x = _rows(n, extra * d, g).to(DTYPES[case["x"]]).view(n, extra, d)[:, :h]
        st = dict(case=case, x=x)
        if case["residual"] != "none":
            st["residual"] = (3.0 * _rows(n, h * d, g)).to(DTYPES[case["residual"]]).view(n, h, d)
        if case["weight"] != "none":
            st["weight"] = (1.0 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(DTYPES[case["weight"]])
        return st
    if case["op"] == "quant":
        d = case["dim"]
        x = torch.randn((n, d), generator=g, device="cuda") * d ** -0.5 if case["weight"] else _rows(n, d, g)
        return dict(case=case, x=x.to(DTYPES[case["x"]]))
    a, a_scales = _quant_rows(_rows(n, case["k"], g))
    w, w_scales = _quant_weight(torch.randn((case["n"], case["k"]), generator=g, device="cuda") * case["k"] ** -0.5)
    return dict(case=case, a=a, a_scales=a_scales, w=w, w_scales=w_scales)


# ---- one pass ----------------------------------------------------------------------

_lib = {}


def _ours():
    """The framework's context, made once."""
    if not _lib:
        import expert_streaming_ffn_gb300 as moe

        _lib["moe"], _lib["ctx"] = moe, moe.moe_ctx_create(0)
    return _lib["moe"], _lib["ctx"]


def run(state):
    case = state["case"]
    if not own:
        return {"norm": _norm, "quant": _quant, "matmul": _matmul}[case["op"]](state)
    moe, ctx = _ours()
    if case["op"] == "norm":
        out, total, codes, scales = moe.moe_rms_norm(ctx, state["x"], state.get("weight"), EPS, residual=state.get("residual"),
                                                     dtype=DTYPES.get(case["out"]), f8=case["f8"])
        got = dict(sum=total, out=out, codes=codes, scales=scales)
        return {name: t for name, t in got.items() if t is not None}
    if case["op"] == "quant":
        codes, scales = (moe.moe_f8_quant_weight if case["weight"] else moe.moe_f8_quant_rows)(ctx, state["x"])
        return dict(codes=codes, scales=scales)
    return moe.moe_f8_matmul(ctx, state["a"], state["a_scales"], state["w"], state["w_scales"], dtype=DTYPES[case["out"]])


# ---- in 64 bits ----------------------------------------------------------------------


def _exact_blocks(x, rows):
    """x [n][d] fp64 in blocks of `rows` by 128: the quotients that the codes round, and the scales [row block][column block]."""
    n, d = x.shape
    q, s = torch.empty_like(x), x.new_empty((-(-n // rows), _blocks(d)))
    for j in range(_blocks(d)):
        part = x[:, 128 * j:128 * j + 128]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.stack([t.amax() for t in top.split(rows)])
        s[:, j] = torch.maximum(top, torch.full_like(top, LEAST)) / TOP
        q[:, 128 * j:128 * j + 128] = part / s[:, j].repeat_interleave(rows)[:n, None]
    return q, s


def exact(case, seed):
    """Codes as the quotients that they round."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        got = {}
        x = st["x"].double()
        if "residual" in st:
            x = x + st["residual"].double()
            got["sum"] = x
        y = x / (torch.einsum("nhd,nhd->nh", x, x) / case["dim"] + EPS).sqrt()[..., None]
        if "weight" in st:
            y = y * st["weight"].double()
        if case["out"] != "none":
            got["out"] = y
        if case["f8"]:
            got["codes"], scales = _exact_blocks(y[:, 0], 1)
            got["scales"] = scales.t()
        return got
    if case["op"] == "quant":
        codes, scales = _exact_blocks(st["x"].double(), 128 if case["weight"] else 1)
        return dict(codes=codes, scales=scales if case["weight"] else scales.t())
    n = case["n"]
    y = torch.zeros((case["tokens"], n), dtype=torch.float64, device="cuda")
    for j in range(_blocks(case["k"])):
        cols = slice(128 * j, 128 * j + 128)
        part = st["a"][:, cols].double() @ st["w"][:, cols].double().t()
        part *= st["a_scales"][j].double()[:, None]
        part *= st["w_scales"][:, j].double().repeat_interleave(128)[:n]
        y += part
    return y
