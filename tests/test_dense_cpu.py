"""Refusals of the norm, quantisation and matrix-product calls: arguments are checked before the context or a device is
touched, so a block of zeros serves as the context here, and a call that is not refused ends in MOE_ECUDA, no device."""
import ctypes
import struct

import pytest

import expert_streaming_ffn_gb300 as moe

CTX = ctypes.create_string_buffer(1 << 16)
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def norm_args(**kw):
    a = moe.moe_norm_args(x=P, x_token_stride=256, x_head_stride=0, out=P, out_token_stride=256, out_head_stride=0, n_tokens=2,
                          n_heads=1, dim=256, eps=1e-6, x_dtype=moe.MOE_BF16, out_dtype=moe.MOE_BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def matmul_args(**kw):
    a = moe.moe_f8_matmul_args(a=P, a_stride=256, a_scales=P, a_scale_stride=4, w=P, w_stride=256, w_scales=P, w_scale_stride=2,
                               out=P, out_stride=100, m=4, n=100, k=256, out_dtype=moe.MOE_BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_structures_match_what_is_packed():
    assert struct.calcsize("@PqqPqqPPqqPqqPqPqiiif4i") == ctypes.sizeof(moe.moe_norm_args)
    assert struct.calcsize("@PqPqPqPqPqiiii") == ctypes.sizeof(moe.moe_f8_matmul_args)


NORM = [dict(x=None), dict(x=P + 8), dict(x_token_stride=252), dict(x_head_stride=4, n_heads=2), dict(dim=250), dict(dim=0),
        dict(dim=8), dict(dim=32784), dict(n_tokens=-1), dict(n_heads=0), dict(n_tokens=1 << 30, n_heads=2), dict(eps=-1.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(out=None), dict(out=P + 2), dict(out_token_stride=257), dict(x_dtype=3),
        dict(x_dtype=-1), dict(out_dtype=7), dict(weight=P, weight_dtype=5), dict(weight=P + 4), dict(sum=P),
        dict(residual=P, residual_dtype=9), dict(residual=P + 2, residual_dtype=1), dict(residual=P, residual_dtype=0, residual_token_stride=2),
        dict(residual=P, sum=P + 4), dict(codes=P), dict(codes=P, scales=P, code_stride=256, scale_stride=2, n_heads=2),
        dict(codes=P, scales=P, code_stride=250, scale_stride=2), dict(codes=P, scales=P, code_stride=240, scale_stride=2),
        dict(codes=P + 8, scales=P, code_stride=256, scale_stride=2), dict(codes=P, scales=P + 2, code_stride=256, scale_stride=2),
        dict(codes=P, scales=P, code_stride=256, scale_stride=1)]
MATMUL = [dict(a=None), dict(w=None), dict(out=None), dict(a_scales=None), dict(w_scales=None), dict(m=-1), dict(n=0), dict(k=0),
          dict(k=250), dict(a=P + 8), dict(w=P + 1), dict(a_stride=264), dict(w_stride=264), dict(a_stride=240), dict(w_stride=0),
          dict(a_stride=1 << 41), dict(a_scales=P + 1), dict(w_scales=P + 2), dict(out=P + 1), dict(out=P + 2, out_dtype=0),
          dict(out_stride=99), dict(out_dtype=3), dict(a_scale_stride=3), dict(w_scale_stride=1, n=200, out_stride=200), dict(w_scale_stride=-2, n=200, out_stride=200), dict(m=(1 << 31) - 1, n=(1 << 31) - 1, out_stride=1 << 31), dict(k=(1 << 30) + 16)]


@pytest.mark.parametrize("bad", NORM)
def test_norm_refuses(lib, bad):
    assert lib.moe_rms_norm(CTX, ctypes.byref(norm_args(**bad)), None) == moe.MOE_EINVAL
    assert moe.moe_last_error().startswith("moe_rms_norm")


@pytest.mark.parametrize("bad", MATMUL)
def test_matmul_refuses(lib, bad):
    assert lib.moe_f8_matmul(CTX, ctypes.byref(matmul_args(**bad)), None) == moe.MOE_EINVAL
    assert moe.moe_last_error().startswith("moe_f8_matmul")


@pytest.mark.parametrize("fn", ["moe_f8_quant_rows", "moe_f8_quant_weight"])
def test_quant_refuses(lib, fn):
    def call(x=P, stride=512, dtype=1, n=300, k=512, codes=P, code_stride=512, scales=P, scale_stride=300, ctx=CTX):
        return getattr(lib, fn)(ctx, x, stride, dtype, n, k, codes, code_stride, scales, scale_stride, None)

    for bad in (dict(ctx=None), dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=3), dict(n=-1), dict(k=0), dict(k=520 + 4),
                dict(x=P + 8), dict(stride=508), dict(codes=P + 8), dict(code_stride=520), dict(code_stride=496), dict(scales=P + 2),
                dict(scale_stride=3), dict(n=(1 << 31) - 1, k=1 << 20, stride=1 << 20, code_stride=1 << 20, scale_stride=1 << 31)):
        assert call(**bad) == moe.MOE_EINVAL, bad
        assert moe.moe_last_error().startswith(fn)
    assert call(n=0) == moe.MOE_OK


def test_null_context_and_empty_calls(lib):
    assert lib.moe_rms_norm(None, ctypes.byref(norm_args()), None) == moe.MOE_EINVAL
    assert lib.moe_rms_norm(CTX, None, None) == moe.MOE_EINVAL
    assert lib.moe_f8_matmul(None, ctypes.byref(matmul_args()), None) == moe.MOE_EINVAL
    assert lib.moe_f8_matmul(CTX, None, None) == moe.MOE_EINVAL
    assert lib.moe_rms_norm(CTX, ctypes.byref(norm_args(n_tokens=0, x=None)), None) == moe.MOE_OK
    assert lib.moe_f8_matmul(CTX, ctypes.byref(matmul_args(m=0, a=None)), None) == moe.MOE_OK


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 256))
    c, s = x.to(torch.float8_e4m3fn), torch.ones((2, 2))
    for call in (lambda: moe.moe_rms_norm(0, x), lambda: moe.moe_f8_quant_rows(0, x), lambda: moe.moe_f8_quant_weight(0, x),
                 lambda: moe.moe_f8_matmul(0, c, s, c, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


TOP = (1 << 31) - 1024  # the most rows


def taken(call):
    """A call that is not refused, which must not find a device: its addresses are none."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the call would be launched")
    assert call() == moe.MOE_ECUDA


@pytest.mark.parametrize("fn", ["moe_f8_quant_rows", "moe_f8_quant_weight"])
@pytest.mark.parametrize("n,k", [(1, (1 << 31) - 16), (1, (1 << 31) - 112), (1, (1 << 31) - 128), (1, (1 << 30) + 16), ((1 << 31) - 1, 16),
                                 ((1 << 31) - 128, 16), (TOP + 1, 16)])
def test_quant_refuses_sizes_that_32_bits_do_not_hold_rounded_up(lib, fn, n, k):
    """Rounded up to blocks and tiles, and a part of a tile further, sizes stay below 2^31."""
    assert getattr(lib, fn)(CTX, P, k, moe.MOE_F16, n, k, P, k, P, n, None) == moe.MOE_EINVAL
    assert "at most" in moe.moe_last_error()


@pytest.mark.parametrize("fn", ["moe_f8_quant_rows", "moe_f8_quant_weight"])
@pytest.mark.parametrize("n,k", [(1, 1 << 30), (3, 1 << 30)])
def test_quant_takes_the_largest_rows(lib, fn, n, k):
    taken(lambda: getattr(lib, fn)(CTX, P, k, moe.MOE_F16, n, k, P, k, P, k, None))


@pytest.mark.parametrize("size", [dict(m=(1 << 31) - 1), dict(m=(1 << 31) - 255), dict(m=TOP + 1), dict(n=(1 << 31) - 1),
                                  dict(n=(1 << 31) - 15), dict(n=TOP + 1)])
def test_matmul_refuses_sizes_that_32_bits_do_not_hold_rounded_up(lib, size):
    big = 1 << 31
    bad = dict(dict(m=1, n=1, k=16, a_stride=16, w_stride=16, a_scale_stride=big, w_scale_stride=big, out_stride=big), **size)
    assert lib.moe_f8_matmul(CTX, ctypes.byref(matmul_args(**bad)), None) == moe.MOE_EINVAL
    assert "at most" in moe.moe_last_error()


@pytest.mark.parametrize("size", [dict(m=TOP), dict(n=TOP), dict(k=1 << 30, a_stride=1 << 30, w_stride=1 << 30, w_scale_stride=1 << 23)])
def test_matmul_takes_the_largest_sizes(lib, size):
    big = 1 << 31
    args = dict(dict(m=1, n=1, k=16, a_stride=16, w_stride=16, a_scale_stride=big, w_scale_stride=big, out_stride=big), **size)
    taken(lambda: lib.moe_f8_matmul(CTX, ctypes.byref(matmul_args(**args)), None))


def test_check_and_injection_refuse_no_context(lib):
    assert lib.moe_f8_check(None) == moe.MOE_EINVAL
    assert lib.moe_ctx_inject_f8_timeout(None) == moe.MOE_EINVAL
