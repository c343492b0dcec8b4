"""Pins of the cache oracle (oracle/kv.py) on small cases, and the library's
host-side checks that need no GPU."""
import ctypes

import numpy as np
import pytest

import expert_streaming_ffn_gb300 as moe
from oracle import kv


def test_quantise_known_groups():
    x = np.zeros((4, 64), np.float32)
    x[0, :16] = np.arange(16)  # 0..15 in steps of 1: codes are the values
    x[1, :] = -3.0  # constant: scale 0, bias -3
    x[2, 0], x[2, 1] = 1e30, -1e30  # held as +-65504
    x[3, 0], x[3, 1] = 7.5, 15.0  # 7.5 is a tie, to even
    c, s, b = kv.quantise(x)
    assert (c[0, 0, :16] == np.arange(16)).all() and s[0, 0] == 1 and b[0, 0] == 0
    assert (c[1] == 0).all() and s[1, 0] == 0 and b[1, 0] == -3
    v = kv.values(c, s, b)
    assert v[2, 1] == -65504 and abs(v[2, 0] - 65504) <= s[2, 0] / 2
    assert c[3, 0, 0] == 8 and c[3, 0, 1] == 15


@pytest.mark.parametrize("seed", range(4))
def test_quantise_within_half_a_step(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((200, 128)) * np.exp(rng.uniform(-12, 8, (200, 1))) + rng.uniform(-50, 50, (200, 1))).astype(np.float32)
    c, s, b = kv.quantise(x)
    assert c.max() <= 15
    err = np.abs(kv.values(c, s, b) - x).reshape(200, 2, 64)
    # half a step, and the fp32 rounding of (x - bias) / scale, at most 2^-19 of a step
    assert (err <= s.astype(np.float64)[..., None] * (0.5 + 2.0 ** -19)).all()


def test_directed_rounding_against_neighbours():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(1000) * np.exp(rng.uniform(-18, 10, 1000)), [0.0, -0.0, 1e-9, -1e-9, 65504, -65504]]).astype(np.float32)
    lo, hi = kv.f16_down(x).astype(np.float64), kv.f16_up(x).astype(np.float64)
    assert (lo <= x).all() and (hi >= x).all()
    assert (np.nextafter(kv.f16_down(x), np.float16(np.inf)).astype(np.float64) > x).all()


def test_layout_of_one_row():
    d = 128
    pages = kv.empty_pages(2, 3, d, 32, 0xEE)
    k = np.zeros((1, 3, d), np.float32)
    k[0, 2] = np.arange(d) % 64 // 4  # group of 0..15: codes equal values, scale 1, bias 0
    kv.append(pages, 32, k, np.zeros_like(k), [32 + 16 + 5])
    rec = pages[1, 2, 1]
    words = rec[5 * 64:6 * 64].view(np.uint32)
    for i in range(8):
        want = [(8 * i + e) // 4 for e in range(8)]
        got = [0] * 8
        for n in range(8):
            got[kv.NIBBLE_ELEMENT[n]] = int(words[2 * i] >> (4 * n)) & 15
        assert got == want and words[2 * i] == words[2 * i + 1]
    aff = rec[16 * d + 5 * 8:16 * d + 6 * 8].view(np.float16)
    assert aff.tolist() == [1, 0, 1, 0]
    assert (pages[0] == 0xEE).all() and (rec[:5 * 64] == 0xEE).all()
    K, V = kv.read(pages, 32, [53, -1])
    assert (K[0, 2] == k[0, 2]).all() and (K[1] == 0).all() and (V == 0).all()


def test_attend_closed_forms():
    d, P = 64, 16
    pages = kv.empty_pages(1, 1, d, P)
    rng = np.random.default_rng(0)
    k, v = np.zeros((3, 1, d), np.float32), rng.standard_normal((3, 1, d)).astype(np.float32)
    kv.append(pages, P, k, v, [0, 1, 2])
    _, V = kv.read(pages, P, [0, 1, 2])
    q = rng.standard_normal((3, 2, d))
    table = np.zeros((1, 1), np.int64)
    out, lse, _ = kv.attend(pages, P, q, table, [3], [0, 3], 0.3)
    for i in range(3):  # equal keys: the mean of the values seen
        np.testing.assert_allclose(out[i], np.broadcast_to(V[:i + 1, 0].mean(0), (2, d)), atol=1e-12)
        np.testing.assert_allclose(lse[i], np.log(i + 1), atol=1e-12)
    out, lse, _ = kv.attend(pages, P, q, table, [3], [0, 3], 0.3, window=1)
    np.testing.assert_allclose(out[:, 0], V[:, 0], atol=1e-12)
    out, lse, _ = kv.attend(pages, P, q, table, [2], [0, 3], 0.3)  # position -1 sees nothing
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()
    out, _, _ = kv.attend(pages, P, q, table, [3], [0, 3], 0.3, causal=False)
    np.testing.assert_allclose(out[0, 0], V[:, 0].mean(0), atol=1e-12)


def test_cache_bytes():
    assert moe.moe_kv_cache_bytes(8, 128, 64, 10) == 10 * 8 * 4 * 18 * 128
    assert moe.moe_kv_cache_bytes(1, 64, 16, 1) == 18 * 64
    for bad in ((0, 128, 64, 1), (8, 96, 64, 1), (8, 128, 48, 1), (8, 128, 8, 1), (8, 128, 512, 1), (8, 128, 64, 0),
                (8, 128, 256, 1 << 23)):
        assert moe.moe_kv_cache_bytes(*bad) == 0, bad


def test_calls_refuse_null_context():
    lib = moe.load()
    c = moe.moe_kv_cache(8, 128, 64, 1, 4096)
    assert lib.moe_kv_append(None, ctypes.byref(c), None, 0, 0, None, 0, 0, moe.MOE_BF16, None, 0, None) == moe.MOE_EINVAL
    assert lib.moe_kv_read(None, ctypes.byref(c), None, 0, None, 0, 0, None, 0, 0, moe.MOE_BF16, None) == moe.MOE_EINVAL
    a = moe.moe_kv_attend_args()
    assert lib.moe_kv_attend(None, ctypes.byref(c), ctypes.byref(a), None) == moe.MOE_EINVAL
    assert lib.moe_kv_check(None) == moe.MOE_EINVAL
    assert "ctx" in moe.moe_last_error()
