"""Pins of the attention oracle (oracle/attn.py) on hand values and closed forms (CPU)."""
import numpy as np

from oracle import attn as A


def test_rope_hand_values():
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    q = np.float64(np.pi / 2)
    out = A.rope(x, None, [1], [q, 0.0], 0.0, False)[0, 0]   # pairs (0, 2), (1, 3); the rest stays
    assert np.allclose(out, [-2, 1, 0, 3, 4, 5, 6, 7], atol=1e-15)
    out = A.rope(x, None, [1], [q, 0.0], 0.0, True)[0, 0]    # pairs (0, 1), (2, 3)
    assert np.allclose(out, [-1, 0, 2, 3, 4, 5, 6, 7], atol=1e-15)
    out = A.rope(x, None, [-1], [q, 0.0], 0.0, True)[0, 0]
    assert np.allclose(out, [1, 0, 2, 3, 4, 5, 6, 7], atol=1e-15)


def test_rope_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    dots = [(A.rope(q, None, [p + 7], f, 0.0, False) * A.rope(k, None, [p], f, 0.0, False)).sum()
            for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0], rtol=1e-9)
    n = A.rope(q, np.ones(64), [3], f, 0.0, True)
    assert np.isclose((n * n).mean(), 1.0)


def test_bf16_rounding_ties_to_even():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, np.inf, -0.0], np.float32)
    assert A.to_bf16(x).tolist() == [1.0, 1.0, 1 + 2.0 ** -6, np.inf, 0.0]


def test_kv4_codes_of_a_ramp_and_of_special_rows():
    x = np.zeros((6, 64), np.float32)
    x[0, :16] = np.arange(16)           # step 1, low 0
    x[1] = 5.0                          # a constant: step 0
    x[2, 3] = np.nan
    x[3, 3] = np.inf
    x[4, 0], x[4, 1] = 3e38, -3e38      # the spread overflows
    x[5, 0] = 2.0 ** -130               # below the smallest step
    codes, s, m = A.kv4_encode(x)
    assert codes[0, :16].tolist() == list(range(16)) and s[0] == 1 and m[0] == 0
    assert s[1] == 0 and m[1] == 5 and not codes[1].any()
    for r in (2, 3, 4):
        assert np.isnan(s[r]) and np.isnan(m[r]) and not codes[r].any()
    assert s[5] == 0 and m[5] == 0
    assert np.array_equal(A.kv4_values(codes[:2], s[:2], m[:2]), x[:2].astype(np.float64))


def test_kv4_error_is_within_half_a_step_and_its_rounding():
    x = np.random.default_rng(1).standard_normal((500, 128)).astype(np.float32) * 3
    codes, s, m = A.kv4_encode(x)
    # half a step; at the ends the low end's and the step's bf16 roundings (2^-8 of each)
    lim = 0.5 * s[:, None] + 15 * s[:, None] * 2.0 ** -8 + np.abs(m)[:, None] * 2.0 ** -8
    assert np.all(np.abs(A.kv4_values(codes, s, m) - x) <= lim)


def test_kv4_pack_places_nibbles_and_pairs():
    cache = np.zeros((2, 1, 2, 64 * 36), np.uint8)
    codes = (np.arange(64) % 16).astype(np.uint8)
    A.kv4_pack(cache, 1, 5, 0, 1, codes, np.float32(1.0), np.float32(-2.0))
    blk = cache[1, 0, 1]
    assert blk[5 * 32] == 0x10 and blk[5 * 32 + 7] == 0xFE
    assert blk[64 * 32 + 20:64 * 32 + 24].tolist() == [0x80, 0x3F, 0x00, 0xC0]
    c, s, m = A.kv4_unpack(cache, 1, 5, 0, 1)
    assert np.array_equal(c, codes) and s == 1.0 and m == -2.0
    assert not cache[0].any() and not cache[1, 0, 0].any()


def test_attend_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 5, 8))
    q = rng.standard_normal((3, 8))
    out = A.attend(q, k, v, [-1, 0, 4], 0.0)
    assert not out[0].any() and np.allclose(out[1], v[0]) and np.allclose(out[2], v.mean(0))
    out = A.attend(np.stack([1e3 * k[2]]), k / np.linalg.norm(k, axis=1)[:, None], v, [4], 1.0)
    assert np.allclose(out[0], v[2])
