"""Pins of the oracle's 4-bit KV rows and of its sampler: worked blocks, bounds
and invariants (no GPU)."""
import numpy as np
import pytest

from oracle import qw3_oracle as orc


def test_kv_q4_worked_block():
    x = np.zeros(32)
    x[:6] = [-4.0, 3.5, 0.24, 0.26, 3.9, -0.25]     # m = -4: d = 0.5
    codes, scales = orc.kv_q4_encode(x)
    assert scales.dtype == np.float16 and scales.tolist() == [0.5]
    # x / d = -8, 7, 0.48, 0.52, 7.8 (clamped), -0.5 (up to 0)
    assert codes[:6].tolist() == [0, 15, 8, 9, 15, 8] and set(codes[6:]) == {8}
    assert orc.kv_q4_decode(codes, scales)[:6].tolist() == [-4.0, 3.5, 0.0, 0.5, 3.5, 0.0]


def test_kv_q4_sign_rule_and_zero_block():
    x = np.zeros((2, 32))
    x[0, 3], x[0, 9] = -2.0, 2.0                       # opposite equals: the positive one decides
    codes, scales = orc.kv_q4_encode(x)
    assert scales[0, 0] == -0.25 and codes[0, 9] == 0 and codes[0, 3] == 15
    assert scales[1, 0] == 0 and set(codes[1]) == {8}


def test_kv_q4_error_bound():
    """|x - value| <= d / 2 + 8 |d - f16(d)|, and d at the clamped end (code 15
    stands for 7 of up to 8 steps)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 128)) * np.exp(rng.standard_normal((64, 1)) * 3)
    codes, scales = orc.kv_q4_encode(x)
    b = x.reshape(64, 4, 32)
    d = np.abs(b).max(-1) / 8
    err = np.abs(orc.kv_q4_decode(codes, scales).astype(np.float64).reshape(b.shape) - b)
    slack = 8 * np.abs(d - np.abs(scales.astype(np.float64)))
    end = codes.reshape(b.shape) == 15
    assert np.all(err <= np.where(end, d[..., None], d[..., None] / 2) + slack[..., None] + 1e-12)


def test_kv_q4_blocks_that_cannot_be_held_are_zeros():
    x = np.ones((6, 64))
    x[0, 3], x[1, 3], x[2, 3], x[3, 3], x[4, 3], x[5, 3] = np.nan, np.inf, -np.inf, 524160.0, -524160.0, 524159.0
    codes, scales = orc.kv_q4_encode(x)
    assert not scales[:5, 0].any() and np.all(codes[:5, :32] == 8)
    assert scales[5, 0] == np.float16(-65504)              # under 65520: still the largest f16
    assert np.all(scales[:, 1] == np.float16(-0.125)) and np.all(orc.kv_q4_decode(codes, scales)[:, 32:] == 1.0)


def test_kv_q4_scales_round_to_nearest_even():
    """d at the middle between two f16 values, normal and subnormal."""
    for d, want in ((1 + 2.0 ** -11, 1.0), (1 + 3 * 2.0 ** -11, 1 + 2.0 ** -9), (2.5 * 2.0 ** -24, 2 * 2.0 ** -24),
                    (3.5 * 2.0 ** -24, 4 * 2.0 ** -24), (0.5 * 2.0 ** -24, 0.0), (0.75 * 2.0 ** -24, 2.0 ** -24)):
        x = np.zeros(32)
        x[7] = -8 * d
        assert orc.kv_q4_encode(x)[1].tolist() == [want]


def test_kv_q4_row_bytes_places():
    """Two blocks: K bytes go word by word, V bytes halfword by halfword."""
    codes = np.concatenate([np.arange(32) % 16, (np.arange(32) + 5) % 16])
    b0 = [(2 * j % 16) | ((2 * j + 1) % 16) << 4 for j in range(16)]
    b1 = [((2 * j + 5) % 16) | ((2 * j + 6) % 16) << 4 for j in range(16)]
    k, v = orc.kv_q4_row_bytes(codes, False).tolist(), orc.kv_q4_row_bytes(codes, True).tolist()
    assert k == [x for w in range(4) for blk in (b0, b1) for x in blk[4 * w:4 * w + 4]]
    assert v == [x for w in range(8) for blk in (b0, b1) for x in blk[2 * w:2 * w + 2]]


def test_kv_q4_cache_reads_dequantised_rows():
    rng = np.random.default_rng(5)
    c = orc.KvCache(1, 2, 64, 8, "q4")
    k, v = rng.standard_normal((2, 3, 2, 64)).astype(np.float32)
    c.append_layer(0, k, v)
    c.advance(3)
    got, _ = c.layer_rows(0, 3)
    assert np.array_equal(got, orc.kv_q4_decode(*orc.kv_q4_encode(k))) and not np.array_equal(got, k)


LOGITS = np.log(np.array([0.1, 0.4, 0.2, 0.05, 0.25]))


@pytest.mark.parametrize("kw,u,token,prob", [
    (dict(), 0.0, 0, 0.1), (dict(), 0.0999, 0, 0.1), (dict(), 0.11, 1, 0.4), (dict(), 0.999, 4, 0.25),
    (dict(top_k=2), 0.3, 1, 0.4 / 0.65), (dict(top_k=2), 0.7, 4, 0.25 / 0.65), (dict(top_k=1), 0.99, 1, 1.0),
    (dict(top_p=0.64), 0.7, 4, 0.25 / 0.65), (dict(top_p=0.66), 0.6, 2, 0.2 / 0.85), (dict(top_p=0.0), 0.5, 1, 1.0),
    # top-p works on the sum that top-k left: 0.6 of 0.65 needs one token only
    (dict(top_k=2, top_p=0.6), 0.99, 1, 1.0),
    (dict(min_p=0.55), 0.5, 1, 0.4 / 0.65), (dict(min_p=5.0), 0.5, 1, 1.0),
    (dict(temperature=0.5), 0.0, 0, 0.01 / (0.01 + 0.16 + 0.04 + 0.0025 + 0.0625)),
    (dict(temperature=0.0), 0.9, 1, 1.0), (dict(temperature=-1.0), 0.0, 1, 1.0),
])
def test_sample_worked(kw, u, token, prob):
    t, p, _ = orc.sample_token(LOGITS, u, **kw)
    assert t == token and p == pytest.approx(prob, rel=1e-12)


def test_sample_ties_go_to_the_lowest_index():
    lg = np.zeros(6)
    assert [orc.sample_token(lg, u, top_k=3)[0] for u in (0.0, 0.4, 0.9)] == [0, 1, 2]
    assert [orc.sample_token(lg, u, top_p=0.5)[0] for u in (0.0, 0.4, 0.99)] == [0, 1, 2]


def test_sample_frequencies_follow_the_distribution():
    n = 4000
    got = np.bincount([orc.sample_token(LOGITS, (i + 0.5) / n)[0] for i in range(n)], minlength=5) / n
    assert np.allclose(got, np.exp(LOGITS), atol=1.0 / n)


def test_sample_skips_minus_inf_and_refuses_what_has_no_answer():
    lg = np.array([-np.inf, 1.0, -np.inf, 1.0])
    assert orc.sample_token(lg, 0.0)[0] == 1 and orc.sample_token(lg, 0.9999999)[0] == 3
    for bad in (np.full(3, -np.inf), np.array([0.0, np.nan]), np.array([0.0, np.inf])):
        with pytest.raises(orc.NonFiniteValue):
            orc.sample_token(bad, 0.5)


def test_sample_refuses_settings_that_are_not_numbers():
    for kw in (dict(temperature=np.nan), dict(temperature=np.inf), dict(temperature=-np.inf), dict(top_p=np.nan),
               dict(min_p=np.nan)):
        with pytest.raises(orc.NonFiniteValue):
            orc.sample_token(LOGITS, 0.5, **kw)
    assert orc.sample_token(LOGITS, 0.5, temperature=0.0, top_p=np.nan, min_p=np.nan)[0] == 1
