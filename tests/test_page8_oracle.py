"""The oracle of the page-scaled cache and of eviction, pinned by closed forms
and brute force (no GPU)."""

import math

import numpy as np
import pytest

from oracle import mla_oracle as O
from oracle import page8_oracle as P


@pytest.mark.parametrize("amax,e", [(0.0, -64), (448.0, 0), (448.0000001, 1), (224.0, -1),
                                    (224.1, 0), (1.0, -8), (0.875, -9), (3.5, -7), (1e30, 64),
                                    (1e-30, -64)])
def test_scale_is_the_least_power_of_two_that_holds_amax(amax, e):
    assert P.scale_for(amax) == math.ldexp(1.0, e)


def test_recode_by_a_power_of_two_is_exact_until_subnormal():
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    v = O.e4m3_decode(codes)
    for k in (1, 3, 6):
        w = O.e4m3_decode(P.recode(codes, 2.0 ** -k))
        normal = np.abs(v) * 2.0 ** -k >= 2.0 ** -6
        assert np.all(w[normal] == v[normal] * 2.0 ** -k)
        assert np.all(np.abs(w - v * 2.0 ** -k) <= 2.0 ** -10)   # half a subnormal step
    assert P.recode(np.array([0x7F, 0xFF], np.uint8), 0.5).tolist() == [0x7F, 0xFF]


def _empty(nb, bs):
    return np.zeros((nb, bs, 512), np.uint8), np.zeros((nb, bs, 64)), np.zeros(nb)


def test_write_grows_a_page_and_keeps_its_values():
    rng = np.random.default_rng(0)
    w = np.ones(512)
    c, r, s = _empty(3, 16)
    x1 = rng.standard_normal((4, 512))
    c1, r1, s1 = P.write(c, r, s, x1, np.zeros((4, 64)), np.arange(4), [16, 17, 18, 19], w, 1e-6, 1e4)
    x2 = np.zeros((1, 512))
    x2[0, 3] = 1.0                       # RMSNorm makes it sqrt(512) = 22.6
    c2, r2, s2 = P.write(c1, r1, s1, x2, np.zeros((1, 64)), [4], [20], w, 1e-6, 1e4)
    assert s1[1] < s2[1] and s2[0] == s2[2] == 0
    old, new = P.rows_of(c1, r1, s1)[1, :4], P.rows_of(c2, r2, s2)[1, :4]
    assert np.max(np.abs(old - new)) <= s2[1] * 2.0 ** -10
    assert P.rows_of(c2, r2, s2)[1, 4, 3] == pytest.approx(math.sqrt(512), rel=2.0 ** -4)


def test_a_repeated_slot_goes_to_the_later_token():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 512))
    c, r, s = _empty(2, 16)
    both = P.write(c, r, s, x, np.zeros((3, 64)), [0, 1, 2], [5, -1, 5], np.ones(512), 1e-6, 1e4)
    last = P.write(c, r, s, x[2:], np.zeros((1, 64)), [2], [5], np.ones(512), 1e-6, 1e4)
    assert np.array_equal(both[0], last[0]) and np.array_equal(both[2], last[2])


def test_mass_of_one_row_sums_to_the_heads():
    rng = np.random.default_rng(2)
    c, r, s = _empty(4, 16)
    c, r, s = P.write(c, r, s, rng.standard_normal((40, 512)), rng.standard_normal((40, 64)),
                      np.arange(40), np.arange(40) + 16, np.ones(512), 1e-6, 1e4)
    mass = np.full((4, 16), 8.0)
    out, m = P.decode(rng.standard_normal((1, 16, 576)), P.rows_of(c, r, s), [[1, 2, 3]], [37], [0, 1],
                      0.07, rng.standard_normal((16, 512, 128)), mass, 0.5)
    live = m.reshape(-1)[16:53]
    assert live.sum() == pytest.approx(37 * 4 + 16)
    assert np.all(m.reshape(-1)[:16] == 8) and np.all(m.reshape(-1)[53:] == 8)


def test_select_keeps_sinks_recent_and_the_heaviest_with_ties_to_the_lower_index():
    mass = np.array([[5, 1, 1, 9, 1, np.nan, 0, 2]], float)
    keep, n = P.select(mass, [[0]], [8], 1, 1, 5)
    assert keep.tolist() == [[0, 1, 2, 3, 7]] and n.tolist() == [5]
    keep, n = P.select(mass, [[0]], [7], 0, 0, 7)
    assert keep.tolist() == [[0, 1, 2, 3, 4, 5, 6]]
    keep, n = P.select(mass, [[0]], [8], 0, 0, 7)      # all but the NaN
    assert keep.tolist() == [[0, 1, 2, 3, 4, 6, 7]]


def test_attention_after_compaction_is_attention_over_the_kept_tokens():
    rng = np.random.default_rng(3)
    c, r, s = _empty(6, 16)
    c, r, s = P.write(c, r, s, rng.standard_normal((40, 512)) * np.exp(rng.standard_normal((40, 1))),
                      rng.standard_normal((40, 64)), np.arange(40), np.arange(40), np.ones(512), 1e-6, 1e4)
    keep = np.array([[0, 3, 4, 17, 20, 39]])
    c2, r2, s2, m2 = P.compact(c, r, s, np.zeros((6, 16)), [[0, 1, 2]], keep, [6], [[5]])
    q, w = rng.standard_normal((1, 16, 576)), rng.standard_normal((16, 512, 128))
    got, _ = P.decode(q, P.rows_of(c2, r2, s2), [[5]], [6], [0, 1], 0.07, w)
    kv = P.rows_of(c, r, s).reshape(-1, 576)[keep[0]]
    o, _ = O.latent_attention(q, kv, [5], 0.07)
    # recoding moves a latent by at most S 2^-10 (half a subnormal step); a
    # convex sum of those, through 512 weights, by at most that times sum |w|;
    # the scores move by scale * sum |q| S 2^-10 (first order, both signs)
    d = s2[5] * 2.0 ** -10
    ds = 0.07 * d * np.abs(q[0, :, :512]).sum(1)
    big = np.abs(kv[:, :512]).max()
    bound = (d + 2 * ds * big)[:, None] * np.abs(w).sum(1)
    assert np.all(np.abs(got - O.out_proj(o, w))[0] <= bound + 1e-12)
