"""Pins of the attention oracle: closed forms, brute force, the 4-bit format's own rules."""
import numpy as np
import pytest

from oracle import attention as A


def test_attend_closed_forms():
    v = np.array([[1.0, 2.0], [3.0, 6.0]])
    o, l, w, a, _ = A.attend(np.zeros(2), np.ones((2, 2)), v, 1.0, np.array([True, True]))
    assert np.allclose(o, [2.0, 4.0]) and np.isclose(l, np.log(2.0)) and np.allclose(w, 0.5)
    o, l, w, _, _ = A.attend(np.ones(2), np.array([[0.0, 0.0], [1.0, 1.0]]), v, 0.5 * np.log(3.0), [1, 1])
    assert np.allclose(w, [0.25, 0.75]) and np.allclose(o, [2.5, 5.0]) and np.isclose(l, np.log(4.0))
    o, l, w, _, _ = A.attend(np.ones(2), np.ones((2, 2)), v, 1.0, [0, 0])
    assert np.all(o == 0) and l == -np.inf and np.all(w == 0)
    o2, l2, _, _, _ = A.attend(np.ones(2), np.array([[0.5, 1.0]]), v[:1], 1.0, [2])      # listed twice
    assert np.allclose(o2, v[0]) and np.isclose(l2, 1.5 + np.log(2.0))


def test_prompt_first_query_sees_one_key():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    out, lse, _, _ = A.prompt(q, k, v, [3, 2], [3, 6], 0.3)
    for h in range(4):
        assert np.allclose(out[0, h], v[0, h // 2]) and np.isclose(lse[0, h], 0.3 * q[0, h] @ k[0, h // 2])


def test_mx_values_survive():
    """Every code and scale encodes to itself when the block holds a code above half the range."""
    for e in (1, 2, 100, 127, 200, 253):
        x = np.concatenate([A.GRID, -A.GRID, np.full(16, 6.0)]) * np.ldexp(1.0, e - 127)
        c, s = A.mx_encode(x)
        assert s[0] == e
        assert np.array_equal(A.mx_decode(c, s), x)


def test_mx_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(200, 64)) * np.exp(rng.normal(size=(200, 1)) * 4)
    c, s = A.mx_encode(x)
    y = A.mx_decode(c, s)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, -1)
    a = np.abs(x) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert np.all(a < 7) and np.all(np.abs(x - y) <= step / 2 * unit)
    # and the scale is the smallest that allows it
    assert np.all(np.abs(x).reshape(200, 2, 32).max(-1) >= 3.5 * np.ldexp(1.0, s.astype(int) - 127))


def test_mx_borders():
    one = lambda v: int(A.mx_encode(np.array([v] + [4.0] + [0.0] * 30))[0][0] & 15)
    assert [one(v) for v in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] == [0, 2, 2, 4, 4, 6, 6]
    assert one(-0.75) == 10 and one(-0.25) == 8
    for top, e in ((7.0, 128), (np.nextafter(7.0, 0), 127), (3.5, 127), (np.nextafter(3.5, 0), 126), (0.0, 1)):
        assert A.mx_encode(np.array([top] + [0.0] * 31))[1][0] == e, top


@pytest.mark.parametrize("seed", range(20))
def test_evict_keeps_the_best(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 60))
    keep = int(rng.integers(0, n + 1))
    acc = rng.integers(0, 6, n).astype(float)        # many ties
    pos = rng.permutation(2 * n)[:n]
    prefix, window = 0, 0
    if keep > 4:
        prefix, window = 2, 2
    src = A.evict(acc, n, keep, prefix, window, pos, 2 * n)
    assert len(set(src.tolist())) == keep
    safe = (pos < prefix) | (pos >= 2 * n - window)
    assert set(np.flatnonzero(safe).tolist()) <= set(src.tolist())
    rest = [j for j in range(n) if j not in set(src.tolist())]
    for j in rest:
        for i in src:
            assert safe[i] or acc[i] > acc[j] or (acc[i] == acc[j] and i < j)
    for j, i in enumerate(src):
        assert i == j or (i >= keep and j in rest)


def test_evict_moves_nothing_to_an_index_without_a_page():
    acc = [5.0, 1.0, 2.0, 9.0, 8.0, 7.0, 3.0, 6.0]
    there = np.array([True, False, True, True, True, False, True, True])
    # places 0, 2, 3 are left in front of 4: of the keys with a page 9, 8 and 6 stay
    assert A.evict(acc, 8, 4, 0, 0, there=there).tolist() == [4, 1, 7, 3]
    # a protected key of small weight takes a place
    assert A.evict(acc, 8, 4, 1, 1, there=there).tolist() == [0, 1, 7, 3]
    # more protected keys than places: the lowest indices
    assert A.evict(acc, 8, 4, 2, 2, there=np.array([False, False, False, True, True, True, True, True])).tolist() == [0, 1, 2, 6]
