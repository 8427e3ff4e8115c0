"""The float64 definitions of the paged operators, pinned by hand examples and other formulas."""
import numpy as np

from oracle import attention as A
from oracle import pages as P


def test_assign_by_hand():
    """Pages of 16: 20 -> 33 opens the third page, 0 -> 17 the first two, the third sequence none."""
    table = np.full((3, 4), -1)
    table[0, :2], table[2, 0] = [7, 3], 5
    free = np.array([9, 1, 0, 2, 0, 0])
    t, s, p, left = P.assign(table, free, 4, [13, 17, 2], [33, 17, 6], 16, 10)
    assert t.tolist() == [[7, 3, 2, -1], [0, 1, -1, -1], [5, -1, -1, -1]] and left == 1
    assert s.tolist() == [3 * 16 + i for i in range(4, 16)] + [32] + list(range(16)) + [16] + [84, 85]
    assert p.tolist() == list(range(20, 33)) + list(range(17)) + [4, 5]
    t2, f2, n2 = P.release(t, free, left, [20, 0, 6], [33, 17, 6], 16)
    assert t2.tolist() == table.tolist() and n2 == 4 and f2[:4].tolist() == [9, 1, 0, 2]


def test_grid():
    for x, codes, e in (([0.0, 0.0], [0, 0], -126), ([127.0, -1.5], [127, -2], 0), ([127.5, 0.5], [64, 0], 1),
                        ([127.49, 2.5], [127, 2], 0), ([63.75, 0.0], [64, 0], 0), ([63.74, -0.25], [127, 0], -1),
                        ([2.0 ** -130, 0.0], [0, 0], -126)):
        c, got = P.to_grid(x)
        assert c.tolist() == codes and got == e, x


def test_select_by_hand():
    """Blocks of 16, one kv head with two query heads: the maximum over the heads decides, ties go to the lower."""
    codes = np.zeros((4, 1, 1, 64), np.int64)
    codes[:, 0, 0, 0], codes[:, 0, 0, 1] = [5, 2, 2, 9], [0, 3, 3, 0]
    scales = np.full((4, 1, 1), 127)
    q = np.zeros((1, 2, 64))
    q[0, 0, 0], q[0, 1, 1] = -100, 100
    table = np.array([[0, 1, 2, 3]])
    got = lambda **k: P.select(q, codes, scales, table, [1], [60], 16, 16, **k)[0, 0].tolist()
    assert got(topn=2, sinks=0, local=1) == [1, 3]              # 0, 300, 300 for blocks 0, 1, 2
    assert got(topn=3, sinks=0, local=1) == [1, 2, 3]
    assert got(topn=2, sinks=1, local=1) == [0, 3]
    assert got(topn=6, sinks=1, local=1) == [0, 1, 2, 3, -1, -1]


def test_attention_over_pages_is_prompt_attention():
    rng = np.random.default_rng(0)
    ql, kl, hq, hk, d, page = [3, 20], [25, 20], 4, 2, 8, 16
    table = np.array([[3, 1], [0, 4]])
    q, kp, vp = rng.normal(size=(23, hq, d)), rng.normal(size=(5, page, hk, d)), rng.normal(size=(5, page, hk, d))
    at = np.concatenate([A.slots(table, b, n, page, 5) for b, n in enumerate(kl)])
    want = A.prompt(q, kp.reshape(-1, hk, d)[at], vp.reshape(-1, hk, d)[at], ql, kl, 0.3)
    for idx, block in ((None, 0), (np.broadcast_to(np.array([1, 0, -1]), (23, hk, 3)), 16)):
        got = P.pages_attention(q, kp, vp, table, ql, kl, 0.3, idx, block)
        for a, b in zip(got, want):
            assert np.allclose(a, b, atol=1e-12)
    twice = P.pages_attention(q, kp, vp, table, ql, kl, 0.3, np.broadcast_to(np.array([0, 0]), (23, hk, 2)), 16)
    once = P.pages_attention(q, kp, vp, table, ql, kl, 0.3, np.broadcast_to(np.array([0]), (23, hk, 1)), 16)
    assert np.allclose(twice[0], once[0]) and np.allclose(twice[1], once[1] + np.log(2.0))


def test_numbers_that_are_not_finite():
    most = float(np.finfo(np.float32).max)
    row, e = P.to_grid([np.inf, -np.inf, np.nan, most, 0.0, 2.0 ** 122])
    assert row.tolist() == [64, -64, 0, 64, 0, 1] and e == 122
    k = np.zeros((1, 16, 1, 4))
    k[0, 3, 0] = [np.inf, -np.inf, np.nan, 16.0]
    k[0, 5, 0] = [1.0, -np.inf, 2.0, 0.0]
    k[0, 6, 0] = [-np.inf, 5.0, 2.0, 0.0]
    c, s = P.summaries(k, np.zeros((1, 1), int), [16], [16], 16, np.zeros((1, 1, 1, 4)), np.zeros((1, 1, 1)))
    assert c.ravel().tolist() == [0, -64, 0, 0] and s.ravel().tolist() == [249]
