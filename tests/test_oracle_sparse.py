"""Properties of the restated block bounds, scores and choice."""
import numpy as np
import pytest

from oracle import bf16, sparse


def _bits(x):
    return bf16.from_f64(np.asarray(x, np.float64))


@pytest.mark.parametrize("a,e", [(0.0, -32), (127 * 2.0 ** -32, -32), (127.5 * 2.0 ** -32, -31), (126.0, 0), (127.0, 0),
                                 (127.5, 1), (1.0, -6), (1.984375, -6), (1.9921875, -5), (127 * 2.0 ** 16, 16),
                                 (2.0 ** 100, 16), (np.inf, 16)])
def test_exponent(a, e):
    assert sparse.exponent(a) == e


@pytest.mark.parametrize("size", [1e-12, 1e-3, 1.0, 50.0, 1e6])
def test_scores_bound_the_products(size):
    """No product of the query's codes with a key of the block exceeds the block's score."""
    rng = np.random.default_rng(int(size * 7) % 1000)
    for rows in (1, 5, 64):
        K, Q = _bits(size * rng.standard_normal((rows, 128))), _bits(3 * rng.standard_normal((6, 128)))
        codes, scale = sparse.bounds(K)
        s = sparse.scores(Q, codes[None], np.array([scale]))[0]
        best = max((sparse.query(q)[0] * sparse.query(q)[1] * bf16.to_f64(k)).sum() for q in Q for k in K)
        assert best <= s


def test_scores_are_exact_in_any_order():
    """fp32 sums in two orders and the fp64 sum agree."""
    rng = np.random.default_rng(3)
    codes, scale = zip(*(sparse.bounds(_bits(2 * rng.standard_normal((64, 128)))) for _ in range(20)))
    Q = _bits(3 * rng.standard_normal((6, 128)))
    want = sparse.scores(Q, np.stack(codes), np.array(scale))
    c, two = zip(*(sparse.query(q) for q in Q))
    for order in (np.arange(128), np.arange(128)[::-1]):
        got = []
        for code, s in zip(codes, scale):
            each = [np.float32(0)] * 6
            for h in range(6):
                for d in order:
                    each[h] += np.float32(max(c[h][d] * float(code[0, d]), c[h][d] * float(code[1, d])))
            got.append(max(np.float32(e * np.float32(t)) for e, t in zip(each, two)) * np.float32(s))
        assert np.array_equal(np.array(got, np.float64), want)


def test_not_finite_keys():
    K = np.zeros((3, 128))
    bits = _bits(K)
    bits[0, 0], bits[1, 1], bits[2, 2], bits[0, 3] = 0x7F80, 0xFF80, 0x7FC0, 0xFFC0
    codes, scale = sparse.bounds(bits)
    assert scale == 2.0 ** 16
    assert codes[:, 0].tolist() == [127, 0] and codes[:, 1].tolist() == [0, -127]
    assert codes[:, 2].tolist() == [127, 0] and codes[:, 3].tolist() == [0, -127]


def test_choice():
    s = np.array([1.0, 5.0, 5.0, 2.0, 5.0, 0.0])
    assert sparse.choose(s, 2, 0, 0) == [1, 2]
    assert sparse.choose(s, 3, 1, 1) == [0, 1, 5]
    assert sparse.choose(s, 4, 0, 2) == [1, 2, 4, 5]
    assert sparse.choose(s, 9, 1, 1) == list(range(6))
    assert sparse.choose(s[:1], 2, 1, 1) == [0]


def test_rows_of_lists():
    assert sparse.rows_of([1, -1, 0], 70).tolist() == list(range(64, 70)) + list(range(64))
    assert sparse.rows_of([-1, -1], 70).size == 0
    assert sparse.at(np.array([7, 3]), np.array([0, 127, 128])).tolist() == [896, 1023, 384]
