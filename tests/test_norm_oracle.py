"""The residual norm's oracle: the generator's published answers, gradients against differences."""
import numpy as np
import pytest

from oracle import residual_norm as rn


@pytest.mark.parametrize("counter,key,want", [  # the generator's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator(counter, key, want):
    assert tuple(int(v) for v in rn.philox(np.array(counter, dtype=np.uint64), key)) == want


def test_share_of_dropped_values():
    T, K = 400, 512
    for p in (0.1, 0.5):
        kept = rn.keep(T, K, p, 77, 5, 2)
        n = T * K
        d = rn.below(p) / 65536
        assert abs((kept == 0).sum() - n * d) < 6 * np.sqrt(n * d * (1 - d))
        assert abs(kept.mean() - 1) < 6 * np.sqrt(d / (1 - d) / n)
    a, b = rn.keep(T, K, 0.5, 77, 5, 2), rn.keep(T, K, 0.5, 77, 5, 3)
    assert 0.45 < ((a == 0) == (b == 0)).mean() < 0.55  # another stream, other numbers


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    T, K, eps = 3, 16, 1e-3
    x, res, w = rng.standard_normal((T, K)), rng.standard_normal((T, K)), rng.standard_normal(K)
    do, dst = rng.standard_normal((T, K)), rng.standard_normal((T, K))
    kept, mask = rn.keep(T, K, 0.3, 1, 2, 3), np.array([1, 0, 1], np.uint8)

    def loss(x, res, w):
        s, n = rn.forward(x, res, w, eps, kept, mask)
        return (do * n)[mask != 0].sum() + (dst * s)[mask != 0].sum()

    s, _ = rn.forward(x, res, w, eps, kept, mask)
    got = dict(zip(("res", "x", "w"), rn.backward(do, dst, s, w, eps, kept, mask)))
    h = 1e-6
    for name, a in (("x", x), ("res", res), ("w", w)):
        for i in np.ndindex(a.shape):
            lo, hi = a.copy(), a.copy()
            lo[i] -= h
            hi[i] += h
            args = {"x": x, "res": res, "w": w}
            d = (loss(**{**args, name: hi}) - loss(**{**args, name: lo})) / (2 * h)
            assert abs(got[name][i] - d) < 1e-7 * (1 + abs(d))


def test_row_scales():
    n = np.array([[0.0, 0.0], [448.0, -1.0], [1e-3, 2e-3]])
    codes, scale = rn.row_quantize(n)
    assert scale[0] == 2.0 ** -120 and scale[1] == 1.0 and np.isclose(scale[2], 2e-3 / 448)
    assert list(codes[0]) == [0, 0] and codes[1][0] == 0x7E and codes[2][1] == 0x7E
