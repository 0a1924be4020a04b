"""Pins of the MXFP4 and dropout oracle (oracle/mx.py) against independent
restatements: exact rationals, published generator vectors, the storage rule
byte by byte, and finite differences."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx as O

LEVELS = [Fraction(n, 2) for n in (0, 1, 2, 3, 4, 6, 8, 12)]


def _brute_block(block):
    """(codes, byte) of 32 exact rationals by search."""
    m = max(abs(v) for v in block)
    b = 0
    if m > 0:
        e = -400
        while Fraction(2) ** (e + 1) <= m:
            e += 1
        b = max(e - 2 + 127, 0)
    scale = Fraction(2) ** (b - 127)
    codes = []
    for v in block:
        a = abs(v) / scale
        best = min(range(8), key=lambda i: (abs(a - LEVELS[i]), i % 2))
        codes.append(best + (8 if v < 0 else 0))
    return codes, b


@pytest.mark.parametrize("std", [1e-40, 1e-3, 1.0, 1e30])
def test_quantise_against_exact_rationals(std):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4, 64)) * std).astype(np.float32)
    x[1, :32] = 0
    codes, s = O.mx_quantize(x)
    for r in range(4):
        for b in range(2):
            want, byte = _brute_block([Fraction(float(v)) for v in x[r, 32 * b:32 * b + 32]])
            assert s[r, b] == byte
            got = [int(c) for c in codes[r, 32 * b:32 * b + 32]]
            assert [c for c in got if c != 8] == [w for w, c in zip(want, got) if c != 8]  # 8: a rounded -0


def test_ties_go_to_the_even_code_and_large_values_saturate():
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 7.9, -5.0, -0.25]
    codes, s = O.mx_quantize(x)
    assert s[0, 0] == 127
    assert list(codes[0, :12]) == [6, 0, 2, 2, 4, 4, 6, 6, 7, 7, 14, 8]


def test_non_finite_block_is_nan_and_leaves_its_neighbour():
    x = np.ones((1, 64))
    x[0, 5] = np.inf
    codes, s = O.mx_quantize(x)
    v = O.mx_values(codes, s)
    assert list(s[0]) == [255, 125] and np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_scale_tiles_byte_by_byte():
    s = np.arange(130 * 5, dtype=np.int64).reshape(130, 5).astype(np.uint8)
    t = O.mx_tile_scales(s)
    assert t.size == 2 * 2 * 512
    for i in range(130):
        for j in range(5):
            tile = t[((i // 128) * 2 + j // 4) * 512:][:512]
            assert tile[(i % 128 % 32) * 16 + (i % 128 // 32) * 4 + j % 4] == s[i, j]


def test_generator_against_published_vectors():
    f = 0xFFFFFFFF
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for ctr, key, want in cases:
        assert tuple(int(v) for v in O.philox4x32(ctr, key)) == want


def test_dropout_keeps_the_right_share_and_masks_differ():
    n = 1 << 18
    for p in (0.0, 0.05, 0.5, 0.9):
        k = O.dropout_keep(n, p, 0x123456789ABCDEF0, 7)
        assert abs(k.mean() - (1 - p)) < 5 * np.sqrt(max(p * (1 - p), 1e-9) / n) + 2 ** -17
    a, b, c = (O.dropout_keep(4096, 0.5, s, o) for s, o in ((1, 0), (1, 1), (1 << 32, 0)))
    assert (a != b).any() and (a != c).any()
    assert np.array_equal(a[:1001], O.dropout_keep(1001, 0.5, 1, 0))


def test_linear_gradients_against_differences():
    """With quantisation taken as the identity the backward is the gradient
    of the forward: checked on values that MXFP4 holds exactly."""
    rng = np.random.default_rng(5)
    M, N, K, r, s = 3, 32, 32, 8, 0.5
    X = rng.choice(O.E2M1, (M, K)) * rng.choice([-1, 1], (M, K))
    X[:, 0] = 4.0
    dY = rng.choice(O.E2M1, (M, N)) * rng.choice([-1, 1], (M, N))
    dY[:, 0] = 6.0
    W = rng.choice(O.E2M1, (N, K))
    L1, L2 = rng.standard_normal((K, r)), rng.standard_normal((r, N))
    mask = O.dropout_keep(M * K, 0.25, 9, 1).reshape(M, K) * O.dropout_scale(0.25)

    def loss(X_, L1_, L2_):
        T = (X_ * mask) @ L1_
        return float(((X_ @ W.T + s * T @ L2_) * dY).sum())

    _, T = O.mx_linear_fwd(X, W, L1, L2, s, mask)
    dX, dL1, dL2 = O.mx_linear_bwd(dY, X, T, W.T, L1, L2, s, mask)
    eps = 1e-4
    for arr, grad, pos in ((X, dX, 0), (L1, dL1, 1), (L2, dL2, 2)):
        for _ in range(6):
            i = tuple(rng.integers(0, d) for d in arr.shape)
            args = [X.copy(), L1.copy(), L2.copy()]
            args[pos][i] += eps
            up = loss(*args)
            args[pos][i] -= 2 * eps
            assert abs((up - loss(*args)) / (2 * eps) - grad[i]) < 1e-6 * (1 + abs(grad[i]))
