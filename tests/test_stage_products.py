"""What tells the two ways of multiplying in 8 bits apart, on the CPU: sums of
cut products (oracle.stage.cut_products) in the place of exact ones fail on the
inputs that the GPU tests of fp32 outputs use."""
import numpy as np

from oracle import stage


def test_cut_products_by_hand():
    a, b = np.zeros((1, 16)), np.zeros((1, 16))
    a[0, :3], b[0, :3] = [256, 256, 3], [256, -256, 4]
    assert stage.cut_products(a, b) == 8           # 12 to a multiple of 2^(16 - 13)
    b[0, 2] = -4
    assert stage.cut_products(a, b) == -8          # towards zero
    a[0, 9], b[0, 9] = 3, 4
    assert stage.cut_products(a, b) == 4           # the next 8 columns have a largest of their own
    assert stage.cut_products(np.zeros((2, 8)), np.ones((3, 8))).any() == False  # noqa: E712


def test_cut_products_are_within_their_bound():
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((20, 64)), rng.standard_normal((30, 64))
    p = a[:, None, :] * b[None, :, :]
    top = np.abs(p).reshape(20, 30, 8, 8).max(axis=3).sum(axis=2)
    err = np.abs(stage.cut_products(a, b) - a @ b.T)
    assert (err <= 8 * 2.0 ** -13 * top).all() and err.max() > 0


def test_small_terms_beside_cancelling_large_ones_show_a_cut():
    rng = np.random.default_rng(1)
    M, N, K = 20, 30, 200
    a, b = rng.integers(-8, 9, (M, K)) / 8, rng.integers(-4, 5, (N, K)) / 4
    a[:, 0::8] = a[:, 1::8] = b[:, 0::8] = 256.0
    b[:, 1::8] = -256.0
    exact = a @ b.T
    # every small term lies below 2^(16 - 13): all of them are lost
    assert not stage.cut_products(a, b).any()
    assert (exact != 0).mean() > 0.9
    # and no fp32 partial sum rounds: a running sum in fp32, in order
    s = np.zeros((M, N), dtype=np.float32)
    for k in range(K):
        s += (a[:, k, None] * b[None, :, k]).astype(np.float32)
    assert np.array_equal(s, exact)


def test_the_cut_follows_the_exponents_not_the_product():
    a, b = np.zeros((1, 8)), np.zeros((1, 8))
    a[0, :3], b[0, :3] = [448, 448, 3], [448, -448, 4]  # 448 * 448 is 3.0625 * 2^16
    assert stage.cut_products(a, b) == 8
