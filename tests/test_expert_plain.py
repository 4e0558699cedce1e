"""The plain forms that the GPU tests compare with, against published and worked values."""
import numpy as np

import expert_plain as plain


def test_philox_published_values():
    """Known answers that come with the generator's paper: counter and key 0, and all ones."""
    words = lambda c, k, r: ["%08x" % int(w) for w in plain.philox(c, k, r)]
    assert words([0] * 4, (0, 0), 10) == ["6627e8d5", "e169c58d", "bc57ac4c", "9b00dbd8"]
    m = 0xFFFFFFFF
    assert words([m] * 4, (m, m), 10) == ["408f276d", "41c83b0e", "a20bc7c6", "6d5451fd"]


def test_share_that_stays():
    # 2^20 draws, keep probability q: five standard deviations of the share
    n = 1 << 20
    for threshold in (0, 6554, 32768, 65535, 65536):
        q = 1 - threshold / 65536
        share = plain.keep(n, 3, 12345, 678, threshold).mean()
        assert abs(share - q) <= 5 * (q * (1 - q) / n) ** 0.5


def test_masks_differ_by_each_number():
    base = plain.keep(4096, 0, 1, 1, 32768)
    for args in ((1, 1, 1), (0, 2, 1), (0, 1, 2), (0, 1 + (1 << 32), 1), (0, 1, 1 + (1 << 32))):
        assert abs((plain.keep(4096, *args, 32768) == base).mean() - 0.5) < 5 * 0.5 / 64


def test_e2m1_nearest_and_ties():
    x = [0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, -0.75, -0.1, 0.0]
    assert plain.e2m1(np.array(x)).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 10, 8, 0]


def test_plan_worked():
    o, a, r, s = plain.plan([[2, 0], [-1, 2], [0, 5]], 4)
    assert o.tolist() == [0, 2, 2, 4, 4]
    assert a.tolist() == [2, 0, 2, -1, -1]
    assert r.tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert s.tolist() == [1, 4, 0, 3, -1, -1]


def test_f4_scales():
    w = np.zeros((1, 130))
    w[0, 0], w[0, 32], w[0, 64], w[0, 96] = 6.0, 6.0001, 2.0 ** -140, np.inf
    w[0, 128] = 3e38
    codes, scales = plain.f4(w)
    assert scales[0].tolist() == [127, 128, 2, 255, 252, 2, 2, 2]
    assert codes[0, [0, 32, 64, 96, 128]].tolist() == [7, 5, 0, 0, 7]
