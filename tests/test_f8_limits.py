"""How large a block-scaled quantization or product may be: what the header promises
to take is not refused, through the C ABI and without a GPU (a workspace of none is
refused after the sizes are)."""
import pytest

import newton_schulz_03_amd as nsa
from newton_schulz_03_amd._binding import _i64_array, _ptr_array

FAKE = 0x7f0000000000
UNSUPPORTED, WORKSPACE = 2, 3
TOP = nsa.F8_MAX_DIM


def product(shapes):
    m, n = (_i64_array([s[i] for s in shapes]) for i in (0, 1))
    p = _ptr_array([FAKE] * len(shapes))
    return nsa.load_library().muon_f8_matmul_batched(len(shapes), m, n, _i64_array([128] * len(shapes)), p, p,
                                                     p, p, p, 0, 0, None, 0, None)


def quantize(shapes):
    rows, cols = (_i64_array([s[i] for s in shapes]) for i in (0, 1))
    p = _ptr_array([FAKE] * len(shapes))
    return nsa.load_library().muon_f8_quantize_batched(len(shapes), rows, cols, p, 0, 1, p, p, None, None, None,
                                                       0, None)


def cdiv(a, b):
    return -(-a // b)


# each just below 2^24 blocks of 16 x 64 outputs
FIT = [[(1, TOP)] * 1023, [(16, TOP)] * 1023, [(17, TOP)] * 511, [(1, TOP), (33, TOP)] * 255, [(TOP, 64)] * 255,
       [(TOP, 1)] * 255, [(4096, 4096)] * 1023, [(64, 65536)] * 4095, [(1, 1)] * 100000, [(TOP, 16320)]]


@pytest.mark.parametrize("shapes", FIT, ids=lambda s: f"{len(s)} of {s[0]}")
def test_products_that_fit(shapes):
    assert sum(cdiv(m, 16) * cdiv(n, 64) for m, n in shapes) < 1 << 24
    assert product(shapes) == WORKSPACE, nsa.last_error_detail()


def test_products_that_do_not():
    for shapes in ([(1, TOP)] * 4097, [(TOP, TOP)], [(17, TOP), (1, TOP)] * 2048):
        assert product(shapes) == UNSUPPORTED, shapes[0]
        assert "2^24" in nsa.last_error_detail()


def test_quantizations():
    assert quantize([(128, 128 * 8192)] * 2047) == WORKSPACE
    assert quantize([(1, TOP)] * 2047) == WORKSPACE
    assert quantize([(TOP, 2047 * 128)]) == WORKSPACE
    for shapes in ([(128, 128 * 8192)] * 2048, [(1, TOP)] * 2048, [(TOP, 2048 * 128)]):
        assert quantize(shapes) == UNSUPPORTED, shapes[0]
