"""Arguments that the token sort, dispatch, combine, dropout and the 4-bit weights refuse,
through the C ABI and the binding, without a GPU: every call fails validation (or
has nothing to do) before the library touches the HIP runtime, so aligned
pointers that are never dereferenced are enough."""
import ctypes
import math

import pytest
import torch

import newton_schulz_03_amd as nsa
from newton_schulz_03_amd._binding import DropoutParams, _i64_array, _ptr_array

FAKE = 0x7f0000000000
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
MAX = ctypes.c_size_t(-1).value
SLOTS = nsa.MOE_MAX_SLOTS


@pytest.fixture(scope="module")
def lib():
    return nsa.load_library()


def at(i):
    return FAKE + (i << 20)


def test_workspaces(lib):
    assert nsa.f4_workspace_bytes(1) == 256 and nsa.f4_workspace_bytes(384) == 8 * 384
    assert lib.muon_f4_workspace_bytes(0) == MAX
    assert lib.muon_f4_workspace_bytes(nsa.MOE_MAX_EXPERTS + 1) == MAX
    for bad in ((-1, 8, 4), (1, 0, 4), (1, nsa.MOE_MAX_TOP_K + 1, 4), (1, 8, 0),
                (1, 8, nsa.MOE_MAX_EXPERTS + 1), (SLOTS // 8 + 1, 8, 4), (1 << 62, 8, 4)):
        assert lib.muon_moe_workspace_bytes(*bad) == MAX
        with pytest.raises(nsa.MuonError):
            nsa.moe_workspace_bytes(*bad)
    with pytest.raises(nsa.MuonError):
        nsa.f4_workspace_bytes(0)
    assert nsa.moe_workspace_bytes(0, 1, 1) >= 0


def test_sort_refusals(lib):
    def call(t=5, k=2, e=4, ids=at(0), size=4, o=at(1), a=at(2), r=at(3), s=at(4), ws=at(5), wsb=1 << 30):
        return lib.muon_moe_sort(t, k, e, ids, size, o, a, r, s, ws, wsb, None)

    assert call(t=-1) == INVALID
    assert call(k=0) == INVALID
    assert call(k=nsa.MOE_MAX_TOP_K + 1) == UNSUPPORTED
    assert call(t=SLOTS // 2 + 1) == UNSUPPORTED
    assert call(e=0) == INVALID
    assert call(e=nsa.MOE_MAX_EXPERTS + 1) == UNSUPPORTED
    for size in (0, 2, 16):
        assert call(size=size) == INVALID
    assert call(size=8, ids=at(0) + 4) == INVALID
    for name in ("ids", "o", "a", "r", "s"):
        for bad in (0, FAKE + 2):
            assert call(**{name: bad}) == INVALID
    # a long list needs its workspace
    n = nsa.moe_workspace_bytes(SLOTS // 2, 2, 4)
    if n > 0:
        assert call(t=SLOTS // 2, ws=0) == WORKSPACE
        assert call(t=SLOTS // 2, wsb=n - 1) == WORKSPACE
        assert call(t=SLOTS // 2, ws=at(5) + 16) == INVALID


def test_row_refusals(lib):
    def dispatch(t=5, k=2, c=8, x=at(0), r=at(1), n=10, out=at(2), dt=0):
        return lib.muon_moe_dispatch(t, k, c, x, r, n, out, dt, None)

    def combine(t=5, k=2, c=8, n=10, x=at(0), r=at(1), w=at(3), out=at(2), dt=0):
        return lib.muon_moe_combine(t, k, c, n, x, r, w, out, dt, None)

    def backward(t=5, k=2, c=8, d=at(4), n=10, x=at(0), r=at(1), w=at(3), out=at(2), dw=at(5), dt=0):
        return lib.muon_moe_combine_backward(t, k, c, d, n, x, r, w, out, dw, dt, None)

    for call in (dispatch, combine, backward):
        assert call(t=-1) == INVALID
        assert call(k=0) == INVALID
        assert call(k=nsa.MOE_MAX_TOP_K + 1) == UNSUPPORTED
        assert call(t=SLOTS) == UNSUPPORTED
        assert call(c=-1) == INVALID
        assert call(c=nsa.F8_MAX_DIM + 1) == UNSUPPORTED
        assert call(n=-1) == INVALID
        assert call(n=SLOTS + 1) == UNSUPPORTED
        assert call(dt=2) == INVALID
        for name in ("x", "out"):
            for bad in (0, FAKE + 8):
                assert call(**{name: bad}) == INVALID
        for bad in (0, FAKE + 2):
            assert call(r=bad) == INVALID
        assert call(out=at(0)) == INVALID
        assert "another buffer" in nsa.last_error_detail()
    assert combine(w=FAKE + 2) == INVALID
    for bad in (0, FAKE + 2):
        assert backward(w=bad) == INVALID
        assert backward(dw=bad) == INVALID
    for bad in (0, FAKE + 8):
        assert backward(d=bad) == INVALID
    assert backward(out=at(4)) == INVALID
    assert backward(dw=at(3)) == INVALID
    # nothing to do
    for call in (dispatch, combine):
        assert call(t=0, x=0, r=0, out=0, n=0) == OK
        assert call(c=0, x=0, out=0) == OK
    assert dispatch(n=0, out=0) == OK
    assert backward(t=0, d=0, x=0, r=0, w=0, out=0, dw=0, n=0) == OK


def test_dropout_refusals(lib):
    def call(n=(5, 7), x=(at(0), at(1)), dt=(0, 1), out=(at(2), at(3)), odt=(0, 1), p=0.5, rng=0,
             ws=at(4), wsb=1 << 20, batch=2, params=True):
        i32 = ctypes.c_int32 * 2
        prm = DropoutParams(p, 1, 2)
        return lib.muon_dropout_batched(batch, _i64_array(n), None if x is None else _ptr_array(x), i32(*dt),
                                        None if out is None else _ptr_array(out), i32(*odt),
                                        ctypes.byref(prm) if params else None, rng, ws, wsb, None)

    assert call(batch=-1) == INVALID
    assert call(batch=0) == OK
    assert call(params=False) == INVALID
    for p in (-0.1, 1.0001, math.nan, math.inf):
        assert call(p=p) == INVALID
    assert call(rng=FAKE + 4) == INVALID
    assert call(n=(5, -1)) == INVALID
    assert call(n=(5, 1 << 35)) == UNSUPPORTED
    assert call(n=(5, (1 << 35) - 1), wsb=16) == WORKSPACE
    assert call(x=None) == INVALID
    assert call(out=None) == INVALID
    assert call(dt=(0, 2)) == INVALID
    assert call(odt=(3, 1)) == INVALID
    for bad in (0, FAKE + 8):
        assert call(x=(at(0), bad)) == INVALID
        assert call(out=(bad, at(1))) == INVALID
    assert call(out=(at(0), at(1)), odt=(1, 1)) == INVALID  # in place, another type
    assert call(ws=0) == WORKSPACE
    assert call(wsb=nsa.grad_workspace_bytes([5, 7]) - 1) == WORKSPACE
    assert call(ws=at(4) + 16) == INVALID


def test_f4_quantize_refusals(lib):
    def call(count=2, r=5, c=7, w=(at(0), at(1)), dt=0, tr=0, q=at(2), s=at(3), ws=at(4), wsb=1 << 20):
        return lib.muon_f4_quantize(count, r, c, None if w is None else _ptr_array(w), dt, tr, q, s, ws, wsb,
                                    None)

    assert call(count=0) == INVALID
    assert call(count=nsa.MOE_MAX_EXPERTS + 1) == UNSUPPORTED
    for dim in ("r", "c"):
        assert call(**{dim: -1}) == INVALID
        assert call(**{dim: nsa.F8_MAX_DIM + 1}) == UNSUPPORTED
    assert call(r=nsa.F8_MAX_DIM, c=nsa.F8_MAX_DIM) == UNSUPPORTED  # 2^29 tiles
    assert call(dt=2) == INVALID
    assert call(tr=2) == INVALID
    assert call(w=None) == INVALID
    for bad in (0, FAKE + 8):
        assert call(w=(at(0), bad)) == INVALID
        assert call(q=bad) == INVALID
        assert call(s=bad) == INVALID
    assert call(ws=0) == WORKSPACE
    assert call(wsb=255) == WORKSPACE
    assert call(ws=at(4) + 16) == INVALID
    assert call(r=0, w=None, q=0, s=0) == OK
    assert call(c=0, w=None, q=0, s=0) == OK


def test_f4_matmul_refusals(lib):
    def call(count=2, r=5, c=7, q=at(0), s=at(1), m=3, x=at(2), xr=3, o=at(3), a=at(4), sl=0, k=1,
             y=at(5), dt=0):
        return lib.muon_f4_matmul(count, r, c, q, s, m, x, xr, o, a, sl, k, y, dt, None)

    assert call(count=0) == INVALID
    assert call(count=nsa.MOE_MAX_EXPERTS + 1) == UNSUPPORTED
    for dim in ("r", "c"):
        assert call(**{dim: -1}) == INVALID
        assert call(**{dim: nsa.F8_MAX_DIM + 1}) == UNSUPPORTED
    assert call(r=nsa.F8_MAX_DIM, c=nsa.F8_MAX_DIM) == UNSUPPORTED
    for dim in ("m", "xr"):
        assert call(**{dim: -1}) == INVALID
        assert call(**{dim: SLOTS + 1}) == UNSUPPORTED
    assert call(dt=2) == INVALID
    assert call(o=0) == INVALID
    assert call(a=0) == INVALID
    assert call(o=0, a=0) == INVALID  # two matrices
    assert call(count=1, o=0, a=0, sl=at(6)) == INVALID
    assert call(xr=2) == INVALID
    assert call(sl=at(6), xr=0) == INVALID
    for k in (0, -1, nsa.MOE_MAX_TOP_K + 1):
        assert call(sl=at(6), k=k) == INVALID
    for name in ("o", "a", "sl"):
        assert call(**{name: FAKE + 2}) == INVALID
    for name in ("q", "s", "x", "y"):
        for bad in (0, FAKE + 8):
            assert call(**{name: bad}) == INVALID
    assert call(y=at(2)) == INVALID
    assert call(m=0, x=0, y=0, xr=0) == OK
    assert call(r=0, q=0, s=0, y=0) == OK


def test_binding_refusals():
    ids = torch.zeros((2, 2), dtype=torch.int32)
    plan = nsa.moe_empty_plan(2, 2, 3, "cpu")
    assert [tuple(t.shape) for t in plan] == [(4,), (4,), (2, 2), (4,)]
    x = torch.zeros((2, 8))
    w = nsa.f4_empty(1, 16, 128, "cpu")
    assert w.q.shape == (1, 1, 1, 64, 16) and w.scales.shape == (1, 1, 1, 16, 16)
    assert nsa.f4_empty(3, 17, 1000, "cpu").q.shape == (3, 2, 8, 64, 16)
    for call in (lambda: nsa.moe_sort(ids, 3), lambda: nsa.moe_dispatch(x, plan),
                 lambda: nsa.moe_combine(x, plan), lambda: nsa.moe_combine_backward(x, x, plan, x),
                 lambda: nsa.dropout_batched([x], 0.5), lambda: nsa.f4_quantize([x]),
                 lambda: nsa.f4_quantize([]), lambda: nsa.f4_quantize([x, x[:1]]),
                 lambda: nsa.f4_matmul(x.bfloat16(), w),
                 lambda: nsa.dropout_batched([x], 0.5, seed=-1),
                 lambda: nsa.dropout_batched([x], 0.5, offset=1 << 64),
                 lambda: nsa.dropout_batched([x], 0.5, seed=1, rng=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    assert nsa.dropout_batched([], 0.5) == []


def test_sizes_of_a_plan():
    plan = nsa.MoePlan(torch.tensor([0, 2, 2, 5], dtype=torch.int32), None, None, None)
    assert plan.sizes() == [2, 0, 3]
