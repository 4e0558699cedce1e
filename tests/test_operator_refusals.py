"""Arguments that the gradient norm, clip, scaled steps and block-scaled e4m3
entry points refuse, through the C ABI and the binding, without a GPU: every
call fails validation (or is the empty batch) before the library touches the
HIP runtime, so aligned pointers that are never dereferenced are enough."""
import ctypes
import math

import pytest
import torch

import newton_schulz_03_amd as nsa
from newton_schulz_03_amd._binding import (AdamWParams, GradNormParams, NsParams, StepParams,
                                           _i64_array, _ptr_array)

FAKE = 0x7f0000000000
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return nsa.load_library()


def _i32_array(vals):
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


def up(x, a):
    return (x + a - 1) // a * a


def params(kind=0, clip=1, max_norm=1.0, eps=1e-6):
    return GradNormParams(kind, clip, max_norm, eps)


def norm_call(lib, numels=(5, 7), g=None, dtype=None, p=None, result=FAKE, ws=FAKE, ws_bytes=1 << 20):
    n = len(numels)
    g = [FAKE + 4096 * i for i in range(n)] if g is None else g
    return lib.muon_grad_norm_batched(n, _i64_array(numels), _ptr_array(g),
                                      _i32_array([0] * n if dtype is None else dtype),
                                      ctypes.byref(params() if p is None else p), result, ws, ws_bytes,
                                      None)


def clip_call(lib, numels=(5, 7), g=None, dtype=None, out=None, out_dtype=None, p=None, result=FAKE,
              ws=FAKE, ws_bytes=1 << 20):
    n = len(numels)
    g = [FAKE + 4096 * i for i in range(n)] if g is None else g
    return lib.muon_grad_clip_batched(
        n, _i64_array(numels), _ptr_array(g), _i32_array([0] * n if dtype is None else dtype),
        _ptr_array(g if out is None else out),
        _i32_array([0] * n if out_dtype is None else out_dtype),
        ctypes.byref(params() if p is None else p), result, ws, ws_bytes, None)


def test_grad_workspace(lib):
    def want(n):
        return up(16 * (n + 1), 256) + up(8 * n, 256) + 8 * 2048

    for numels in ([], [0], [1], [5, 0, 16384 * 3 + 1], [7] * 300):
        assert nsa.grad_workspace_bytes(numels) == want(len(numels))
    with pytest.raises(nsa.MuonError):
        nsa.grad_workspace_bytes([-1])
    assert lib.muon_grad_workspace_bytes(-1, _i64_array([1])) == ctypes.c_size_t(-1).value
    assert lib.muon_grad_workspace_bytes(1, None) == ctypes.c_size_t(-1).value
    # more chunks than a launch can number
    assert lib.muon_grad_workspace_bytes(2, _i64_array([1 << 45, 1])) == ctypes.c_size_t(-1).value
    assert lib.muon_grad_workspace_bytes(1, _i64_array([(1 << 63) - 1])) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("call", [norm_call, clip_call])
def test_norm_and_clip_refusals(lib, call):
    assert call(lib, numels=(5, -1)) == INVALID
    assert call(lib, g=[FAKE, 0]) == INVALID
    assert call(lib, g=[FAKE, FAKE + 8]) == INVALID
    assert call(lib, dtype=[0, 2]) == INVALID
    for bad in (params(kind=2), params(kind=-1), params(clip=2), params(max_norm=-1.0),
                params(max_norm=math.inf), params(max_norm=math.nan), params(eps=-1.0),
                params(eps=math.nan)):
        assert call(lib, p=bad) == INVALID
    assert call(lib, result=0) == INVALID
    assert call(lib, result=FAKE + 2) == INVALID
    assert call(lib, ws=0) == WORKSPACE
    assert call(lib, ws_bytes=nsa.grad_workspace_bytes([5, 7]) - 1) == WORKSPACE
    assert call(lib, ws=FAKE + 128) == INVALID
    assert "256-byte" in nsa.last_error_detail()
    assert call(lib, numels=(1 << 45, 1)) == UNSUPPORTED


def test_clip_refusals(lib):
    assert clip_call(lib, p=params(clip=0)) == INVALID
    assert clip_call(lib, out=[FAKE, 0]) == INVALID
    assert clip_call(lib, out=[FAKE, FAKE + 4]) == INVALID
    assert clip_call(lib, out_dtype=[0, 5]) == INVALID
    assert clip_call(lib, out_dtype=[1, 0]) == INVALID  # in place, another type
    assert "in place" in nsa.last_error_detail()
    n, num = 2, _i64_array([5, 7])
    g, d = _ptr_array([FAKE, FAKE + 4096]), _i32_array([0, 0])
    p = params()
    assert lib.muon_grad_clip_batched(n, num, g, d, None, d, ctypes.byref(p), FAKE, FAKE, 1 << 20,
                                      None) == INVALID
    assert lib.muon_grad_clip_batched(n, num, g, d, g, None, ctypes.byref(p), FAKE, FAKE, 1 << 20,
                                      None) == INVALID
    assert lib.muon_grad_clip_batched(n, num, None, d, g, d, ctypes.byref(p), FAKE, FAKE, 1 << 20,
                                      None) == INVALID
    assert lib.muon_grad_clip_batched(n, num, g, d, g, d, None, FAKE, FAKE, 1 << 20, None) == INVALID


def test_scale_refusals(lib):
    def call(scale=FAKE, out=(FAKE, FAKE + 4096), odt=(0, 0), ws_bytes=1 << 20, batch=2):
        return lib.muon_grad_scale_batched(batch, _i64_array([5, 7]),
                                           _ptr_array([FAKE, FAKE + 4096]), _i32_array([0, 0]),
                                           None if out is None else _ptr_array(out),
                                           _i32_array(odt), scale, FAKE, ws_bytes, None)

    assert call(scale=0) == INVALID
    assert call(scale=FAKE + 1) == INVALID
    assert call(out=None) == INVALID
    assert call(out=(FAKE, 0)) == INVALID
    assert call(odt=(1, 0)) == INVALID
    assert call(ws_bytes=16) == WORKSPACE
    assert call(batch=-1) == INVALID
    assert call(batch=0) == OK


def test_scaled_steps_refuse_a_missing_factor(lib):
    one = _i64_array([16])
    p = [_ptr_array([FAKE + 4096 * i]) for i in range(4)]
    prm = AdamWParams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1)
    sp = StepParams(0.02, 0.95, 0, NsParams(5, 3.4445, -4.775, 2.0315, 1e-7, 0, 0), 0)
    for bad in (None, FAKE + 2):
        assert lib.muon_adamw_batched_scaled(1, one, *p, 0, ctypes.byref(prm), bad, FAKE, 1 << 20,
                                             None) == INVALID
        assert "grad_scale" in nsa.last_error_detail()
        assert lib.muon_step_batched_scaled(1, one, one, *p[:3], 0, ctypes.byref(sp), bad, FAKE,
                                            1 << 30, None) == INVALID
        assert "grad_scale" in nsa.last_error_detail()
    # the other checks are those of the plain calls
    assert lib.muon_adamw_batched_scaled(1, one, *p, 0, ctypes.byref(prm), FAKE, FAKE, 16,
                                         None) == WORKSPACE
    assert lib.muon_step_batched_scaled(1, one, one, *p[:3], 0, ctypes.byref(sp), FAKE, FAKE, 16,
                                        None) == WORKSPACE


def test_f8_workspace():
    for n in (0, 1, 7, 384):
        assert nsa.f8_workspace_bytes(n) == up(56 * n, 256) + up(4 * 4 * (n + 1), 256)
    with pytest.raises(nsa.MuonError):
        nsa.f8_workspace_bytes(-1)


def test_quantize_refusals(lib):
    def call(rows=(5,), cols=(7,), x=(FAKE,), dtype=0, br=1, q=(FAKE,), s=(FAKE,), qt=None, st=None,
             ws=FAKE, wsb=1 << 20, batch=1):
        arr = [None if v is None else _ptr_array(v) for v in (q, s, qt, st)]
        return lib.muon_f8_quantize_batched(batch, _i64_array(rows), _i64_array(cols), _ptr_array(x),
                                            dtype, br, *arr, ws, wsb, None)

    assert call(batch=-1) == INVALID
    assert call(batch=0) == OK
    assert call(dtype=2) == INVALID
    for br in (0, 2, 64, 129, -1):
        assert call(br=br) == INVALID
    assert call(q=None, s=None) == INVALID
    assert call(q=None) == INVALID
    assert call(qt=(FAKE,)) == INVALID
    assert call(rows=(-1,)) == INVALID
    assert call(cols=(-1,)) == INVALID
    assert call(rows=(nsa.F8_MAX_DIM + 1,)) == UNSUPPORTED
    assert call(cols=(nsa.F8_MAX_DIM + 1,)) == UNSUPPORTED
    assert call(rows=(1 << 40,)) == UNSUPPORTED
    # 2^26 tiles of 128 x 128: more threads than one launch holds
    assert call(rows=(nsa.F8_MAX_DIM,), cols=(nsa.F8_MAX_DIM,)) == UNSUPPORTED
    for bad in (0, FAKE + 8):
        assert call(x=(bad,)) == INVALID
        assert call(q=(bad,)) == INVALID
        assert call(s=(bad,)) == INVALID
        assert call(qt=(bad,), st=(FAKE,)) == INVALID
        assert call(qt=(FAKE,), st=(bad,)) == INVALID
    assert call(ws=0) == WORKSPACE
    assert call(wsb=511) == WORKSPACE
    assert call(ws=FAKE + 16) == INVALID


def test_matmul_refusals(lib):
    def call(m=(5,), n=(7,), k=(9,), a=(FAKE,), sa=(FAKE,), b=(FAKE,), sb=(FAKE,), c=(FAKE,),
             dtype=0, acc=0, ws=FAKE, wsb=1 << 20, batch=1):
        arr = [None if v is None else _ptr_array(v) for v in (a, sa, b, sb, c)]
        return lib.muon_f8_matmul_batched(batch, _i64_array(m), _i64_array(n), _i64_array(k), *arr,
                                          dtype, acc, ws, wsb, None)

    assert call(batch=-1) == INVALID
    assert call(batch=0) == OK
    assert call(dtype=7) == INVALID
    assert call(acc=2) == INVALID
    for dim in ("m", "n", "k"):
        assert call(**{dim: (-1,)}) == INVALID
        assert call(**{dim: (nsa.F8_MAX_DIM + 1,)}) == UNSUPPORTED
    assert call(m=(nsa.F8_MAX_DIM,), n=(nsa.F8_MAX_DIM,)) == UNSUPPORTED
    for arr in ("a", "sa", "b", "sb", "c"):
        assert call(**{arr: None}) == INVALID
        assert call(**{arr: (0,)}) == INVALID
        assert call(**{arr: (FAKE + 8,)}) == INVALID
    assert call(ws=0) == WORKSPACE
    assert call(wsb=511) == WORKSPACE
    assert call(ws=FAKE + 16) == INVALID


def test_binding_refusals():
    cpu = [torch.zeros(4)]
    with pytest.raises(ValueError):
        nsa.grad_norm_batched(cpu)
    with pytest.raises(ValueError):
        nsa.grad_norm_batched([])
    with pytest.raises(ValueError):
        nsa.grad_norm_batched(cpu, norm_type=1)
    with pytest.raises(ValueError):
        nsa.grad_clip_batched(cpu, None)
    with pytest.raises(ValueError):
        nsa.grad_clip_batched(cpu, 1.0)
    with pytest.raises(ValueError):
        nsa.grad_scale_batched(cpu, torch.ones(1))
    assert nsa.grad_scale_batched([], torch.ones(1)) == []
    with pytest.raises(ValueError):
        nsa.f8_quantize_batched([torch.zeros(2, 3)])
    with pytest.raises(ValueError):
        nsa.f8_quantize_batched([torch.zeros(2, 3)], normal=False)
    assert nsa.f8_quantize_batched([]) == []
    assert nsa.f8_quantize_batched([], transpose=True) == ([], [])
    op = nsa.f8_empty(3, 200, "cpu")
    assert op.q.shape == (3, 256) and op.scales.shape == (2, 16)
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched([op], [op])
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched([op], [])
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched([op], [op], accumulate=True)
    assert nsa.f8_matmul_batched([], []) == []
