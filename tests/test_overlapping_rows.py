"""Outputs of the expert layers' operators that share memory with what the call reads
are refused, wherever in it they begin; neighbours in one allocation are taken."""
import pytest
import torch

import newton_schulz_03_amd as nsa

FAKE = 0x7f0000000000
INVALID = 1
T, K, C, N = 6, 2, 40, 12  # tokens, choices, columns, sorted rows: rows of 80 bytes (bf16)


def at(i):
    return FAKE + (i << 20)


def refused(status):
    return status == INVALID and "another buffer" in nsa.last_error_detail()


@pytest.mark.parametrize("off", [-T * C * 2 + 16, -16, 0, 16, 160, N * C * 2 - 16])
def test_sorted_rows_beside_tokens(off):
    """A sorted rows' buffer N rows long, at `off` ... from a tokens' buffer of T rows."""
    lib = nsa.load_library()
    tokens, rows = at(1) + off, at(1)
    assert refused(lib.muon_moe_dispatch(T, K, C, tokens, at(2), N, rows, 0, None))
    assert refused(lib.muon_moe_combine(T, K, C, N, rows, at(2), at(3), tokens, 0, None))
    assert refused(lib.muon_moe_combine_backward(T, K, C, tokens, N, at(4), at(2), at(3), rows, at(5), 0, None))


@pytest.mark.parametrize("off", [-N * C * 2 + 16, -16, 0, 16, N * C * 2 - 16])
def test_gradient_rows_and_weights(off):
    lib = nsa.load_library()
    assert refused(lib.muon_moe_combine_backward(T, K, C, at(0), N, at(1) + off, at(2), at(3), at(1), at(5), 0, None))
    for w in (-T * K * 4 + 4, -4, 0, 4, T * K * 4 - 4):
        assert refused(lib.muon_moe_combine_backward(T, K, C, at(0), N, at(4), at(2), at(3) + w, at(1), at(3), 0,
                                                     None))


@pytest.mark.parametrize("off", [-3 * 40 * 2 + 16, 0, 16, 3 * 20 * 4 - 16])
def test_product(off):
    """3 rows of 40 bf16, 3 of 20 fp32."""
    lib = nsa.load_library()
    assert refused(lib.muon_f4_matmul(1, 20, 40, at(0), at(1), 3, at(2) + off, 3, None, None, None, 1, at(2), 1, None))


@pytest.mark.gpu
def test_neighbours():
    ids = torch.tensor([[0, 1], [2, 0], [1, 2], [1, 0]], dtype=torch.int32, device="cuda")
    plan = nsa.moe_sort(ids, 3)
    for order in (0, 1):  # the tokens' rows first, then the sorted ones, and the other way round
        def pair(rows):
            buf = torch.zeros((4 + rows, 40), device="cuda").bfloat16()
            return (buf[:4], buf[4:]) if order == 0 else (buf[rows:], buf[:rows])

        x, xs = pair(8)
        x.copy_(torch.randn(4, 40))
        nsa.moe_dispatch(x, plan, out=xs)
        assert torch.equal(xs, nsa.moe_dispatch(x.clone(), plan))
        out, ys = pair(8)
        ys.copy_(torch.randn(8, 40))
        nsa.moe_combine(ys, plan, out=out)
        assert torch.equal(out, nsa.moe_combine(ys.clone(), plan))
        dout, dys = pair(8)
        dout.copy_(torch.randn(4, 40))
        both = torch.rand((8, 2), device="cuda")
        w, dw = both[4 * order:4 * order + 4], both[4 - 4 * order:8 - 4 * order]
        nsa.moe_combine_backward(dout, ys, plan, w, dys=dys, dweights=dw)
        want = nsa.moe_combine_backward(dout.clone(), ys, plan, w)
        assert torch.equal(dys, want[0]) and torch.equal(dw, want[1])
    op = nsa.f4_quantize([torch.randn((40, 40), device="cuda")])
    buf = torch.randn((6, 40), device="cuda").bfloat16()
    x = buf[:3]
    want = nsa.f4_matmul(x, op)
    assert torch.equal(nsa.f4_matmul(x, op, out=buf[3:]), want)
    with pytest.raises(nsa.MuonError, match="another buffer"):
        nsa.f4_matmul(buf[:4], op, out=buf[2:])
