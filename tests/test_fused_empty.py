"""Calls of the fused products without rows, columns or a sum, as the header says."""
import pytest

from test_fused_abi import DEQUANT, FAKE, GATED, GATED_GRAD, INV, LINEAR, LINEAR_GRAD, OK, QUANT, call


@pytest.mark.parametrize("fn,args", [("qgemm_a8w8_linear", LINEAR), ("qgemm_a8w8_gated", GATED)])
def test_products(fn, args):
    for kw in (dict(M=0), dict(N=0), dict(M=0, N=0), dict(M=0, K=0), dict(N=0, K=0)):
        assert call(fn, args, kw) == OK
    assert call(fn, args, dict(K=0)) == INV


@pytest.mark.parametrize("fn,args", [("qgemm_a8w8_linear_grad", LINEAR_GRAD), ("qgemm_a8w8_gated_grad", GATED_GRAD)])
def test_gradients(fn, args):
    for kw in (dict(M=0), dict(M=0, N=0), dict(M=0, K=0), dict(M=0, N=0, K=0)):
        assert call(fn, args, kw) == OK
    for kw in (dict(K=0), dict(N=0), dict(N=0, K=0)):
        assert call(fn, args, kw) == INV
        if fn == "qgemm_a8w8_linear_grad":
            assert call(fn, args, dict(kw, db=FAKE)) == INV
    assert call("qgemm_a8w8_linear_grad", LINEAR_GRAD, dict(M=0, N=0, db=FAKE)) == OK


@pytest.mark.parametrize("fn,args", [("int8_quantize", QUANT), ("int8_dequantize", DEQUANT)])
def test_quantisers(fn, args):
    for block, lds in ((0, 1), (32, 2)):
        assert call(fn, args, dict(M=0, block=block, lds=lds)) == OK
        for m in (0, 4):
            assert call(fn, args, dict(M=m, n=0, block=block, lds=lds)) == INV
