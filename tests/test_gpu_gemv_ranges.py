"""nvfp4_gemv on rows and weights near the ends of fp32's range, whose products lie within it.  Tolerances are those of
test_gpu_gemv.py."""
import pytest
import torch

from tests.test_gpu_gemv import L, Weights, _check, _x  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,N,K", [(3, 64, 128), (8, 64, 14336), (16, 128, 4096)])
@pytest.mark.parametrize("x_log2,w_log2", [(118, 0), (118, -40), (-110, 110), (100, -110), (-60, 60)])
def test_ends_of_the_range(L, rows, N, K, x_log2, w_log2):  # noqa: F811
    W = Weights(1, N, K, seed=rows)
    W.ts[:, 2] *= 2.0 ** w_log2
    W.w *= 2.0 ** w_log2
    x = (_x(rows, K, rows).float() * 2.0 ** x_log2).bfloat16()
    assert x.isfinite().all()
    out = _check(L, W, x, rows, epi="f32")
    assert out.isfinite().all()
