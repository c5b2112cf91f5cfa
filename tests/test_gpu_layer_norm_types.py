"""Layer norm of fp16 rows with fp32 parameters, both passes (the other pairs of types are
in test_gpu_layer_norm.py, whose references and tolerances these use)."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from test_gpu_layer_norm import SHAPES, _check_backward, _check_forward, _inputs, _saved

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_fp16_rows_fp32_parameters(rows, cols):
    x, w, b, _ = _inputs(rows, cols, torch.float16, torch.float32, rows * 31 + cols)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, w, b, eps=1e-5, stats=True)
    assert y.dtype == torch.float16
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("rows,cols", SHAPES + [(2000, 96), (5000, 8)])
def test_backward_fp16_rows_fp32_parameters(rows, cols):
    x, w, _, dy = _inputs(rows, cols, torch.float16, torch.float32, rows * 17 + cols)
    mean, rstd = _saved(x)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.dtype == torch.float16 and dw.dtype == db.dtype == torch.float32
    _check_backward(dy, x, mean, rstd, w, dx, dw, db)
