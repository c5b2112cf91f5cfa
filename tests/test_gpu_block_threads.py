"""The layer norm from two host threads that share a GPU and nothing else: each thread's
widths use the same kernels with different amounts of shared memory."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from test_gpu_layer_norm import _check_backward, _check_forward, _inputs, _saved

pytestmark = pytest.mark.gpu


def _forward(cols, p):
    x, w, b, _ = _inputs(3, cols, torch.bfloat16, p, cols)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, w, b, eps=1e-5, stats=True)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


def _backward(cols, p):
    x, w, _, dy = _inputs(9, cols, torch.bfloat16, p, cols)
    mean, rstd = _saved(x)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy, x, mean, rstd, w)
    _check_backward(dy, x, mean, rstd, w, dx, dw, db)


# pairs of widths of one kernel each, both above the 48 KB every kernel may use:
# whole 16-byte rows, and rows off 16-byte boundaries
@pytest.mark.parametrize("run,wide,narrow", [(_forward, 32768, 24576), (_forward, 8191, 7001),
                                             (_backward, 8192, 5120), (_backward, 8191, 5001)])
@pytest.mark.parametrize("p", [torch.bfloat16, torch.float32])
def test_two_threads_alternate_two_widths(run, wide, narrow, p):
    with ThreadPoolExecutor(1) as a, ThreadPoolExecutor(1) as b:
        for _ in range(2):
            a.submit(run, wide, p).result()
            b.submit(run, narrow, p).result()
        a.submit(run, narrow, p).result()
        b.submit(run, wide, p).result()
        a.submit(run, wide, p).result()


def test_two_threads_at_once():
    def loop(widths):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            for cols in widths * 4:
                _forward(cols, torch.float32)
                _backward(cols, torch.float32)

    with ThreadPoolExecutor(2) as pool:
        for f in [pool.submit(loop, [8192, 5120, 8191]), pool.submit(loop, [5120, 8192, 5001])]:
            f.result()
