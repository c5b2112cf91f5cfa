"""CPU checks of the block operators' binding: what it refuses before the library sees it."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as pkg
from rope_tcgen05_mxfp8_gb300 import build as b


@pytest.fixture(scope="module", autouse=True)
def _built():
    b.build()


def test_binding_refuses_transposed_shapes():
    """Shapes whose elements would be read in another order (checked before any address)."""
    i32 = dict(dtype=torch.int32)
    rope = pkg.QkvCteRopeAxes(24, (8, 8, 8))
    host = torch.device("cpu")
    ok = rope._where(2, 10, torch.zeros(10, 3, **i32), None, host)
    assert ok[1] == 0 and rope._where(2, 10, torch.zeros(2, 10, 3, **i32), None, host)[1] == 30
    assert rope._where(2, 10, torch.zeros(30, **i32), None, host)[1] == 0
    for bad in ((3, 10), (1, 30), (10, 2, 3), (2, 3, 10), (3, 10, 1)):
        with pytest.raises(ValueError):
            rope._where(2, 10, torch.zeros(*bad, **i32), None, host)
    rope._where(2, 10, None, torch.zeros(2, 3, **i32), host)
    rope._where(2, 10, None, torch.zeros(6, **i32), host)
    with pytest.raises(ValueError):
        rope._where(2, 10, None, torch.zeros(3, 2, **i32), host)
    one = pkg.QkvCteRopeAxes(8, (8,))                    # one axis: no order to mistake
    assert one._where(1, 10, torch.zeros(1, 10, **i32), None, host)[1] == 0
    with pytest.raises(ValueError, match="CUDA"):
        rope.tables(1, 10, positions=torch.zeros(10, 3, **i32))


def test_numbers_beyond_the_c_types_are_refused():
    """ctypes keeps the low 32 bits of a number: 2^32 + 64 columns are not 64."""
    big = 2 ** 32
    calls = [lambda: pkg.qkv_cte_layer_norm_backward_workspace(8, big + 64),
             lambda: pkg.qkv_cte_layer_norm_backward_workspace(2 ** 64 + 8, 64),
             lambda: pkg.QkvCteRopeAxes(big + 8, (8,)), lambda: pkg.QkvCteRopeAxes(8, (big + 8,)),
             lambda: pkg.QkvCteRopeAxes(8, (8,), spectrum=big), lambda: pkg.QkvCteRopeAxes(8, (8,), pairing=-big),
             lambda: pkg.QkvCteLinear(4, big + 64, 32), lambda: pkg.QkvCteLinear(4, 64, big + 32),
             lambda: pkg.QkvCteLinear(2 ** 64 + 4, 64, 32), lambda: pkg.QkvCteLinear(4, 64, 32, act=big),
             lambda: pkg.QkvCteLinear(4, 64, 32, flags=big), lambda: pkg.QkvCteLinear(4, 64, 32, input_layout=big)]
    for call in calls:
        with pytest.raises(pkg.QkvCteError) as ei:
            call()
        assert ei.value.code == pkg.QKV_CTE_ERR_UNSUPPORTED
