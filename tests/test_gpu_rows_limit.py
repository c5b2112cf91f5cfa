"""The producer kernels at the largest token count, where a row index and the step to the
next row add up past 2^31 (about 112 GB of device memory)."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, H, TAIL = 2 ** 31 - 1, 16, 8192


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB of free device memory")
    yield
    torch.cuda.empty_cache()


def _check(A, s, want_A, want_s):
    assert torch.equal(A[T - TAIL:], want_A) and torch.equal(s[T - TAIL:], want_s)
    assert torch.equal(A[:TAIL], want_A.flip(0)) and torch.equal(s[:TAIL], want_s.flip(0))
    step = T // 7
    for i in range(step, T - TAIL, step):                          # rows of zeros between
        assert not bool(A[i: i + 99].any()) and bool((s[i: i + 99] == 1.0).all())


def test_row_quantize_at_the_limit(room):
    tail = torch.randn(TAIL, H, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    want_A, want_s, _ = lib.qkv_cte_row_quantize(tail)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[T - TAIL:], x[:TAIL] = tail, tail.flip(0)
    A, s, _ = lib.qkv_cte_row_quantize(x)
    _check(A, s, want_A, want_s)


def test_unpack_rows_at_the_limit(room):
    tail = torch.randint(0, 256, (TAIL, H + 4), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV,
                         dtype=torch.int32).to(torch.uint8)
    tail[:, H:] = torch.rand(TAIL, device=DEV).view(torch.uint8).view(TAIL, 4)
    want_A, want_s = lib.qkv_cte_unpack_rows(tail)
    packed = torch.zeros(T, H + 4, dtype=torch.uint8, device=DEV)
    packed[:, H + 2], packed[:, H + 3] = 0x80, 0x3F                # the scale 1.0
    packed[T - TAIL:], packed[:TAIL] = tail, tail.flip(0)
    A, s = lib.qkv_cte_unpack_rows(packed)
    _check(A, s, want_A, want_s)
