"""rt_linear_int8_workspace looks at m, n and k each, not at m n (no GPU): on both
sides of the largest product it gives the same kind of size, and the call refuses
what lies above before anything runs."""
import pytest

from top_search_resident_amd import ResidentTopKError, _lib, linear_int8_workspace

P = 0x10000
LIMIT = 2 ** 37


@pytest.mark.parametrize("m,n", [(2 ** 20, 2 ** 17), (2 ** 20, 2 ** 17 + 1), (2 ** 20 + 1, 2 ** 17), (2 ** 31 - 1, 64),
                                 (2 ** 31 - 1, 65), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("k", [1, 777, 65536])
def test_products_on_both_sides_of_the_limit(m, n, k):
    lib = _lib.load()
    need = lib.rt_linear_int8_workspace(m, n, k)
    padded = (k + 127) // 128 * 128
    assert need == m * padded + (4 * m + 15) // 16 * 16 == linear_int8_workspace(m, n, k)
    fine = lib.rt_check_matmul_int8(P, k, P, P, k, P, None, P, _lib.RT_DTYPE_FLOAT32, n, m, n, k)
    assert fine == (_lib.RT_OK if m * n <= LIMIT else _lib.RT_EINVAL)
    if m * n > LIMIT:
        assert lib.rt_linear_int8(P, _lib.RT_DTYPE_FLOAT32, k, P, k, P, None, P, _lib.RT_DTYPE_FLOAT32, n, m, n, k, P,
                                  need, None) == _lib.RT_EINVAL


def test_each_size_alone_is_refused():
    for bad in ((2 ** 31, 1, 64), (1, 2 ** 31, 64), (1, 1, 65537), (-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(ResidentTopKError):
            linear_int8_workspace(*bad)
