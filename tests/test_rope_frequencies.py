"""The rotary frequencies of the paged calls and the backward pass against 50 decimal digits (CPU):
relative error within (5 |ln base| + 7) 2^-53, the bound that their arithmetic gives."""
import ctypes
from decimal import Decimal, getcontext

import pytest

import pose_retrieved_kv_b200 as P

PI = Decimal("3.14159265358979323846264338327950288419716939937510582")


def _frequencies(base, dims):
    fn = getattr(P._lib._lib, "_ZN6prsink16rope_frequenciesEdiPd")    # (internal: by its C++ name)
    fn.argtypes, fn.restype = [ctypes.c_double, ctypes.c_int, ctypes.c_void_p], None
    out = (ctypes.c_double * 65)(*([-1.0] * 65))
    fn(base, dims, ctypes.addressof(out))
    assert all(x == -1.0 for x in out[dims // 2:])
    return list(out[:dims // 2])


@pytest.mark.parametrize("base", [0.5, 2.0, 100.0, 10000.0, 500000.0, 1e9])
def test_frequencies(base):
    getcontext().prec = 50
    b = Decimal(base)
    bound = (5 * abs(b.ln()) + 7) / Decimal(2) ** 53
    if base == 10000.0:
        assert bound < Decimal(2) ** -47
    for dims in (2, 16, 20, 24, 32, 42, 44, 64, 128):
        for j, x in enumerate(_frequencies(base, dims)):
            want = (b.ln() * -2 * j / dims).exp() / PI
            assert abs(Decimal(x) - want) <= bound * want, (dims, j)
