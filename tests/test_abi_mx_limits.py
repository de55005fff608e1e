"""Limits of the microscaled products, on the CPU: what a grid cannot hold is refused before a launch."""
import ctypes

import pytest

from test_abi_mx_route_grads import err, shape
from test_abi_residual import at, lib  # noqa: F401  (lib: fixture)

BY = ctypes.byref


@pytest.mark.parametrize("kw,status", [
    (dict(T=1024, E=1024, N=1 << 20), 2), (dict(T=1024, E=1024, N=1 << 20, out=1), 2),
    (dict(T=16384, E=1000, N=1 << 20, gather=0), 2), (dict(T=1000, E=1000, N=1 << 20), 0),
    (dict(T=1024, E=1024, N=1 << 20, swiglu=0), 0), (dict(T=16384, E=0, N=1 << 20, gather=0), 0),
    (dict(T=1 << 14, E=1024, N=1 << 19), 0),
])
def test_grids(lib, kw, status):  # noqa: F811
    n = ctypes.c_size_t()
    s = shape(**{**dict(K=32, k=1), **kw})
    assert lib.moe_mx_linear_workspace_bytes(BY(s), BY(n)) == status
    if status:
        assert "grid" in err(lib)
        assert lib.moe_mx_linear(BY(s), *(at(i) for i in range(8)), None, 0, None) == status
