"""The microscaled products with long reductions on every tile size: the ring of stages goes round several
times, and the scales' second place is filled, read and filled again. Every block of 32 has a scale of its
own, so that a scale of another block or stage shows. References and tolerances are those of
test_gpu_mx_linear.py (the operands' spread goes into them through the operands)."""
import numpy as np
import pytest

import test_gpu_mx_linear as base
from oracle import microscale as X

pytestmark = pytest.mark.gpu


def _operand(rng, shape, fmt, std=1.0):
    rows, K = int(np.prod(shape[:-1])), shape[-1]
    x = rng.standard_normal((rows, K // 32, 32), dtype=np.float32) * np.float32(std)
    x *= np.exp2(rng.integers(-3, 4, size=(rows, K // 32, 1))).astype(np.float32)
    codes, scales = X.quantize(x.reshape(rows, K), fmt)
    val = X.dequantize(codes, scales, fmt).reshape(shape)
    return X.pack(codes, fmt).reshape(*shape[:-1], -1), scales.reshape(*shape[:-1], -1), val


# stages of 128 elements: 8.25, 9.25 or 22.5
CASES = [  # T, K, N, out, act, E, k, gather
    (13, 2880, 96, "bf16", "none", 0, 1, False), (9, 1184, 64, "mx8", "swiglu", 8, 2, True),    # few rows
    (300, 1056, 1096, "bf16", "none", 0, 1, False), (300, 2880, 1088, "mx8", "swiglu", 0, 1, False),  # 64 x 128
    (300, 1184, 320, "f16", "none", 6, 3, True), (301, 1056, 352, "mx8", "swiglu", 6, 3, True),
    (300, 1056, 352, "mx8", "none", 6, 3, False),
    (2056, 1056, 1600, "f16", "none", 0, 1, False), (2056, 1184, 1600, "mx8", "none", 0, 1, False),  # 128 x 128
    (1100, 1056, 1536, "bf16", "none", 4, 2, True), (1100, 1184, 768, "mx8", "swiglu", 4, 2, True),
    (4200, 1056, 3104, "mx8", "none", 0, 1, False), (2300, 1184, 3136, "bf16", "swiglu", 0, 1, False),  # 256 x 256
    (1500, 1056, 2240, "mx8", "swiglu", 3, 2, True),
    (4100, 1184, 4104, "f16", "none", 0, 1, False), (2056, 1056, 4128, "mx8", "none", 2, 2, True),  # 256 x 192
]


@pytest.mark.parametrize("T,K,N,out,act,E,k,gather", CASES)
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_long_reductions(monkeypatch, T, K, N, out, act, E, k, gather, fmt):
    monkeypatch.setattr(base, "_operand", _operand)
    base.check(T, K, N, fmt, out, act, E, k, gather)
