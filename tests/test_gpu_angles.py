"""The angles of qk_norm_rope_fwd at near and far positions, against angles in
60 digits (a double-precision oracle is itself off at far positions by as much
as the kernels are)."""
from decimal import Decimal, localcontext
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def angle(pos, base, i, dim):
    """pos base^(-2i / dim) mod 2 pi, as a double."""
    with localcontext() as c:
        c.prec = 60
        return float((Decimal(pos) * Decimal(base) ** (Decimal(-2 * i) / dim)) % TWO_PI)


@pytest.mark.parametrize("base,dim", [(10000.0, 64), (500000.0, 128), (1.0, 32), (3.0e38, 64), (0.5, 64)])
def test_angles(base, dim):
    """Rows of (1, 0) pairs come out as (cos, sin).  Tolerance: the angle's
    stated error, and 7 2^-24 for the rest (an eighth of a turn at most in fp32,
    three roundings of it; the series; the products)."""
    import transformer_attention_backward_gb300 as abw
    given, base = base, float(np.float32(base))             # a C float: the formula's base (3e38 is none itself)
    rng = np.random.default_rng(dim)
    pos = np.concatenate([[0, 1, -1, 4095, 2 ** 24, -2 ** 24, 2 ** 31 - 1, -2 ** 31], rng.integers(-2 ** 31, 2 ** 31, 24)])
    x = torch.zeros(1, len(pos), 1, dim, device="cuda")
    x[..., 0::2] = 1.0
    y, _ = abw.qk_norm_rope_fwd(x, None, rope_base=given, positions=torch.from_numpy(pos.astype(np.int32))[None].cuda())
    y = y[0, :, 0].double().cpu().numpy()
    for t, p in enumerate(int(n) for n in pos):
        for i in range(dim // 2):
            a = angle(p, base, i, dim)
            turns = abs(p) * base ** (-2.0 * i / dim) / (2 * math.pi)
            off = abs(p) * 2.0 ** -54 if base >= 1 else turns * (4 + abs(math.log(base))) * 2.0 ** -53
            tol = 2 * math.pi * (off + 2.0 ** -31) + 7 * 2.0 ** -24
            assert abs(y[t, 2 * i] - math.cos(a)) <= tol and abs(y[t, 2 * i + 1] - math.sin(a)) <= tol, (p, i)
