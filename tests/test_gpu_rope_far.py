"""Rotary positions in fp32 up to the last position, against angles in 50 decimal digits.

The table's words come from fp64: the exponent -2 i / r is off by half a step, which the power turns into
ln(1 / theta_i) 2^-53 of theta_i; the power itself by a step, pi by half of one and the division by half: in all
(ln(1 / theta_i) + 4) 2^-53 of theta_i.  Then they are cut to units of 2^-64 turns.  At position p the angle is off by p
times both, 2^-20 radians at most at 2^31; sine, cosine, products and sum add 2^-21 a (|x1| + |x2|) as at small positions."""
import decimal
import math

import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")
POSITIONS = [0, 1, -1, 4095, 2 ** 20, 2 ** 24 + 1, 12345678, 2 ** 28 + 3, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("r,base", [(64, 10000), (16, 500000), (128, 2)])
def test_far_positions(r, base, layout, inverse):
    build.build()
    g = torch.Generator().manual_seed(r)
    n, heads = len(POSITIONS), 3
    x = torch.randn(n, heads, r, generator=g)
    table = torch.empty(r // 2, dtype=torch.int64, device="cuda")
    abi.csa2_rope_table(abi.RopeSpec(scaling=abi.ROPE_PLAIN, base=float(base), factor=1.0), r, table)
    y = torch.empty(n, heads, r, device="cuda")
    abi.csa2_rope(x.cuda(), y, torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"), table, inverse=inverse,
                  layout=abi.ROPE_HALF if layout == "half" else abi.ROPE_INTERLEAVED)
    torch.cuda.synchronize()
    with decimal.localcontext() as c:
        c.prec = 50
        theta = [(D(base).ln() * D(-2 * i) / D(r)).exp() for i in range(r // 2)]
        turn = np.array([[float((D(p) * t / (2 * PI)) % 1) for t in theta] for p in POSITIONS])   # within 2^-53 turns
    theta = np.array([float(t) for t in theta])
    xd = x.double().numpy()
    half = r // 2
    x1, x2 = (xd[..., :half], xd[..., half:]) if layout == "half" else (xd[..., 0::2], xd[..., 1::2])
    z = (x1 + 1j * x2) * np.exp((-2j if inverse else 2j) * math.pi * turn)[:, None, :]
    got = y.double().cpu().numpy()
    got = got[..., :half] + 1j * got[..., half:] if layout == "half" else got[..., 0::2] + 1j * got[..., 1::2]
    p = np.abs(np.array(POSITIONS, dtype=np.float64))[:, None]
    angle = p * theta * (np.log(1 / theta) + 4) * 2.0 ** -53 + 2 * math.pi * p * 2.0 ** -64
    tol = (angle[:, None, :] + 2.0 ** -21) * (np.abs(x1) + np.abs(x2))
    tol = tol + (np.abs(x1) + np.abs(x2) + tol) * 2.0 ** -24
    assert np.all(np.abs(got.real - z.real) <= tol) and np.all(np.abs(got.imag - z.imag) <= tol)
    assert abi.csa2_get_status() == 0
