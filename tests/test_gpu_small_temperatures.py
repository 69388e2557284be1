"""Token probabilities at temperatures so small that 1 / T passes 32 bits."""
import math

import numpy as np
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv
from serve_ref import U32, probs

pytestmark = pytest.mark.gpu

TINY = [2e-38, 1e-38, 4.3e-39, 4.2e-39, 4e-39, 1e-39, 3e-42, 1.4e-45]


def check(z, t, got):
    """Off by a factor of 1 + (|y| + 1) 2^-21 and 140 roundings for y = (z - m) log2(e) / T, as for other temperatures."""
    for i in range(z.shape[0]):
        zi = z[i].double().cpu().numpy()
        want = probs(zi, float(t[i]))
        y = np.where(want > 0, (zi.max() - zi) / float(t[i]) * 1.4427, 0.0)
        tol = want * ((2 * (y + 1) + 2) * 2.0 ** -22 * 0.7 + 140 * U32) + 1.2e-38
        assert (np.abs(got[i].double().cpu().numpy() - want) <= tol).all(), (i, float(t[i]))


@pytest.mark.parametrize("rows, V", [(8, 1000), (8, 20000), (8, 300000), (48, 20000), (48, 50000)])
def test_small_temperatures(rows, V):
    """Ordinary logits (everything on the largest one, or shared by equal ones), and logits as small as T."""
    g = torch.Generator(device="cuda").manual_seed(V)
    t = torch.tensor((TINY * 6)[:rows], device="cuda")
    z = torch.randn(rows, V, generator=g, device="cuda")
    z[1, [5, V - 1]] = z[3, [7, 8]] = 9.0
    p = sv.token_probs(z, t)
    check(z, t, p)
    assert (p.amax(1) >= 0.5).all() and p[1, 5] == p[1, V - 1] == 0.5
    z[0, 3] = math.nan
    z[1] = -math.inf
    assert (sv.token_probs(z, t)[:2] == 0).all()
    x = torch.rand(rows, V, generator=g, device="cuda").double() * 6 * t.double()[:, None]
    x[:, ::3] = -math.inf
    x = x.float()
    check(x, t, sv.token_probs(x, t))
