"""append_paged's codes at the ends of the float range: the nearest code to the
exact quotient also where scale and values are a few thousand times the
smallest float, and next to the largest."""
import numpy as np
import pytest
import torch

import attention_split_attn_b200 as A
from test_parity_paged import _codes64, i32

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149


def _next_to_ties(rng, fmt, rows, D, unit):
    """Rows whose scale is n units exactly and whose values are whole units on and beside the borders of the codes."""
    top, ties = (127, np.arange(126) + 0.5) if fmt == "i8" else (448, None)
    if ties is None:
        vals = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        ties = (vals[1:] + vals[:-1]) / 2
    factor = 127 if fmt == "i8" else 7              # top n is a float while factor n has 24 bits
    n = rng.integers(2 ** 24 // factor // 16, 2 ** 24 // factor, size=(rows, 1))
    m = np.floor(rng.choice(ties, size=(rows, D)) * n) + rng.integers(0, 2, size=(rows, D))
    m = np.where(m < 2 ** 24, m, np.floor(m / 2 ** 6) * 2 ** 6)     # (floats: units are whole multiples there)
    m[:, 0] = top * n[:, 0]
    x = torch.from_numpy(m * rng.choice([-1.0, 1.0], size=m.shape) * unit)
    assert torch.equal(x.float().double(), x)
    return x.float(), torch.from_numpy(n[:, 0] * unit)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("unit", [TINY, TINY * 2.0 ** 30, TINY * 2.0 ** 49, 2.0 ** -20, 2.0 ** 80, 2.0 ** 98])
def test_codes_at_the_ends_of_the_range(cuda_lib, fmt, unit):
    rows, D, P = 1024, 256, 16
    rng = np.random.default_rng(5)
    x, scale = _next_to_ties(rng, fmt, rows, D, unit)
    want_s, want = _codes64(x, fmt)
    assert torch.equal(want_s.double(), scale)
    dt = torch.int8 if fmt == "i8" else torch.float8_e4m3fn
    k = torch.zeros(rows // P, P, 1, D, dtype=torch.int8, device="cuda").view(dt)
    v = k.clone()
    ks, vs = torch.zeros(rows, 1, device="cuda"), torch.zeros(rows, 1, device="cuda")
    new = x.view(rows, 1, D).cuda()
    A.append_paged(new, -new, i32(np.arange(rows)).cuda(), k, v, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for got, s, w in ((k, ks, want), (v, vs, -want)):
        assert torch.equal(s[:, 0].cpu(), want_s)
        got = got.cpu().view(rows, D).double()
        off = got != w
        assert not off.any(), (int(off.sum()), off.nonzero()[:5], got[off][:5], w[off][:5])
