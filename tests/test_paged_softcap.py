"""The cap c tanh(u / c) of decode_shared's tensor-core form over the whole
range of c and u: caps far above the scores (the cap does nothing there), far
below them (all scores end at +-c), and warps that hold both kinds.

Tolerances are those of the other attention tests: a logit is off by at most
8e-7 of itself plus 3.7e-7 c where |u| is between c / 16 and 0.4 c, and by a
few roundings (2^-24 of itself) below that; scores here are of size 1 beside
caps above 3, so logits are good to 2e-6 and outputs to 4e-6 relative, far
below the 16-bit rounding that sets the tolerance."""
import math

import pytest
import torch

import attention_split_attn_b200 as A
from parity import compare
from test_paged_groups import run_shared
from test_parity_paged import Case

pytestmark = pytest.mark.gpu

ENDS, GROUPS = [500, 520, 640, 505, 90], [(4, 500)]


def _check(c):
    want = c.expected()
    run_shared(c.args(A.OP_DECODE_SHARED))
    A.check_device_status()
    compare(c.dev["out"], want, 1e-5, 2e-2)


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("cap", [0.05, 1.0, 3e3, 1e5, 1e6, 1e12, 1e30, 3e38])
def test_caps(cuda_lib, cap, D, cache):
    _check(Case(51, ENDS, P=32, D=D, cache=cache, softcap=cap, groups=GROUPS))


@pytest.mark.parametrize("cap", [30.0, 2e3, 1e5])
@pytest.mark.parametrize("sign", [-1, 1])
def test_one_score_far_above_the_cap_beside_small_ones(cuda_lib, cap, sign):
    """One key is so long that its score passes the cap: negative for row 0, it has no weight there, and the small
    scores beside it decide; the other rows of the warp do not see it."""
    c = Case(52, ENDS, P=16, Hq=4, Hkv=2, D=64, softcap=cap, groups=GROUPS, begins=[0, 200, 200, 200, 0])
    page, at = int(c.table[0, 100 // 16]), 100 % 16
    for g in range(2):
        q = c.q[0, 2 * g].float()
        c.k[page, at, g] = (sign * 4 * cap * q / (q @ q) * math.sqrt(64)).to(c.k.dtype)
    _check(c)
    u = (c.q[0, 0].float() @ c.k[page, at, 0].float()).item() * c.kw["scale"]
    assert sign * u > cap


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-12, 3.0])
def test_scales_under_a_cap(cuda_lib, scale):
    _check(Case(53, ENDS, P=16, Hq=4, Hkv=2, D=64, softcap=4e4, scale=scale, groups=GROUPS))
