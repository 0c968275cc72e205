"""csa2_kv8_attn where scales and weights lie far apart: what the softmax sum, small weights beside a
dominating key and scores near the end of fp32 are held to.  max_q 1 takes the kernel of few rows per
key head, max_q 40 the f16 one."""
import math

import pytest
import torch

import kv8_ref as ref
from sparse_attention_fp4_pack_b200 import csa2
from test_gpu_kv8 import BF, HF, attn_inputs, run_attn

pytestmark = pytest.mark.gpu

ROWS = [(1, [1, 3]), (40, [40, 3])]


def check_lse(lse, want, what):
    """lse against the 64-bit one, with the bound of ref.assert_attn: the scores' error and 2^-19 of
    the value for exp2, the fp32 sums and the logarithm."""
    _, exact, _, smax = want
    rows = ~torch.isnan(exact[:, 0])
    tol = 2.0 ** -17 * smax + 2.0 ** -20 + 2.0 ** -19 * (1.0 + exact.abs())
    err = (lse.cpu().double() - exact).abs()
    assert (err <= tol)[rows].all(), f"{what}: lse off by {float(err[rows].max()):.3g}"


@pytest.mark.parametrize("max_q,news", ROWS)
@pytest.mark.parametrize("length", [200, 2000])
@pytest.mark.parametrize("scales", [(2.0 ** 60, 2.0 ** -60), (2.0 ** 120, 1.0), (2.0 ** -64, 2.0 ** 100, 3.0), (1.0, 2.0 ** -20, 2.0 ** 118)])
def test_softmax_sum_with_value_scales_far_apart(max_q, news, length, scales):
    """The sum of the weights does not depend on the value scales: keys on pages of small scale count
    in it whatever the other pages' scales are, and lower the share of the others."""
    args = list(attn_inputs(21, [length, 90], news, 4, 2, 64, 16, BF))
    vs, table = args[4], args[5]
    for r, n in enumerate((length, 90)):
        for j in range(-(-n // 16)):
            vs[table[r, j].long()] = scales[j % len(scales)]
    out, lse = run_attn(args, 0.125, max_q=max_q)
    want = ref.attn(*args, 0.125, 0, 0.0)
    check_lse(lse, want, f"scales {scales}")
    ref.assert_attn(out, None, want, 0.0, length, f"scales {scales}")
