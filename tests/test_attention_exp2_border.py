"""2^x on the FMA pipe where the attention kernels hold it (csrc/attn_prims.cuh, kLowest): a masked weight has to be
zero as bf16, or it multiplies whatever lies in the masked place.  Replays the header's fp32 steps in numpy."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "test_rnn_layer_b200", "csrc")
POLY = open(os.path.join(CSRC, "fma_exp2.cuh")).read()
PRIMS = open(os.path.join(CSRC, "attn_prims.cuh")).read()
BORDERS = {"kC4": "ex2_poly2_fine", "kC3": "ex2_cubic2"}     # the polynomial and the function that holds x


def _lowest(name):
    body = PRIMS[PRIMS.index(f"void {name}("):]
    held = re.search(r"max_nan\(x0, ([^)]+)\)", body).group(1)
    if held == "kLowest":
        held = re.search(r"constexpr float kLowest = (\S+);", PRIMS).group(1)
    return np.float32(held.rstrip("f"))


def _ex2(x, poly, lowest):
    """The steps in fp32; each fma is rounded once (computed in fp64, then rounded)."""
    got = dict(re.findall(r"(" + poly + r"_\d) = ([0-9.eE+-]+)f", POLY))
    c = [np.float32(got[f"{poly}_{k}"]) for k in range(len(got))]
    x = np.maximum(np.asarray(x, dtype=np.float32), lowest)
    shift = np.float32(12582912.0)
    t = x + shift
    f = x - (t - shift)
    p = np.full_like(f, c[-1])
    for k in range(len(c) - 2, -1, -1):
        p = (p.astype(np.float64) * f + c[k]).astype(np.float32)
    bits = (p.view(np.int32).astype(np.int64) + (t.view(np.int32).astype(np.int64) << 23)) & 0xFFFFFFFF
    return bits.astype(np.uint32).view(np.float32)


@pytest.mark.parametrize("poly", BORDERS)
def test_what_a_masked_score_gets_is_zero_as_bf16(poly):
    low = _lowest(BORDERS[poly])
    got = _ex2([-np.inf, -1e30, -200.0, -127.0, low], poly, low).astype(np.float64)
    # half of the least bf16 value above zero (2^-133); ties go to the even 0
    assert np.all(got >= 0) and np.all(got < 2.0 ** -134)


@pytest.mark.parametrize("poly", BORDERS)
def test_the_way_there_has_no_jump(poly):
    """Every fp32 value in [-127.5, -125.5]: never negative, off by less than 2^-126, falling."""
    low = _lowest(BORDERS[poly])
    x = -np.arange(np.float32(125.5).view(np.int32), np.float32(127.5).view(np.int32) + 1, dtype=np.int32).view(np.float32)
    got = _ex2(x, poly, low).astype(np.float64)
    want = np.exp2(x.astype(np.float64))
    assert np.all(got >= 0) and np.all(np.abs(got - want) < 2.0 ** -126)
    assert np.all(np.diff(got) <= 2.0 ** -126 * 1e-4)      # falls with x (to the polynomial's error)


def test_a_nan_comes_out_finite():
    """CUDA's arithmetic makes 0x7fffffff of any NaN.  Shifted left by 23 and added to itself it is the largest finite
    number, which is why the kernels look for NaN in their rows' maxima and inputs."""
    bits = 0x7fffffff
    got = np.array([(bits + (bits << 23)) & 0xFFFFFFFF], dtype=np.uint32).view(np.float32)
    assert np.isnan(np.array([bits], dtype=np.uint32).view(np.float32)[0]) and got[0] == np.finfo(np.float32).max
