"""Biases of drafted trees at the ends of their types' range: a row whose keys all carry the lowest value is still a softmax."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import check
from tests.tree_common import Step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def check_ties(out, lse, ref, rows, label):
    """Rows whose largest biases are so far from the others, and so large, that scores are lost in their rounding: the mean of V
    over the keys that share the largest bias.  Weights of 1 and 0 are exact in bf16; sums are fp32 (at most a truncation of 2^-23 of
    the magnitudes a key, here less than 2^-10) and the output is rounded once (2^-8 of its value); lse is the bias, off by 2^-22 of it."""
    want, want_lse, mag = ref[:3]
    got, got_lse = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    assert np.isfinite(got).all() and np.isfinite(got_lse).all(), f"{label}: not finite"
    excess = np.abs(got - want[rows]) - 2.0 ** -8 * np.abs(want[rows]) - 2.0 ** -10 * mag[rows]
    assert excess.max() <= 0, f"{label}: out off by {excess.max():.3e} over its bound"
    ex = np.abs(got_lse - want_lse[rows]) - 2.0 ** -22 * np.abs(want_lse[rows])
    assert ex.max() <= 0, f"{label}: lse off by {ex.max():.3e} over its bound"


CASES = [
    # heads, dim, page, tokens, history, window, extent: whole histories, windows, pieces side by side and cut ones, an odd extent
    ((8, 2), 128, 64, [13, 30, 1], [900, 70, 300], -1, 256), ((16, 16), 64, 16, [7] * 20, [300] * 20, 200, 200),
    ((16, 2), 128, 64, [16, 40], [5000, 3000], -1, 1024), ((8, 2), 64, 64, [9, 5], [500, 90], -1, 61)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("bias,value", [(F32, torch.finfo(F32).min), (BF16, torch.finfo(BF16).min), (F32, -1e30), (F32, 1e30),
                                        (BF16, -2.0 ** 70), (F32, torch.finfo(F32).max)])
def test_rows_whose_keys_all_have_it(cuda_device, case, softcap, bias, value):
    """Every second token's bias is `value` at all distances; the others' are ordinary."""
    heads, dim, page, n, history, window, extent = CASES[case]
    step = Step(heads, dim, page, n, history, 80 + case, cuda_device, window=window, extent=extent, bias=bias)
    rows = np.arange(step.prob.total_q) % 2 == 1
    rel = step.rel.clone()
    rel[1::2] = value
    step.rel = rel
    out, lse, ws = step.call(softcap=softcap)
    assert binding.inkling_attn_read_device_error(ws) == 0
    check_ties(out, lse, step.reference(), rows, f"case {case}, {value}")
    want = step.reference(softcap=softcap)
    out[1::2], lse[1::2] = 7.0, 7.0
    check(out, lse, [np.where(rows.reshape(-1, *[1] * (x.ndim - 1)), np.nan if i == 1 else 0.0, x) for i, x in enumerate(want)],
          f"case {case}, the other rows")


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("bias", [F32, BF16])
def test_rows_of_lowest_and_less_low_values(cuda_device, case, bias):
    """By token: the lowest value but for a few distances of half of it; the lowest at near distances and a quarter of it from some
    distance on (the last value, which far tiles take for a whole row); the other way round; the lowest everywhere but at distance 0."""
    heads, dim, page, n, history, window, extent = CASES[case]
    step = Step(heads, dim, page, n, history, 90 + case, cuda_device, window=window, extent=extent, bias=bias)
    low, E = torch.finfo(bias).min, extent
    rel = torch.full_like(step.rel, low)
    rel[0::4, :, 5::37] = low / 2
    rel[1::4, :, E // 2:] = low / 4
    rel[2::4, :, : E // 2] = low / 4
    rel[3::4, :, 0] = 0.5
    step.rel = rel
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == 0
    rows = np.arange(step.prob.total_q) % 4 != 3
    check_ties(out, lse, step.reference(), rows, f"case {case}")
    # the others see but themselves: the lowest value weighs exactly nothing, so bounds go by the scores without a bias
    want = step.reference()
    step.rel = None
    smag = step.reference()[3] + 0.5
    out[torch.from_numpy(rows).to(cuda_device)] = 7.0
    lse[torch.from_numpy(rows).to(cuda_device)] = 7.0
    check(out, lse, (want[0], np.where(rows[:, None], np.nan, want[1]), want[2], smag), f"case {case}, the others")


def test_slopes_that_leave_one_key(cuda_device):
    """A slope of -1e25 times the distance: the farthest key has all the weight; one of 1e25: the nearest."""
    step = Step((8, 2), 128, 64, [9, 30, 1], [3000, 70, 0], 97, cuda_device)
    slopes = torch.tensor([1e25, -1e25] * 4, device=cuda_device)
    out, lse, ws = step.call(slopes=slopes)
    assert binding.inkling_attn_read_device_error(ws) == 0
    # (siblings of one distance do not see one another; every distance is another weight)
    want, want_lse, mag, _ = step.reference(slopes=slopes)
    far = np.arange(8) % 2 == 1
    check_ties(out[:, far], lse[:, far], (want[:, far], want_lse[:, far], mag[:, far]), slice(0, 39), "the farthest key")
    step.rel = None
    smag = step.reference()[3] + 0.5
    near = ~far
    check(out[:, near], lse[:, near], (want[:, near], want_lse[:, near], mag[:, near], smag[:, near]), "the nearest key")


@pytest.mark.parametrize("value", [-1e9, -1e10, -3e12, 1e10, 1e15])
@pytest.mark.parametrize("heads,dim,n,history", [((8, 2), 128, [13, 30], [900, 70]), ((16, 2), 64, [16, 40], [5000, 3000])])
def test_weights_add_up_whatever_the_size(cuda_device, value, heads, dim, n, history):
    """A bias that swallows some of a score's bits: which ones is rounding, but weights add up to 1 and lse stays beside the bias."""
    step = Step(heads, dim, 64, n, history, 95, cuda_device, extent=300, bias=F32)
    step.rel[:] = value
    step.prob.v_cache.fill_(1.0)
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == 0
    assert (out.float() - 1.0).abs().max() <= 2.0 ** -7     # of numerators and output
    # scores here are below 40, the logarithm of the number of keys below 9; the rest is rounding
    assert (lse.double() - value).abs().max() <= 49.0 + 2.0 ** -21 * abs(value)
