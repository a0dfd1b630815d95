"""Attention of drafted trees where V holds infinities and NaN in many places: the check of V is then what its tiles wait for."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import check
from tests.tree_common import Step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def check_other_channels(out, lse, ref, label):
    """Infinities and NaN are where the oracle has them; everything else is within its bound."""
    want, want_lse, mag, smag = ref
    got = out.double().cpu().numpy()
    odd = ~np.isfinite(want)
    assert odd.any() and not odd.all(-1).any(), label
    assert np.array_equal(np.isnan(want), np.isnan(got)), f"{label}: NaN elsewhere"
    assert np.array_equal(want[np.isinf(want)], got[np.isinf(want)]), f"{label}: infinities"
    clean = torch.from_numpy(np.where(odd, 0.0, got)).float()
    check(clean, lse, (np.where(odd, 0.0, want), want_lse, np.where(odd, 0.0, mag), smag), label)


def spread(step, by, seed):
    """Positions up to `by` beyond the tree's: the rows' windows begin at as many places."""
    rng = np.random.default_rng(seed)
    at = step.positions_np + rng.integers(0, by, step.prob.total_q)
    step.positions = torch.from_numpy(at.astype(np.int32)).to(step.device)


CASES = [
    # two row tiles; pieces of about the same length side by side; pieces of very different lengths, each for itself
    ((8, 1), 64, [400, 500], [9000, 5000], 3000, 2500), ((8, 2), 16, [12] * 80, list(range(2800, 3600, 10)), 2500, 2000),
    ((8, 2), 64, [9] * 60, [700, 4500] * 30, 4000, 3500)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dim,bias", [(64, None), (64, F32), (128, None), (128, BF16)])
def test_every_tile_checked(cuda_device, case, dim, bias):
    """An infinity and a NaN in every row of V: each tile at the windows' beginnings and behind the history takes the check of V
    longer than its products take.  No wait runs out, and every call gives the same bits."""
    heads, page, n, history, window, by = CASES[case]
    step = Step(heads, dim, page, n, history, 60 + case, cuda_device, window=window, extent=256, bias=bias)
    spread(step, by, 61)
    step.prob.v_cache[..., 3] = float("inf")
    step.prob.v_cache[..., 40] = float("nan")
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    out, lse, _ = step.call(workspace=ws)
    assert binding.inkling_attn_read_device_error(ws) == 0
    with np.errstate(invalid="ignore"):
        check_other_channels(out, lse, step.reference(), f"case {case}")
    for i in range(30):
        a, b, _ = step.call(workspace=ws)
        assert torch.equal(a.view(torch.int16), out.view(torch.int16)) and torch.equal(b, lse), f"call {i}"
    assert binding.inkling_attn_read_device_error(ws) == 0
