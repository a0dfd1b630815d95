"""Attention of drafted trees in batches of thousands of sequences, most of which draft nothing or a token."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import check
from tests.tree_common import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,dim,window,bias", [((4, 2), 64, -1, None), ((2, 1), 128, 60, None), ((4, 2), 128, -1, torch.float32)])
def test_thousands_of_sequences(cuda_device, heads, dim, window, bias):
    """Sequences without a token, without a history, of one to five tokens, of lengths from one tile to a few dozen; two that are
    refused, far from one another."""
    rng = np.random.default_rng(40)
    B = 2900
    n = np.where(rng.random(B) < 0.3, 0, np.where(rng.random(B) < 0.6, 1, rng.integers(1, 6, B))).tolist()
    history = np.where(rng.random(B) < 0.05, 0, np.where(rng.random(B) < 0.02, rng.integers(500, 2000, B), rng.integers(1, 150, B))).tolist()
    n[1000] = n[2800] = 3
    step = Step(heads, dim, 16, n, history, 41, cuda_device, window=window, extent=64, bias=bias)
    step.prob.seq_lens[1000] = 2
    step.prob.seq_lens[2800] = 1
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_QLEN_EXCEEDS_KV
    check(out, lse, step.reference(), "thousands")
