"""Weights of the masked operators where the result is known exactly."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import call, options, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0, 500.0])
@pytest.mark.parametrize("heads,dim,page,q_lens,seq_lens", [
    ((8, 8), 128, 64, [400, 130], [700, 130]), ((8, 2), 64, 16, [300], [300]), ((8, 1), 128, 64, [9, 20], [9, 6000])])
@pytest.mark.parametrize("decode", [False, True])
def test_a_row_of_one_key_is_that_keys_value(cuda_device, decode, softcap, heads, dim, page, q_lens, seq_lens):
    """Rows of one key among rows that see their whole history: its weight is 1, whatever the score."""
    if decode:
        q_lens = [1] * len(q_lens)
    prob = problem(heads, dim, page, q_lens, seq_lens, 80, cuda_device, q_std=2.0)
    p = np.concatenate([np.arange(L - n, L) for n, L in zip(q_lens, seq_lens)])
    b = np.repeat(np.arange(len(q_lens)), q_lens)
    rng = np.random.default_rng(81)
    lone = (np.arange(len(p)) % 3 == 0) | decode
    key = rng.integers(0, p + 1)
    begin, end = np.where(lone, key, 0), np.where(lone, key + 1, p + 1)
    out, lse, ws = call(prob, options(prob, softcap=softcap, begin=begin, end=end), decode)
    assert binding.inkling_attn_read_device_error(ws) == 0
    table = prob.block_table.long().cpu()
    rows = torch.as_tensor(np.nonzero(lone)[0])
    k = torch.as_tensor(key)[rows]
    v = prob.v_cache.cpu()[table[torch.as_tensor(b)[rows], k // page], :, k % page]   # [rows, Hkv, D]
    want = v.repeat_interleave(heads[0] // heads[1], 1)
    assert torch.equal(out.cpu()[rows].float(), want.float())
