"""Requests whose rows lie outside the rows there are: skipped and reported by the norm and write as by the
attention that reads its cache."""
import numpy as np
import pytest
import torch

from oracle import masked as oracle
from paged_attention_relative_gqa_gb300 import binding, rotary
from tests.masked_common import bits, options, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,written", [
    ([0, 5, 12, 20], [0, 1, 2]),       # as it should be
    ([0, 5, 12, 26], [0, 1]),          # the last request ends behind the last row
    ([0, 5, 20, 24], [0, 1]),          # ... and lies behind it whole
    ([0, 20, 20, 21], [0]),            # ... behind one without rows
    ([-3, 5, 12, 20], [1, 2]),         # the first begins before row 0
    ([0, 5, 2**31 - 1, 20], None),     # offsets that go down
])
def test_requests_outside_the_rows(cuda_device, cu, written):
    dev, T, D, page = cuda_device, 20, 64, 16
    prob = problem((8, 2), D, page, [5, 7, 8], [30, 40, 50], 95, dev)
    params = binding.params_of(prob)
    q, k, v = (torch.randn(T, h, D, device=dev).to(torch.bfloat16) for h in (8, 2, 2))
    f = rotary.inv_freq(D, device=dev)[0]
    ws = binding.alloc_masked_workspace(params, False, dev)
    q_out = torch.full_like(q, 7.0)
    before = [prob.k_cache.clone(), prob.v_cache.clone()]
    offsets = torch.tensor(cu, dtype=torch.int32, device=dev)
    binding.inkling_attn_qk_norm_rope_write(params, q, k, v, offsets, prob.seq_lens, prob.block_table, q_out, prob.k_cache,
                                            prob.v_cache, ws, inv_freq=f)
    err = binding.inkling_attn_read_device_error(ws)
    assert err == (0 if written == [0, 1, 2] else binding.DEVERR_BAD_ROWS)
    out = torch.full_like(q, 7.0)
    binding.inkling_attn_prefill_masked(params, q_out, offsets, prob.k_cache, prob.v_cache, prob.block_table, prob.seq_lens,
                                        out, ws, **options(prob))
    assert binding.inkling_attn_read_device_error(ws) == err
    if written is None:
        return
    table, L = prob.block_table.cpu().numpy(), prob.seq_lens.cpu().numpy()
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in written])
    pos = np.concatenate([np.arange(L[b] - (cu[b + 1] - cu[b]), L[b]) for b in written])
    seq = np.concatenate([np.full(cu[b + 1] - cu[b], b) for b in written])
    rest = np.setdiff1d(np.arange(T), rows)
    assert (q_out[rest] == 7.0).all() and (out[rest] == 7.0).all() and not (q_out[rows] == 7.0).all(-1).any()
    y, mag = oracle.norm_rope(k[rows].double().cpu().numpy(), pos, None, 0.0, f.double().cpu().numpy(), "half", 1.0)
    at = table[seq, pos // page], slice(None), pos % page
    assert (np.abs(prob.k_cache.double().cpu().numpy()[at] - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag + 1e-30).all()
    assert np.array_equal(bits(prob.v_cache)[at], bits(v[rows]))
    for now, old in ((prob.k_cache, before[0]), (prob.v_cache, before[1])):
        n = bits(now).copy()
        n[at] = bits(old)[at]
        assert np.array_equal(n, bits(old))
