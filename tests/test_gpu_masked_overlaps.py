"""Buffers of the masked operators that lie side by side in one allocation are taken, and shared inputs too."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding, rotary
from tests.masked_common import check, options, problem, reference

pytestmark = pytest.mark.gpu


def side_by_side(device, sizes):
    """uint8 views of the given sizes, each right behind the one before (sizes are multiples of 256)."""
    whole = torch.zeros(sum(sizes), dtype=torch.uint8, device=device)
    return [x for x in whole.split(sizes)]


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("order", [(0, 1, 2, 3), (2, 0, 3, 1), (3, 2, 1, 0)])
def test_attention(cuda_device, decode, order):
    lens = [300, 40, 7, 129]
    prob = problem((16, 2), 128, 16, [1] * 4 if decode else [8, 8, 4, 12], lens, 90, cuda_device)
    params = binding.params_of(prob)
    T = prob.total_q
    need = binding.inkling_attn_masked_workspace_bytes(params, decode)
    sizes = [T * 16 * 256, T * 16 * 256, T * 16 * 4, need]   # q, out, lse, workspace
    parts = side_by_side(cuda_device, [sizes[i] for i in order])
    q, out, lse, ws = (parts[order.index(i)] for i in range(4))
    q = q.view(torch.bfloat16).view(T, 16, 128)
    q.copy_(prob.q)
    out, lse = out.view(torch.bfloat16).view(T, 16, 128), lse.view(torch.float32).view(T, 16)
    binding.inkling_attn_workspace_init(ws)
    opts = options(prob)
    end = opts["key_begin"] = torch.full((T,), 3, dtype=torch.int32, device=cuda_device)
    opts["key_end"] = end * 2   # a range of three keys
    for shared in (False, True):
        if shared:
            opts["key_end"] = end   # one buffer for both: nothing is seen
        args = (prob.k_cache, prob.v_cache, prob.block_table, prob.seq_lens, out, ws)
        if decode:
            binding.inkling_attn_decode_masked(params, q, *args, lse=lse, **opts)
        else:
            binding.inkling_attn_prefill_masked(params, q, prob.cu_q_lens, *args, lse=lse, **opts)
        assert binding.inkling_attn_read_device_error(ws) == 0
        check(out, lse, reference(prob, opts), f"order {order}")
        assert torch.equal(q, prob.q)


def test_norm_and_write(cuda_device):
    prob = problem((8, 2), 64, 16, [20, 5], [20, 60], 91, cuda_device)
    params = binding.params_of(prob)
    pool = prob.k_cache.numel() * 2
    q, k, v = (torch.randn(25, h, 64, device=cuda_device).to(torch.bfloat16) for h in (8, 2, 2))
    f = rotary.inv_freq(64, device=cuda_device)[0]
    size = 25 * 8 * 64 * 2
    kc, ws, q_out, vc = side_by_side(cuda_device, [pool, 256, size, pool])
    got = [t.view(torch.bfloat16).view(s) for t, s in ((q_out, q.shape), (kc, prob.k_cache.shape), (vc, prob.v_cache.shape))]
    want = [torch.zeros_like(q), torch.zeros_like(prob.k_cache), torch.zeros_like(prob.v_cache)]
    for (o, a, b), w in ((got, ws), (want, binding.alloc_masked_workspace(params, False, cuda_device))):
        binding.inkling_attn_qk_norm_rope_write(params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table, o, a, b, w,
                                                inv_freq=f)
        assert binding.inkling_attn_read_device_error(w) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(got[1].abs().sum()) > 0
