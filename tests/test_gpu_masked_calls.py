"""Calls of the masked operators that the header allows and that no model makes often."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding, rotary
from tests.masked_common import call, check, options, problem, reference

pytestmark = pytest.mark.gpu


def _problem(decode, device, seed=110, heads=(8, 2), dim=128):
    q_lens, seq_lens = ([1, 1, 1], [700, 3, 129]) if decode else ([300, 3, 60], [700, 3, 4000])
    return problem(heads, dim, 64, q_lens, seq_lens, seed, device)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("scale", [0.0, -0.1, -3.0, 1e-30, 1e-6, 2.0, 100.0])
@pytest.mark.parametrize("decode", [False, True])
def test_scales_of_any_sign_and_size(cuda_device, decode, scale, softcap):
    prob = _problem(decode, cuda_device)
    prob.sm_scale = scale
    opts = options(prob, softcap=softcap)
    out, lse, ws = call(prob, opts, decode)
    assert binding.inkling_attn_read_device_error(ws) == 0
    want, want_lse, mag, _ = reference(prob, opts)
    prob.sm_scale = abs(scale)   # (the magnitudes that went into a score)
    check(out, lse, (want, want_lse, mag, reference(prob, opts)[3]), f"scale {scale}")


@pytest.mark.parametrize("decode", [False, True])
def test_without_lse_and_on_streams_given_by_handle(cuda_device, decode):
    prob = _problem(decode, cuda_device)
    params, opts = binding.params_of(prob), options(prob, softcap=30.0)
    want, _, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        out = torch.full_like(prob.q, 7.0)
        torch.cuda.synchronize()
        args = (prob.k_cache, prob.v_cache, prob.block_table, prob.seq_lens, out, ws)
        if decode:
            binding.inkling_attn_decode_masked(params, prob.q, *args, stream=stream, **opts)
        else:
            binding.inkling_attn_prefill_masked(params, prob.q, prob.cu_q_lens, *args, stream=stream, **opts)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert binding.inkling_attn_read_device_error(ws) == 0


@pytest.mark.parametrize("decode", [False, True])
def test_thousands_of_sequences(cuda_device, decode):
    B = 5000
    rng = np.random.default_rng(111)
    seq_lens = rng.integers(1, 60, B).tolist()
    q_lens = [1] * B if decode else [int(rng.integers(0, min(4, L) + 1)) for L in seq_lens]
    prob = problem((4, 2), 64, 8, q_lens, seq_lens, 112, cuda_device)
    opts = options(prob, slopes=[0.1, 0.2, 0.3, 0.4])
    out, lse, ws = call(prob, opts, decode)
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), "thousands of sequences")


def test_a_captured_write_and_attention_replayed_with_other_lengths(cuda_device):
    """One graph of a decode step: write, attend.  Each replay with new rows and one token more."""
    dev, B, D, heads = cuda_device, 5, 128, (16, 2)
    lens = [100, 1, 63, 64, 700]
    prob = problem(heads, D, 16, [1] * B, lens, 113, dev, max_pages=60)
    pages = torch.randperm(B * 60, device=dev).to(torch.int32).view(B, 60).contiguous()
    kc, vc = (torch.randn(B * 60, 2, 16, D, device=dev).to(torch.bfloat16) for _ in range(2))
    prob.block_table, prob.k_cache, prob.v_cache = pages, kc, vc
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, True, dev)
    rows = torch.zeros(B, (16 + 4) * D, dtype=torch.bfloat16, device=dev)
    q, k, v = (x.unflatten(-1, (h, D)) for x, h in zip(rows.split([16 * D, 2 * D, 2 * D], -1), (16, 2, 2)))
    f = rotary.inv_freq(D, device=dev)[0]
    w = torch.rand(D, device=dev) + 0.5
    out, lse = torch.zeros_like(prob.q), torch.zeros(B, 16, device=dev)

    def step():
        binding.inkling_attn_qk_norm_rope_write(params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table, prob.q, kc,
                                                vc, ws, w_q=w, w_k=w, inv_freq=f)
        binding.inkling_attn_decode_masked(params, prob.q, kc, vc, prob.block_table, prob.seq_lens, out, ws, softcap=30.0,
                                           lse=lse)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        rows.copy_(torch.randn_like(rows, dtype=torch.float32))
        prob.seq_lens += 1
        prob.seq_lens_list = [L + 1 for L in prob.seq_lens_list]
        graph.replay()
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == 0
        got, got_lse, got_q = out.clone(), lse.clone(), prob.q.clone()
        check(got, got_lse, reference(prob, options(prob, softcap=30.0)), f"replay {i}")
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(lse, got_lse) and torch.equal(prob.q, got_q)
