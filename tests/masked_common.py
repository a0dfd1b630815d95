"""Shared by the tests of the masked attention and of the head norm, rotation and cache write."""
import numpy as np
import torch

from oracle import masked as oracle
from paged_attention_relative_gqa_gb300 import binding
from paged_attention_relative_gqa_gb300 import workloads as W


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def problem(heads, dim, page, q_lens, seq_lens, seed, device, window=-1, q_std=1.0, max_pages=None):
    prob = W.make_problem(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, rel_extent=1,
                          window=window, q_lens=q_lens, seq_lens=seq_lens, seed=seed, device=device, max_pages=max_pages)
    if q_std != 1.0:
        prob.q = (prob.q.float() * q_std).to(torch.bfloat16)
    return prob


def options(prob, *, begin=None, end=None, slopes=None, softcap=0.0):
    dev = prob.q.device
    to = lambda v, t: None if v is None else torch.as_tensor(np.asarray(v), dtype=t).to(dev)
    return dict(softcap=softcap, key_begin=to(begin, torch.int32), key_end=to(end, torch.int32),
                slopes=to(slopes, torch.float32))


def reference(prob, opts):
    num = lambda v: None if v is None else v.cpu().numpy()
    return oracle.attention(num_q_heads=prob.num_q_heads, num_kv_heads=prob.num_kv_heads, head_dim=prob.head_dim,
                            page_size=prob.page_size, window=prob.window, sm_scale=prob.sm_scale,
                            cu_q=prob.cu_q_lens.cpu().numpy(), seq_lens=prob.seq_lens.cpu().numpy(),
                            q_bits=bits(prob.q), k_bits=bits(prob.k_cache), v_bits=bits(prob.v_cache),
                            block_table=prob.block_table.cpu().numpy(), softcap=opts["softcap"],
                            key_begin=num(opts["key_begin"]), key_end=num(opts["key_end"]), slopes=num(opts["slopes"]))


def call(prob, opts, decode, workspace=None, stream=None):
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, decode, prob.q.device) if workspace is None else workspace
    out = torch.full_like(prob.q, 7.0)
    lse = torch.full(prob.q.shape[:2], 7.0, dtype=torch.float32, device=prob.q.device)
    if decode:
        binding.inkling_attn_decode_masked(params, prob.q, prob.k_cache, prob.v_cache, prob.block_table, prob.seq_lens,
                                           out, ws, lse=lse, stream=stream, **opts)
    else:
        binding.inkling_attn_prefill_masked(params, prob.q, prob.cu_q_lens, prob.k_cache, prob.v_cache,
                                            prob.block_table, prob.seq_lens, out, ws, lse=lse, stream=stream, **opts)
    return out, lse, ws


def check(out, lse, ref, label=""):
    """Bounds, per element.  A score is a sum of D products added in fp32 by the tensor cores (at
    most D + 16 roundings or truncations of 2^-23 of the summed magnitudes), then capped, shifted
    and exponentiated with a few more roundings: off by at most d = 2^-15 (1 + smag).  A softmax
    weight is then off by a factor 1 +- 2 d and rounded to bf16 once (2^-8) before it multiplies V;
    the output is rounded to bf16 once (2^-8 of its value).  lse is off by d and a few roundings of
    its own value."""
    want, want_lse, mag, smag = ref
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(want_lse)
    assert np.all(got[~rows] == 7.0) and np.all(got_lse[~rows] == 7.0), f"{label}: rows of no sequence were written"
    d = 2.0 ** -15 * (1.0 + smag)
    tol = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -8 + 2.0 * d[..., None]) + 1e-30
    nothing = np.isneginf(want_lse)
    assert np.all(got[nothing] == 0.0) and np.all(np.isneginf(got_lse[nothing])), f"{label}: rows that see nothing"
    rows &= ~nothing
    assert np.isfinite(got[rows]).all() and np.isfinite(got_lse[rows]).all(), f"{label}: not finite"
    excess = (np.abs(got - want) - tol)[rows]
    assert excess.size == 0 or excess.max() <= 0, f"{label}: out off by {excess.max():.3e} over its bound"
    tol_l = (d + 2.0 ** -20 * (1.0 + np.abs(want_lse)))[rows]
    ex = np.abs(got_lse[rows] - want_lse[rows]) - tol_l
    assert ex.size == 0 or ex.max() <= 0, f"{label}: lse off by {ex.max():.3e} over its bound"
