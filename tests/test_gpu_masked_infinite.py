"""One infinity of V in a long history: the rows that see it get it, and finding it takes no time that a wait
would run out in."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import call, check, options, problem, reference

pytestmark = pytest.mark.gpu


def history(device, L, tokens, heads, dim, behind, seed=120):
    """A history of L keys from a small pool; page 0 is named once, at the key `behind` keys before the end."""
    page, pages = 64, 100
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(pages, heads[1], page, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    width = (L + page - 1) // page
    table = torch.randint(1, pages, (1, width), generator=g, dtype=torch.int32)
    at = L - behind
    table[0, at // page] = 0
    v[0, :, at % page] = 0
    q = torch.randn(tokens, heads[0], dim, generator=g).to(torch.bfloat16)
    params = binding.make_params(num_seqs=1, num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page,
                                 max_pages_per_seq=width, num_pages=pages, rel_extent=1, window=-1, sm_scale=dim ** -0.5)
    lens, cu = torch.tensor([L], dtype=torch.int32), torch.tensor([0, tokens], dtype=torch.int32)
    return params, [x.to(device) for x in (q, cu, k, v, table, lens)], at


@pytest.mark.parametrize("L,tokens,heads,softcap", [(3_000_000, 20, (8, 1), 0.0), (3_000_000, 300, (16, 2), 30.0), (40_000, 33, (5, 1), 0.0)])
def test_it_is_found_at_once(cuda_device, L, tokens, heads, softcap):
    params, (q, cu, k, v, table, lens), at = history(cuda_device, L, tokens, heads, 128, 10)
    ws = binding.alloc_masked_workspace(params, False, cuda_device)
    seen = torch.arange(L - tokens, L, device=cuda_device) >= at
    outs = []
    for value in (0.0, float("inf"), float("nan")):
        v[0, :, at % 64, 3] = value
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda_device)
        binding.inkling_attn_prefill_masked(params, q, cu, k, v, table, lens, out, ws, softcap=softcap, lse=lse)
        assert binding.inkling_attn_read_device_error(ws) == 0
        outs.append((out.float(), lse))
    rest = [c for c in range(128) if c != 3]
    for out, lse in outs[1:]:
        assert torch.equal(lse, outs[0][1])
        assert torch.equal(out[..., rest], outs[0][0][..., rest]) and torch.equal(out[~seen], outs[0][0][~seen])
    assert torch.isposinf(outs[1][0][seen][..., 3]).all() and torch.isnan(outs[2][0][seen][..., 3]).all()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("heads,dim,page,q_lens,seq_lens", [
    ((8, 2), 64, 16, [150, 40], [150, 300]), ((8, 8), 128, 64, [300], [500]), ((8, 1), 128, 64, [20, 3], [6000, 4000])])
def test_the_other_channels_keep_their_values(cuda_device, decode, softcap, heads, dim, page, q_lens, seq_lens):
    """Infinities and NaN in some channels of some keys, near the rows' own positions: every other channel of every
    row against the oracle, which sums over those keys too."""
    if decode:
        q_lens = [1] * len(q_lens)
    prob = problem(heads, dim, page, q_lens, seq_lens, 121, cuda_device)
    rng = np.random.default_rng(122)
    table = prob.block_table.cpu().numpy()
    for b, (n, L) in enumerate(zip(q_lens, seq_lens)):
        for _ in range(4):
            k = int(rng.integers(max(0, L - n - 3), L))
            for value in (float("inf"), -float("inf"), float("nan")):
                prob.v_cache[int(table[b, k // page]), :, k % page, int(rng.integers(dim))] = value
    opts = options(prob, softcap=softcap)
    out, lse, ws = call(prob, opts, decode)
    assert binding.inkling_attn_read_device_error(ws) == 0
    with np.errstate(invalid="ignore"):
        want, want_lse, mag, smag = reference(prob, opts)
    got = out.double().cpu().numpy()
    odd = ~np.isfinite(want)
    assert odd.any() and not odd.all(-1).any()
    assert np.array_equal(np.isnan(want), np.isnan(got)) and np.array_equal(want[np.isinf(want)], got[np.isinf(want)])
    clean = torch.from_numpy(np.where(odd, 0.0, got)).float()
    check(clean, lse, (np.where(odd, 0.0, want), want_lse, np.where(odd, 0.0, mag), smag), "other channels")
