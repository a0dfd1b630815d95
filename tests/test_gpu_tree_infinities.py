"""Attention of drafted trees where V holds infinities and NaN in many places: the check of V is then what its tiles wait for."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import check
from tests.test_gpu_wait_limits import DEFAULT_LIMIT_NS, limit
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


@pytest.mark.parametrize("dim,tokens", [(64, 9), (128, 40)])
def test_an_infinity_at_both_ends_of_a_long_window(cuda_device, limit, dim, tokens):
    """One at the first keys that some rows see and one in a drafted token, 300,000 keys apart, on every SM: found without a look
    at the keys between, so that no wait comes near its limit.  Rows take what they see; everything else keeps its bits."""
    dev, B, Hkv, G, page, L, window = cuda_device, 38, 16, 2, 256, 310_000, 300_000
    g = torch.Generator(device=dev).manual_seed(62)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev).to(BF16)
    width, pages = (L + page - 1) // page, 82
    k, v = randn(pages, Hkv, page, dim), randn(pages, Hkv, page, dim)
    table = torch.randint(2, pages, (B, width), generator=g, device=dev, dtype=torch.int32)
    H, T = L - tokens, B * tokens
    first, last = H - window + 3, L - 1            # keys with an infinity, on pages that are named there alone
    table[:, first // page], table[:, last // page] = 0, 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    params = binding.make_params(num_seqs=B, num_q_heads=Hkv * G, num_kv_heads=Hkv, head_dim=dim, page_size=page,
                                 max_pages_per_seq=width, num_pages=pages, rel_extent=1, window=window, sm_scale=dim ** -0.5)
    q = randn(T, Hkv * G, dim)
    cu, lens, parents = ints([tokens * b for b in range(B + 1)]), ints([L] * B), ints(list(range(-1, tokens - 1)) * B)
    words = (tokens + 31) // 32
    pos, anc = torch.empty(T, dtype=torch.int32, device=dev), torch.empty(T, words, dtype=torch.int32, device=dev)
    ws = binding.alloc_tree_workspace(params, dev)
    binding.inkling_attn_tree_plan(params, cu, lens, parents, pos, anc, ws)
    outs = []
    for value in (0.0, float("inf"), float("nan")):
        v[0, :, first % page, 3] = value
        v[1, :, last % page, dim - 1] = value
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
        binding.inkling_attn_tree(params, q, cu, k, v, table, lens, pos, anc, out, ws, lse=lse)   # (the first loads the kernel)
        limit(20_000_000)
        binding.inkling_attn_tree(params, q, cu, k, v, table, lens, pos, anc, out, ws, lse=lse)
        assert binding.inkling_attn_read_device_error(ws) == 0, value
        limit(DEFAULT_LIMIT_NS)
        outs.append((out.float().view(B, tokens, -1, dim), lse))
    place = torch.arange(tokens, device=dev)
    begin, end = place + H - window + 1 <= first, place + H >= last
    assert 0 < begin.sum() < tokens and end.sum() == 1
    want = outs[0][0]
    for (out, lse), odd in zip(outs[1:], (torch.isposinf, torch.isnan)):
        assert torch.equal(lse, outs[0][1])
        assert odd(out[:, begin][..., 3]).all() and odd(out[:, end][..., dim - 1]).all()
        out[:, begin, :, 3], out[:, end, :, dim - 1] = want[:, begin, :, 3], want[:, end, :, dim - 1]
        assert torch.equal(out, want)
