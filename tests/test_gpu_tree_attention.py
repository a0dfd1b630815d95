"""Attention of drafted trees over the paged cache on the GPU against the fp64 oracle, element by element."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import check
from tests.tree_common import Step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
CASES = [
    # heads, dim, page, tokens, history, kind, window, extent, bias, options
    ((8, 2), 64, 16, [1], [0], "chain", -1, 1, None, ""),
    ((8, 2), 64, 16, [1, 0, 7, 3], [0, 4, 300, 1], "tree", -1, 1, None, ""),
    ((8, 2), 64, 16, [5, 2, 16], [130, 0, 700], "tree", -1, 64, F32, ""),
    ((64, 8), 128, 64, [16, 9, 1], [1000, 129, 2000], "tree", -1, 4096, F32, ""),
    ((64, 16), 128, 64, [8, 5, 3], [2000, 700, 100], "tree", 512, 512, F32, ""),
    ((64, 8), 128, 64, [61, 17], [1500, 40], "tree", -1, 1, None, ""),
    ((64, 8), 128, 64, [61, 33], [515, 90], "forest", -1, 300, BF16, ""),
    ((12, 4), 128, 32, [40, 90], [200, 333], "tree", 37, 20, F32, "cap"),
    ((14, 2), 64, 8, [20, 1, 64], [77, 1000, 5], "forest", 3, 1, None, "slopes"),
    ((16, 1), 128, 128, [30, 4], [900, 127], "tree", -1, 100, BF16, "cap+slopes"),
    ((40, 8), 128, 256, [26, 51], [255, 300], "tree", 1, 77, F32, ""),
    ((5, 5), 64, 32, [128, 129, 3], [64, 63, 65], "flat", -1, 1, None, "cap"),
    ((130, 1), 64, 64, [3, 1], [200, 0], "chain", -1, 9, F32, "slopes"),
    ((4, 4), 128, 16, [512, 300], [0, 10], "forest", -1, 50, F32, ""),
    ((8, 1), 64, 64, [300], [3000], "chain", 100, 1, None, "cap_small"),
    ((8, 2), 128, 64, [2, 2], [20000, 9000], "tree", -1, 1024, F32, ""),
    ((8, 8), 64, 16, [9] * 50, list(range(0, 500, 10)), "tree", -1, 33, BF16, "slopes"),
    ((2, 1), 128, 64, [3], [70000], "chain", -1, 1, None, "cap_large"),
]


def options(heads, kind, device):
    kw = {}
    if "cap" in kind:
        kw["softcap"] = {"cap": 30.0, "cap_small": 1.5, "cap_large": 500.0}[[w for w in kind.split("+") if w.startswith("cap")][0]]
    if "slopes" in kind:
        kw["slopes"] = torch.pow(2.0, -8.0 * (torch.arange(heads[0], device=device) + 1) / heads[0])
    return kw


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_oracle(cuda_device, case):
    heads, dim, page, n, history, kind, window, extent, bias, opts = CASES[case]
    step = Step(heads, dim, page, n, history, 700 + case, cuda_device, kind, window, extent, bias,
                q_std=3.0 if "cap" in opts else 1.0)
    kw = options(heads, opts, cuda_device)
    out, lse, ws = step.call(**kw)
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, step.reference(**kw), f"case {case}")


def test_a_chain_is_a_prefill_and_one_token_a_decode(cuda_device):
    """The same rows through the masked entry points, within twice their bound of one another."""
    for n in ([7, 20], [1, 1]):
        step = Step((8, 2), 128, 64, n, [300, 1000], 5, cuda_device, "chain", window=100)
        p = step.prob
        out, lse, _ = step.call(softcap=20.0)
        ws = binding.alloc_masked_workspace(step.params, False, cuda_device)
        other, other_lse = torch.empty_like(out), torch.empty_like(lse)
        binding.inkling_attn_prefill_masked(step.params, p.q, p.cu_q_lens, p.k_cache, p.v_cache, p.block_table, p.seq_lens,
                                            other, ws, softcap=20.0, lse=other_lse)
        ref = step.reference(softcap=20.0)
        check(out, lse, ref, "tree")
        check(other, other_lse, ref, "prefill")


def test_any_bits_and_positions_will_do(cuda_device):
    """Bits that no tree has (of later tokens, none at all, past the sequence's tokens), positions below the history and far
    beyond it."""
    step = Step((8, 2), 64, 16, [40, 3, 20], [50, 0, 333], 9, cuda_device, window=60, extent=40, bias=F32)
    rng = np.random.default_rng(1)
    T = step.prob.total_q
    step.ancestors = torch.from_numpy(rng.integers(-2**31, 2**31, (T, step.words)).astype(np.int32)).to(cuda_device)
    step.ancestors[5] = 0
    step.ancestors[41] = 0      # no history either: sees nothing
    step.ancestors[44] = 0
    at = step.positions_np + rng.integers(-70, 70, T)
    at[50] = 2**31 - 1
    at[51] = -2**31
    step.positions = torch.from_numpy(at.astype(np.int32)).to(cuda_device)
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, step.reference(), "any bits")


def test_rows_behind_the_last_sequence_and_empty_ones(cuda_device):
    step = Step((8, 2), 64, 16, [5, 0, 9, 3], [100, 30, 0, 7], 11, cuda_device)
    p = step.prob
    p.q = torch.cat((p.q, torch.full((6, 8, 64), float("nan"), device=cuda_device, dtype=BF16)))
    pad = lambda x: torch.cat((x, torch.full((6, *x.shape[1:]), -1, dtype=x.dtype, device=cuda_device)))
    step.positions, step.ancestors = pad(step.positions), pad(step.ancestors)
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, step.reference(), "rows behind the last sequence")


def test_sequences_that_do_not_fit(cuda_device):
    """More tokens than length or than bits: zero rows; rows that are not there: skipped; the others are right."""
    step = Step((8, 2), 64, 16, [5, 33, 9], [100, 30, 50], 12, cuda_device)
    p = step.prob
    step.ancestors = step.ancestors[:, :1].contiguous()
    step.words = 1
    p.seq_lens[0] = 4
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_QLEN_EXCEEDS_KV | binding.DEVERR_QLEN_EXCEEDS_MAX
    ref = step.reference()
    assert np.isneginf(ref[1][:38]).all()
    check(out, lse, ref, "do not fit")
    p.seq_lens[0] = 105
    p.cu_q_lens[3] = 48
    out, lse, _ = step.call(workspace=ws)
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_BAD_ROWS | binding.DEVERR_QLEN_EXCEEDS_MAX
    assert (out[38:] == 7.0).all() and (lse[38:] == 7.0).all()
    p.cu_q_lens[3] = 47
    full = step.reference()
    check(out[:38], lse[:38], [x[:38] for x in full], "beside one that is skipped")


@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("bias", [None, F32])
def test_pages_outside_the_pool(cuda_device, page, bias):
    """Their keys are as if masked, drafted ones among them; table entries past the last key are never read."""
    step = Step((8, 2), 128, page, [20, 9], [700, 300], 13, cuda_device, extent=100, bias=bias)
    p = step.prob
    p.block_table[0, 3 if page < 256 else 1] = -5
    p.block_table[0, (719 // page)] = p.num_pages
    p.block_table[1, 0] = 2**31 - 1
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE
    check(out, lse, step.reference(), "bad pages")


def test_lengths_past_the_table(cuda_device):
    step = Step((8, 2), 64, 16, [6], [200], 14, cuda_device)
    step.prob.block_table = step.prob.block_table[:, :8].contiguous()
    step.params = binding.params_of(step.prob)
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE
    check(out, lse, step.reference(), "past the table")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -3.3895e38])
@pytest.mark.parametrize("bias,softcap", [(None, 0.0), (F32, 0.0), (None, 20.0)])
def test_values_in_masked_places_do_not_reach_the_output(cuda_device, bad, bias, softcap):
    """K and V of siblings, of keys before the window and of slots behind the last token hold `bad`; rows that
    see none of them are as before."""
    step = Step((8, 2), 128, 16, [12, 7, 30], [200, 97, 0], 15, cuda_device, "chain", window=40, extent=64, bias=bias)
    p = step.prob
    # tokens 3 and 5 of every sequence are seen by nobody but themselves
    anc = step.ancestors_np.copy()
    cu = p.cu_q_lens.cpu().numpy()
    alone = np.concatenate([c + np.array([3, 5]) for c in cu[:-1]])
    keep = np.ones(len(anc), bool)
    keep[alone] = False
    anc[keep] &= ~np.uint32(1 << 3 | 1 << 5)
    step.ancestors = torch.from_numpy(anc.view(np.int32)).to(cuda_device)
    want = step.reference(softcap=softcap)
    table = p.block_table.cpu().numpy()
    for b, (n, L) in enumerate(zip(p.q_lens, p.seq_lens_list)):
        H = L - n
        for k in list(range(0, max(0, H - 40))) + [H + 3, H + 5] + list(range(L, (L + 15) // 16 * 16)):
            p.k_cache[int(table[b, k // 16]), :, k % 16] = bad
            p.v_cache[int(table[b, k // 16]), :, k % 16] = bad
    out, lse, ws = step.call(softcap=softcap)
    assert binding.inkling_attn_read_device_error(ws) == 0
    rows = torch.from_numpy(keep).to(cuda_device)
    ref = [np.where(keep.reshape(-1, *[1] * (x.ndim - 1)), x, np.nan if i == 1 else 0.0) for i, x in enumerate(want)]
    out[~rows], lse[~rows] = 7.0, 7.0   # (rows that do see one)
    check(out, lse, ref, f"{bad} in masked places")


@pytest.mark.parametrize("bias", [None, BF16])
@pytest.mark.parametrize("heads,dim,n,history", [((8, 2), 64, [20, 7], [150, 300]), ((8, 1), 128, [40, 3], [6000, 4000])])
def test_the_other_channels_of_an_infinity_keep_their_values(cuda_device, bias, heads, dim, n, history):
    """Infinities and NaN in some channels of V of drafted tokens and of late keys of the history."""
    step = Step(heads, dim, 64, n, history, 16, cuda_device, extent=200, bias=bias)
    p = step.prob
    rng = np.random.default_rng(17)
    table = p.block_table.cpu().numpy()
    for b, (x, L) in enumerate(zip(n, p.seq_lens_list)):
        for k in rng.integers(L - x - 3, L, 4):
            for value in (float("inf"), -float("inf"), float("nan")):
                p.v_cache[int(table[b, k // 64]), :, int(k) % 64, int(rng.integers(dim))] = value
    out, lse, ws = step.call()
    assert binding.inkling_attn_read_device_error(ws) == 0
    with np.errstate(invalid="ignore"):
        want, want_lse, mag, smag = step.reference()
    got = out.double().cpu().numpy()
    odd = ~np.isfinite(want)
    assert odd.any() and not odd.all(-1).any()
    assert np.array_equal(np.isnan(want), np.isnan(got)) and np.array_equal(want[np.isinf(want)], got[np.isinf(want)])
    clean = torch.from_numpy(np.where(odd, 0.0, got)).float()
    check(clean, lse, (np.where(odd, 0.0, want), want_lse, np.where(odd, 0.0, mag), smag), "other channels")


@pytest.mark.parametrize("bias", [None, F32])
def test_results_repeat_bit_for_bit_and_streams_are_kept(cuda_device, bias):
    step = Step((64, 8), 128, 64, [16, 3, 40], [5000, 300, 2000], 18, cuda_device, extent=1000, bias=bias)
    out, lse, ws = step.call()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        torch.cuda.synchronize()
        if stream is None:
            a, b, _ = step.call(workspace=ws)
        else:
            with torch.cuda.stream(side):
                a, b, _ = step.call(workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, lse)
    assert binding.inkling_attn_read_device_error(ws) == 0


def test_a_workspace_serves_calls_of_any_sizes_in_turn(cuda_device):
    """Long and short, wide and narrow, with and without a bias, D = 128 first: what one call leaves changes no other."""
    steps = [Step((64, 8), 128, 64, [61], [9000], 19, cuda_device), Step((8, 2), 128, 16, [1, 1], [10, 4000], 20, cuda_device),
             Step((8, 2), 64, 16, [30, 30], [300, 3], 21, cuda_device, extent=50, bias=F32)]
    ws = binding.alloc_tree_workspace(steps[0].params, cuda_device)
    refs = [s.reference() for s in steps]
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        out, lse, _ = steps[i].call(workspace=ws)
        check(out, lse, refs[i], f"call of step {i}")
    assert binding.inkling_attn_read_device_error(ws) == 0


def test_no_lse_and_workspaces_that_are_not_zeroed(cuda_device):
    """Of a workspace only its error word has to be zero."""
    step = Step((8, 2), 64, 16, [9, 4], [3000, 70], 22, cuda_device, extent=50, bias=F32)
    p = step.prob
    want, lse, _ = step.call()
    n = binding.inkling_attn_tree_workspace_bytes(step.params)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda_device)
    ws[:256] = 0
    out = torch.empty_like(p.q)
    binding.inkling_attn_tree(step.params, p.q, p.cu_q_lens, p.k_cache, p.v_cache, p.block_table, p.seq_lens, step.positions,
                              step.ancestors, out, ws, rel_logits=step.rel)
    assert torch.equal(out, want) and binding.inkling_attn_read_device_error(ws) == 0


@pytest.mark.parametrize("odd", [1, 3])
def test_a_bias_at_any_address(cuda_device, odd):
    """rel_logits behind a few elements of another buffer, rows of an odd length."""
    for bias in (F32, BF16):
        step = Step((8, 2), 128, 64, [10, 3], [500, 90], 23, cuda_device, extent=61, bias=bias)
        want = step.call()
        held = torch.zeros(odd + step.rel.numel(), dtype=bias, device=cuda_device)
        held[odd:] = step.rel.flatten()
        step.rel = held[odd:].view_as(step.rel)
        got = step.call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads,n,history,window", [
    ((8, 8), [5] * 40, list(range(100, 900, 20)), -1), ((16, 16), [7] * 64, [600] * 64, 512), ((64, 8), [9, 30, 4] * 10, [700, 90, 3000] * 10, 300),
    ((8, 2), [3] * 100, list(range(100)), -1), ((64, 8), [16] * 32, [2000 + 97 * i for i in range(32)], -1)])
@pytest.mark.parametrize("bias", [None, F32])
def test_many_short_pieces(cuda_device, heads, n, history, window, bias):
    """Runs of several items of many lengths on every SM: pieces side by side, cut ones, pieces of one tile."""
    step = Step(heads, 128, 64, n, history, 24, cuda_device, window=window, extent=200, bias=bias)
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    ref = step.reference()
    for _ in range(3):
        out, lse, _ = step.call(workspace=ws)
        assert binding.inkling_attn_read_device_error(ws) == 0
        check(out, lse, ref, "many pieces")


REPEATED = [
    # heads, dim, page, tokens, history, window, extent, bias
    ((64, 8), 128, 64, [61, 30, 45], [9000, 500, 4000], -1, 1, None), ((64, 8), 128, 16, [61, 5], [9000, 3000], -1, 1, None),
    ((64, 8), 64, 8, [61, 20], [9000, 3000], -1, 1, None), ((64, 16), 128, 64, [7] * 40, [600] * 40, 512, 1, None),
    ((64, 8), 128, 64, [16, 40], [5000, 3000], -1, 1000, F32), ((64, 16), 128, 16, [7] * 40, [600] * 40, 512, 512, BF16),
    ((64, 8), 64, 64, [16, 40], [5000, 3000], -1, 1000, F32)]


@pytest.mark.parametrize("case", range(len(REPEATED)))
def test_two_hundred_calls_give_the_same_bits(cuda_device, case):
    """What a warp does not wait for shows at one call in a hundred."""
    heads, dim, page, n, history, window, extent, bias = REPEATED[case]
    step = Step(heads, dim, page, n, history, 25, cuda_device, window=window, extent=extent, bias=bias)
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    out, lse, _ = step.call(workspace=ws)
    check(out, lse, step.reference(), f"case {case}")
    for i in range(200):
        a, b, _ = step.call(workspace=ws)
        assert torch.equal(a.view(torch.int16), out.view(torch.int16)) and torch.equal(b, lse), f"call {i}"
    assert binding.inkling_attn_read_device_error(ws) == 0
