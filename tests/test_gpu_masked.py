"""Masked, capped paged attention on the GPU against the fp64 oracle, element by element."""
import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import call, check, options, problem, reference

pytestmark = pytest.mark.gpu


def _opts(prob, kind, seed, decode):
    rng = np.random.default_rng(seed)
    T = prob.total_q
    L = np.repeat(prob.seq_lens_list, prob.q_lens)
    p = np.concatenate([np.arange(b - a, b) for a, b in zip(prob.q_lens, prob.seq_lens_list)]) if T else np.zeros(0, int)
    kw = {}
    if "cap" in kind:
        kw["softcap"] = {"cap": 30.0, "cap_small": 1.5, "cap_large": 500.0}[[w for w in kind.split("+") if w.startswith("cap")][0]]
    if "slopes" in kind:
        kw["slopes"] = 2.0 ** -rng.uniform(0, 8, prob.num_q_heads)
    if "documents" in kind:
        cut = 13
        kw["begin"] = p // cut * cut
    if "prefix" in kind:
        kw["end"] = np.maximum(p + 1, L // 2)
    if "random" in kind:   # anything goes: negative, past the end, empty, reversed
        kw["begin"] = rng.integers(-5, L + 5)
        kw["end"] = rng.integers(-5, L + 40)
    if "nothing" in kind:
        kw["begin"] = np.full(T, 3)
        kw["end"] = np.full(T, 3)
    return options(prob, **kw)


PREFILL = [
    # heads, dim, page, q_lens, seq_lens, window, options
    ((8, 2), 64, 16, [1, 0, 37, 130, 5], [1, 4, 37, 400, 300], -1, ""),
    ((8, 2), 64, 16, [1, 0, 37, 130, 5], [1, 4, 37, 400, 300], -1, "cap+slopes+random"),
    ((8, 8), 128, 64, [257, 3], [257, 700], -1, "cap+prefix"),
    ((8, 8), 64, 8, [90, 300], [95, 300], 37, "slopes"),
    ((3, 1), 128, 32, [129, 1, 2], [129, 515, 2], -1, "cap_small+documents"),
    ((14, 2), 128, 128, [40, 200], [300, 200], 100, "cap"),
    ((16, 1), 64, 256, [33, 9], [700, 9], -1, "slopes+prefix"),
    ((20, 1), 128, 16, [50], [333], 1, "cap_large"),
    ((40, 1), 64, 64, [21], [128], 5, "documents"),
    ((8, 1), 128, 64, [160, 100], [160, 1000], -1, "random"),
    ((4, 2), 128, 16, [64, 64, 64], [64, 65, 1029], 64, "cap+random"),
    ((8, 2), 128, 64, [70], [70], -1, "nothing"),
    ((2, 1), 64, 8, [512], [1100], 512, "cap_small+slopes+documents"),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill_against_the_oracle(cuda_device, case):
    heads, dim, page, q_lens, seq_lens, window, kind = PREFILL[case]
    prob = problem(heads, dim, page, q_lens, seq_lens, 100 + case, cuda_device, window, q_std=3.0 if "cap" in kind else 1.0)
    opts = _opts(prob, kind, case, False)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), f"case {case}")


DECODE = [
    ((8, 2), 64, 16, [1, 5, 64, 65, 700], -1, ""),
    ((8, 8), 128, 64, [1, 129, 1000], -1, "cap"),
    ((16, 1), 128, 8, [300, 17], -1, "cap_small+slopes"),
    ((20, 1), 64, 32, [63, 640], 100, "slopes"),
    ((40, 2), 128, 16, [333, 2], 1, "cap"),
    ((64, 8), 128, 64, [5000, 1, 300, 2048], -1, "slopes+documents"),
    ((8, 2), 64, 256, [255, 256, 257, 4000], 512, "random"),
    ((14, 2), 128, 128, [900, 30, 31, 32, 33], -1, "random"),
    ((8, 1), 64, 64, [100, 200], -1, "nothing"),
    ((8, 1), 128, 64, [20000], -1, "cap_large"),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_against_the_oracle(cuda_device, case):
    heads, dim, page, seq_lens, window, kind = DECODE[case]
    prob = problem(heads, dim, page, [1] * len(seq_lens), seq_lens, 200 + case, cuda_device, window,
                   q_std=3.0 if "cap" in kind else 1.0)
    opts = _opts(prob, kind, case, True)
    out, lse, ws = call(prob, opts, True)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), f"case {case}")


@pytest.mark.parametrize("decode", [False, True])
def test_empty_sequences_and_rows_behind_the_last(cuda_device, decode):
    q_lens, seq_lens = ([1, 1, 1], [5, 0, 40]) if decode else ([5, 0, 9], [5, 0, 40])
    prob = problem((8, 2), 64, 16, [n if L else 0 for n, L in zip(q_lens, seq_lens)], seq_lens, 7, cuda_device)
    rows = len(seq_lens) if decode else prob.total_q + 6
    prob.q = torch.randn(rows, 8, 64, device=cuda_device).to(torch.bfloat16)
    if decode:
        prob.cu_q_lens = torch.arange(4, dtype=torch.int32, device=cuda_device)
    opts = options(prob)
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), "rows behind the last sequence")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -3.3895e38])
@pytest.mark.parametrize("decode", [False, True])
def test_values_in_masked_places_do_not_reach_the_output(cuda_device, decode, bad):
    """Keys past the visible range of a row, and keys that only other rows see, hold `bad` in K and V."""
    seq_lens = [200, 97, 330]
    q_lens = [1, 1, 1] if decode else [200, 60, 70]
    prob = problem((8, 2), 128, 16, q_lens, seq_lens, 8, cuda_device)
    p = np.concatenate([np.arange(b - a, b) for a, b in zip(q_lens, seq_lens)])
    begin = np.where(p >= 60, 60, 0)          # two documents: [0, 60) and [60, L)
    opts = options(prob, begin=begin)
    clean = reference(prob, opts)
    table = prob.block_table.cpu().numpy()
    for b, L in enumerate(seq_lens):
        for k in list(range(20, 40)) + list(range(L, (L + 15) // 16 * 16)):
            prob.k_cache[int(table[b, k // 16]), :, k % 16] = bad
            prob.v_cache[int(table[b, k // 16]), :, k % 16] = bad
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    second = np.nonzero((p >= 60) | (p < 20))[0]   # rows that see none of the poisoned keys
    check(out[second], lse[second], tuple(x[second] for x in clean), "poisoned keys")


def test_non_finite_values_reach_the_rows_that_see_them(cuda_device):
    prob = problem((8, 2), 64, 16, [150], [150], 9, cuda_device)
    table = prob.block_table.cpu().numpy()
    prob.v_cache[int(table[0, 70 // 16]), :, 70 % 16, 5] = float("inf")
    prob.v_cache[int(table[0, 90 // 16]), :, 90 % 16, 6] = float("nan")
    opts = options(prob)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()
    assert np.isfinite(got[:70]).all() and np.isfinite(lse.cpu().numpy()).all()
    assert np.isposinf(got[70:, :, 5]).all() and np.isfinite(got[:, :, 7:]).all()
    assert np.isfinite(got[:90, :, 6]).all() and np.isnan(got[90:, :, 6]).all()


@pytest.mark.parametrize("decode", [False, True])
def test_pages_outside_the_pool_are_masked_and_reported(cuda_device, decode):
    seq_lens = [200, 90]
    prob = problem((8, 2), 64, 16, [1, 1] if decode else [30, 90], seq_lens, 10, cuda_device)
    prob.block_table[0, 3] = prob.num_pages
    prob.block_table[1, 0] = -4
    opts = options(prob, slopes=np.linspace(0, 0.1, 8))
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE
    check(out, lse, reference(prob, opts), "bad pages")


def test_lengths_that_contradict_are_reported(cuda_device):
    prob = problem((8, 2), 64, 16, [8, 4, 6], [20, 9, 30], 11, cuda_device)
    prob.seq_lens[1] = 3   # four new tokens, three keys
    opts = options(prob)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_QLEN_EXCEEDS_KV
    check(out, lse, reference(prob, opts), "contradicting lengths")


@pytest.mark.parametrize("decode", [False, True])
def test_offsets_past_32_bits(cuda_device, decode):
    """Pages at the end of a pool of more than 2^31 elements, another sequence at its start."""
    prob = problem((8, 8), 128, 64, [1, 1] if decode else [5, 40], [100, 150], 12, cuda_device)
    n = (1 << 31) // (8 * 64 * 128) + 64
    big = []
    for c in (prob.k_cache, prob.v_cache):
        pool = torch.zeros(n, 8, 64, 128, dtype=torch.bfloat16, device=cuda_device)
        pool[:2] = c[prob.block_table[0, :2].long()]
        pool[n - 3:] = c[prob.block_table[1, :3].long()]
        big.append(pool)
    small = prob.to("cpu")
    opts = options(prob)
    want = reference(small, options(small))
    prob.k_cache, prob.v_cache = big
    prob.block_table = torch.tensor([[0, 1, n + 7], [n - 3, n - 2, n - 1]], dtype=torch.int32, device=cuda_device)
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, want, "large pool")


@pytest.mark.parametrize("decode", [False, True])
def test_repeats_bit_for_bit_and_from_a_graph_on_another_stream(cuda_device, decode):
    seq_lens = [1500, 3, 700, 2222]
    prob = problem((16, 2), 128, 64, [1] * 4 if decode else [300, 3, 1, 222], seq_lens, 13, cuda_device, q_std=2.0)
    opts = options(prob, softcap=20.0, slopes=np.linspace(0.01, 0.3, 16))
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    first = (out.clone(), lse.clone())
    check(out, lse, reference(prob, opts), "eager")
    params = binding.params_of(prob)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    ws2 = binding.alloc_masked_workspace(params, decode, cuda_device)
    torch.cuda.synchronize()

    def go():
        if decode:
            binding.inkling_attn_decode_masked(params, prob.q, prob.k_cache, prob.v_cache, prob.block_table,
                                               prob.seq_lens, o2, ws2, lse=l2, **opts)
        else:
            binding.inkling_attn_prefill_masked(params, prob.q, prob.cu_q_lens, prob.k_cache, prob.v_cache,
                                                prob.block_table, prob.seq_lens, o2, ws2, lse=l2, **opts)
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        go()
    for _ in range(3):
        o2.zero_()
        l2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, first[0]) and torch.equal(l2, first[1])
    # new lengths and inputs in the captured buffers
    prob.seq_lens.copy_(torch.tensor([1400, 3, 650, 2000], dtype=torch.int32))
    prob.seq_lens_list = [1400, 3, 650, 2000]
    prob.q.copy_(torch.randn_like(prob.q, dtype=torch.float32))
    graph.replay()
    torch.cuda.synchronize()
    check(o2, l2, reference(prob, opts), "replayed with new lengths")


def test_prefill_and_decode_agree_and_parts_join(cuda_device):
    """One token as prefill and as decode, and the outputs over two halves of a history joined by lse."""
    L = 1000
    prob = problem((8, 2), 128, 64, [1], [L], 14, cuda_device)
    whole, wl, _ = call(prob, options(prob), False)
    dec, dl, _ = call(prob, options(prob), True)
    ref = reference(prob, options(prob))
    check(whole, wl, ref, "prefill")
    check(dec, dl, ref, "decode")
    parts = [call(prob, options(prob, begin=[a], end=[b]), True) for a, b in ((0, 450), (450, L))]
    lse = torch.stack([x[1] for x in parts])
    w = torch.softmax(lse, 0)[..., None]
    joined = sum(wi * x[0].float() for wi, x in zip(w, parts))
    # two more bf16 roundings of the parts
    tol = 2.0 ** -7 * sum(wi * x[0].float().abs() for wi, x in zip(w, parts)) + torch.as_tensor(ref[2] * 2.0 ** -7).to(cuda_device)
    assert ((joined - whole.float()).abs() <= tol).all()


def test_calls_on_two_streams_with_their_own_workspaces(cuda_device):
    probs = [problem((8, 2), 64, 16, [1] * 5, [300, 20, 777, 1, 64], 15 + i, cuda_device) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in probs]
    params = [binding.params_of(p) for p in probs]
    ws = [binding.alloc_masked_workspace(p, True, cuda_device) for p in params]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [call(p, options(p), True, workspace=w, stream=s) for p, w, s in zip(probs, ws, streams)]
        torch.cuda.synchronize()
    for p, (out, lse, _) in zip(probs, got):
        check(out, lse, reference(p, options(p)), "two streams")


def test_many_launches_of_a_long_prompt_agree_and_report_nothing(cuda_device):
    """A barrier that lets a warp pass a phase early shows once in a thousand launches: as a wait that
    runs out, or as another result."""
    prob = problem((16, 2), 128, 64, [1500, 700, 40], [1500, 2100, 9000], 16, cuda_device)
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, False, cuda_device)
    opts = options(prob, begin=np.concatenate([np.arange(b - a, b) // 300 * 300 for a, b in zip(prob.q_lens, prob.seq_lens_list)]))
    out, lse, _ = call(prob, opts, False, workspace=ws)
    first = (out.clone(), lse.clone())
    for _ in range(40):
        for _ in range(50):
            binding.inkling_attn_prefill_masked(params, prob.q, prob.cu_q_lens, prob.k_cache, prob.v_cache,
                                                prob.block_table, prob.seq_lens, out, ws, lse=lse, **opts)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert binding.inkling_attn_read_device_error(ws) == 0


def test_long_stretches_of_tokens_that_see_nothing(cuda_device):
    """Whole work items without a key between items with keys: padding inside packed rows, a sequence
    whose lengths contradict, and sequences without new tokens."""
    q_lens, seq_lens = [3000, 0, 900, 2500, 0], [3000, 7, 1000, 2600, 0]
    prob = problem((4, 1), 64, 64, q_lens, seq_lens, 17, cuda_device)
    prob.seq_lens[2] = 100   # 900 new tokens, 100 keys
    p = np.concatenate([np.arange(b - a, b) for a, b in zip(q_lens, seq_lens)])
    end = np.where((p % 1400) < 1300, 0, p + 1)
    begin = np.maximum(p - 5, 0)
    opts = options(prob, begin=begin, end=end)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_QLEN_EXCEEDS_KV
    check(out, lse, reference(prob, opts), "stretches of nothing")


SPLIT = [
    # few new tokens against long histories: the key tiles of an item are cut into pieces
    ((8, 1), 128, 64, [5, 40, 1], [6000, 9111, 700], -1, "cap"),
    ((8, 2), 64, 16, [33, 2], [5000, 4097], -1, "slopes+documents"),
    ((5, 1), 128, 128, [60], [8000], -1, "random"),
    ((4, 4), 64, 64, [200, 1], [7000, 3], 2500, "cap_large+prefix"),
    ((16, 1), 128, 8, [9], [3333], -1, "slopes+cap_small"),
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_prefill_of_few_tokens_against_long_histories(cuda_device, case):
    heads, dim, page, q_lens, seq_lens, window, kind = SPLIT[case]
    prob = problem(heads, dim, page, q_lens, seq_lens, 400 + case, cuda_device, window, q_std=3.0 if "cap" in kind else 1.0)
    opts = _opts(prob, kind, case, False)
    out, lse, ws = call(prob, opts, False)
    ref = reference(prob, opts)
    check(out, lse, ref, f"case {case}")
    again, lse2, _ = call(prob, opts, False, workspace=ws)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_non_finite_values_in_one_piece_of_a_cut_item(cuda_device):
    prob = problem((8, 1), 128, 64, [20], [6000], 18, cuda_device)
    table = prob.block_table.cpu().numpy()
    prob.v_cache[int(table[0, 5990 // 64]), :, 5990 % 64, 3] = float("-inf")
    out, lse, ws = call(prob, options(prob), False)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()   # token i sits at 5980 + i
    assert np.isfinite(got[:10]).all() and np.isneginf(got[10:, :, 3]).all()
    assert np.isfinite(np.delete(got, 3, axis=2)).all() and np.isfinite(lse.cpu().numpy()).all()


@pytest.mark.parametrize("decode", [False, True])
def test_waits_that_run_out_report_a_timeout_and_later_calls_are_right(cuda_device, decode):
    """A zero wait limit makes every wait for data that is not there yet give up.  A prefill workspace
    then refuses further work, with the same error, until it is initialised again."""
    seq_lens = [1500 + 97 * i for i in range(24)] if decode else [900, 5000]
    prob = problem((8, 2), 128, 64, [1] * 24 if decode else [700, 20], seq_lens, 19, cuda_device)
    opts = options(prob, softcap=20.0)
    ws = binding.alloc_masked_workspace(binding.params_of(prob), decode, cuda_device)
    try:
        binding.inkling_attn_set_wait_limit_ns(0)
        call(prob, opts, decode, workspace=ws)
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) & binding.DEVERR_WAIT_TIMEOUT
    finally:
        binding.inkling_attn_set_wait_limit_ns(2_000_000_000)
    if not decode:
        out, lse, _ = call(prob, opts, decode, workspace=ws)
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_WAIT_TIMEOUT
        assert (out == 7.0).all() and (lse == 7.0).all()
        binding.inkling_attn_workspace_init(ws)
    for _ in range(2):
        out, lse, _ = call(prob, opts, decode, workspace=ws)
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == 0
        check(out, lse, reference(prob, opts), "after a timeout")


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 200, 1 << 30])
def test_windows_beyond_every_history_are_no_windows(cuda_device, decode, window):
    """Few rows against long histories, whose pieces are counted from the window and the lengths."""
    prob = problem((8, 1), 128, 64, [1, 1] if decode else [5, 40], [6000, 9111], 20, cuda_device)
    opts = options(prob)
    want, want_lse, _ = call(prob, opts, decode)
    prob.window = window
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), "window beyond the history")
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("tokens,keys", [(20, 6016), (600, 640)])
@pytest.mark.parametrize("length", [2**31 - 1, 2**31 - 100, 1 << 20])
def test_a_length_past_the_block_table_is_reported(cuda_device, tokens, keys, length):
    """Keys end with the table; the rows' positions are those of the length."""
    prob = problem((8, 1), 128, 64, [tokens], [keys], 21, cuda_device, max_pages=keys // 64)
    opts = options(prob, end=np.full(tokens, keys))
    want = reference(prob, opts)
    prob.seq_lens[0] = length
    out, lse, ws = call(prob, options(prob), False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE
    check(out, lse, want, "length past the table")


@pytest.mark.parametrize("softcap", [10.0, 50.0, 300.0])
@pytest.mark.parametrize("power", [-60, 70])
def test_capped_scores_leave_the_range_of_v(cuda_device, softcap, power):
    """V near the ends of its range, scores up to the cap."""
    prob = problem((8, 2), 128, 64, [200, 30], [300, 3000], 22, cuda_device, q_std=30.0)
    prob.v_cache *= 2.0 ** power
    opts = options(prob, softcap=softcap)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), "range of V")


@pytest.mark.parametrize("softcap", [0.0, 50.0, 1000.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_scores_far_to_one_side(cuda_device, softcap, sign):
    """All scores of a row near -20 or near 20: the largest magnitude of a tile is not its largest score."""
    prob = problem((4, 2), 64, 64, [150, 20], [400, 2900], 23, cuda_device)
    prob.k_cache *= 0.1
    prob.k_cache += 1.0
    prob.q = (0.1 * prob.q.float() + sign * 20.0 / 8.0).to(torch.bfloat16)   # 64 products of 2.5 over sqrt(64)
    opts = options(prob, softcap=softcap)
    out, lse, ws = call(prob, opts, False)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), "scores to one side")


@pytest.mark.parametrize("fill", [float("nan"), 1e30])
def test_rows_of_other_sequences_change_no_bit(cuda_device, fill):
    """Rows of a tile past a sequence's own (the next one's, padding) have no say in how it is capped."""
    prob = problem((8, 2), 128, 64, [5, 70, 9], [1000, 70, 40], 24, cuda_device, q_std=2.0)
    opts = options(prob, softcap=50.0)
    want, want_lse, _ = call(prob, opts, False)
    T = prob.total_q
    q = torch.full((T + 40, *prob.q.shape[1:]), fill, dtype=torch.bfloat16, device=cuda_device)
    q[:5] = prob.q[:5]
    q[5 + 70:T] = prob.q[5 + 70:T]
    prob.q = q
    out, lse, _ = call(prob, opts, False)
    torch.cuda.synchronize()
    for part in (slice(0, 5), slice(75, T)):
        assert torch.equal(out[part], want[part]) and torch.equal(lse[part], want_lse[part])
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()


def test_one_workspace_serves_prefills_and_decodes_of_any_sizes(cuda_device):
    """Initialised once, then used in turn by calls of other batch sizes, head counts and kinds."""
    def make(decode, heads, dim, q_lens, seq_lens, seed):
        prob = problem(heads, dim, 64, q_lens, seq_lens, seed, cuda_device)
        opts = options(prob, softcap=40.0)
        return decode, prob, opts, reference(prob, opts)

    wide = [300 + 31 * i for i in range(96)]
    jobs = [make(True, (64, 8), 64, [1] * 96, wide, 25), make(False, (8, 1), 128, [30], [6000], 26),
            make(True, (8, 1), 128, [1, 1], [9000, 7], 27), make(True, (32, 1), 128, [1] * 5, [4000] * 5, 28),
            make(False, (8, 2), 64, [3, 20], [5000, 4000], 29)]
    sizes = [binding.inkling_attn_masked_workspace_bytes(binding.params_of(j[1]), j[0]) for j in jobs]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device=cuda_device)
    ws.fill_(0x5A)
    binding.inkling_attn_workspace_init(ws)
    for order in ((0, 1, 2, 3, 4), (4, 0, 3, 1, 0, 2, 0)):
        for i in order:
            decode, prob, opts, ref = jobs[i]
            out, lse, _ = call(prob, opts, decode, workspace=ws)
            check(out, lse, ref, f"call {i} of {order}")
    assert binding.inkling_attn_read_device_error(ws) == 0


@pytest.mark.parametrize("decode", [False, True])
def test_empty_batches_return_at_once(cuda_device, decode):
    prob = problem((8, 2), 64, 16, [1, 1], [9, 30], 30, cuda_device)
    params, ws = binding.params_of(prob), None
    ws = binding.alloc_masked_workspace(params, decode, cuda_device)
    none = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=cuda_device)
    if decode:
        params.num_seqs = 0
        out = none(0, 8, 64)
        assert binding.inkling_attn_decode_masked(params, none(0, 8, 64), prob.k_cache, prob.v_cache,
                                                  prob.block_table[:0], prob.seq_lens[:0], out, ws) is out
        return
    out = none(0, 8, 64)
    cu = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    assert binding.inkling_attn_prefill_masked(params, none(0, 8, 64), cu, prob.k_cache, prob.v_cache, prob.block_table,
                                               prob.seq_lens, out, ws) is out
    kv = none(0, 2, 64)
    assert binding.inkling_attn_qk_norm_rope_write(params, none(0, 8, 64), kv, kv, cu, prob.seq_lens, prob.block_table, out,
                                                   prob.k_cache, prob.v_cache, ws) is out


MANY = [
    # more query heads per KV head than a row tile holds; more sequences than lanes of a warp
    (False, (200, 1), 128, 64, [3, 40], [900, 40], -1, "cap+documents"),
    (False, (260, 2), 64, 16, [17, 1], [300, 3100], 33, "slopes"),
    (False, (129, 1), 64, 64, [5], [4500], -1, "random"),
    (False, (8, 1), 64, 16, [1 + i % 5 for i in range(70)], [2100 + 7 * i for i in range(70)], -1, "cap"),
    (False, (4, 2), 128, 8, [(5 * i) % 7 for i in range(150)], [(5 * i) % 7 + i for i in range(150)], -1, "slopes"),
    (False, (2, 2), 64, 16, [1], [1], -1, "cap"),
    (True, (200, 1), 128, 64, [1] * 2, [900, 40], -1, "cap"),
    (True, (4, 2), 64, 16, [1] * 300, [1 + (37 * i) % 90 for i in range(300)], 20, "slopes"),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_heads_and_many_sequences(cuda_device, case):
    decode, heads, dim, page, q_lens, seq_lens, window, kind = MANY[case]
    prob = problem(heads, dim, page, q_lens, seq_lens, 500 + case, cuda_device, window, q_std=3.0 if "cap" in kind else 1.0)
    opts = _opts(prob, kind, case, decode)
    out, lse, ws = call(prob, opts, decode)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    check(out, lse, reference(prob, opts), f"case {case}")
    again, lse2, _ = call(prob, opts, decode, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_offsets_that_change_between_replays(cuda_device):
    """A captured prefill of few rows against long histories, replayed with other splits of its rows over
    the sequences, other lengths and other ranges."""
    prob = problem((8, 1), 128, 64, [20, 20, 8], [6000, 3000, 500], 31, cuda_device)
    opts = options(prob, softcap=40.0, begin=np.zeros(48), end=np.full(48, 1 << 30))
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, False, cuda_device)
    out, lse = torch.empty_like(prob.q), torch.empty(48, 8, dtype=torch.float32, device=cuda_device)
    run = lambda: binding.inkling_attn_prefill_masked(params, prob.q, prob.cu_q_lens, prob.k_cache, prob.v_cache,
                                                      prob.block_table, prob.seq_lens, out, ws, lse=lse, **opts)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        run()
    for q_lens, seq_lens, first in (([20, 20, 8], [6000, 3000, 500], 0), ([1, 0, 40], [5999, 3000, 490], 100),
                                    ([48, 0, 0], [4000, 0, 0], 3990), ([0, 0, 0], [6000, 3000, 500], 0)):
        prob.cu_q_lens.copy_(torch.tensor([0, *np.cumsum(q_lens)], dtype=torch.int32))
        prob.seq_lens.copy_(torch.tensor(seq_lens, dtype=torch.int32))
        opts["key_begin"].fill_(first)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == 0
        check(out, lse, reference(prob, opts), f"replayed with {q_lens}")


@pytest.mark.parametrize("softcap", [5.0, 30.0, 50.0, 300.0])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,seq_lens", [([200, 33], [1500, 900]), ([3, 18], [4000, 2500])])
def test_tiles_of_small_and_large_scores_in_turn(cuda_device, softcap, dim, q_lens, seq_lens):
    """The magnitude of the keys changes from one 128-key tile to the next, so that tiles within the short
    polynomial's reach, within the cap and beyond it follow one another in every order; the first rows of a
    sequence begin to see keys at different tiles."""
    prob = problem((8, 2), dim, 64, q_lens, seq_lens, 32, cuda_device, q_std=1.5)
    table = prob.block_table.cpu().numpy()
    factors = [0.1, 3.0, 20.0, 0.3, 0.3, 8.0, 3.0, 3.0, 0.1, 40.0, 20.0]
    for b, L in enumerate(seq_lens):
        for j in range((L + 63) // 64):
            prob.k_cache[int(table[b, j])] *= factors[(j // 2 + 3 * b) % len(factors)]
    rng = np.random.default_rng(33)
    first = np.concatenate([rng.integers(0, L - n + 1, n) for n, L in zip(q_lens, seq_lens)])
    for begin in (None, first):
        opts = options(prob, softcap=softcap, begin=begin)
        out, lse, ws = call(prob, opts, False)
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == 0
        check(out, lse, reference(prob, opts), f"cap {softcap}")
