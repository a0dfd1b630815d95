"""Accepted paths moved in the pools, on the GPU against the oracle: bits, equal; and a whole step."""
import numpy as np
import pytest
import torch

from oracle import tree as oracle
from paged_attention_relative_gqa_gb300 import binding, rotary
from tests.masked_common import bits, check, problem, reference
from tests.tree_common import Step, parents_of

pytestmark = pytest.mark.gpu


def pools_of(heads, dim, page, n, history, layers, seed, device):
    """(params, cu, seq_lens, table, K pools, V pools) with pages of every sequence at random places."""
    prob = problem((heads, heads), dim, page, n, [a + b for a, b in zip(n, history)], seed, device)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    draw = lambda: torch.randint(-32768, 32767, prob.k_cache.shape, generator=g, device=device,
                                 dtype=torch.int16).view(torch.bfloat16)
    params = binding.params_of(prob)
    return params, prob.cu_q_lens, prob.seq_lens, prob.block_table, [draw() for _ in range(layers)], [draw() for _ in range(layers)]


def run(made, paths, lens, width, device, out=True):
    params, cu, L, table, K, V = made
    path = torch.full((len(paths), width), -9, dtype=torch.int32, device=device)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    ws = binding.alloc_tree_workspace(params, device)
    new = torch.full_like(L, 77) if out else None
    binding.inkling_attn_tree_commit(params, cu, L, table, path, torch.tensor(lens, dtype=torch.int32, device=device),
                                     binding.tree_pools(params, K, V), new, ws)
    return new, binding.inkling_attn_read_device_error(ws), path.cpu().numpy()


def expect(made, path, lens):
    params, cu, L, table, K, V = made
    cu, L, table = cu.cpu().numpy(), L.cpu().numpy(), table.cpu().numpy()
    pools, new = [bits(x).copy() for x in K + V], []
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n < 0 or n > L[b]:
            new.append(L[b])
            continue
        took = oracle.accepted(path[b], lens[b], n)
        new.append(L[b] - n + len(took))
        for x in pools:
            oracle.commit(x, table[b], params.page_size, params.num_pages, L[b] - n, took)
    return pools, new


def random_path(n, rng, most):
    m = int(rng.integers(0, min(n, most) + 1))
    return sorted(rng.choice(n, m, replace=False).tolist())


@pytest.mark.parametrize("heads,dim,page,n,history,layers", [
    (2, 64, 16, [1], [0], 1), (8, 128, 64, [9, 0, 33, 2, 1], [100, 5, 63, 0, 64], 3), (1, 64, 8, [300], [3], 2),
    (16, 128, 256, [64, 64], [1000, 0], 1), (5, 64, 32, [512, 40], [70, 9], 2), (8, 128, 64, [32] * 100, [50] * 100, 4),
    (2, 64, 16, [6], [40], 128)])
def test_against_the_oracle(cuda_device, heads, dim, page, n, history, layers):
    rng = np.random.default_rng(len(n) + dim)
    for trial in range(3):
        made = pools_of(heads, dim, page, n, history, layers, 70 + trial, cuda_device)
        paths = [random_path(x, rng, 400) if trial else list(range(x))[x // 2:] for x in n]
        lens = [len(p) for p in paths]
        width = max(lens + [1]) + trial
        want = expect(made, [p + [-9] * (width - len(p)) for p in paths], lens)
        new, err, _ = run(made, paths, lens, width, cuda_device)
        assert err == 0 and new.tolist() == want[1]
        for got, w in zip(made[4] + made[5], want[0]):
            assert np.array_equal(bits(got), w)


def test_paths_that_are_refused_and_sequences_that_are_skipped(cuda_device):
    n = [6] * 8
    made = pools_of(2, 64, 16, n, [20] * 8, 2, 80, cuda_device)
    made[1][7] = 36       # offsets that fall: six more of sequence 6, then minus six
    made[1][8] = 30
    paths = [[0, 3], [3, 3], [2, 1], [-1, 2], [0, 6], [1, 5], [0, 1], [2, 4]]
    lens = [2, 2, 2, 2, 2, 9, 2, 2]
    width = 8
    full = [p + [-9] * (width - len(p)) for p in paths]
    want = expect(made, full, lens)
    new, err, _ = run(made, paths, lens, width, cuda_device)
    assert err == binding.DEVERR_BAD_TREE | binding.DEVERR_BAD_ROWS
    assert new.tolist() == want[1]
    for got, w in zip(made[4] + made[5], want[0]):
        assert np.array_equal(bits(got), w)
    # more tokens than length
    made = pools_of(2, 64, 16, [6, 6], [20, 0], 1, 81, cuda_device)
    made[2][1] = 5
    want = expect(made, [[0, 3], [0, 3]], [2, 2])
    new, err, _ = run(made, [[0, 3], [0, 3]], [2, 2], 2, cuda_device)
    assert err == binding.DEVERR_QLEN_EXCEEDS_KV and new.tolist() == want[1] == [22, 5]
    assert all(np.array_equal(bits(a), b) for a, b in zip(made[4] + made[5], want[0]))


def test_pages_outside_the_pool(cuda_device):
    made = pools_of(2, 64, 8, [30], [5], 2, 82, cuda_device)
    made[3][0, 1] = made[0].num_pages + 7
    made[3][0, 4] = -1
    path = [1, 5, 9, 13, 20, 28]
    want = expect(made, [path], [6])
    new, err, _ = run(made, [path], [6], 6, cuda_device, out=False)
    assert err == binding.DEVERR_PAGE_OUT_OF_RANGE
    assert all(np.array_equal(bits(a), b) for a, b in zip(made[4] + made[5], want[0]))


def test_captured_and_replayed_with_other_paths(cuda_device):
    made = pools_of(4, 128, 64, [20, 20], [50, 3], 2, 83, cuda_device)
    params, cu, L, table, K, V = made
    path, lens = torch.zeros(2, 10, dtype=torch.int32, device=cuda_device), torch.zeros(2, dtype=torch.int32, device=cuda_device)
    new, ws, pools = torch.empty_like(L), binding.alloc_tree_workspace(params, cuda_device), binding.tree_pools(params, K, V)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        binding.inkling_attn_tree_commit(params, cu, L, table, path, lens, pools, new, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.inkling_attn_tree_commit(params, cu, L, table, path, lens, pools, new, ws)
    rng = np.random.default_rng(4)
    for _ in range(4):
        paths = [random_path(20, rng, 10) for _ in range(2)]
        full = [p + [0] * (10 - len(p)) for p in paths]
        m = [len(p) for p in paths]
        torch.cuda.synchronize()
        path.copy_(torch.tensor(full, dtype=torch.int32))
        lens.copy_(torch.tensor(m, dtype=torch.int32))
        want = expect(made, full, m)
        g.replay()
        torch.cuda.synchronize()
        assert new.tolist() == want[1]
        assert all(np.array_equal(bits(a), b) for a, b in zip(K + V, want[0]))


@pytest.mark.parametrize("rotary_model", [True, False])
def test_a_step_with_drafted_trees(cuda_device, rotary_model):
    """Plan, write (or convolution), attention, commit and state of one layer, on the device from the parents and the
    accepted paths alone; then the cache holds, bit for bit, what a step with the accepted tokens alone writes, and the tokens of
    the path were answered as that step answers them."""
    heads, dim, page, n, history = (8, 2), 128, 16, [13, 30, 1, 7], [100, 37, 64, 0]
    step = Step(heads, dim, page, n, history, 90, cuda_device, "tree", window=60, extent=80,
                bias=None if rotary_model else torch.float32)
    p, dev = step.prob, cuda_device
    B, T, Hq, Hkv = len(n), sum(n), *heads
    rng = np.random.default_rng(91)
    g = torch.Generator(device=dev)
    g.manual_seed(92)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)
    rows = randn(T, Hq + 2 * Hkv, dim)
    q, k, v = (x.contiguous() for x in rows.split([Hq, Hkv, Hkv], 1))
    freq, w = rotary.inv_freq(dim, device=dev)[0], torch.rand(dim, generator=g, device=dev) + 0.5
    ks = 4
    w_k, w_v = torch.randn(2, Hkv, dim, ks, generator=g, device=dev)
    state_k, state_v = randn(B, ks - 1, Hkv, dim), randn(B, ks - 1, Hkv, dim)
    ws = binding.alloc_tree_workspace(step.params, dev)
    pos, anc = torch.empty(T, dtype=torch.int32, device=dev), torch.empty(T, step.words, dtype=torch.int32, device=dev)

    def write(params, parents, positions, cu, L, q, k, v, kc, vc):
        if rotary_model:
            q_out = torch.empty_like(q)
            binding.inkling_attn_qk_norm_rope_write(params, q, k, v, cu, L, p.block_table, q_out, kc, vc, ws, w_q=w, w_k=w,
                                                    inv_freq=freq, positions=positions)
            return q_out
        binding.inkling_attn_kv_conv_write_tree(params, k, v, cu, L, p.block_table, parents, w_k, w_v, state_k, state_v, kc, vc,
                                                ws)
        return q

    binding.inkling_attn_tree_plan(step.params, p.cu_q_lens, p.seq_lens, step.parents_t, pos, anc, ws)
    kc, vc = p.k_cache.clone(), p.v_cache.clone()
    q_all = write(step.params, step.parents_t, pos, p.cu_q_lens, p.seq_lens, q, k, v, kc, vc)
    out, lse = torch.empty_like(p.q), torch.empty(T, Hq, device=dev)
    binding.inkling_attn_tree(step.params, q_all, p.cu_q_lens, kc, vc, p.block_table, p.seq_lens, pos, anc, out, ws,
                              rel_logits=step.rel, lse=lse)
    # a path from a token to its root in every sequence
    paths = []
    for tree in step.parents:
        way = [int(rng.integers(len(tree)))]
        while tree[way[-1]] >= 0:
            way.append(tree[way[-1]])
        paths.append(way[::-1])
    m = [len(x) for x in paths]
    path = torch.full((B, max(m)), -1, dtype=torch.int32, device=dev)
    for b, x in enumerate(paths):
        path[b, : len(x)] = torch.tensor(x, dtype=torch.int32)
    lens = torch.tensor(m, dtype=torch.int32, device=dev)
    new = torch.empty_like(p.seq_lens)
    binding.inkling_attn_tree_commit(step.params, p.cu_q_lens, p.seq_lens, p.block_table, path, lens,
                                     binding.tree_pools(step.params, [kc], [vc]), new, ws)
    # the same tokens in a step of their own, as a chain
    took = torch.tensor([sum(n[:b]) + i for b, x in enumerate(paths) for i in x], device=dev)
    cu = torch.tensor([0] + np.cumsum(m).tolist(), dtype=torch.int32, device=dev)
    assert new.tolist() == [h + x for h, x in zip(history, m)]
    chain = torch.tensor([i for x in m for i in range(-1, x - 1)], dtype=torch.int32, device=dev)
    kd, vd = p.k_cache.clone(), p.v_cache.clone()
    q_one = write(step.params, chain, pos[took], cu, new, q[took], k[took], v[took], kd, vd)
    assert torch.equal(q_one, q_all[took])
    table = p.block_table.cpu().numpy()
    for b, L in enumerate(new.tolist()):
        key = np.arange(L)
        at = table[b, key // page], slice(None), key % page
        assert np.array_equal(bits(kc)[at], bits(kd)[at]) and np.array_equal(bits(vc)[at], bits(vd)[at])
    pos1, anc1 = torch.empty(len(took), dtype=torch.int32, device=dev), torch.empty(len(took), 1, dtype=torch.int32, device=dev)
    binding.inkling_attn_tree_plan(step.params, cu, new, chain, pos1, anc1, ws)
    assert torch.equal(pos1, pos[took])
    if not rotary_model:
        old = [(state_k, k), (state_v, v)]
        got = torch.empty_like(state_k), torch.empty_like(state_v)
        binding.inkling_attn_kv_conv_state_tree(step.params, k, v, p.cu_q_lens, path, lens, state_k, state_v, *got, ws)
        cu_n = p.cu_q_lens.cpu().numpy()
        for (s, x), now in zip(old, got):
            for b in range(B):
                assert np.array_equal(bits(now)[b], oracle.conv_state(bits(x)[cu_n[b]: cu_n[b + 1]], bits(s)[b], paths[b]))
    assert binding.inkling_attn_read_device_error(ws) == 0
    # the attention of the tree against the oracle over the cache as it was, and of the chain over the cache as it is
    keep = p.k_cache, p.v_cache, p.q
    kt, vt = p.k_cache.clone(), p.v_cache.clone()
    write(step.params, step.parents_t, pos, p.cu_q_lens, p.seq_lens, q, k, v, kt, vt)
    p.k_cache, p.v_cache, p.q = kt, vt, q_all
    ref = step.reference()
    check(out, lse, ref, "tree")
    p.k_cache, p.v_cache, p.q = keep
    one, one_lse = torch.empty_like(q_one), torch.empty(len(took), Hq, device=dev)
    binding.inkling_attn_tree(step.params, q_one, cu, kc, vc, p.block_table, new, pos1, anc1, one, ws,
                              rel_logits=None if step.rel is None else step.rel[took], lse=one_lse)
    check(one, one_lse, [x[took.cpu().numpy()] for x in ref], "the accepted path alone")
