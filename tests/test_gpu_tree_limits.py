"""Attention of drafted trees at its ends: waits that run out, graphs, the last positions there are, the longest history."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as oracle
from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import bits, check
from tests.test_gpu_wait_limits import limit, sweep
from tests.tree_common import Step, parents_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("heads,dim,page,n,history,window,extent,bias,softcap", [
    ((64, 8), 128, 64, [61, 5, 30], [3000, 900, 2000], -1, 1, None, 0.0), ((8, 2), 64, 16, [7] * 30, [600] * 30, 200, 1, None, 30.0),
    ((64, 8), 128, 64, [16, 40], [3000, 1000], -1, 1000, F32, 0.0), ((16, 16), 128, 16, [7] * 30, [600] * 30, 200, 201, BF16, 0.0)])
def test_waits_that_run_out(cuda_device, limit, heads, dim, page, n, history, window, extent, bias, softcap):
    """The result or the timeout and no other error; the next call with the same workspace is right."""
    step = Step(heads, dim, page, n, history, 30, cuda_device, window=window, extent=extent, bias=bias)
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    out, lse, _ = step.call(workspace=ws, softcap=softcap)
    check(out, lse, step.reference(softcap=softcap), "before")
    sweep(limit, lambda: step.call(workspace=ws, softcap=softcap)[:2], ws)


@pytest.mark.parametrize("bias", [None, F32])
def test_two_graphs_of_one_workspace_replayed_with_other_trees(cuda_device, bias):
    """Plan and attention captured twice, for two steps that share a workspace; replayed with other lengths, trees and pages (entries behind a shorter sequence name no page: permuted, they take keys away and are told)."""
    heads, dim, page, words, E = (16, 2), 128, 64, 2, 300
    rng = np.random.default_rng(31)
    made = []
    s = torch.cuda.Stream()
    ws = None
    for i in range(2):
        step = Step(heads, dim, page, [40, 24], [900, 2000], 32 + i, cuda_device, extent=E, bias=bias, words=words, max_pages=40)
        p = step.prob
        if ws is None:
            ws = binding.alloc_tree_workspace(step.params, cuda_device)
        out, lse = torch.empty_like(p.q), torch.empty(p.q.shape[:2], device=cuda_device)

        def run(step=step, p=p, out=out, lse=lse):
            binding.inkling_attn_tree_plan(step.params, p.cu_q_lens, p.seq_lens, step.parents_t, step.positions, step.ancestors, ws)
            binding.inkling_attn_tree(step.params, p.q, p.cu_q_lens, p.k_cache, p.v_cache, p.block_table, p.seq_lens,
                                      step.positions, step.ancestors, out, ws, rel_logits=step.rel, lse=lse)

        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            run()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                run()
        made.append((step, g, out, lse))
    bad = False
    for n, history in (([40, 24], [900, 2000]), ([3, 61], [2400, 0]), ([64, 0], [64, 500])):
        torch.cuda.synchronize()
        for step, _, out, lse in made:
            p = step.prob
            trees = [parents_of("tree", x, rng) for x in n]
            step.parents_t.copy_(torch.tensor([x for t in trees for x in t], dtype=torch.int32))
            p.cu_q_lens.copy_(torch.tensor([0, n[0], 64], dtype=torch.int32))
            p.seq_lens.copy_(torch.tensor([a + b for a, b in zip(n, history)], dtype=torch.int32))
            p.block_table.copy_(torch.from_numpy(rng.permuted(p.block_table.cpu().numpy(), axis=1)))
            table = p.block_table.cpu().numpy()
            for b in range(2):
                used = table[b, : (n[b] + history[b] + page - 1) // page if n[b] else 0]
                bad |= bool(((used < 0) | (used >= p.num_pages)).any())
            out.fill_(7.0)
            lse.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _, g, _, _ in made:
                g.replay()
        torch.cuda.synchronize()
        for step, _, out, lse in made:
            check(out, lse, step.reference(), f"{n} tokens")
    assert bad and binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE


def test_two_calls_at_once(cuda_device):
    """Two streams, a workspace each: neither call sees the other."""
    steps = [Step((64, 8), 128, 64, [61, 5], [3000, 900], 38, cuda_device),
             Step((16, 4), 128, 16, [7] * 20, [600] * 20, 39, cuda_device, window=200, extent=200, bias=F32)]
    streams = [torch.cuda.Stream() for _ in steps]
    made = [binding.alloc_tree_workspace(x.params, cuda_device) for x in steps]
    want = [x.call(workspace=ws)[:2] for x, ws in zip(steps, made)]
    for x, got in zip(steps, want):
        check(*got, x.reference(), "alone")
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for x, ws, stream in zip(steps, made, streams):
            with torch.cuda.stream(stream):
                outs.append(x.call(workspace=ws, stream=stream)[:2])
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    assert all(binding.inkling_attn_read_device_error(ws) == 0 for ws in made)


def at_the_end(device, L, tokens, heads, dim, page, window, seed, kind="tree"):
    """One sequence that ends at key L and names few pages, all of them at the end."""
    width = (L + page - 1) // page
    g = torch.Generator().manual_seed(seed)
    pools = [torch.randn(80, heads[1], page, dim, generator=g).to(BF16) for _ in range(2)]
    table = torch.full((1, width), -1, dtype=torch.int32)
    table[0, -60:] = torch.randperm(80, generator=g)[:60].to(torch.int32)
    q = torch.randn(tokens, heads[0], dim, generator=g).to(BF16)
    params = binding.make_params(num_seqs=1, num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page,
                                 max_pages_per_seq=width, num_pages=80, rel_extent=1, window=window, sm_scale=dim ** -0.5)
    parents = parents_of(kind, tokens, np.random.default_rng(seed))
    return params, parents, table, [x.to(device) for x in (q, *pools, table, torch.tensor([L], dtype=torch.int32),
                                                           torch.tensor([0, tokens], dtype=torch.int32))]


@pytest.mark.parametrize("tokens,page,window,bias,softcap,bad", [
    (1, 64, 300, None, 0.0, None), (9, 64, 300, None, 30.0, None), (70, 64, 260, F32, 0.0, None), (20, 16, 100, None, 0.0, None),
    (20, 16, 100, BF16, 0.0, None), (9, 16, 300, None, 0.0, float("inf"))])
def test_the_last_key_there_is(cuda_device, tokens, page, window, bias, softcap, bad):
    """A length of 2^31 less a page, the most a table may name.  The oracle takes the last pages alone: only distances count."""
    dev, L, heads, dim = cuda_device, 2**31 - page, (8, 2), 128
    params, parents, table, (q, k, v, table_d, lens, cu) = at_the_end(dev, L, tokens, heads, dim, page, window, 33)
    ints = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)
    par, words = torch.tensor(parents, dtype=torch.int32, device=dev), (tokens + 31) // 32
    pos, anc = ints(tokens), ints(tokens, words)
    if bad is not None:   # the last token's own key, which nobody else sees
        v[int(table[0, -1]), :, (L - 1) % page, 3] = bad
    rel = None
    if bias is not None:
        params.rel_extent = window
        rel = torch.randn(tokens, heads[0], window, generator=torch.Generator().manual_seed(34)).to(bias).to(dev)
    ws = binding.alloc_tree_workspace(params, dev)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=dev)
    binding.inkling_attn_tree_plan(params, cu, lens, par, pos, anc, ws)
    for _ in range(2):
        binding.inkling_attn_tree(params, q, cu, k, v, table_d, lens, pos, anc, out, ws, rel_logits=rel, softcap=softcap, lse=lse)
    assert binding.inkling_attn_read_device_error(ws) == 0
    at, seen = oracle.plan(parents, L - tokens, words)
    assert np.array_equal(pos.cpu().numpy(), at) and np.array_equal(anc.cpu().numpy().view(np.uint32), seen)
    first = (table.shape[1] - 60) * page
    with np.errstate(invalid="ignore"):
        ref = oracle.attention(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, window=window,
                               sm_scale=dim ** -0.5, cu_q=np.array([0, tokens]), seq_lens=np.array([L - first]), q_bits=bits(q),
                               k_bits=bits(k), v_bits=bits(v), block_table=table[:, -60:].numpy(), positions=at - first,
                               ancestors=seen, softcap=softcap, rel=None if rel is None else rel.double().cpu().numpy())
    if bad is not None:
        want = ref[0]
        odd = ~np.isfinite(want)
        assert odd.any() and odd.sum() == heads[0] and np.array_equal(out.double().cpu().numpy()[odd], want[odd])
        out[torch.from_numpy(odd).to(dev)] = 0.0
        ref = (np.where(odd, 0.0, want), ref[1], np.where(odd, 0.0, ref[2]), ref[3])
    check(out, lse, ref, f"window {window}")


@pytest.mark.parametrize("window", [20, 70, 250, 500])
def test_the_last_tile_as_a_run_of_its_own(cuda_device, window):
    """One KV head, pages smaller than a tile, a length of 2^31 less a page: runs are cut so that the last tile stands alone (the
    other chain has no tile, and none would follow)."""
    dev, page, heads, dim, tokens = cuda_device, 16, (8, 1), 128, 9
    L = 2**31 - page
    params, parents, table, (q, k, v, table_d, lens, cu) = at_the_end(dev, L, tokens, heads, dim, page, window, 37)
    ints = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)
    par, pos, anc = torch.tensor(parents, dtype=torch.int32, device=dev), ints(tokens), ints(tokens, 1)
    ws = binding.alloc_tree_workspace(params, dev)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=dev)
    binding.inkling_attn_tree_plan(params, cu, lens, par, pos, anc, ws)
    binding.inkling_attn_tree(params, q, cu, k, v, table_d, lens, pos, anc, out, ws, lse=lse)
    assert binding.inkling_attn_read_device_error(ws) == 0
    at, seen = oracle.plan(parents, L - tokens, 1)
    first = (table.shape[1] - 60) * page
    ref = oracle.attention(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, window=window,
                           sm_scale=dim ** -0.5, cu_q=np.array([0, tokens]), seq_lens=np.array([L - first]), q_bits=bits(q),
                           k_bits=bits(k), v_bits=bits(v), block_table=table[:, -60:].numpy(), positions=at - first, ancestors=seen)
    check(out, lse, ref, f"window {window}")


@pytest.mark.parametrize("tokens", [1, 20])
def test_the_longest_history(cuda_device, tokens):
    """2^31 - 256 keys, all seen.  Keys of zeros weigh the same; values are powers of two, a channel each: sums of up to 2^23 of
    them on a chain are exact in fp32, and so is the output after its rounding to bf16.  lse = log(number of keys), off by a few
    roundings of its value."""
    dev, L, heads, dim, page = cuda_device, 2**31 - 256, (8, 1), 64, 256
    params, parents, table, (q, k, v, table_d, lens, cu) = at_the_end(dev, L, tokens, heads, dim, page, -1, 35, "chain")
    k.zero_()
    value = torch.tensor([1.0, -2.0, 0.5, 0.0], device=dev).repeat(dim // 4)
    v[:] = value
    table_d.clamp_(min=7)
    ints = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)
    par, pos, anc = torch.tensor(parents, dtype=torch.int32, device=dev), ints(tokens), ints(tokens, 1)
    ws = binding.alloc_tree_workspace(params, dev)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=dev)
    binding.inkling_attn_tree_plan(params, cu, lens, par, pos, anc, ws)
    binding.inkling_attn_tree(params, q, cu, k, v, table_d, lens, pos, anc, out, ws, lse=lse)
    assert binding.inkling_attn_read_device_error(ws) == 0
    assert torch.equal(out.float(), value.expand_as(out))
    seen = torch.arange(L - tokens + 1, L + 1, dtype=torch.float64)
    assert ((lse.cpu().double() - seen.log()[:, None]).abs() <= 2.0 ** -20 * (1.0 + math.log(L))).all()


@pytest.mark.parametrize("tokens,heads", [(20, (8, 1)), (3, (16, 2))])
def test_an_infinity_near_the_end_of_a_long_history(cuda_device, tokens, heads):
    """Found at once (no wait runs out), given to the rows that see it and to no other channel."""
    dev, L, page = cuda_device, 3_000_000, 64
    params, parents, table, (q, k, v, table_d, lens, cu) = at_the_end(dev, L, tokens, heads, 128, page, -1, 36, "chain")
    table_d.clamp_(min=1)
    k[0], v[0] = k[1], v[1]
    at = L - 2                 # of a page that is named once
    table_d[table_d == 0] = 1
    table_d[0, at // page] = 0
    ints = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)
    par, pos, anc = torch.tensor(parents, dtype=torch.int32, device=dev), ints(tokens), ints(tokens, 1)
    ws = binding.alloc_tree_workspace(params, dev)
    binding.inkling_attn_tree_plan(params, cu, lens, par, pos, anc, ws)
    seen = torch.arange(L - tokens, L, device=dev) >= at
    outs = []
    for value in (0.0, float("inf"), float("nan")):
        v[0, :, at % page, 3] = value
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
        binding.inkling_attn_tree(params, q, cu, k, v, table_d, lens, pos, anc, out, ws, lse=lse)
        assert binding.inkling_attn_read_device_error(ws) == 0
        outs.append((out.float(), lse))
    rest = [c for c in range(128) if c != 3]
    for out, lse in outs[1:]:
        assert torch.equal(lse, outs[0][1])
        assert torch.equal(out[..., rest], outs[0][0][..., rest]) and torch.equal(out[~seen], outs[0][0][~seen])
    assert torch.isposinf(outs[1][0][seen][..., 3]).all() and torch.isnan(outs[2][0][seen][..., 3]).all()
