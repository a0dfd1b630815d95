"""Positions and visible tokens of drafted trees, on the GPU against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import tree as oracle
from paged_attention_relative_gqa_gb300 import binding
from tests.tree_common import parents_of

pytestmark = pytest.mark.gpu
GUARD = 1234567


def params(B):
    return binding.make_params(num_seqs=B, num_q_heads=2, num_kv_heads=1, head_dim=64, page_size=16, max_pages_per_seq=4,
                               num_pages=4, rel_extent=1, window=-1, sm_scale=1.0)


def run(parents, history, words, device, rows=None, cu=None, seq_lens=None):
    n = [len(p) for p in parents]
    T = sum(n) if rows is None else rows
    flat = [x for p in parents for x in p]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    par = torch.full((T,), -7, dtype=torch.int32, device=device)
    par[: len(flat)] = ints(flat)
    cu = ints([0] + np.cumsum(n).tolist() if cu is None else cu)
    lens = ints([a + b for a, b in zip(n, history)] if seq_lens is None else seq_lens)
    pos = torch.full((T,), GUARD, dtype=torch.int32, device=device)
    anc = torch.full((T, words), GUARD, dtype=torch.int32, device=device)
    P = params(len(parents))
    ws = binding.alloc_tree_workspace(P, device)
    binding.inkling_attn_tree_plan(P, cu, lens, par, pos, anc, ws)
    return pos.cpu().numpy(), anc.cpu().numpy().view(np.uint32), binding.inkling_attn_read_device_error(ws)


@pytest.mark.parametrize("kind", ["chain", "tree", "forest", "flat"])
@pytest.mark.parametrize("n,words", [([1], 1), ([7, 0, 1, 32], 1), ([33, 2, 64], 2), ([5], 16), ([512, 100, 511], 16),
                                     ([90] * 40, 3)])
def test_against_the_oracle(cuda_device, kind, n, words):
    rng = np.random.default_rng(len(n) + words)
    parents = [parents_of(kind, x, rng) for x in n]
    history = rng.integers(0, 100000, len(n)).tolist()
    pos, anc, err = run(parents, history, words, cuda_device)
    assert err == 0
    want = [oracle.plan(p, h, words) for p, h in zip(parents, history)]
    assert np.array_equal(pos, np.concatenate([w[0] for w in want]))
    assert np.array_equal(anc, np.concatenate([w[1] for w in want]))


def test_rows_behind_the_last_sequence_stay(cuda_device):
    pos, anc, err = run([[-1, 0, 0], [-1]], [5, 9], 2, cuda_device, rows=9)
    assert err == 0 and pos.tolist() == [5, 6, 6, 9] + [GUARD] * 5 and (anc[4:] == GUARD).all()


def test_parents_that_no_tree_has(cuda_device):
    """Its own child, a later token, a number below -1: reported, and a root."""
    bad = [-1, 1, 5, 0, -2, 2]
    pos, anc, err = run([bad], [10], 1, cuda_device)
    assert err == binding.DEVERR_BAD_TREE
    want = oracle.plan([-1, -1, -1, 0, -1, 2], 10, 1)
    assert np.array_equal(pos, want[0]) and np.array_equal(anc, want[1])


def test_sequences_that_are_skipped(cuda_device):
    """More tokens than bits, than length, rows that are not there, offsets that fall: reported one by one."""
    tree = [-1, 0, 1, 1]
    for kw, bit in ((dict(parents=[[-1] * 33, tree]), binding.DEVERR_QLEN_EXCEEDS_MAX),
                    (dict(parents=[tree, tree], seq_lens=[3, 14]), binding.DEVERR_QLEN_EXCEEDS_KV),
                    (dict(parents=[tree, tree], cu=[-4, 4, 8]), binding.DEVERR_BAD_ROWS),
                    (dict(parents=[tree, tree], cu=[9, 4, 8]), binding.DEVERR_BAD_ROWS)):
        pos, anc, err = run(history=[10, 10], words=1, device=cuda_device, **kw)
        assert err == bit
        first = len(kw["parents"][0])
        assert (pos[:first] == GUARD).all() and (anc[:first] == GUARD).all()
        want = oracle.plan(tree, 10, 1)
        assert np.array_equal(pos[first:], want[0]) and np.array_equal(anc[first:], want[1])
    pos, anc, err = run([tree, tree], [10, 10], 1, cuda_device, cu=[0, 4, 9])
    assert err == binding.DEVERR_BAD_ROWS and (pos[4:] == GUARD).all()


def test_captured_and_replayed_with_other_trees(cuda_device):
    P = params(2)
    ws = binding.alloc_tree_workspace(P, cuda_device)
    rng = np.random.default_rng(3)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)
    par, cu, lens = ints(parents_of("tree", 40, rng) + parents_of("chain", 24, rng)), ints([0, 40, 64]), ints([50, 60])
    pos, anc = torch.zeros_like(par), torch.zeros(64, 2, dtype=torch.int32, device=cuda_device)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        binding.inkling_attn_tree_plan(P, cu, lens, par, pos, anc, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.inkling_attn_tree_plan(P, cu, lens, par, pos, anc, ws)
    for n in ([40, 24], [3, 61], [64, 0]):
        trees = [parents_of("tree", x, rng) if x else [] for x in n]
        torch.cuda.synchronize()
        par.copy_(ints([x for t in trees for x in t]))
        cu.copy_(ints([0, n[0], 64]))
        lens.copy_(ints([n[0] + 7, n[1] + 1000]))
        g.replay()
        want = [oracle.plan(t, h, 2) for t, h in zip(trees, (7, 1000))]
        assert np.array_equal(pos.cpu().numpy(), np.concatenate([w[0] for w in want]))
        assert np.array_equal(anc.cpu().numpy().view(np.uint32), np.concatenate([w[1] for w in want]))
    assert binding.inkling_attn_read_device_error(ws) == 0
