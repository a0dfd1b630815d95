"""Shared by the tests of the operators on trees of drafted tokens."""
import numpy as np
import torch

from oracle import tree as oracle
from paged_attention_relative_gqa_gb300 import binding
from paged_attention_relative_gqa_gb300 import workloads as W
from tests.masked_common import bits


def parents_of(kind, n, rng):
    """A chain, a random tree, a tree of `wide` levels, several roots, or all tokens beside one another."""
    if n == 0:
        return []
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "flat":
        return [-1] * n
    if kind == "forest":
        return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)]   # "tree"


class Step:
    """A step's drafted tokens: a problem (its q_lens tokens drafted) with their parents, positions and bits."""

    def __init__(self, heads, dim, page, n, history, seed, device, kind="tree", window=-1, extent=1, bias=None,
                 q_std=1.0, words=None, max_pages=None):
        rng = np.random.default_rng(seed)
        self.prob = W.make_problem(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page,
                                   rel_extent=extent, window=window, q_lens=n, seq_lens=[a + b for a, b in zip(n, history)],
                                   seed=seed, device=device, max_pages=max_pages,
                                   bias_dtype=bias or torch.float32)
        if q_std != 1.0:
            self.prob.q = (self.prob.q.float() * q_std).to(torch.bfloat16)
        kinds = [kind] * len(n) if isinstance(kind, str) else kind
        self.parents = [parents_of(k, x, rng) for k, x in zip(kinds, n)]
        self.words = words or max(1, (max(n + [1]) + 31) // 32)
        pos, anc = [], []
        for p, H in zip(self.parents, history):
            a, b = oracle.plan(p, H, self.words)
            pos.append(a)
            anc.append(b)
        self.positions_np = np.concatenate(pos)
        self.ancestors_np = np.concatenate(anc)
        self.rel = self.prob.rel_logits if bias is not None else None
        self.device = device
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device)
        self.positions = to(self.positions_np.astype(np.int32))
        self.ancestors = to(self.ancestors_np.view(np.int32))
        self.parents_t = torch.tensor([x for p in self.parents for x in p], dtype=torch.int32, device=device)
        self.params = binding.params_of(self.prob)

    def reference(self, **opts):
        p = self.prob
        slopes = opts.get("slopes")
        return oracle.attention(num_q_heads=p.num_q_heads, num_kv_heads=p.num_kv_heads, head_dim=p.head_dim,
                                page_size=p.page_size, window=p.window, sm_scale=p.sm_scale, cu_q=p.cu_q_lens.cpu().numpy(),
                                seq_lens=p.seq_lens.cpu().numpy(), q_bits=bits(p.q), k_bits=bits(p.k_cache),
                                v_bits=bits(p.v_cache), block_table=p.block_table.cpu().numpy(),
                                positions=self.positions.cpu().numpy(),
                                ancestors=self.ancestors.cpu().numpy().view(np.uint32),
                                rel=None if self.rel is None else self.rel.double().cpu().numpy(),
                                softcap=opts.get("softcap", 0.0), slopes=None if slopes is None else slopes.cpu().numpy())

    def call(self, workspace=None, stream=None, **opts):
        p = self.prob
        ws = binding.alloc_tree_workspace(self.params, p.q.device) if workspace is None else workspace
        out = torch.full_like(p.q, 7.0)
        lse = torch.full(p.q.shape[:2], 7.0, dtype=torch.float32, device=p.q.device)
        binding.inkling_attn_tree(self.params, p.q, p.cu_q_lens, p.k_cache, p.v_cache, p.block_table, p.seq_lens,
                                  self.positions, self.ancestors, out, ws, rel_logits=self.rel, lse=lse, stream=stream, **opts)
        return out, lse, ws
