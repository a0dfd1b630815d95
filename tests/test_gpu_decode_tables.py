"""The decode's staged slices of the block table: pages smaller than a tile, units of several splits."""
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from paged_attention_relative_gqa_gb300 import workloads as W
from tests.parity import compare, oracle_full

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [8, 16, 32, 64])
@pytest.mark.parametrize("heads,dim", [((32, 2), 64), ((32, 2), 128), ((64, 4), 64), ((8, 4), 128), ((8, 4), 64)])
def test_every_tile_comes_from_its_own_sequence(cuda_device, heads, dim, page):
    """More units than CTAs, of a few tiles each: a loader's lanes that run ahead of the one that reads a
    slice overwrite it."""
    lens = [1500 + 97 * i for i in range(24)]
    prob = W.make_problem(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, rel_extent=512,
                          window=-1, q_lens=[1] * 24, seq_lens=lens, seed=61, device=cuda_device)
    params = binding.params_of(prob)
    ws = binding.alloc_workspace(params, True, cuda_device)
    first = None
    for _ in range(5):
        out = binding.run(prob, out=torch.zeros_like(prob.q), workspace=ws)
        assert binding.inkling_attn_read_device_error(ws) == 0
        if first is None:
            first = out
            compare(out.float().cpu().numpy(), oracle_full(prob), f"page {page}")
        assert torch.equal(out, first)


@pytest.mark.parametrize("page,lens", [(8, [400000, 5, 330011]), (16, [650000]), (64, [2600003])])
def test_units_of_more_entries_than_are_staged(cuda_device, page, lens):
    """A table this long is cut into the most splits there are, each with more pages than the slice that is
    kept in shared memory (576).  The pages are named many times over: the pool is small."""
    prob = W.make_problem(num_q_heads=4, num_kv_heads=1, head_dim=64, page_size=page, rel_extent=16, window=-1,
                          q_lens=[1] * len(lens), seq_lens=[1000] * len(lens), seed=62, device=cuda_device)
    width = (max(lens) + page - 1) // page
    tiles = (width * page + 63) // 64
    assert (tiles + 63) // 64 * 64 // page > 576
    g = torch.Generator().manual_seed(63)
    prob.block_table = torch.randint(0, prob.num_pages, (len(lens), width), generator=g, dtype=torch.int32).to(cuda_device)
    prob.k_cache = torch.randn(prob.k_cache.shape, generator=g).to(torch.bfloat16).to(cuda_device)
    prob.v_cache = torch.randn(prob.v_cache.shape, generator=g).to(torch.bfloat16).to(cuda_device)
    prob.seq_lens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    prob.seq_lens_list = lens
    params = binding.params_of(prob)
    ws = binding.alloc_workspace(params, True, cuda_device)
    out = binding.run(prob, out=torch.zeros_like(prob.q), workspace=ws)
    assert binding.inkling_attn_read_device_error(ws) == 0
    compare(out.float().cpu().numpy(), oracle_full(prob), f"page {page}")
