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
