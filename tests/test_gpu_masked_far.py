"""Masked attention at the end of the positions there are: the last tile before 2^31."""
import numpy as np
import pytest
import torch

from oracle import masked as oracle
from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import bits, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decode,tokens,window,softcap", [(False, 1, 300, 0.0), (False, 9, 300, 30.0), (False, 70, 260, 0.0),
                                                          (False, 5, 3000, 30.0), (False, 5, 3000, 0.0), (True, 1, 700, 0.0)])
def test_the_last_tile_before_2_to_31(cuda_device, decode, tokens, window, softcap):
    """A history of 2^31 - 64 keys: the tile from 2^31 - 128 on is half full.  The table names few pages; all but
    its last entries lie outside the window and the pool."""
    dev, D, page, Hq, Hkv = cuda_device, 128, 64, 8, 2
    width = (1 << 25) - 1
    L = width * page
    g = torch.Generator().manual_seed(70)
    pools = [torch.randn(80, Hkv, page, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    table = torch.full((1, width), -1, dtype=torch.int32)
    table[0, -60:] = torch.randperm(80, generator=g)[:60].to(torch.int32)
    q = torch.randn(tokens, Hq, D, generator=g).to(torch.bfloat16)
    lens, cu = torch.tensor([L], dtype=torch.int32), torch.tensor([0, tokens], dtype=torch.int32)
    params = binding.make_params(num_seqs=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=page,
                                 max_pages_per_seq=width, num_pages=80, rel_extent=1, window=window, sm_scale=D ** -0.5)
    ws = binding.alloc_masked_workspace(params, decode, dev)
    out = torch.full((tokens, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((tokens, Hq), 7.0, device=dev)
    kc, vc, bt, sl, qd = pools[0].to(dev), pools[1].to(dev), table.to(dev), lens.to(dev), q.to(dev)
    # another call first, so that shared memory holds something
    for _ in range(2):
        if decode:
            binding.inkling_attn_decode_masked(params, qd, kc, vc, bt, sl, out, ws, softcap=softcap, lse=lse)
        else:
            binding.inkling_attn_prefill_masked(params, qd, cu.to(dev), kc, vc, bt, sl, out, ws, softcap=softcap, lse=lse)
    assert binding.inkling_attn_read_device_error(ws) == 0
    ref = oracle.attention(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=page, window=window, sm_scale=D ** -0.5,
                           cu_q=np.array([0, tokens]), seq_lens=np.array([L]), q_bits=bits(q), k_bits=bits(pools[0]),
                           v_bits=bits(pools[1]), block_table=table.numpy(), softcap=softcap)
    check(out, lse, ref, f"window {window}")
