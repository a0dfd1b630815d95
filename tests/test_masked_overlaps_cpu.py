"""Buffers of the masked operators that overlap are refused before anything is launched (no GPU; that buffers side
by side are taken is tested on one)."""
import ctypes

import pytest

from paged_attention_relative_gqa_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


T, B, HQ, HKV, D, PAGE, WIDTH, PAGES = 64, 4, 64, 8, 128, 64, 512, 2400
PARAMS = binding.make_params(num_seqs=B, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, page_size=PAGE,
                             max_pages_per_seq=WIDTH, num_pages=PAGES, rel_extent=1, window=-1, sm_scale=0.088)
POOL = PAGES * HKV * PAGE * D * 2
OVERLAP = 2   # INK_ERR_BAD_SHAPE


def where(names):
    """An address of its own, never dereferenced, for each name."""
    return {n: (1 << 40) * (i + 1) for i, n in enumerate(names)}


def attention(lib, decode, at):
    mask = binding.ink_attn_mask_t(0.0, at["key_begin"], at["key_end"], at["slopes"])
    head = [ctypes.byref(PARAMS), ctypes.byref(mask), at["q"]]
    tail = [at[n] for n in ("k_cache", "v_cache", "block_table", "seq_lens", "out", "lse", "workspace")] + [1 << 30, None]
    if decode:
        return lib.inkling_attn_decode_masked(*head, *tail)
    return lib.inkling_attn_prefill_masked(*head, at["cu"], T, *tail)


@pytest.mark.parametrize("decode", [False, True])
def test_attention(lib, decode):
    rows = B if decode else T
    need = binding.inkling_attn_masked_workspace_bytes(PARAMS, decode)
    size = dict(out=rows * HQ * D * 2, lse=rows * HQ * 4, workspace=need, q=rows * HQ * D * 2, k_cache=POOL, v_cache=POOL,
                block_table=B * WIDTH * 4, seq_lens=B * 4, key_begin=rows * 4, key_end=rows * 4, slopes=HQ * 4)
    if not decode:
        size["cu"] = B * 4 + 4
    for w in ("out", "lse", "workspace"):
        for x in size:
            if x == w:
                continue
            step = 256 if "workspace" in (w, x) else 16   # (addresses stay aligned)
            for off in (0, (size[x] - 1) // step * step, -((size[w] - 1) // step * step)):
                at = where(list(size) + ["cu"])
                at[w] = at[x] + off
                assert attention(lib, decode, at) == OVERLAP, (w, x, off)


def write(lib, at):
    rope = binding.ink_norm_rope_t(at["w_q"], at["w_k"], 1e-6, at["inv_freq"], 64, 0, 1.0)
    return lib.inkling_attn_qk_norm_rope_write(
        ctypes.byref(PARAMS), ctypes.byref(rope), at["q"], HQ * D, at["k"], HKV * D, at["v"], HKV * D, at["cu"], T,
        at["seq_lens"], at["block_table"], at["q_out"], at["k_cache"], at["v_cache"], at["workspace"], 1 << 30, None)


def test_norm_and_write(lib):
    size = dict(q_out=T * HQ * D * 2, k_cache=POOL, v_cache=POOL, workspace=256, q=T * HQ * D * 2, k=T * HKV * D * 2,
                v=T * HKV * D * 2, block_table=B * WIDTH * 4, seq_lens=B * 4, cu=B * 4 + 4, w_q=D * 4, w_k=D * 4,
                inv_freq=64 * 2)
    for w in ("q_out", "k_cache", "v_cache", "workspace"):
        for x in size:
            if x == w:
                continue
            step = 256 if "workspace" in (w, x) else 16
            for off in (0, (size[x] - 1) // step * step, -((size[w] - 1) // step * step)):
                at = where(size)
                at[w] = at[x] + off
                if (w, x, off) != ("q_out", "q", 0):   # (in place)
                    assert write(lib, at) == OVERLAP, (w, x, off)
    # in place, k and v are still not written over
    at = where(size)
    at["q_out"] = at["q"]
    at["k"] = at["q"] + 256
    assert write(lib, at) == OVERLAP
