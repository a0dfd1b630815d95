"""Operators on trees of drafted tokens without a GPU: refusals before anything is launched, the oracle's closed
forms."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import masked, tree as oracle
from paged_attention_relative_gqa_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


T, B, HQ, HKV, D, PAGE, WIDTH, PAGES, E, WORDS, PATH, KS = 64, 4, 64, 8, 128, 64, 512, 2400, 100, 2, 10, 4
POOL = PAGES * HKV * PAGE * D * 2
ROW = HKV * D * 2


def params(**kw):
    base = dict(num_seqs=B, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, page_size=PAGE, max_pages_per_seq=WIDTH,
                num_pages=PAGES, rel_extent=E, window=-1, sm_scale=0.088)
    base.update(kw)
    return binding.make_params(**base)


# the buffers of each call with their sizes, what is written first; addresses are made up and never dereferenced
def plan_sizes():
    return dict(positions=T * 4, ancestors=T * WORDS * 4, workspace=256, cu=B * 4 + 4, seq_lens=B * 4, parents=T * 4), 3


def attention_sizes():
    rows = T * HQ * D * 2
    return dict(out=rows, lse=T * HQ * 4, workspace=binding.inkling_attn_tree_workspace_bytes(params()), q=rows, k_cache=POOL,
                v_cache=POOL, block_table=B * WIDTH * 4, seq_lens=B * 4, cu=B * 4 + 4, positions=T * 4, ancestors=T * WORDS * 4,
                slopes=HQ * 4, rel=T * HQ * E * 4), 3


def conv_sizes():
    return dict(k_cache=POOL, v_cache=POOL, workspace=256, k=T * ROW, v=T * ROW, cu=B * 4 + 4, seq_lens=B * 4,
                block_table=B * WIDTH * 4, parents=T * 4, w_k=HKV * D * KS * 4, w_v=HKV * D * KS * 4,
                state_k=B * (KS - 1) * ROW, state_v=B * (KS - 1) * ROW), 3


def state_sizes():
    state = B * (KS - 1) * ROW
    return dict(out_k=state, out_v=state, workspace=256, state_k=state, state_v=state, k=T * ROW, v=T * ROW, cu=B * 4 + 4,
                path=B * PATH * 4, path_lens=B * 4), 3


def commit_sizes():
    return dict(k_cache=POOL, v_cache=POOL, k2=POOL, v2=POOL, new_lens=B * 4, workspace=256, cu=B * 4 + 4, seq_lens=B * 4,
                block_table=B * WIDTH * 4, path=B * PATH * 4, path_lens=B * 4), 6


def write_sizes():
    return dict(q_out=T * HQ * D * 2, k_cache=POOL, v_cache=POOL, workspace=256, positions=T * 4), 4


def addresses(names):
    return {n: (1 << 40) * (i + 1) for i, n in enumerate(names)}


def plan(lib, at, p=None, total=T, words=WORDS, ws=1 << 30):
    return lib.inkling_attn_tree_plan(ctypes.byref(p or params()), at["cu"], total, at["seq_lens"], at["parents"], words,
                                      at["positions"], at["ancestors"], at["workspace"], ws, None)


def attention(lib, at, p=None, total=T, words=WORDS, ws=1 << 30, softcap=0.0, bf16=0, no_tree=False):
    tree = binding.ink_attn_tree_t(at["positions"], at["ancestors"], words)
    opts = binding.ink_attn_tree_options_t(softcap, at["slopes"], at["rel"], bf16)
    return lib.inkling_attn_tree(ctypes.byref(p or params()), None if no_tree else ctypes.byref(tree), ctypes.byref(opts),
                                 at["q"], at["cu"], total, at["k_cache"], at["v_cache"], at["block_table"], at["seq_lens"],
                                 at["out"], at["lse"], at["workspace"], ws, None)


def conv(lib, at, p=None, total=T, ks=KS, ws=1 << 30):
    return lib.inkling_attn_kv_conv_write_tree(ctypes.byref(p or params()), at["k"], at["v"], at["cu"], total, at["seq_lens"],
                                               at["block_table"], at["parents"], at["w_k"], at["w_v"], ks, at["state_k"],
                                               at["state_v"], at["k_cache"], at["v_cache"], at["workspace"], ws, None)


def state(lib, at, p=None, total=T, ks=KS, width=PATH, ws=1 << 30):
    return lib.inkling_attn_kv_conv_state_tree(ctypes.byref(p or params()), at["k"], at["v"], at["cu"], total, at["path"],
                                               at["path_lens"], width, ks, at["state_k"], at["state_v"], at["out_k"],
                                               at["out_v"], at["workspace"], ws, None)


def commit(lib, at, p=None, width=PATH, pools=2, ws=1 << 30):
    two = ctypes.c_void_p * 2
    return lib.inkling_attn_tree_commit(ctypes.byref(p or params()), at["cu"], at["seq_lens"], at["block_table"], at["path"],
                                        at["path_lens"], width, pools, two(at["k_cache"], at["k2"]),
                                        two(at["v_cache"], at["v2"]), at["new_lens"], at["workspace"], ws, None)


def write(lib, at, p=None, total=T, ws=1 << 30):
    rope = binding.ink_norm_rope_t(None, None, 1e-6, 1 << 20, 64, 0, 1.0)
    far = [ctypes.c_void_p((1 << 50) + (1 << 40) * i) for i in range(3)]
    small = ctypes.c_void_p(1 << 21)
    return lib.inkling_attn_qk_norm_rope_write_at(ctypes.byref(p or params()), ctypes.byref(rope), at["positions"], far[0],
                                                  HQ * D, far[1], HKV * D, far[2], HKV * D, small, total, small, small,
                                                  at["q_out"], at["k_cache"], at["v_cache"], at["workspace"], ws, None)


CALLS = {"plan": (plan, plan_sizes), "attention": (attention, attention_sizes), "conv": (conv, conv_sizes),
         "state": (state, state_sizes), "commit": (commit, commit_sizes), "write": (write, write_sizes)}
OPTIONAL = {("attention", "lse"), ("attention", "slopes"), ("attention", "rel"), ("commit", "new_lens")}


@pytest.mark.parametrize("name", CALLS)
def test_overlaps_are_refused(lib, name):
    call, sizes = CALLS[name]
    size, written = sizes()
    for w in list(size)[:written]:
        for x in size:
            if x == w:
                continue
            step = 256 if "workspace" in (w, x) else 16   # (addresses stay aligned)
            for off in {0, (size[x] - 1) // step * step, -((size[w] - 1) // step * step)}:
                at = addresses(size)
                at[w] = at[x] + off
                assert call(lib, at) == 2, (w, x, off)


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned_pointers_are_refused(lib, name):
    call, sizes = CALLS[name]
    size, _ = sizes()
    for x in size:
        if (name, x) not in OPTIONAL:
            assert call(lib, dict(addresses(size), **{x: None})) == 1, x
        assert call(lib, dict(addresses(size), **{x: addresses(size)[x] + 1})) == 5, x
    if name == "attention":
        assert call(lib, addresses(size), no_tree=True) == 1


@pytest.mark.parametrize("name", CALLS)
def test_bad_sizes_are_refused(lib, name):
    call, sizes = CALLS[name]
    at = addresses(sizes()[0])
    assert call(lib, at, p=params(head_dim=96)) == 2 and call(lib, at, p=params(num_kv_heads=7)) == 2
    assert call(lib, at, p=params(page_size=24)) == 3
    assert call(lib, at, ws=100) == 4
    if name != "commit":
        assert call(lib, at, total=-1) == 2
    if name in ("plan", "attention"):
        assert call(lib, at, words=0) == 2 and call(lib, at, words=17) == 2
    if name in ("conv", "state"):
        assert call(lib, at, ks=0) == 2 and call(lib, at, ks=9) == 2
    if name in ("state", "commit"):
        assert call(lib, at, width=0) == 2
    if name == "commit":
        assert call(lib, at, pools=0) == 2 and call(lib, at, pools=129) == 2
    if name == "attention":
        need = binding.inkling_attn_tree_workspace_bytes(params())
        assert need > 0 and call(lib, at, ws=need - 1) == 4
        assert binding.inkling_attn_tree_workspace_bytes(params(head_dim=32)) == 0
        for cap in (-1.0, 1e-7, 1e7, float("nan"), float("inf")):
            assert call(lib, at, softcap=cap) == 2
        assert call(lib, at, total=1 << 26) == 7
        odd = dict(at, rel=at["rel"] + 2)
        assert call(lib, odd) == 5 and call(lib, dict(odd, out=odd["rel"] - 2), bf16=1) == 2   # (bf16 may lie there)


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do_launches_nothing(lib, name):
    call, sizes = CALLS[name]
    at = addresses(sizes()[0])
    assert call(lib, at, p=params(num_seqs=0)) == 0
    if name not in ("state", "commit"):
        assert call(lib, at, total=0) == 0
    if name == "state":
        assert call(lib, at, ks=1) == 0


def test_binding_checks_before_the_library(lib):
    p = params(num_seqs=1, num_q_heads=2, num_kv_heads=1, head_dim=64, page_size=16, max_pages_per_seq=2, num_pages=3)
    q, cache = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    one, two, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    bits, table = one.view(1, 1), two.view(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.inkling_attn_tree_plan(p, two, one, one, one, bits, ws)
    with pytest.raises(TypeError):
        binding.inkling_attn_tree_plan(p, two, one, None, one, bits, ws)
    with pytest.raises(ValueError, match="CUDA"):
        binding.inkling_attn_tree(p, q, two, cache, cache, table, one, one, bits, q, ws)
    with pytest.raises(ValueError, match="CUDA"):
        binding.inkling_attn_kv_conv_write_tree(p, q, q, two, one, table, one, None, None, None, None, cache, cache, ws)
    with pytest.raises(ValueError, match="CUDA"):
        binding.inkling_attn_kv_conv_state_tree(p, q, q, two, bits, one, q, q, q, q, ws)
    with pytest.raises(ValueError, match="CUDA"):
        binding.tree_pools(p, [cache], [cache])
    with pytest.raises(ValueError, match="equally many"):
        binding.tree_pools(p, [cache], [])
    with pytest.raises(ValueError, match="equally many"):
        binding.tree_pools(p, [], [])
    with pytest.raises(TypeError, match="tree_pools"):
        binding.inkling_attn_tree_commit(p, two, one, table, bits, one, [cache], one, ws)


# ------------------------------------------------------------------ the oracle


def test_oracle_plan_and_path():
    pos, bits = oracle.plan([-1, 0, 0, 1, 3, -1], 10, 1)
    assert pos.tolist() == [10, 11, 11, 12, 13, 10]
    assert bits[:, 0].tolist() == [1, 3, 5, 11, 27, 32]
    pos, bits = oracle.plan(list(range(-1, 40)), 0, 2)
    assert pos.tolist() == list(range(41)) and bits[40].tolist() == [2**32 - 1, 2**9 - 1]
    assert oracle.accepted([0, 2, 5, -1], 3, 6) == [0, 2, 5]
    for path, m, n in (([0, 0], 2, 6), ([3, 1], 2, 6), ([0, 6], 2, 6), ([-1, 0], 2, 6), ([0], 2, 6), ([0, 1], -1, 6)):
        assert oracle.accepted(path, m, n) == []


def test_oracle_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(0)
    raw = lambda *s: (rng.normal(size=s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    kw = dict(num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=8, sm_scale=0.1, cu_q=np.array([0, 5, 6]),
              seq_lens=np.array([17, 9]), q_bits=raw(6, 4, 64), k_bits=raw(6, 2, 8, 64), v_bits=raw(6, 2, 8, 64),
              block_table=np.array([[0, 3, 1], [4, 2, 99]]), softcap=2.0, slopes=np.array([0.1, 0.2, 0.0, 1.0]))
    pos, bits = zip(oracle.plan([-1, 0, 1, 2, 3], 12, 1), oracle.plan([-1], 8, 1))
    pos, bits = np.concatenate(pos), np.concatenate(bits)
    for window in (-1, 3, 14):
        a = oracle.attention(window=window, positions=np.concatenate([np.arange(12, 17), [8]]),
                             ancestors=np.array([[1], [3], [7], [15], [31], [1]], np.uint32), **kw)
        b = masked.attention(window=window, **kw)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


def test_oracle_attention_weighs_by_position():
    """Equal scores: siblings are not seen, a bias goes by the depth."""
    kw = dict(num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=8, window=-1, sm_scale=1.0, cu_q=np.array([0, 3]),
              seq_lens=np.array([5]), q_bits=np.zeros((3, 1, 64), np.uint16), block_table=np.array([[0]]),
              k_bits=np.zeros((1, 1, 8, 64), np.uint16),
              v_bits=(np.arange(8, dtype=np.float32)[None, None, :, None].repeat(64, 3).view(np.uint32) >> 16).astype(np.uint16))
    pos, bits = oracle.plan([-1, 0, 0], 2, 1)
    out, lse, _, _ = oracle.attention(positions=pos, ancestors=bits, **kw)
    assert np.allclose(out[:, 0, 0], [1.0, 1.5, 7 / 4]) and np.allclose(lse[:, 0], np.log([3, 4, 4]))
    rel = np.log(np.array([1.0, 2.0, 4.0]))[None, None].repeat(3, 0)
    _, lse, _, _ = oracle.attention(positions=pos, ancestors=bits, rel=rel, **kw)
    assert np.allclose(lse[:, 0], np.log([1 + 2 + 4, 1 + 2 + 4 + 4, 1 + 2 + 4 + 4]))
    _, lse, _, _ = oracle.attention(positions=pos, ancestors=bits, **dict(kw, window=2))
    assert np.allclose(lse[:, 0], np.log([2, 2, 2]))


def test_oracle_convolution_follows_the_tree():
    one = lambda v: (np.float32(v).reshape(1).view(np.uint32) >> 16).astype(np.uint16)[0]
    x = np.array([one(v) for v in (1, 2, 4, 8)], np.uint16).reshape(4, 1, 1)
    st = np.array([one(v) for v in (16, 32)], np.uint16).reshape(2, 1, 1)
    w = np.array([100.0, 10.0, 1.0]).reshape(1, 1, 3)
    y, _ = oracle.conv(x, st, [-1, 0, 0, 2], w)
    assert y.ravel().tolist() == [1 + 320 + 1600, 2 + 10 + 3200, 4 + 10 + 3200, 8 + 40 + 100]
    assert oracle.conv_state(x, st, [0, 2, 3]).ravel().tolist() == x.ravel()[[2, 3]].tolist()
    assert oracle.conv_state(x, st, [1]).ravel().tolist() == [st.ravel()[1], x.ravel()[1]]
    assert np.array_equal(oracle.conv_state(x, st, []), st)


def test_oracle_commit():
    cache = np.arange(32).reshape(4, 1, 8, 1).copy()
    oracle.commit(cache, [2, 0], 8, 4, 6, [1, 3, 4])   # rows 7, 9, 10 to 6, 7, 8
    line = np.concatenate((cache[2].ravel(), cache[0].ravel()))
    want = np.concatenate((np.arange(16, 24), np.arange(8)))
    want[[6, 7, 8]] = want[[7, 9, 10]]
    assert line.tolist() == want.tolist()
