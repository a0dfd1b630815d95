"""Refusals of the masked attention and of the norm, rotation and write (no GPU: validation comes
before any launch), the frequency tables, and closed forms of the fp64 oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import masked as oracle
from paged_attention_relative_gqa_gb300 import binding, build, rotary

OK = ctypes.c_void_p(1 << 20)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def params(**kw):
    base = dict(num_seqs=4, num_q_heads=64, num_kv_heads=8, head_dim=128, page_size=64, max_pages_per_seq=512,
                num_pages=2400, rel_extent=1, window=-1, sm_scale=0.088)
    base.update(kw)
    return binding.make_params(**base)


def prefill(lib, p=None, mask=None, q=OK, cu=OK, total=64, lse=OK, ws=OK, ws_bytes=1 << 30, out=OK, seq=OK):
    p = params() if p is None else p
    m = None if mask is None else ctypes.byref(mask)
    return lib.inkling_attn_prefill_masked(ctypes.byref(p), m, q, cu, total, OK, OK, OK, seq, out, lse, ws, ws_bytes, None)


def decode(lib, p=None, mask=None, q=OK, lse=OK, ws=OK, ws_bytes=1 << 30):
    p = params() if p is None else p
    m = None if mask is None else ctypes.byref(mask)
    return lib.inkling_attn_decode_masked(ctypes.byref(p), m, q, OK, OK, OK, OK, OK, lse, ws, ws_bytes, None)


def mask(softcap=0.0, begin=None, end=None, slopes=None):
    return binding.ink_attn_mask_t(softcap, begin, end, slopes)


@pytest.mark.parametrize("bad,code", [(dict(num_q_heads=12), 2), (dict(head_dim=96), 2), (dict(page_size=48), 3),
                                      (dict(num_pages=1 << 24), 7), (dict(sm_scale=float("nan")), 2)])
def test_bad_params(lib, bad, code):
    p = params(**bad)
    assert binding.inkling_attn_masked_workspace_bytes(p, True) == 0
    assert binding.inkling_attn_masked_workspace_bytes(p, False) == 0
    assert prefill(lib, p) == code and decode(lib, p) == code


def test_bad_options(lib):
    for cap in (-1.0, float("nan"), float("inf"), 1e31):
        assert prefill(lib, mask=mask(cap)) == 2 and decode(lib, mask=mask(cap)) == 2
    odd = (1 << 20) + 2
    for m in (mask(begin=odd), mask(end=odd), mask(slopes=odd)):
        assert prefill(lib, mask=m) == 5 and decode(lib, mask=m) == 5


def test_bad_pointers_sizes_and_workspaces(lib):
    null, odd = ctypes.c_void_p(0), ctypes.c_void_p((1 << 20) + 8)
    assert prefill(lib, q=null) == 1 and prefill(lib, cu=null) == 1 and prefill(lib, seq=null) == 1
    assert prefill(lib, ws=null) == 1 and decode(lib, q=null) == 1 and decode(lib, ws=null) == 1
    assert prefill(lib, q=odd) == 5 and decode(lib, q=odd) == 5 and prefill(lib, out=odd) == 5
    assert prefill(lib, lse=ctypes.c_void_p((1 << 20) + 1)) == 5 and prefill(lib, ws=odd) == 5
    assert prefill(lib, total=-1) == 2
    assert prefill(lib, total=1 << 26) == 7
    for dec in (False, True):
        need = binding.inkling_attn_masked_workspace_bytes(params(), dec)
        assert need > 0
        assert (decode if dec else prefill)(lib, ws_bytes=need - 1) == 4


def test_nothing_to_do_launches_nothing(lib):
    p = params(num_seqs=0)
    assert prefill(lib, p) == 0 and decode(lib, p) == 0 and prefill(lib, total=0) == 0
    # lse and the options may be absent
    assert prefill(lib, p, lse=None) == 0 and decode(lib, p, mask=mask(), lse=None) == 0


def rope(lib, p=None, r=None, q=OK, qs=64 * 128, ks=8 * 128, vs=8 * 128, q_out=None, total=64, ws_bytes=1 << 30):
    p = params() if p is None else p
    r = rope_opts() if r is None else r
    return lib.inkling_attn_qk_norm_rope_write(ctypes.byref(p), ctypes.byref(r), q, qs, OK, ks, OK, vs, OK, total, OK, OK,
                                               ctypes.c_void_p(1 << 24) if q_out is None else q_out, OK, OK, OK, ws_bytes, None)


def rope_opts(w_q=None, w_k=None, eps=1e-6, inv_freq=1 << 20, rot=64, layout=0, scale=1.0):
    return binding.ink_norm_rope_t(w_q, w_k, eps, inv_freq, rot, layout, scale)


def test_norm_rope_refusals(lib):
    for rot in (-16, 8, 24, 144):
        assert rope(lib, r=rope_opts(rot=rot)) == 2
    assert rope(lib, r=rope_opts(layout=2)) == 2 and rope(lib, r=rope_opts(eps=-1.0)) == 2
    assert rope(lib, r=rope_opts(eps=float("nan"))) == 2 and rope(lib, r=rope_opts(scale=float("nan"))) == 2
    assert rope(lib, r=rope_opts(inv_freq=None)) == 1 and rope(lib, q=ctypes.c_void_p(0)) == 1
    assert rope(lib, qs=64 * 128 - 8) == 2 and rope(lib, ks=8) == 2 and rope(lib, vs=0) == 2
    assert rope(lib, qs=64 * 128 + 4) == 5 and rope(lib, q=ctypes.c_void_p((1 << 20) + 8)) == 5
    assert rope(lib, r=rope_opts(w_q=(1 << 20) + 4)) == 5
    assert rope(lib, total=-1) == 2 and rope(lib, ws_bytes=16) == 4
    assert rope(lib, p=params(head_dim=96)) == 2 and rope(lib, p=params(page_size=12)) == 3
    # in place only when a row of q is as long as a row of q_out
    assert rope(lib, qs=64 * 128 + 8, q_out=OK) == 2
    assert rope(lib, total=0, q_out=OK) == 0 and rope(lib, p=params(num_seqs=0)) == 0


def test_buffers_that_overlap_are_refused(lib):
    at = lambda n: ctypes.c_void_p((1 << 20) + n)
    row, rows = 64 * 128 * 2, 64 * 64 * 128 * 2
    for off in (0, 16, row, rows - 16):
        assert prefill(lib, out=at(off)) == 2
        assert prefill(lib, q=at(off), out=OK) == 2
    assert decode(lib) == 2   # q and out are one buffer
    # norm and write: q_out against k and v, the caches against everything
    big = [ctypes.c_void_p((1 << 40) * i) for i in range(1, 7)]

    def write(q=big[0], k=big[1], v=big[2], q_out=big[3], k_cache=big[4], v_cache=big[5], qs=64 * 128):
        p, r = params(), rope_opts()
        return lib.inkling_attn_qk_norm_rope_write(ctypes.byref(p), ctypes.byref(r), q, qs, k, 8 * 128, v, 8 * 128, OK, 64,
                                                   OK, OK, q_out, k_cache, v_cache, OK, 1 << 30, None)

    behind = ctypes.c_void_p(big[0].value + row)
    assert write(q_out=behind) == 2 and write(q_out=behind, qs=80 * 128) == 2
    assert write(k=big[3]) == 2 and write(v=behind, q_out=big[0]) == 2
    for name in ("q", "k", "v", "q_out", "v_cache"):
        assert write(**{name: ctypes.c_void_p(big[4].value + row)}) == 2
    assert write(v_cache=big[0]) == 2


def test_binding_checks_before_the_library(lib):
    p = params(num_seqs=1, num_q_heads=2, num_kv_heads=1, head_dim=64, page_size=16, max_pages_per_seq=2, num_pages=3)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.inkling_attn_prefill_masked(p, q, ints, cache, cache, ints.view(1, 2), ints[:1], q, ws)
    with pytest.raises(ValueError):
        binding.inkling_attn_decode_masked(p, q, cache, cache, ints.view(1, 2), ints[:1], q, ws)
    with pytest.raises(ValueError, match="layout"):
        binding.inkling_attn_qk_norm_rope_write(p, q, q, q, ints, ints, ints, q, cache, cache, ws, layout="pairs")
    with pytest.raises(ValueError):
        binding.inkling_attn_qk_norm_rope_write(p, q, q, q, ints, ints, ints, q, cache, cache, ws)


def test_frequency_tables():
    f, s = rotary.inv_freq(8, base=10000.0)
    assert s == 1.0 and f.dtype == torch.float32
    assert torch.allclose(f.double(), torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=2.0 ** -24)
    g, s = rotary.inv_freq(8, scaling="linear", factor=4.0)
    assert s == 1.0 and torch.allclose(g * 4, f, rtol=2.0 ** -22)
    y, s = rotary.inv_freq(64, scaling="yarn", factor=8.0, original_len=4096)
    f, _ = rotary.inv_freq(64)
    turns = 4096 * f.double() / (2 * math.pi)
    assert s == pytest.approx(0.1 * math.log(8.0) + 1.0)
    assert torch.equal(y[turns > 32], f[turns > 32])
    assert torch.allclose(y[turns < 1] * 8, f[turns < 1], rtol=2.0 ** -22)
    assert ((y <= f) & (y >= f / 8 * 0.999999)).all()
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, factor=0.5)):
        with pytest.raises(ValueError):
            rotary.inv_freq(**bad)


def _bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_oracle_closed_forms():
    """Equal scores average the visible values; a cap bounds a score; a slope weighs by distance."""
    q = _bits(np.zeros((3, 1, 64)))
    v = np.arange(8, dtype=np.float32)[None, None, :, None] * np.ones((1, 1, 8, 64), np.float32)
    kw = dict(num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=8, window=-1, sm_scale=1.0, cu_q=np.array([0, 3]),
              seq_lens=np.array([6]), k_bits=_bits(np.ones((1, 1, 8, 64))), v_bits=_bits(v), block_table=np.array([[0]]))
    out, lse, _, _ = oracle.attention(q_bits=q, **kw)
    assert np.allclose(out[:, 0, 0], [1.5, 2.0, 2.5]) and np.allclose(lse[:, 0], np.log([4, 5, 6]))
    out, lse, _, _ = oracle.attention(q_bits=q, key_begin=np.array([2, 5, -3]), key_end=np.array([3, 5, 99]), **kw)
    assert np.allclose(out[:, 0, 0], [2.0, 0.0, 2.5]) and np.isneginf(lse[1, 0]) and np.allclose(lse[0, 0], 0)
    big = _bits(np.full((3, 1, 64), 64.0))
    _, lse, _, _ = oracle.attention(q_bits=big, softcap=2.0, **kw)
    assert np.allclose(lse[:, 0], 2.0 + np.log([4, 5, 6]))
    _, lse, _, _ = oracle.attention(q_bits=q, slopes=np.array([0.5]), **dict(kw, window=2))
    assert np.allclose(lse[:, 0], np.log(1 + np.exp(-0.5)))


def test_oracle_rotation_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(0)
    f = rotary.inv_freq(32)[0].double().numpy()
    for layout in ("half", "interleaved"):
        x, z = rng.normal(size=(2, 1, 1, 64))
        at = lambda u, p: oracle.norm_rope(u, np.array([p]), None, 0.0, f, layout, 1.0)[0]
        assert np.isclose((at(x, 5) ** 2).sum(), (x ** 2).sum()) and np.array_equal(at(x, 9)[..., 32:], x[..., 32:])
        assert np.isclose((at(x, 100) * at(z, 93)).sum(), (at(x, 17) * at(z, 10)).sum())
    y, _ = oracle.norm_rope(x, np.array([0]), np.full(64, 2.0), 0.0, None, "half", 1.0)
    assert np.isclose((y ** 2).mean(), 4.0)
