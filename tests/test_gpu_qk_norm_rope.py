"""Head norm, rotation and paged K/V write on the GPU against the fp64 oracle, and the three
operators of a step run together."""
import numpy as np
import pytest
import torch

from oracle import masked as oracle
from paged_attention_relative_gqa_gb300 import binding, rotary
from tests.masked_common import bits, call, check, options, problem, reference

pytestmark = pytest.mark.gpu


def _step(prob, seed, device, fused=True):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    T, D, Hq, Hkv = prob.total_q, prob.head_dim, prob.num_q_heads, prob.num_kv_heads
    if fused:
        rows = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g, device=device).to(torch.bfloat16)
        parts = rows.split([Hq * D, Hkv * D, Hkv * D, 8], -1)[:3]
        return [x.unflatten(-1, (h, D)) for x, h in zip(parts, (Hq, Hkv, Hkv))]
    return [torch.randn(T, h, D, generator=g, device=device).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]


def _expect(prob, q, k, v, kw):
    """(q_out, its bound, K rows, their bound) in fp64, and each row's sequence and position."""
    cu, L = prob.cu_q_lens.cpu().numpy(), prob.seq_lens.cpu().numpy()
    T = int(cu[-1])
    b = np.searchsorted(cu, np.arange(T), side="right") - 1
    pos = (L[b] - (cu[b + 1] - cu[b]) + np.arange(T) - cu[b]).astype(np.int64)
    num = lambda t: None if t is None else t.double().cpu().numpy()
    res = []
    for x, w in ((q, kw.get("w_q")), (k, kw.get("w_k"))):
        y, mag = oracle.norm_rope(x[:T].double().cpu().numpy(), pos, num(w), kw.get("eps", 1e-6), num(kw.get("inv_freq")),
                                  kw.get("layout", "half"), kw.get("rot_scale", 1.0))
        # one rounding to bf16; the fp32 sums of the norm (D / 2 + 20 roundings of 2^-24, half of the
        # mean square's), the angle (a few 2^-22 of a turn) and the products stay below 2^-16
        res += [y, 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag + 1e-30]
    return res, b, pos


def _check(prob, q, k, v, kw, q_out, kc, vc, before):
    (yq, tq, yk, tk), b, pos = _expect(prob, q, k, v, kw)
    T = len(b)
    assert (np.abs(q_out[:T].double().cpu().numpy() - yq) <= tq).all()
    page = prob.block_table.cpu().numpy()[b, pos // prob.page_size]
    slot = pos % prob.page_size
    got = kc.double().cpu().numpy()[page, :, slot]
    assert (np.abs(got - yk) <= tk).all()
    assert np.array_equal(bits(vc)[page, :, slot], bits(v[:T]))
    for now, old in ((kc, before[0]), (vc, before[1])):   # every other slot as it was
        n, o = bits(now).copy(), bits(old)
        n[page, :, slot] = o[page, :, slot]
        assert np.array_equal(n, o)


CASES = [
    # heads, dim, page, q_lens, seq_lens, norm, rot, layout, rot_scale, fused
    ((8, 2), 64, 16, [1], [1], True, 64, "half", 1.0, True),
    ((8, 2), 64, 16, [37, 0, 1, 130], [37, 4, 90, 400], True, 64, "half", 1.0, True),
    ((64, 8), 128, 64, [1] * 33, list(range(1, 331, 10)), True, 128, "half", 1.2079, True),
    ((64, 16), 128, 64, [50, 20], [50, 300], False, 64, "interleaved", 1.0, True),
    ((5, 5), 64, 8, [33], [100], True, 16, "interleaved", 1.0, False),
    ((7, 1), 128, 128, [9, 8], [9, 900], True, 96, "half", 0.5, True),
    ((3, 3), 128, 256, [70], [257], True, 112, "interleaved", 1.0, False),
    ((12, 4), 64, 32, [20, 1], [20, 5], True, 0, "half", 1.0, True),
    ((12, 4), 64, 32, [20, 1], [20, 5], False, 0, "half", 1.0, False),
    ((8, 2), 128, 16, [2000], [2100], True, 128, "interleaved", 1.0, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_oracle(cuda_device, case):
    heads, dim, page, q_lens, seq_lens, norm, rot, layout, rot_scale, fused = CASES[case]
    prob = problem(heads, dim, page, q_lens, seq_lens, 300 + case, cuda_device)
    q, k, v = _step(prob, case, cuda_device, fused)
    kw = dict(layout=layout, rot_scale=rot_scale, eps=1e-5)
    if norm:
        kw["w_q"], kw["w_k"] = torch.rand(dim, device=cuda_device) + 0.5, torch.randn(dim, device=cuda_device)
    if rot:
        kw["inv_freq"] = rotary.inv_freq(rot, device=cuda_device)[0]
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, False, cuda_device)
    before = (prob.k_cache.clone(), prob.v_cache.clone())
    q_out = torch.empty(prob.total_q, heads[0], dim, dtype=torch.bfloat16, device=cuda_device)
    binding.inkling_attn_qk_norm_rope_write(params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table, q_out,
                                            prob.k_cache, prob.v_cache, ws, **kw)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    _check(prob, q, k, v, kw, q_out, prob.k_cache, prob.v_cache, before)


@pytest.mark.parametrize("length", [4095, 70001, (1 << 24) + 3, (1 << 30) + 77, (1 << 31) - 1 - 65536])
def test_far_positions(cuda_device, length):
    page = 1 << 16
    width = (length + page - 1) // page
    D, dev = 64, cuda_device
    params = binding.make_params(num_seqs=1, num_q_heads=2, num_kv_heads=1, head_dim=D, page_size=page,
                                 max_pages_per_seq=width, num_pages=2, rel_extent=1, window=-1, sm_scale=1.0)
    table = torch.full((1, width), 9, dtype=torch.int32, device=dev)
    last = (length - 1) // page
    table[0, last] = 1
    if (length - 3) // page != last:
        table[0, last - 1] = 0
    lens = torch.tensor([length], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    q, k, v = (torch.randn(3, h, D, device=dev).to(torch.bfloat16) for h in (2, 1, 1))
    f = rotary.inv_freq(D, device=dev)[0]
    kc, vc = (torch.zeros(2, 1, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = binding.alloc_masked_workspace(params, False, dev)
    q_out = torch.empty_like(q)
    binding.inkling_attn_qk_norm_rope_write(params, q, k, v, cu, lens, table, q_out, kc, vc, ws, inv_freq=f)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == 0
    pos = np.arange(length - 3, length)
    for x, got in ((q, q_out), (k, torch.stack([kc[int(table[0, p // page]), :, p % page] for p in pos]))):
        y, mag = oracle.norm_rope(x.double().cpu().numpy(), pos, None, 0.0, f.double().cpu().numpy(), "half", 1.0)
        assert (np.abs(got.double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag).all()


def test_in_place_and_rows_behind_the_last_request(cuda_device):
    prob = problem((8, 2), 64, 16, [5, 9], [5, 40], 20, cuda_device)
    dev = cuda_device
    q, k, v = (torch.randn(14 + 6, h, 64, device=dev).to(torch.bfloat16) for h in (8, 2, 2))
    orig = q.clone()
    kw = dict(w_q=torch.rand(64, device=dev), w_k=torch.rand(64, device=dev), inv_freq=rotary.inv_freq(64, device=dev)[0])
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, False, dev)
    before = (prob.k_cache.clone(), prob.v_cache.clone())
    binding.inkling_attn_qk_norm_rope_write(params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table, q,
                                            prob.k_cache, prob.v_cache, ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q[14:], orig[14:])
    _check(prob, orig, k, v, kw, q, prob.k_cache, prob.v_cache, before)


def test_bad_pages_and_contradicting_lengths_are_skipped_and_reported(cuda_device):
    dev = cuda_device
    prob = problem((8, 2), 64, 16, [20, 7, 6], [20, 9, 30], 21, dev)
    q, k, v = _step(prob, 5, dev)
    params = binding.params_of(prob)
    ws = binding.alloc_masked_workspace(params, False, dev)
    before = (prob.k_cache.clone(), prob.v_cache.clone())
    q_out = torch.full((33, 8, 64), 7.0, dtype=torch.bfloat16, device=dev)
    good = prob.block_table.clone()
    prob.block_table[0, 1] = prob.num_pages      # positions 16 .. 19 of request 0
    prob.seq_lens[1] = 5                         # seven new rows, five keys
    args = (params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table, q_out, prob.k_cache, prob.v_cache, ws)
    binding.inkling_attn_qk_norm_rope_write(*args)
    torch.cuda.synchronize()
    assert binding.inkling_attn_read_device_error(ws) == binding.DEVERR_PAGE_OUT_OF_RANGE | binding.DEVERR_QLEN_EXCEEDS_KV
    assert (q_out[20:27] == 7.0).all()
    assert torch.equal(q_out[:20], q[:20]) and torch.equal(q_out[27:], q[27:])
    for now, old, rows in ((prob.k_cache, before[0], k), (prob.v_cache, before[1], v)):
        want = bits(old).copy()
        t = good.cpu().numpy()
        for i in range(16):
            want[t[0, 0], :, i] = bits(rows[i])
        for i in range(6):
            p = 24 + i
            want[t[2, p // 16], :, p % 16] = bits(rows[27 + i])
        assert np.array_equal(bits(now), want)


def test_a_prompt_then_tokens_through_the_three_operators(cuda_device):
    """Write a prompt and attend, then one token at a time: norm, rotate, write, attend; every attention
    is checked on the cache as the write left it, and the cache against the oracle's rows."""
    dev = cuda_device
    heads, D, page = (16, 2), 128, 16
    start, steps = [70, 5, 131], 3
    prob = problem(heads, D, page, start, start, 30, dev, max_pages=16)
    # room for the tokens to come: pages of its own for every table entry
    n = 3 * 16
    prob.k_cache = torch.full((n, 2, page, D), float("nan"), dtype=torch.bfloat16, device=dev)
    prob.v_cache = torch.full((n, 2, page, D), float("nan"), dtype=torch.bfloat16, device=dev)
    prob.block_table = torch.randperm(n, device=dev).to(torch.int32).view(3, 16).contiguous()
    f, scale = rotary.inv_freq(D, scaling="yarn", factor=4.0, original_len=64, device=dev)
    kw = dict(w_q=torch.rand(D, device=dev) + 0.5, w_k=torch.rand(D, device=dev) + 0.5, inv_freq=f, rot_scale=scale)
    for step in range(steps + 1):
        if step:
            prob.q_lens = [1] * 3
            prob.seq_lens_list = [L + 1 for L in prob.seq_lens_list]
            prob.seq_lens += 1
            prob.cu_q_lens = torch.arange(4, dtype=torch.int32, device=dev)
        q, k, v = _step(prob, 40 + step, dev)
        params = binding.params_of(prob)
        ws = binding.alloc_masked_workspace(params, step > 0, dev)
        before = (prob.k_cache.clone(), prob.v_cache.clone())
        prob.q = torch.empty(prob.total_q, heads[0], D, dtype=torch.bfloat16, device=dev)
        binding.inkling_attn_qk_norm_rope_write(params, q, k, v, prob.cu_q_lens, prob.seq_lens, prob.block_table,
                                                prob.q, prob.k_cache, prob.v_cache, ws, **kw)
        opts = options(prob, softcap=25.0)
        out, lse, _ = call(prob, opts, step > 0, workspace=ws)
        torch.cuda.synchronize()
        assert binding.inkling_attn_read_device_error(ws) == 0
        _check(prob, q, k, v, kw, prob.q, prob.k_cache, prob.v_cache, before)
        check(out, lse, reference(prob, opts), f"step {step}")
