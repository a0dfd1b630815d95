"""What a step writes for its drafted tokens, on the GPU against the fp64 oracle: norm and rotation at given
positions, and the K/V short convolution along each token's way to the root with its state."""
import numpy as np
import pytest
import torch

from oracle import masked as rope_oracle
from oracle import tree as oracle
from paged_attention_relative_gqa_gb300 import binding, rotary
from paged_attention_relative_gqa_gb300 import workloads as W
from tests.masked_common import bits
from tests.tree_common import Step, parents_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation at positions


def rope_inputs(step, seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    p = step.prob
    rows = torch.randn(p.total_q, p.num_q_heads + 2 * p.num_kv_heads, p.head_dim, generator=g, device=device).to(torch.bfloat16)
    return rows.split([p.num_q_heads, p.num_kv_heads, p.num_kv_heads], 1)


def slots(step):
    cu, L = step.prob.cu_q_lens.cpu().numpy(), step.prob.seq_lens.cpu().numpy()
    b = np.searchsorted(cu, np.arange(cu[-1]), side="right") - 1
    key = (L[b] - (cu[b + 1] - cu[b]) + np.arange(cu[-1]) - cu[b]).astype(np.int64)
    return step.prob.block_table.cpu().numpy()[b, key // step.prob.page_size], key % step.prob.page_size


@pytest.mark.parametrize("heads,dim,page,n,history,rot,layout,norm", [
    ((8, 2), 64, 16, [5], [3001], 64, "half", True), ((64, 8), 128, 64, [33, 1, 8], [100, 0, 5000], 128, "half", True),
    ((40, 8), 128, 32, [20, 17], [9, 300], 64, "interleaved", True), ((3, 3), 64, 8, [30], [0], 16, "interleaved", False),
    ((8, 2), 128, 64, [12], [70], 0, "half", True)])
def test_rotation_at_positions(cuda_device, heads, dim, page, n, history, rot, layout, norm):
    step = Step(heads, dim, page, n, history, 30, cuda_device)
    p = step.prob
    q, k, v = rope_inputs(step, 31, cuda_device)
    at = step.positions.clone()
    at[0] = -9                       # counts as 0
    at[-1] = 2**31 - 1
    w = torch.rand(dim, device=cuda_device) + 0.5 if norm else None
    freq = rotary.inv_freq(rot, device=cuda_device)[0] if rot else None
    kc, vc, q_out = p.k_cache.clone(), p.v_cache.clone(), torch.empty_like(p.q)
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    binding.inkling_attn_qk_norm_rope_write(step.params, q, k, v, p.cu_q_lens, p.seq_lens, p.block_table, q_out, kc, vc, ws,
                                            w_q=w, w_k=w, inv_freq=freq, layout=layout, rot_scale=1.25, positions=at)
    assert binding.inkling_attn_read_device_error(ws) == 0
    pos = np.maximum(at.cpu().numpy().astype(np.int64), 0)
    num = lambda t: None if t is None else t.double().cpu().numpy()
    page_of, slot = slots(step)
    for x, got in ((q, q_out.double().cpu().numpy()), (k, kc.double().cpu().numpy()[page_of, :, slot])):
        y, mag = rope_oracle.norm_rope(x.double().cpu().numpy(), pos, num(w), 1e-6, num(freq), layout, 1.25)
        # one rounding to bf16; norm, angle (2^-25 of a turn) and products in fp32 below 2^-16 of what is added
        assert (np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag + 1e-30).all()
    assert np.array_equal(bits(vc)[page_of, :, slot], bits(v))
    for now, old in ((kc, p.k_cache), (vc, p.v_cache)):   # every other slot as it was
        a, b = bits(now).copy(), bits(old)
        a[page_of, :, slot] = b[page_of, :, slot]
        assert np.array_equal(a, b)


@pytest.mark.parametrize("heads,dim,n", [((64, 8), 128, [20] * 85), ((64, 8), 128, [30] * 110), ((8, 2), 64, [29] * 128),
                                         ((64, 8), 128, [40] * 25), ((8, 2), 128, [41] * 100)])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 32)])
def test_rows_do_not_depend_on_how_many_there_are(cuda_device, heads, dim, n, layout, rot):
    """However a token's heads are shared out over warps: the call for all sequences gives the bits of calls for a few of them."""
    step = Step(heads, dim, 64, n, [100 + i for i in range(len(n))], 34, cuda_device)
    p = step.prob
    q, k, v = rope_inputs(step, 35, cuda_device)
    w, freq = torch.rand(dim, device=cuda_device) + 0.5, rotary.inv_freq(rot, device=cuda_device)[0]
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    outs = []
    for most in (len(n), 3):
        kc, vc, q_out = p.k_cache.clone(), p.v_cache.clone(), torch.zeros_like(p.q)
        for b in range(0, len(n), most):
            few = slice(b, min(b + most, len(n)))
            t = slice(sum(n[: few.start]), sum(n[: few.stop]))
            params = binding.params_of(p)
            params.num_seqs = few.stop - few.start
            binding.inkling_attn_qk_norm_rope_write(params, q[t], k[t], v[t], p.cu_q_lens[b: few.stop + 1] - t.start, p.seq_lens[few],
                                                    p.block_table[few], q_out[t], kc, vc, ws, w_q=w, w_k=w, inv_freq=freq,
                                                    layout=layout, positions=step.positions[t])
        outs.append((q_out, kc, vc))
    assert binding.inkling_attn_read_device_error(ws) == 0
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(*outs))
    assert all(outs[0][0].abs().sum(-1).flatten() > 0)


def test_positions_of_the_slots_change_nothing(cuda_device):
    step = Step((8, 2), 128, 64, [33, 4], [100, 9], 32, cuda_device, "chain")
    p = step.prob
    q, k, v = rope_inputs(step, 33, cuda_device)
    freq = rotary.inv_freq(128, device=cuda_device)[0]
    ws = binding.alloc_tree_workspace(step.params, cuda_device)
    got = []
    for at in (None, step.positions):
        kc, vc, q_out = p.k_cache.clone(), p.v_cache.clone(), torch.empty_like(p.q)
        binding.inkling_attn_qk_norm_rope_write(step.params, q, k, v, p.cu_q_lens, p.seq_lens, p.block_table, q_out, kc, vc,
                                                ws, inv_freq=freq, positions=at)
        got.append([bits(x) for x in (q_out, kc, vc)])
    assert all(np.array_equal(a, b) for a, b in zip(*got))


# ------------------------------------------------------------------ convolution


class Conv:
    def __init__(self, heads, dim, page, n, history, ks, seed, device, kind):
        rng = np.random.default_rng(seed)
        self.s = W.make_kv_step(num_kv_heads=heads, head_dim=dim, page_size=page, kernel_size=ks, q_lens=n,
                                seq_lens=[a + b for a, b in zip(n, history)], seed=seed, device=device)
        s = self.s
        self.parents = [parents_of(kind, x, rng) if x else [] for x in n]
        self.parents_t = torch.tensor([x for p in self.parents for x in p], dtype=torch.int32, device=device)
        self.params = binding.make_params(num_seqs=s.num_seqs, num_q_heads=heads, num_kv_heads=heads, head_dim=dim,
                                          page_size=page, max_pages_per_seq=s.max_pages, num_pages=s.num_pages, rel_extent=1,
                                          window=-1, sm_scale=1.0)
        self.ws = binding.alloc_tree_workspace(self.params, device)
        self.ks = ks

    def write(self, parents=None):
        s = self.s
        kc, vc = s.k_cache.clone(), s.v_cache.clone()
        state = (s.state_k, s.state_v) if self.ks > 1 else (None, None)
        binding.inkling_attn_kv_conv_write_tree(self.params, s.k_new, s.v_new, s.cu_q_lens, s.seq_lens, s.block_table,
                                                self.parents_t if parents is None else parents, s.w_k, s.w_v, *state, kc, vc,
                                                self.ws)
        return kc, vc

    def check(self, caches, skip=(), parents=None):
        s = self.s
        cu, table = s.cu_q_lens.cpu().numpy(), s.block_table.cpu().numpy()
        for name, cache, old in (("k", caches[0], s.k_cache), ("v", caches[1], s.v_cache)):
            x, w = bits(getattr(s, name + "_new")), getattr(s, "w_" + name).double().cpu().numpy()
            state = bits(getattr(s, "state_" + name)) if self.ks > 1 else np.zeros((s.num_seqs, 0, *x.shape[1:]), np.uint16)
            got, rest = bits(cache).copy(), bits(old)
            for b, (n, L) in enumerate(zip(s.q_lens, s.seq_lens_list)):
                if b in skip or n == 0:
                    continue
                y, mag = oracle.conv(x[cu[b]: cu[b + 1]], state[b], (parents or self.parents)[b], w)
                key = np.arange(L - n, L)
                page, slot = table[b, key // s.page_size], key % s.page_size
                val = (got[page, :, slot].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
                # ks products added in fp32 (a rounding each), then one rounding to bf16
                assert (np.abs(val - y) <= 2.0 ** -8 * np.abs(y) + self.ks * 2.0 ** -23 * mag + 1e-38).all(), (name, b)
                got[page, :, slot] = rest[page, :, slot]
            assert np.array_equal(got, rest), "other slots"


CONV = [(2, 64, 16, [1], [0], 4, "chain"), (2, 64, 16, [5, 0, 33, 2], [3, 9, 100, 0], 4, "tree"),
        (16, 128, 64, [32, 17, 9], [500, 63, 64], 4, "forest"), (8, 128, 8, [100], [7], 8, "chain"),
        (3, 64, 32, [40, 40], [10, 11], 2, "tree"), (1, 128, 128, [64], [1], 3, "flat"), (5, 64, 16, [9, 8], [30, 2], 1, "tree"),
        (8, 128, 64, [30] * 64, [70] * 64, 4, "tree"), (2, 128, 16, [20], [5], 5, "forest"), (2, 64, 16, [20], [5], 6, "tree"),
        (2, 64, 16, [20], [5], 7, "forest")]


@pytest.mark.parametrize("heads,dim,page,n,history,ks,kind", CONV)
def test_convolution_along_the_ways_to_the_root(cuda_device, heads, dim, page, n, history, ks, kind):
    c = Conv(heads, dim, page, n, history, ks, 40 + ks, cuda_device, kind)
    got = c.write()
    assert binding.inkling_attn_read_device_error(c.ws) == 0
    c.check(got)


def test_a_chain_gives_the_bits_of_the_step_without_a_tree(cuda_device):
    c = Conv(8, 128, 64, [9, 1, 30], [100, 5, 64], 4, 50, cuda_device, "chain")
    s = c.s
    tree = c.write()
    kc, vc, sk, sv = s.k_cache.clone(), s.v_cache.clone(), torch.empty_like(s.state_k), torch.empty_like(s.state_v)
    binding.inkling_attn_kv_conv_write(c.params, s.k_new, s.v_new, s.cu_q_lens, s.seq_lens, s.block_table, s.w_k, s.w_v,
                                       s.state_k, s.state_v, sk, sv, kc, vc, c.ws)
    assert np.array_equal(bits(tree[0]), bits(kc)) and np.array_equal(bits(tree[1]), bits(vc))
    # all tokens accepted: the state too
    path = torch.tensor([list(range(30))] * 3, dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([9, 1, 30], dtype=torch.int32, device=cuda_device)
    tk, tv = torch.empty_like(sk), torch.empty_like(sv)
    binding.inkling_attn_kv_conv_state_tree(c.params, s.k_new, s.v_new, s.cu_q_lens, path, lens, s.state_k, s.state_v, tk, tv,
                                            c.ws)
    assert np.array_equal(bits(tk), bits(sk)) and np.array_equal(bits(tv), bits(sv))
    assert binding.inkling_attn_read_device_error(c.ws) == 0


def test_convolution_errors(cuda_device):
    """A bad parent is a root, a sequence that does not fit is skipped, so is a row on a bad page."""
    c = Conv(2, 64, 16, [6, 5, 7], [20, 30, 3], 4, 51, cuda_device, "chain")
    s = c.s
    bad = c.parents_t.clone()
    bad[3] = 3
    got = c.write(bad)
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_BAD_TREE
    c.check(got, parents=[[-1, 0, 1, -1, 3, 4]] + c.parents[1:])
    s.seq_lens[1] = 4
    got = c.write()
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_QLEN_EXCEEDS_KV
    c.check(got, skip=(1,))
    s.seq_lens[1] = 35
    s.cu_q_lens[3] = 19
    got = c.write()
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_BAD_ROWS
    c.check(got, skip=(2,))
    s.cu_q_lens[3] = 18
    s.block_table[2, 0] = s.num_pages
    got = c.write()
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_PAGE_OUT_OF_RANGE
    c.check(got, skip=(2,))


@pytest.mark.parametrize("ks", [2, 4, 8])
def test_state_behind_a_path(cuda_device, ks):
    n = [9, 1, 40, 0, 6, 5, 7]
    c = Conv(3, 64, 16, n, [20] * 7, ks, 52 + ks, cuda_device, "tree")
    s = c.s
    paths = [[0, 2, 5], [0], list(range(0, 40, 2)), [], [], [0, 4], [3, 2, 5]]
    lens = [3, 1, 20, 0, 0, 22, 3]     # the last but one longer than the table, the last not increasing
    width = 20
    path = torch.tensor([p + [-3] * (width - len(p)) for p in paths], dtype=torch.int32, device=cuda_device)
    out = torch.empty_like(s.state_k), torch.empty_like(s.state_v)
    binding.inkling_attn_kv_conv_state_tree(c.params, s.k_new, s.v_new, s.cu_q_lens, path,
                                            torch.tensor(lens, dtype=torch.int32, device=cuda_device), s.state_k, s.state_v,
                                            *out, c.ws)
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_BAD_TREE
    cu, table = s.cu_q_lens.cpu().numpy(), path.cpu().numpy()
    for x, old, new in ((s.k_new, s.state_k, out[0]), (s.v_new, s.state_v, out[1])):
        for b in range(len(n)):
            took = oracle.accepted(table[b], lens[b], n[b])
            assert took == ([] if b >= 5 else paths[b])
            assert np.array_equal(bits(new)[b], oracle.conv_state(bits(x)[cu[b]: cu[b + 1]], bits(old)[b], took)), b


def test_state_of_rows_that_are_not_there(cuda_device):
    c = Conv(2, 64, 16, [4, 4], [9, 9], 4, 60, cuda_device, "chain")
    s = c.s
    s.cu_q_lens[2] = 9
    path = torch.tensor([[0, 1], [2, 4]], dtype=torch.int32, device=cuda_device)
    lens = torch.tensor([2, 2], dtype=torch.int32, device=cuda_device)
    out = torch.empty_like(s.state_k), torch.empty_like(s.state_v)
    binding.inkling_attn_kv_conv_state_tree(c.params, s.k_new, s.v_new, s.cu_q_lens, path, lens, s.state_k, s.state_v, *out,
                                            c.ws)
    assert binding.inkling_attn_read_device_error(c.ws) == binding.DEVERR_BAD_ROWS
    assert np.array_equal(bits(out[0])[1], bits(s.state_k)[1])
    assert np.array_equal(bits(out[1])[0], oracle.conv_state(bits(s.v_new)[:4], bits(s.state_v)[0], [0, 1]))
