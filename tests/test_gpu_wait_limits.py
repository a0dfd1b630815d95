"""Waits that run out somewhere in a call: limits between none and the default.

A call ends in any case.  Without an error bit it gives what it gives otherwise, bit for bit; with one
it reports the timeout and no other error, and the next calls are right."""
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from paged_attention_relative_gqa_gb300 import workloads as W
from tests.masked_common import call, check, options, problem, reference
from tests.parity import compare, oracle_full
from tests.test_gpu_kv_conv import check as kv_check, run_gpu as run_kv

pytestmark = pytest.mark.gpu
LIMITS = [0, 1, 300, 1000, 2000, 4000, 8000, 16000, 40000]
DEFAULT_LIMIT_NS = 2_000_000_000


@pytest.fixture
def limit():
    yield binding.inkling_attn_set_wait_limit_ns
    torch.cuda.synchronize()
    binding.inkling_attn_set_wait_limit_ns(DEFAULT_LIMIT_NS)


def sweep(limit, run, ws):
    """`run` (its outputs as a tuple) under every limit, three times each."""
    want = [x.clone() for x in run()]
    assert binding.inkling_attn_read_device_error(ws) == 0
    ran_out = 0
    for ns in LIMITS:
        for _ in range(3):
            limit(ns)
            got = run()
            err = binding.inkling_attn_read_device_error(ws)
            assert err in (0, binding.DEVERR_WAIT_TIMEOUT)
            ran_out += err != 0
            if not err:
                assert all(torch.equal(a, b) for a, b in zip(got, want)), f"limit {ns} ns"
            limit(DEFAULT_LIMIT_NS)
            got = run()
            assert binding.inkling_attn_read_device_error(ws) == 0
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"after a limit of {ns} ns"
    assert ran_out


@pytest.mark.parametrize("heads,dim,page,softcap", [((8, 2), 128, 64, 0.0), ((16, 1), 128, 16, 20.0), ((8, 8), 64, 8, 0.0)])
def test_masked_decode(cuda_device, limit, heads, dim, page, softcap):
    seq_lens = [1500 + 97 * i for i in range(24)]
    prob = problem(heads, dim, page, [1] * 24, seq_lens, 50, cuda_device)
    opts = options(prob, softcap=softcap)
    ws = binding.alloc_masked_workspace(binding.params_of(prob), True, cuda_device)
    out, lse, _ = call(prob, opts, True, workspace=ws)
    check(out, lse, reference(prob, opts), "before")
    sweep(limit, lambda: call(prob, opts, True, workspace=ws)[:2], ws)


@pytest.mark.parametrize("heads,dim,page,window", [((16, 4), 128, 64, 512), ((32, 2), 64, 16, -1), ((16, 4), 128, 8, -1)])
def test_decode_with_a_bias(cuda_device, limit, heads, dim, page, window):
    prob = W.make_problem(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, rel_extent=512,
                          window=window, q_lens=[1] * 24, seq_lens=[1500 + 97 * i for i in range(24)], seed=51,
                          device=cuda_device)
    params = binding.params_of(prob)
    ws = binding.alloc_workspace(params, True, cuda_device)
    run = lambda: (binding.run(prob, out=torch.zeros_like(prob.q), workspace=ws),)
    compare(run()[0].float().cpu().numpy(), oracle_full(prob), "before")
    sweep(limit, run, ws)


@pytest.mark.parametrize("form,heads,dim,page,extent", [
    ("lowrank", (8, 2), 128, 64, 1024), ("lowrank", (4, 4), 64, 16, 300), ("fp32", (8, 2), 128, 64, 1024),
    ("fp32", (4, 2), 64, 8, 301), ("bf16", (8, 8), 128, 64, 1024), ("bf16", (3, 1), 64, 32, 96)])
def test_prefill_with_a_bias(cuda_device, limit, form, heads, dim, page, extent):
    kw = {"lowrank": dict(lowrank_d=64), "fp32": {}, "bf16": dict(bias_dtype=torch.bfloat16)}[form]
    prob = W.make_problem(num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=dim, page_size=page, rel_extent=extent,
                          window=-1, q_lens=[300, 130], seq_lens=[300, 900], seed=52, device=cuda_device, **kw)
    params = binding.params_of(prob)
    ws = binding.alloc_workspace(params, True, cuda_device)
    run = lambda: (binding.run(prob, out=torch.zeros_like(prob.q), workspace=ws),)
    compare(run()[0].float().cpu().numpy(), oracle_full(prob), "before")
    sweep(limit, run, ws)


@pytest.mark.parametrize("heads,dim,kernel_size", [(8, 128, 4), (2, 64, 8)])
def test_kv_write(cuda_device, limit, heads, dim, kernel_size):
    step = W.make_kv_step(num_kv_heads=heads, head_dim=dim, page_size=64, kernel_size=kernel_size, q_lens=[1024] * 4,
                          seq_lens=[1024] * 4, seed=53, device=cuda_device)
    kv_check(step, run_kv(step), "before")
    params = binding.make_params(num_seqs=4, num_q_heads=heads, num_kv_heads=heads, head_dim=dim, page_size=64,
                                 max_pages_per_seq=step.max_pages, num_pages=step.num_pages, rel_extent=1, window=-1,
                                 sm_scale=1.0)
    ws = binding.alloc_workspace(params, False, cuda_device)

    def run():
        kc, vc = step.k_cache.clone(), step.v_cache.clone()
        sk, sv = torch.empty_like(step.state_k), torch.empty_like(step.state_v)
        binding.inkling_attn_kv_conv_write(params, step.k_new, step.v_new, step.cu_q_lens, step.seq_lens,
                                           step.block_table, step.w_k, step.w_v, step.state_k, step.state_v, sk, sv,
                                           kc, vc, ws)
        return tuple(x.view(torch.int16) for x in (kc, vc, sk, sv))

    sweep(limit, run, ws)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("q_lens,seq_lens", [([700, 300], [700, 900]), ([20, 3], [6000, 9000])])
def test_masked_prefill(cuda_device, limit, softcap, q_lens, seq_lens):
    """After a timeout its workspace has to be initialised again."""
    prob = problem((8, 2), 128, 64, q_lens, seq_lens, 54, cuda_device)
    opts = options(prob, softcap=softcap)
    ws = binding.alloc_masked_workspace(binding.params_of(prob), False, cuda_device)
    want = call(prob, opts, False, workspace=ws)[:2]
    check(*want, reference(prob, opts), "before")
    ran_out = 0
    for ns in LIMITS:
        for _ in range(3):
            limit(ns)
            got = call(prob, opts, False, workspace=ws)[:2]
            err = binding.inkling_attn_read_device_error(ws)
            assert err in (0, binding.DEVERR_WAIT_TIMEOUT)
            limit(DEFAULT_LIMIT_NS)
            if err:
                ran_out += 1
                binding.inkling_attn_workspace_init(ws)
                got = call(prob, opts, False, workspace=ws)[:2]
                assert binding.inkling_attn_read_device_error(ws) == 0
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"limit {ns} ns"
    assert ran_out
