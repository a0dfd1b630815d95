"""The capped score of the masked operators, with the cap's own error apart from that of the product.

tests/masked_common.check counts the whole cap among the magnitudes that go into a score: with caps of
hundreds it would pass a cap that is off by a per cent.  Here a score may be off by

    2^-15 (1 + m)   the product, m the sum of the magnitudes of its terms (and of the slope's), as there
    2^-20 |s|       the polynomials: 2^-20.7 of the score by approximation (six terms), a few 2^-24 by rounding
    2^-21 C         beyond the cap: C (1 - 2 / (1 + e^2y)) with e^2y off by 2^-20 of itself, of which at most a
                    fifth arrives, a reciprocal and two roundings
"""
import math

import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding
from tests.masked_common import call, options, problem, reference

pytestmark = pytest.mark.gpu


def check_tight(out, lse, ref, softcap, label):
    want, want_lse, mag, smag = ref
    m = smag - softcap
    d = 2.0 ** -15 * (1 + m) + 2.0 ** -20 * np.minimum(softcap, m) + np.where(m > softcap, 2.0 ** -21 * softcap, 0.0)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -8 + 2.0 * d[..., None]) + 1e-30
    excess = np.abs(got - want) - tol
    assert excess.max() <= 0, f"{label}: out off by {excess.max():.3e} over its bound"
    excess = np.abs(got_lse - want_lse) - d - 2.0 ** -20 * (1 + np.abs(want_lse))
    assert excess.max() <= 0, f"{label}: lse off by {excess.max():.3e} over its bound"


@pytest.mark.parametrize("softcap", [10.0, 300.0, 1000.0, 1e5, 1e6])
@pytest.mark.parametrize("dim,q_std", [(128, 1.0), (64, 6.0)])
@pytest.mark.parametrize("decode", [False, True])
def test_large_caps(cuda_device, decode, dim, q_std, softcap):
    q_lens, seq_lens = ([1, 1], [3000, 77]) if decode else ([150, 40], [700, 2100])
    prob = problem((8, 2), dim, 64, q_lens, seq_lens, 100, cuda_device, q_std=q_std)
    for slopes in (None, np.linspace(0.0, 0.2, 8)):
        opts = options(prob, softcap=softcap, slopes=slopes)
        out, lse, ws = call(prob, opts, decode)
        assert binding.inkling_attn_read_device_error(ws) == 0
        check_tight(out, lse, reference(prob, opts), softcap, f"cap {softcap}")


@pytest.mark.parametrize("softcap", [1e-3, 1.0, 30.0, 50.0, 1000.0, 1e6])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens", [[384, 1], [40, 40]])
@pytest.mark.parametrize("decode", [False, True])
def test_the_cap_itself(cuda_device, decode, q_lens, dim, softcap):
    """Keys that are all one unit vector: the score of a row is its first channel, exactly, up to four times the
    cap, and its lse that score's cap and the logarithm of the number of keys.  Rows are ordered by the score's
    size, so that tiles come inside the short polynomial's reach, inside the cap and beyond it."""
    seq_lens = [n + 260 for n in q_lens]
    if decode:
        q_lens = [1] * 130
        seq_lens = [1 + 3 * i for i in range(130)]
    prob = problem((2, 1), dim, 64, q_lens, seq_lens, 101, cuda_device)
    T = prob.total_q
    g = torch.Generator().manual_seed(102)
    y = torch.cat([torch.logspace(-3, math.log10(4.0), n) if n > 1 else torch.tensor([0.7]) for n in (q_lens if not decode else [T])])
    y = y[:, None] * torch.where(torch.rand(T, 2, generator=g) < 0.5, -1.0, 1.0)
    prob.q = torch.zeros(T, 2, dim, dtype=torch.bfloat16)
    prob.q[:, :, 0] = (y * softcap).to(torch.bfloat16)
    x = prob.q[:, :, 0].double()
    prob.q = prob.q.to(cuda_device)
    prob.k_cache.zero_()
    prob.k_cache[..., 0] = 1.0
    prob.sm_scale = 1.0
    p = torch.cat([torch.arange(L - n, L) for n, L in zip(q_lens, seq_lens)])
    s = softcap * torch.tanh(x / softcap)
    bound = 2.0 ** -20 * s.abs() + torch.where(x.abs() > softcap, 2.0 ** -21 * softcap, 0.0)
    for begin, keys in ((None, p + 1), (p, torch.ones_like(p))):
        out, lse, ws = call(prob, options(prob, softcap=softcap, begin=begin), decode)
        assert binding.inkling_attn_read_device_error(ws) == 0
        want = s + torch.log(keys.double())[:, None]
        err = (lse.double().cpu() - want).abs() - bound - 2.0 ** -20 * (1 + want.abs())
        assert err.max() <= 0, f"off by {err.max():.3e} over its bound at {x.flatten()[err.argmax()]:.6g}"
