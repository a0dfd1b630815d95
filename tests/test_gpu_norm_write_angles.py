"""The rotation's angle at far positions, seen where a cosine or a sine is nearly zero.

There bf16's rounding is that of the small value itself, and an error of the angle shows in full: elsewhere it
would have to reach 2^-9 to be seen."""
from fractions import Fraction
import math
import random

import numpy as np
import pytest
import torch

from paged_attention_relative_gqa_gb300 import binding

pytestmark = pytest.mark.gpu
# 1 / (2 pi) to 40 digits
INV_2PI = Fraction(1591549430918953357688837633725143620344, 10 ** 40)


def turns(p, f):
    """p f / (2 pi) less the nearest quarter turn, and that quarter (0 .. 3)."""
    t = Fraction(float(f)) * p * INV_2PI
    quarter = round(4 * t)
    return float(t - Fraction(quarter, 4)), quarter % 4


def near_quarters(p, low, high, n, rng):
    """Frequencies at which position p lies within 2^-16 of a turn of a quarter turn."""
    found = []
    scale = int(INV_2PI * 2 ** 80)
    while len(found) < n:
        f = np.float32(math.exp(rng.uniform(math.log(low), math.log(high))))
        num, den = float(f).as_integer_ratio()
        part = (4 * p * num * scale // den) & (2 ** 80 - 1)
        if min(part, 2 ** 80 - part) < 2 ** (80 - 14):
            found.append(f)
    return np.array(found, dtype=np.float32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("p,low,high", [(5, 0.2, 1.0), (70001, 1e-4, 1.0), ((1 << 24) + 3, 1e-4, 1.0), ((1 << 28) + 12345, 1e-4, 1.0),
                                        (1999999993, 1e-4, 1.0), ((1 << 31) - 65538, 1e-4, 1.0), ((1 << 31) - 65538, 1.0, 50.0)])
def test_angles_keep_their_precision(cuda_device, p, low, high, layout):
    """Bound: 2^-26 of a turn from the turn's float and 2^-32 from its integers, 2 pi times that in the value; the
    sine of a float is good to 2^-21 of itself, bf16 to 2^-8."""
    dev, D, page = cuda_device, 128, 1 << 16
    f = near_quarters(p, low, high, D // 2, random.Random(p))
    if p == (1 << 31) - 65538:   # frequencies may be negative
        f[::2] = -f[::2]
    width = p // page + 1
    params = binding.make_params(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=D, page_size=page,
                                 max_pages_per_seq=width, num_pages=1, rel_extent=1, window=-1, sm_scale=1.0)
    table = torch.zeros(1, width, dtype=torch.int32, device=dev)
    i = torch.arange(D // 2)
    ia, ib = (i, i + D // 2) if layout == "half" else (2 * i, 2 * i + 1)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16)
    q[..., ia] = 1.0
    q = q.to(dev)
    kc, vc = (torch.zeros(1, 1, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = binding.alloc_masked_workspace(params, False, dev)
    q_out = torch.empty_like(q)
    binding.inkling_attn_qk_norm_rope_write(
        params, q, q, q, torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.tensor([p + 1], dtype=torch.int32, device=dev),
        table, q_out, kc, vc, ws, inv_freq=torch.from_numpy(f).to(dev), layout=layout)
    assert binding.inkling_attn_read_device_error(ws) == 0
    got = q_out.double().cpu().numpy()[0, 0]
    assert np.array_equal(kc[0, 0, p % page].double().cpu().numpy(), got)
    for x in range(D // 2):
        r, quarter = turns(p, f[x])
        small = 2 * math.pi * r                       # sine of the rest, to its cube
        cos, sin = [(1.0, small), (-small, 1.0), (-1.0, -small), (small, -1.0)][quarter]
        for value, want in ((got[ia[x]], cos), (got[ib[x]], sin)):
            bound = 2.0 ** -8 * abs(want) + 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + 2.0 ** -21 * abs(want) + 2.0 ** -40
            assert abs(value - want) <= bound, (p, float(f[x]), value, want)


@pytest.mark.parametrize("f", [0.0, 1e-45, 1e-39, 1e-30, 3e-12, 1e-9, 3e7, 1e20, 3e38, float("inf"), float("nan")])
def test_odd_frequencies(cuda_device, f):
    dev, D, page, p = cuda_device, 64, 1 << 16, 40000
    params = binding.make_params(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=D, page_size=page,
                                 max_pages_per_seq=1, num_pages=1, rel_extent=1, window=-1, sm_scale=1.0)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=dev)
    q[..., :8] = 1.0
    kc, vc = (torch.zeros(1, 1, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = binding.alloc_masked_workspace(params, False, dev)
    q_out = torch.empty_like(q)
    table = torch.full((8,), f, dtype=torch.float32, device=dev)
    binding.inkling_attn_qk_norm_rope_write(
        params, q, q, q, torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.tensor([p + 1], dtype=torch.int32, device=dev),
        torch.zeros(1, 1, dtype=torch.int32, device=dev), q_out, kc, vc, ws, inv_freq=table)
    got = q_out.double().cpu().numpy()[0, 0]
    if not math.isfinite(f):
        assert np.isnan(got[:16]).all()
        return
    f32 = float(np.float32(f))
    # (the 40 digits of 1 / (2 pi) reach 3e38 turns no more: only that the pair keeps its length is asked there)
    if f32 < 1e30:
        r = float(Fraction(f32) * p * INV_2PI % 1) if f32 < 1e10 else None
        if r is not None:
            want = math.cos(2 * math.pi * r), math.sin(2 * math.pi * r)
            assert (abs(got[:8] - want[0]) <= 2.0 ** -8 * abs(want[0]) + 2.0 ** -22).all()
            assert (abs(got[8:16] - want[1]) <= 2.0 ** -8 * abs(want[1]) + 2.0 ** -22).all()
    assert (abs(got[:8] ** 2 + got[8:16] ** 2 - 1.0) <= 2.0 ** -6).all()
