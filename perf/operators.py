"""The operators around the paged cache that carry no per-token bias tensor, as a serving step uses them.

Three operators, each in a plain form (elementary torch operations in 32 bits) and as calls of the library:

* ``rope``: per-head RMS norm of queries and keys, the position rotation, and the write of K and V into
  the paged cache, from the rows of a fused QKV projection;
* ``prefill``: attention of packed new tokens over the paged cache, each token seeing the keys
  ``[key_begin, key_end)`` of its sequence (causal, sliding window, packed documents, a bidirectional
  prefix), with scores capped by a tanh and a bias that falls linearly with the distance;
* ``decode``: the same for one new token per sequence.
"""
import math
import random

import torch

own = False

# (query heads, KV heads): the window and global layers of the model, their tiny form, and layouts without
# grouping or with odd groups.
HEADS = ((64, 8), (64, 16), (16, 2), (8, 2), (8, 8), (12, 4), (14, 2), (40, 8))


def _attn(name, op, batch, new, ctx, heads, dim, page, lens, window=-1, softcap=0.0, mask="causal", slopes=False):
    """New tokens per sequence in [new/2, new] and history before them in [ctx/2, ctx], drawn by `lens`."""
    return dict(name=name, op=op, batch=batch, new=new, ctx=ctx, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                page=page, window=window, softcap=softcap, mask=mask, slopes=slopes, lens=lens)


def _rope(name, batch, new, ctx, heads, dim, page, lens, norm=True, layout="half", rot=0, scaling="none"):
    return dict(name=name, op="rope", batch=batch, new=new, ctx=ctx, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                page=page, norm=norm, layout=layout, rot=rot, scaling=scaling, lens=lens)


def listed():
    return [
        # a few short requests of a small model with a bidirectional prefix: launch latency counts
        _attn("prefill_prefix_small", "prefill", 6, 130, 90, (8, 2), 64, 16, 1, mask="prefix", slopes=True),
        # prompts of a global layer with capped scores
        _attn("prefill_capped", "prefill", 2, 9000, 0, (64, 8), 128, 64, 2, softcap=50.0),
        # training-style packing of documents in one long row, a window layer
        _attn("prefill_documents_window", "prefill", 1, 12000, 0, (64, 16), 128, 64, 3, window=512, mask="documents"),
        # a chunk of a prompt (or drafted tokens to check) against a long history
        _attn("prefill_chunk_long", "prefill", 3, 70, 40000, (64, 8), 128, 64, 4),
        # one request, short history, small model
        _attn("decode_one_short", "decode", 1, 1, 1555, (8, 2), 64, 16, 5, softcap=30.0),
        # a decode step of a window layer
        _attn("decode_window_batch", "decode", 64, 1, 8192, (64, 16), 128, 64, 6, window=512, softcap=50.0),
        # a decode step of a global layer
        _attn("decode_global_batch", "decode", 32, 1, 32768, (64, 8), 128, 64, 7, slopes=True),
        # one request with a very long history
        _attn("decode_one_long", "decode", 1, 1, 131075, (64, 8), 128, 64, 8),
        # one token of a small model
        _rope("rope_one", 1, 1, 3001, (8, 2), 64, 16, 9, layout="half", rot=64),
        # a decode step, half layout, scaled to long contexts
        _rope("rope_decode_batch", 64, 1, 131072, (64, 8), 128, 64, 10, layout="half", rot=128, scaling="yarn"),
        # ragged prompts of a model that rotates half of each head, pairs interleaved
        _rope("rope_ragged", 9, 777, 300, (40, 8), 128, 32, 11, layout="interleaved", rot=64),
        # the step's prompts of a model without rotation (norm only)
        _rope("rope_prompts", 4, 12000, 0, (64, 8), 128, 64, 12, layout="half", rot=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "decode", "decode", "rope"))
    heads = rng.choice(HEADS)
    dim = rng.choice((64, 128, 128))
    page = rng.choice((8, 16, 32, 64, 64, 128, 256))
    lens = rng.randrange(1 << 20)
    if op == "rope":
        new = _log(rng, 1, 8000)
        batch = min(_log(rng, 1, 256), max(1, 40000 // new))
        rot = rng.choice((0, 16, dim // 2, dim, dim))
        return {k: v for k, v in _rope("", batch, new, rng.choice((0, _log(rng, 1, 4000))), heads, dim, page, lens,
                                       norm=rng.random() < 0.7 or rot == 0, layout=rng.choice(("half", "interleaved")),
                                       rot=rot, scaling=rng.choice(("none", "linear", "yarn"))).items() if k != "name"}
    window = rng.choice((-1, -1, 512, _log(rng, 1, 3000)))
    cap = rng.choice((0.0, 0.0, 30.0, 50.0, 100.0))
    if op == "decode":
        ctx = _log(rng, 1, 100000)
        batch = min(_log(rng, 1, 200), max(1, 360000 // ctx))
        mask = rng.choice(("causal", "causal", "documents"))
        new = 1
    else:
        new = _log(rng, 1, 5000)
        ctx = rng.choice((0, 0, _log(rng, 1, 20000)))
        batch = max(1, min(_log(rng, 1, 40), 50_000_000 // (new * (new + ctx))))
        mask = rng.choice(("causal", "documents", "prefix"))
    return {k: v for k, v in _attn("", op, batch, new, ctx, heads, dim, page, lens, window=window, softcap=cap,
                                   mask=mask, slopes=rng.random() < 0.3).items() if k != "name"}


# ------------------------------------------------------------------ sizes that follow from a case alone


def _lengths(case):
    """(new tokens, length with them) of each sequence, and the generator that drew them."""
    r = random.Random(case["lens"])
    got = []
    for _ in range(case["batch"]):
        n = r.randint((case["new"] + 1) // 2, case["new"])
        c = r.randint(case["ctx"] // 2, case["ctx"])
        got.append((n, n + c))
    return got, r


def _visible(case):
    """Per sequence, the lists of first and last-plus-one visible key of its new tokens."""
    lens, r = _lengths(case)
    got = []
    for n, L in lens:
        first = L - n
        lo = [0] * n
        hi = [p + 1 for p in range(first, L)]
        if case["mask"] == "documents":
            # documents of 32 to 2000 tokens; the last few tokens of a prompt are padding and see nothing
            start, at = 0, 0
            ends = []
            while at < L:
                at = min(L, at + int(round(math.exp(r.uniform(math.log(32), math.log(2000))))))
                ends.append((start, at))
                start = at
            k = 0
            for i in range(n):
                while first + i >= ends[k][1]:
                    k += 1
                lo[i] = ends[k][0]
            if n > 16:
                for i in range(n - r.randint(1, 8), n):
                    hi[i] = lo[i]
        elif case["mask"] == "prefix":
            cut = r.randint(0, L)
            hi = [max(h, cut) for h in hi]
        got.append((lo, hi))
    return got


def _windowed(case, n, L, lo, hi):
    w = case["window"]
    if w > 0:
        lo = [max(a, L - n + i - w + 1) for i, a in enumerate(lo)]
    return lo, hi


def work(case):
    lens, _ = _lengths(case)
    D, Hq, Hkv = case["dim"], case["q_heads"], case["kv_heads"]
    T = sum(n for n, _ in lens)
    if case["op"] == "rope":
        # rows of the projection in, q and the cache slots out
        return {"bytes": 2.0 * T * (Hq + 2 * Hkv) * D * 2 + T * 8, "flops": 8.0 * T * (Hq + Hkv) * D}
    pairs, keys = 0, 0
    for (n, L), (lo, hi) in zip(lens, _visible(case)):
        lo, hi = _windowed(case, n, L, lo, hi)
        pairs += sum(max(0, b - a) for a, b in zip(lo, hi))
        seen = [(a, b) for a, b in zip(lo, hi) if b > a]
        reach = 0
        for a, b in sorted(seen):
            keys += max(0, b - max(a, reach))
            reach = max(reach, b)
    return {"bytes": 2.0 * T * Hq * D * 2 + T * Hq * 4 + keys * Hkv * D * 4.0, "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs


def _table(lens, page, gen_host, dev):
    """Pages of a sequence at random places of a pool with spare pages; entries past a sequence's own
    pages name no page at all."""
    need = [(L + page - 1) // page for _, L in lens]
    total = sum(need)
    pages = total + max(1, total // 10)
    perm = torch.randperm(pages, generator=gen_host).to(torch.int32)
    width = max(need)
    col = torch.arange(width)
    count = torch.tensor(need)
    start = torch.cumsum(count, 0) - count
    own_page = col[None, :] < count[:, None]
    at = (start[:, None] + col[None, :]).clamp_(max=total - 1)
    table = torch.where(own_page, perm[at], torch.tensor(pages + 7, dtype=torch.int32))
    return table.contiguous().to(dev), pages, perm[total:].to(dev).long()


def _int(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed + 77)
    lens, _ = _lengths(case)
    B, D, P, Hq, Hkv = case["batch"], case["dim"], case["page"], case["q_heads"], case["kv_heads"]
    table, pages, spare = _table(lens, P, host, dev)
    n = [a for a, _ in lens]
    T = sum(n)
    s = dict(case=case, table=table, seq_lens=_int([L for _, L in lens], dev), T=T, n_max=max(n),
             L_max=max(L for _, L in lens))
    s["cu"] = _int([0] + torch.cumsum(torch.tensor(n), 0).tolist(), dev)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    if case["op"] == "rope":
        # the rows of one fused projection: q, k and v are strided views of it
        rows = randn(T, (Hq + 2 * Hkv) * D, std=1.5)
        s["q"] = rows[:, : Hq * D].view(T, Hq, D)
        s["k"] = rows[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = rows[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["k_cache"] = torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device=dev)
        s["v_cache"] = torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device=dev)
        s["w_q"] = s["w_k"] = s["inv_freq"] = None
        s["rot_scale"] = 1.0
        if case["norm"]:
            s["w_q"] = torch.rand(D, generator=gen, device=dev) + 0.5
            s["w_k"] = torch.rand(D, generator=gen, device=dev) + 0.5
        if case["rot"]:
            s["inv_freq"], s["rot_scale"] = _frequencies(case["rot"], case["scaling"], dev)
    else:
        # capped models have larger scores than the others
        s["q"] = randn(T, Hq, D, std=4.0 if case["softcap"] else 1.0)
        s["k_cache"] = randn(pages, Hkv, P, D)
        s["v_cache"] = randn(pages, Hkv, P, D)
        s["k_cache"][spare] = float("nan")
        s["v_cache"][spare] = float("nan")
        s["key_begin"] = s["key_end"] = s["slopes"] = None
        if case["mask"] != "causal":
            vis = _visible(case)
            s["key_end"] = _int([b for _, hi in vis for b in hi], dev)
            if case["mask"] == "documents":
                s["key_begin"] = _int([a for lo, _ in vis for a in lo], dev)
        if case["slopes"]:
            s["slopes"] = torch.pow(2.0, -8.0 * (torch.arange(Hq, device=dev) + 1) / Hq)
    if own:
        from paged_attention_relative_gqa_gb300 import binding
        s["params"] = binding.make_params(num_seqs=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=P,
                                          max_pages_per_seq=table.shape[1], num_pages=pages, rel_extent=1,
                                          window=case.get("window", -1), sm_scale=D ** -0.5)
        s["workspace"] = binding.alloc_masked_workspace(s["params"], case["op"] == "decode", dev)
    return s


def _frequencies(rot, scaling, dev):
    """Rotation frequencies of base 10000, plain or stretched for eight times the trained length."""
    f = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if scaling == "linear":
        f = f / 8.0
    elif scaling == "yarn":
        # frequencies that turn often over 4096 positions stay, slow ones are interpolated
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / 8.0 * (1 - keep)
        scale = 0.1 * math.log(8.0) + 1.0
    return f.float().to(dev), scale


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if case["op"] == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    return _own_attention(s) if own else _plain_attention(s)


def _own_rope(s):
    from paged_attention_relative_gqa_gb300 import binding
    c = s["case"]
    q_out = torch.empty(s["T"], c["q_heads"], c["dim"], dtype=torch.bfloat16, device=s["q"].device)
    binding.inkling_attn_qk_norm_rope_write(
        s["params"], s["q"], s["k"], s["v"], s["cu"], s["seq_lens"], s["table"], q_out, s["k_cache"], s["v_cache"],
        s["workspace"], w_q=s["w_q"], w_k=s["w_k"], eps=1e-6, inv_freq=s["inv_freq"], layout=c["layout"],
        rot_scale=s["rot_scale"])
    return {"q": q_out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    from paged_attention_relative_gqa_gb300 import binding
    c = s["case"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=out.device)
    more = dict(softcap=c["softcap"], key_begin=s["key_begin"], key_end=s["key_end"], slopes=s["slopes"], lse=lse)
    if c["op"] == "decode":
        binding.inkling_attn_decode_masked(s["params"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                           out, s["workspace"], **more)
    else:
        binding.inkling_attn_prefill_masked(s["params"], s["q"], s["cu"], s["k_cache"], s["v_cache"], s["table"],
                                            s["seq_lens"], out, s["workspace"], **more)
    return {"out": out, "lse": lse}


def _rows(s):
    """Sequence and position of each packed new token."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b + 1] + s["seq_lens"].long()[b]


def _turn(x, cos, sin, rot, layout):
    """The first `rot` channels rotated in pairs."""
    y = x.clone()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2] = a * cos - b * sin
        y[..., rot // 2: rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _plain_rope(s):
    c = s["case"]
    b, p = _rows(s)
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["w_q"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["w_k"]
    if c["rot"]:
        angle = p.double()[:, None, None] * s["inv_freq"].double()   # far positions need 64 bits
        cos, sin = (torch.cos(angle) * s["rot_scale"]).float(), (torch.sin(angle) * s["rot_scale"]).float()
        q, k = _turn(q, cos, sin, c["rot"], c["layout"]), _turn(k, cos, sin, c["rot"], c["layout"])
    page = s["table"][b, p // c["page"]].long()
    s["k_cache"][page, :, p % c["page"]] = k.to(torch.bfloat16)
    s["v_cache"][page, :, p % c["page"]] = s["v"]
    return {"q": q.to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _limits(s):
    """First and last-plus-one visible key of each packed new token, its sequence and position."""
    c = s["case"]
    T, dev = s["T"], s["q"].device
    if c["op"] == "decode":
        b = torch.arange(T, device=dev)
        p = s["seq_lens"].long() - 1
    else:
        b, p = _rows(s)
    lo = torch.zeros_like(p) if s["key_begin"] is None else s["key_begin"].long()
    hi = p + 1 if s["key_end"] is None else s["key_end"].long()
    if c["window"] > 0:
        lo = torch.maximum(lo, p - c["window"] + 1)
    return b, p, lo.clamp(min=0), torch.minimum(hi, s["seq_lens"].long()[b])


def _plain_attention(s):
    c = s["case"]
    B, D, Hq, Hkv, L, n = c["batch"], c["dim"], c["q_heads"], c["kv_heads"], s["L_max"], s["n_max"]
    G = Hq // Hkv
    b, p, lo, hi = _limits(s)
    i = torch.arange(s["T"], device=b.device) - s["cu"].long()[b]   # row of the token in its sequence
    key = torch.arange(L, device=b.device)
    # keys and values of each sequence in order, rows past its end zero
    table = torch.where(s["table"] < s["k_cache"].shape[0], s["table"], 0).long()
    real = (key[None, :] < s["seq_lens"][:, None])[:, None, :, None]
    k = s["k_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    v = s["v_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    k, v = torch.where(real, k, 0.0), torch.where(real, v, 0.0)
    q = torch.zeros(B, n, Hq, D, device=b.device)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, G, n, L).mul_(D ** -0.5)
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    see = torch.zeros(B, n, L, dtype=torch.bool, device=b.device)
    see[b, i] = (key[None, :] >= lo[:, None]) & (key[None, :] < hi[:, None])
    if s["slopes"] is not None:
        far = torch.zeros(B, n, L, device=b.device)
        far[b, i] = (p[:, None] - key[None, :]).abs().float()
        x.sub_(s["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None])
    x.masked_fill_(~see[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * n, L), v).view(B, Hkv, G, n, D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[b, i]
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[b, i].contiguous()}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)


def _exact_rope(s):
    c = s["case"]
    lens, _ = _lengths(c)
    P, D, rot = c["page"], c["dim"], c["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q_all = torch.empty(s["T"], c["q_heads"], D, dtype=torch.float64, device=kc.device)
    t0 = 0
    for b, (n, L) in enumerate(lens):
        pos = torch.arange(L - n, L, device=kc.device)
        got = []
        for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])):
            x = x[t0: t0 + n].double()
            if c["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            if rot:
                # a pair of channels as a complex number times exp(i p f)
                if c["layout"] == "half":
                    z = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot])
                else:
                    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2])
                angle = pos.double()[:, None] * s["inv_freq"].double()[None, :]
                z = z * torch.polar(torch.full_like(angle, s["rot_scale"]), angle)[:, None, :]
                pair = (z.real, z.imag)
                turned = torch.cat(pair, -1) if c["layout"] == "half" else torch.stack(pair, -1).flatten(-2)
                x = torch.cat((turned, x[..., rot:]), -1)
            got.append(x)
        q_all[t0: t0 + n] = got[0]
        page = s["table"][b].long()[pos // P]
        kc[page, :, pos % P] = got[1]
        vc[page, :, pos % P] = s["v"][t0: t0 + n].double()
        t0 += n
    return {"q": q_all, "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    c = s["case"]
    lens, _ = _lengths(c)
    P, D, Hq, Hkv = c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    G = Hq // Hkv
    dev = s["q"].device
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], Hq), float("-inf"), dtype=torch.float64, device=dev)
    t0 = 0
    for b, ((n, L), (lo, hi)) in enumerate(zip(lens, _visible(c))):
        lo, hi = _windowed(c, n, L, lo, hi)
        lo, hi = torch.tensor(lo, device=dev), torch.tensor(hi, device=dev)
        key = torch.arange(L, device=dev)
        page, slot = s["table"][b].long()[key // P], key % P
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            a, z = max(0, int(lo[i0:i1].min())), min(L, int(hi[i0:i1].max()))
            if z <= a:
                continue
            hidden = (key[None, a:z] < lo[i0:i1, None]) | (key[None, a:z] >= hi[i0:i1, None])
            away = (torch.arange(L - n + i0, L - n + i1, device=dev)[:, None] - key[None, a:z]).abs().double()
            k, v = s["k_cache"][page[a:z], :, slot[a:z]].double(), s["v_cache"][page[a:z], :, slot[a:z]].double()
            for g in range(Hkv):
                x = torch.einsum("ihd,kd->hik", s["q"][t0 + i0: t0 + i1, g * G: (g + 1) * G].double(), k[:, g]) / math.sqrt(D)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][g * G: (g + 1) * G].double()[:, None, None] * away
                x = torch.where(hidden[None], float("-inf"), x)
                total = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(torch.isinf(total), 0.0, total)[..., None])
                out[t0 + i0: t0 + i1, g * G: (g + 1) * G] = torch.einsum("hik,kd->ihd", w, v[:, g])
                lse[t0 + i0: t0 + i1, g * G: (g + 1) * G] = total.T
        t0 += n
    return {"out": out, "lse": lse}
