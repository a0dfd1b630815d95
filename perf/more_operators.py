"""The operators of a serving step that checks a tree of drafted tokens over the paged cache.

Such a step writes its drafted tokens behind each sequence's history, siblings side by side: a token's slot
is no longer its position, and it sees the history and its own ancestors only.  Five operators, each in a plain
form (elementary torch operations in 32 bits) and as calls of the library:

* ``plan``: from each token's parent its position and the bits of the drafted tokens it sees, once a step;
* ``write``: norm and rotation at those positions, and the write of K and V behind the history;
* ``conv``: the short convolution of K and V along each token's path to the root, written to the cache, and the
  convolution state along the path that was accepted;
* ``attend``: attention of the drafted tokens over history and ancestors, with a window, capped scores, a bias
  per token and distance, or a bias that falls linearly with the distance;
* ``commit``: the K and V rows of the accepted path moved behind the history, in the pools of all layers.
"""
import math
import random

import torch

own = False

# (query heads, KV heads): the window and global layers of the model, their tiny form, and layouts without
# grouping, with odd groups or with one KV head.
HEADS = ((64, 8), (64, 16), (8, 2), (8, 8), (12, 4), (14, 2), (40, 8), (16, 1))


def _base(name, op, batch, nodes, ctx, heads, dim, page, shape, lens):
    """Drafted tokens per sequence in [nodes/2, nodes], history before them in [ctx/2, ctx], by `lens`."""
    return dict(name=name, op=op, batch=batch, nodes=nodes, ctx=ctx, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                page=page, shape=shape, lens=lens)


def _attend(*a, window=-1, extent=0, bias="none", softcap=0.0, slopes=False):
    return dict(_base(*a), window=window, extent=extent, bias=bias, softcap=softcap, slopes=slopes)


def _write(*a, norm=True, layout="half", rot=0):
    return dict(_base(*a), norm=norm, layout=layout, rot=rot)


def listed():
    return [
        # one request that drafts a few tokens: a launch
        _base("plan_one", "plan", 1, 7, 500, (8, 2), 64, 16, "chain", 1),
        # a full batch with wide trees
        _base("plan_batch", "plan", 128, 64, 4000, (64, 8), 128, 64, "tree", 2),
        # one request of a small model that drafts a chain
        _attend("attend_chain_small", "attend", 1, 3, 1555, (8, 2), 64, 16, "chain", 3, softcap=30.0),
        # a global layer of the model, trees of up to 16 tokens
        _attend("attend_global_bias", "attend", 16, 16, 16384, (64, 8), 128, 64, "tree", 4, extent=4096, bias="float32"),
        # a window layer of the model, trees of up to 8 tokens
        _attend("attend_window_bias", "attend", 64, 8, 8192, (64, 16), 128, 64, "tree", 5, window=512, extent=512,
                bias="float32"),
        # large trees of a rotary model against long histories
        _attend("attend_long", "attend", 4, 61, 65536, (64, 8), 128, 64, "tree", 6),
        # a drafted chain of one request of a small rotary model
        _write("write_one", "write", 1, 5, 3001, (8, 2), 64, 16, "chain", 7, rot=64),
        # the trees of a batch, heads normed and rotated
        _write("write_batch", "write", 64, 32, 2000, (64, 8), 128, 64, "tree", 8, rot=128),
        # a drafted chain of one request of the tiny form of the model
        dict(_base("conv_one", "conv", 1, 4, 300, (8, 2), 64, 16, "chain", 9), taps=4),
        # the trees of a batch, window layers
        dict(_base("conv_batch", "conv", 64, 32, 500, (64, 16), 128, 64, "tree", 10), taps=4),
        # one request, one layer
        dict(_base("commit_one", "commit", 1, 9, 1000, (8, 2), 64, 16, "tree", 11), pools=1),
        # a batch, the pools of the global layers
        dict(_base("commit_layers", "commit", 64, 32, 300, (64, 8), 128, 64, "tree", 12), pools=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "plan", "write", "conv", "commit"))
    heads = rng.choice(HEADS)
    dim = rng.choice((64, 128, 128))
    page = rng.choice((8, 16, 32, 64, 64, 128, 256))
    nodes = _log(rng, 1, 100)
    shape = rng.choice(("chain", "tree", "tree"))
    lens = rng.randrange(1 << 20)
    if op == "attend":
        ctx = _log(rng, 1, 60000)
        bias = rng.choice(("none", "none", "float32", "float32", "bfloat16"))
        extent = 0 if bias == "none" else rng.choice((64, 512, 1024, 4096, _log(rng, 1, 3000)))
        batch = max(1, min(_log(rng, 1, 100), 1_500_000 // (ctx * heads[1]), 12_000_000 // (ctx * nodes), 2000 // nodes,
                           80_000_000 // (nodes * heads[0] * max(1, min(extent, ctx)))))
        case = _attend("", op, batch, nodes, ctx, heads, dim, page, shape, lens,
                       window=rng.choice((-1, -1, 512, _log(rng, 1, 2500))), extent=extent, bias=bias,
                       softcap=rng.choice((0.0, 0.0, 30.0, 50.0)), slopes=rng.random() < 0.25)
    else:
        batch = max(1, min(_log(rng, 1, 128), 4000 // nodes))
        case = _base("", op, batch, nodes, _log(rng, 1, 600), heads, dim, page, shape, lens)
        if op == "write":
            rot = rng.choice((0, 16, dim // 2, dim, dim))
            case.update(norm=rng.random() < 0.7 or rot == 0, layout=rng.choice(("half", "interleaved")), rot=rot)
        elif op == "conv":
            case.update(taps=rng.choice((2, 3, 4, 4, 8)))
        elif op == "commit":
            case.update(pools=rng.choice((1, 2, 5, 11)))
    del case["name"]
    return case


# ------------------------------------------------------------------ sizes that follow from a case alone


def _lengths(case):
    """(drafted tokens, history) of each sequence, and the generator that drew them."""
    r = random.Random(case["lens"])
    return [(r.randint((case["nodes"] + 1) // 2, case["nodes"]), r.randint((case["ctx"] + 1) // 2, case["ctx"]))
            for _ in range(case["batch"])], r


def _parents(case, seed=None):
    """Each token's parent within its sequence (-1: the last token of the history), parents first.

    A chain, or levels of 2 to 8 tokens whose parents are drawn from the level before; the first
    token, which the last step has sampled, is the root of them all."""
    lens, r = _lengths(case)
    if seed is not None:
        r = random.Random(seed)
    got = []
    for n, _ in lens:
        if case["shape"] == "chain":
            got.append(list(range(-1, n - 1)))
            continue
        p, level = [-1], [0]
        while len(p) < n:
            below = range(len(p), min(n, len(p) + r.randint(2, 8)))
            p.extend(sorted(r.choice(level) for _ in below))
            level = list(below)
        got.append(p)
    return got


def _paths(case):
    """An accepted path from the root of each sequence.

    A path that moves a row from a slot that it also fills is left out, so that a second pass over the
    same pools finds the same rows."""
    r = random.Random(case["lens"] + 1)
    got = []
    for p in _parents(case):
        path = [0]
        for _ in range(20):
            way = [r.randrange(len(p))]
            while p[way[-1]] >= 0:
                way.append(p[way[-1]])
            way.reverse()
            if all(i == j or i >= len(way) for j, i in enumerate(way)):
                path = way
                break
        got.append(path)
    return got


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _words(case):
    return (case["nodes"] + 31) // 32


def work(case):
    lens, _ = _lengths(case)
    D, Hq, Hkv = case["dim"], case["q_heads"], case["kv_heads"]
    T = sum(n for n, _ in lens)
    op = case["op"]
    if op == "plan":
        return {"bytes": 4.0 * T * (2 + _words(case)), "flops": 0.0}
    if op == "write":
        return {"bytes": 2.0 * T * (Hq + 2 * Hkv) * D * 2 + T * 12, "flops": 8.0 * T * (Hq + Hkv) * D}
    if op == "conv":
        ks, row = case["taps"], Hkv * D * 2
        return {"bytes": 2.0 * (2 * T * row + 3 * len(lens) * (ks - 1) * row + Hkv * D * ks * 4) + T * 8,
                "flops": 4.0 * T * Hkv * D * ks}
    if op == "commit":
        moved = sum(sum(i != j for j, i in enumerate(path)) for path in _paths(case))
        return {"bytes": 2.0 * 2 * case["pools"] * moved * Hkv * D * 2 + 4.0 * T, "flops": 0.0}
    pairs, keys, biases = 0, 0, 0
    W = case["window"]
    for (n, H), parents in zip(lens, _parents(case)):
        first = H
        for d in _depths(parents):
            lo = max(0, H + d - W + 1) if W > 0 else 0
            first = min(first, lo)
            near = min(d + 1, W) if W > 0 else d + 1
            seen = max(0, H - lo) + near
            pairs += seen
            biases += min(seen, case["extent"])
        keys += H - first + n
    size = {"none": 0, "float32": 4, "bfloat16": 2}[case["bias"]]
    return {"bytes": 2.0 * T * Hq * D * 2 + T * Hq * 4 + keys * Hkv * D * 4.0 + float(biases) * Hq * size,
            "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs


def _table(lens, page, host, dev):
    """Pages of a sequence at random places of a pool with spare pages; entries past a sequence's own
    pages name no page at all."""
    need = [(n + h + page - 1) // page for n, h in lens]
    total = sum(need)
    pages = total + max(1, total // 10)
    perm = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((len(lens), max(need)), pages + 7, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = perm[at: at + c]
        at += c
    return table.to(dev), pages, perm[total:].long().to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed + 77)
    lens, _ = _lengths(case)
    parents = _parents(case)
    if case["op"] == "plan":   # its inputs are the trees and the lengths
        parents = _parents(case, seed)
        r = random.Random(seed)
        lens = [(n, r.randint((case["ctx"] + 1) // 2, case["ctx"])) for n, _ in lens]
    D, P, Hq, Hkv = case["dim"], case["page"], case["q_heads"], case["kv_heads"]
    T = sum(n for n, _ in lens)
    table, pages, spare = _table(lens, P, host, dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    def pool():
        x = randn(pages, Hkv, P, D)
        x[spare] = float("nan")
        return x

    s = dict(case=case, T=T, table=table, n_max=max(n for n, _ in lens), L_max=max(n + h for n, h in lens))
    s["seq_lens"] = ints([n + h for n, h in lens])
    s["cu"] = ints([0] + torch.cumsum(torch.tensor([n for n, _ in lens]), 0).tolist())
    s["parents"] = ints([p for ps in parents for p in ps])
    op = case["op"]
    if op in ("write", "attend"):
        s["positions"] = ints([h + d for (_, h), ps in zip(lens, parents) for d in _depths(ps)])
    if op == "write":
        # the rows of one fused projection: q, k and v are strided views of it
        rows = randn(T, (Hq + 2 * Hkv) * D, std=1.5)
        s["q"] = rows[:, : Hq * D].view(T, Hq, D)
        s["k"] = rows[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = rows[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["k_cache"], s["v_cache"] = pool(), pool()
        s["w_q"] = s["w_k"] = s["inv_freq"] = None
        if case["norm"]:
            s["w_q"] = torch.rand(D, generator=gen, device=dev) + 0.5
            s["w_k"] = torch.rand(D, generator=gen, device=dev) + 0.5
        if case["rot"]:
            s["inv_freq"] = torch.pow(10000.0, -torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64)
                                      / case["rot"]).float()
    elif op == "attend":
        # capped models have larger scores than the others
        s["q"] = randn(T, Hq, D, std=4.0 if case["softcap"] else 1.0)
        s["k_cache"], s["v_cache"] = pool(), pool()
        s["ancestors"] = _bits(parents, _words(case)).to(dev)
        s["rel"] = s["slopes"] = None
        if case["bias"] != "none":
            s["rel"] = (torch.randn(T, Hq, case["extent"], generator=gen, device=dev) * 0.5).to(getattr(torch, case["bias"]))
        if case["slopes"]:
            s["slopes"] = torch.pow(2.0, -8.0 * (torch.arange(Hq, device=dev) + 1) / Hq)
    elif op == "conv":
        ks = case["taps"]
        s["k"], s["v"] = randn(T, Hkv, D), randn(T, Hkv, D)
        s["w_k"] = torch.randn(Hkv, D, ks, generator=gen, device=dev) * ks ** -0.5
        s["w_v"] = torch.randn(Hkv, D, ks, generator=gen, device=dev) * ks ** -0.5
        s["state_k"], s["state_v"] = randn(len(lens), ks - 1, Hkv, D), randn(len(lens), ks - 1, Hkv, D)
        s["k_cache"], s["v_cache"] = pool(), pool()
    elif op == "commit":
        s["k_caches"], s["v_caches"] = [pool() for _ in range(case["pools"])], [pool() for _ in range(case["pools"])]
    if op in ("conv", "commit"):
        paths = _paths(case)
        width = max(len(p) for p in paths)
        s["path"] = ints([p + [-1] * (width - len(p)) for p in paths])
        s["path_lens"] = ints([len(p) for p in paths])
    if own:
        from paged_attention_relative_gqa_gb300 import binding
        s["params"] = binding.make_params(num_seqs=len(lens), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=P,
                                          max_pages_per_seq=table.shape[1], num_pages=pages,
                                          rel_extent=max(1, case.get("extent", 1)), window=case.get("window", -1),
                                          sm_scale=D ** -0.5)
        s["workspace"] = binding.alloc_tree_workspace(s["params"], dev)
        if op == "commit":
            s["pools"] = binding.tree_pools(s["params"], s["k_caches"], s["v_caches"])
    return s


def _bits(parents, words):
    """Ancestors of each token, itself among them, a bit each (int32 words)."""
    rows = []
    for ps in parents:
        own_bits = []
        for i, p in enumerate(ps):
            own_bits.append((own_bits[p] if p >= 0 else 0) | 1 << i)
        rows.extend(own_bits)
    raw = b"".join(x.to_bytes(4 * words, "little") for x in rows)
    return torch.frombuffer(bytearray(raw), dtype=torch.int32).view(len(rows), words)


# ------------------------------------------------------------------ one pass


def run(s):
    return _RUN[s["case"]["op"]][own](s)


def _own_plan(s):
    from paged_attention_relative_gqa_gb300 import binding
    positions = torch.empty_like(s["parents"])
    ancestors = torch.empty(s["T"], _words(s["case"]), dtype=torch.int32, device=positions.device)
    binding.inkling_attn_tree_plan(s["params"], s["cu"], s["seq_lens"], s["parents"], positions, ancestors, s["workspace"])
    return {"positions": positions, "ancestors": ancestors}


def _own_write(s):
    from paged_attention_relative_gqa_gb300 import binding
    c = s["case"]
    q_out = torch.empty(s["T"], c["q_heads"], c["dim"], dtype=torch.bfloat16, device=s["q"].device)
    binding.inkling_attn_qk_norm_rope_write(
        s["params"], s["q"], s["k"], s["v"], s["cu"], s["seq_lens"], s["table"], q_out, s["k_cache"], s["v_cache"],
        s["workspace"], w_q=s["w_q"], w_k=s["w_k"], eps=1e-6, inv_freq=s["inv_freq"], layout=c["layout"],
        positions=s["positions"])
    return {"q": q_out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_conv(s):
    from paged_attention_relative_gqa_gb300 import binding
    binding.inkling_attn_kv_conv_write_tree(s["params"], s["k"], s["v"], s["cu"], s["seq_lens"], s["table"], s["parents"],
                                            s["w_k"], s["w_v"], s["state_k"], s["state_v"], s["k_cache"], s["v_cache"],
                                            s["workspace"])
    state_k, state_v = torch.empty_like(s["state_k"]), torch.empty_like(s["state_v"])
    binding.inkling_attn_kv_conv_state_tree(s["params"], s["k"], s["v"], s["cu"], s["path"], s["path_lens"], s["state_k"],
                                            s["state_v"], state_k, state_v, s["workspace"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "state_k": state_k, "state_v": state_v}


def _own_attend(s):
    from paged_attention_relative_gqa_gb300 import binding
    c = s["case"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=out.device)
    binding.inkling_attn_tree(s["params"], s["q"], s["cu"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                              s["positions"], s["ancestors"], out, s["workspace"], rel_logits=s["rel"],
                              softcap=c["softcap"], slopes=s["slopes"], lse=lse)
    return {"out": out, "lse": lse}


def _own_commit(s):
    from paged_attention_relative_gqa_gb300 import binding
    seq_lens = torch.empty_like(s["seq_lens"])
    binding.inkling_attn_tree_commit(s["params"], s["cu"], s["seq_lens"], s["table"], s["path"], s["path_lens"],
                                     s["pools"], seq_lens, s["workspace"])
    return {"seq_lens": seq_lens, "k": s["k_caches"], "v": s["v_caches"]}


def _rows(s):
    """Sequence of each packed token, its place in it, and the sequence's history."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b], (s["seq_lens"].long() - cu.diff())[b]


def _slot(s, b, key):
    """Page and place of key `key` of sequence b."""
    P = s["case"]["page"]
    return s["table"][b, key // P].long(), key % P


def _plain_plan(s):
    c = s["case"]
    b, i, hist = _rows(s)
    words = _words(c)
    n = s["n_max"]
    # the tokens of each sequence as a matrix that says who sees whom, joined along ever longer paths
    see = torch.zeros(c["batch"], n, 32 * words, dtype=torch.bool, device=b.device)
    see[b, i, i] = True
    up = torch.full((c["batch"], n), -1, dtype=torch.long, device=b.device)
    up[b, i] = s["parents"].long()
    step = 1
    while step < n:
        at = up.clamp(min=0)
        there = (up >= 0)[..., None] & see.gather(1, at[..., None].expand_as(see))
        see = see | there
        up = torch.where(up >= 0, up.gather(1, at), up)
        step *= 2
    see = see[b, i]
    bit = torch.pow(2, torch.arange(32, device=b.device))
    w = (see.view(s["T"], words, 32).long() * bit).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w)
    return {"positions": (hist + see.sum(-1) - 1).int(), "ancestors": w.int()}


def _turn(x, cos, sin, rot, layout):
    """The first `rot` channels rotated in pairs."""
    y = x.clone()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_write(s):
    c = s["case"]
    b, i, hist = _rows(s)
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["w_q"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["w_k"]
    if c["rot"]:
        angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()   # far positions need 64 bits
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q, k = _turn(q, cos, sin, c["rot"], c["layout"]), _turn(k, cos, sin, c["rot"], c["layout"])
    page, at = _slot(s, b, hist + i)
    s["k_cache"][page, :, at] = k.to(torch.bfloat16)
    s["v_cache"][page, :, at] = s["v"]
    return {"q": q.to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_conv(s):
    c = s["case"]
    ks, T, B = c["taps"], s["T"], c["batch"]
    b, i, hist = _rows(s)
    start = s["cu"].long()[b]
    page, at = _slot(s, b, hist + i)
    got = {}
    # rows of the step, then those of the states: the row of the ancestor at each distance
    node = i.clone()
    rows = []
    back = torch.full_like(i, ks - 1)     # the state's row that comes next
    for d in range(ks):
        live = node >= 0
        rows.append(torch.where(live, start + node, T + b * (ks - 1) + back.clamp(min=0)))
        node = torch.where(live, s["parents"].long()[(start + node).clamp(min=0)], node)
        back = torch.where(node < 0, back - 1, back)
    # the accepted path behind the state, its last ks - 1 rows
    m = s["path_lens"].long()
    col = m[:, None] + torch.arange(ks - 1, device=m.device)[None, :]
    on_path = s["path"].long().gather(1, (col - (ks - 1)).clamp(min=0, max=s["path"].shape[1] - 1))
    keep = torch.where(col >= ks - 1, s["cu"].long()[:-1, None] + on_path,
                       T + torch.arange(B, device=m.device)[:, None] * (ks - 1) + col.clamp(max=max(ks - 2, 0)))
    for name in ("k", "v"):
        x = torch.cat((s[name], s["state_" + name].reshape(-1, c["kv_heads"], c["dim"])))
        w = s["w_" + name]
        y = sum(x[rows[d]].float() * w[..., ks - 1 - d] for d in range(ks))
        s[name + "_cache"][page, :, at] = y.to(torch.bfloat16)
        got[name + "_cache"] = s[name + "_cache"]
        got["state_" + name] = x[keep]
    return {k: got[k] for k in ("k_cache", "v_cache", "state_k", "state_v")}


def _plain_attend(s):
    c = s["case"]
    B, D, Hq, Hkv, L, n = c["batch"], c["dim"], c["q_heads"], c["kv_heads"], s["L_max"], s["n_max"]
    G, W, T = Hq // Hkv, c["window"], s["T"]
    b, i, hist = _rows(s)
    dev = b.device
    key = torch.arange(L, device=dev)
    # keys and values of each sequence in order, rows past its end zero
    table = torch.where(s["table"] < s["k_cache"].shape[0], s["table"], 0).long()
    real = (key[None, :] < s["seq_lens"][:, None])[:, None, :, None]
    k = s["k_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    v = s["v_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    k, v = torch.where(real, k, 0.0), torch.where(real, v, 0.0)
    # positions of the keys of each sequence, and what each token sees
    pos = key.expand(B, L).clone()
    pos[b, hist + i] = s["positions"].long()
    bit = (s["ancestors"].long()[:, :, None] >> torch.arange(32, device=dev)) & 1
    bit = bit.view(T, -1).bool()
    slot = key[None, :] - hist[:, None]
    see = (slot < 0) | ((slot < bit.shape[1]) & bit.gather(1, slot.clamp(0, bit.shape[1] - 1)))
    see &= key[None, :] < s["seq_lens"][b][:, None]
    away = (s["positions"].long()[:, None] - pos[b]).abs()
    if W > 0:
        see &= s["positions"].long()[:, None] - pos[b] < W
    q = torch.zeros(B, n, Hq, D, device=dev)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, Hq, n, L)[b, :, i].mul_(D ** -0.5)   # [T, Hq, L]
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if s["slopes"] is not None:
        x.sub_(s["slopes"][None, :, None] * away.float()[:, None])
    if s["rel"] is not None:
        x.add_(s["rel"].float().gather(2, away.clamp(max=c["extent"] - 1)[:, None].expand(T, Hq, L)))
    x.masked_fill_(~see[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    w = torch.zeros(B, Hq, n, L, device=dev)
    w[b, :, i] = x / torch.where(total > 0, total, 1.0)
    o = torch.matmul(w.view(B, Hkv, G * n, L), v).view(B, Hq, n, D)[b, :, i]
    return {"out": o.to(torch.bfloat16), "lse": (top + torch.log(total))[..., 0]}


def _plain_commit(s):
    hist = s["seq_lens"].long() - s["cu"].long().diff()
    j = torch.arange(s["path"].shape[1], device=hist.device)
    here = (j[None, :] < s["path_lens"][:, None]) & (s["path"] >= 0)
    b, j = here.nonzero(as_tuple=True)
    src = _slot(s, b, hist[b] + s["path"].long()[b, j])
    dst = _slot(s, b, hist[b] + j)
    for pool in s["k_caches"] + s["v_caches"]:
        pool[dst[0], :, dst[1]] = pool[src[0], :, src[1]]
    return {"seq_lens": (hist + s["path_lens"]).int(), "k": s["k_caches"], "v": s["v_caches"]}


_RUN = {"plan": (_plain_plan, _own_plan), "write": (_plain_write, _own_write), "conv": (_plain_conv, _own_conv),
        "attend": (_plain_attend, _own_attend), "commit": (_plain_commit, _own_commit)}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    if case["op"] == "plan":   # whole numbers
        return None
    return {"write": _exact_write, "conv": _exact_conv, "attend": _exact_attend,
            "commit": _exact_commit}[case["op"]](prepare(case, seed))


def _exact_write(s):
    c = s["case"]
    P, D, rot = c["page"], c["dim"], c["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q_all = torch.empty(s["T"], c["q_heads"], D, dtype=torch.float64, device=kc.device)
    t0 = 0
    for b, ((n, H), parents) in enumerate(zip(_lengths(c)[0], _parents(c))):
        pos = torch.tensor([H + d for d in _depths(parents)], device=kc.device, dtype=torch.float64)
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
                angle = pos[:, None] * s["inv_freq"].double()[None, :]
                z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
                pair = (z.real, z.imag)
                turned = torch.cat(pair, -1) if c["layout"] == "half" else torch.stack(pair, -1).flatten(-2)
                x = torch.cat((turned, x[..., rot:]), -1)
            got.append(x)
        q_all[t0: t0 + n] = got[0]
        key = torch.arange(H, H + n, device=kc.device)
        page = s["table"][b].long()[key // P]
        kc[page, :, key % P] = got[1]
        vc[page, :, key % P] = s["v"][t0: t0 + n].double()
        t0 += n
    return {"q": q_all, "k_cache": kc, "v_cache": vc}


def _exact_conv(s):
    c = s["case"]
    ks, P = c["taps"], c["page"]
    got = {}
    for name in ("k", "v"):
        cache, w = s[name + "_cache"].double(), s["w_" + name].double()
        new_state = torch.empty_like(s["state_" + name], dtype=torch.float64)
        t0 = 0
        for b, ((n, H), parents, path) in enumerate(zip(_lengths(c)[0], _parents(c), _paths(c))):
            x, state = s[name][t0: t0 + n].double(), s["state_" + name][b].double()
            # the raw rows on the way from the oldest state row to each token
            ways = []
            for i, p in enumerate(parents):
                ways.append((ways[p] if p >= 0 else []) + [i])
            pick = torch.tensor([([*range(-(ks - 1), 0)] + way)[-ks:] for way in ways], device=x.device)
            both = torch.cat((state, x))
            y = torch.einsum("njhd,hdj->nhd", both[pick + ks - 1], w)
            key = torch.arange(H, H + n, device=x.device)
            cache[s["table"][b].long()[key // P], :, key % P] = y
            new_state[b] = both[torch.tensor(([*range(-(ks - 1), 0)] + path)[len(path):], device=x.device) + ks - 1]
            t0 += n
        got[name + "_cache"], got["state_" + name] = cache, new_state
    return {k: got[k] for k in ("k_cache", "v_cache", "state_k", "state_v")}


def _exact_attend(s):
    c = s["case"]
    P, D, Hq, Hkv, W, E = c["page"], c["dim"], c["q_heads"], c["kv_heads"], c["window"], c["extent"]
    G, dev = Hq // Hkv, s["q"].device
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], Hq), float("-inf"), dtype=torch.float64, device=dev)
    t0 = 0
    for b, ((n, H), parents) in enumerate(zip(_lengths(c)[0], _parents(c))):
        depth = _depths(parents)
        a = max(0, H + min(depth) - W + 1) if W > 0 else 0
        hidden = torch.zeros(n, H + n, dtype=torch.bool)
        hidden[:, H:] = True
        for i in range(n):
            j = i
            while j >= 0:
                hidden[i, H + j] = False
                j = parents[j]
        where = torch.cat((torch.arange(H), H + torch.tensor(depth)))
        far = where[H:, None] - where[None, :]
        if W > 0:
            hidden |= far >= W
        hidden, far = hidden[:, a:].to(dev), far[:, a:].abs().to(dev)
        key = torch.arange(a, H + n, device=dev)
        page, at = s["table"][b].long()[key // P], key % P
        k, v = s["k_cache"][page, :, at].double(), s["v_cache"][page, :, at].double()
        for g in range(Hkv):
            heads = slice(g * G, (g + 1) * G)
            x = torch.einsum("ihd,kd->hik", s["q"][t0: t0 + n, heads].double(), k[:, g]) / math.sqrt(D)
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][heads].double()[:, None, None] * far.double()
            if s["rel"] is not None:
                rel = s["rel"][t0: t0 + n, heads].double().transpose(0, 1)
                x = x + torch.take_along_dim(rel, far.clamp(max=E - 1)[None], 2)
            x = torch.where(hidden[None], float("-inf"), x)
            total = torch.logsumexp(x, -1)
            out[t0: t0 + n, heads] = torch.einsum("hik,kd->ihd", torch.exp(x - total[..., None]), v[:, g])
            lse[t0: t0 + n, heads] = total.T
        t0 += n
    return {"out": out, "lse": lse}


def _exact_commit(s):
    c = s["case"]
    P = c["page"]
    table = s["table"].tolist()
    lens = []
    k, v = [x.double() for x in s["k_caches"]], [x.double() for x in s["v_caches"]]
    for b, ((n, H), path) in enumerate(zip(_lengths(c)[0], _paths(c))):
        for j, i in enumerate(path):
            if i != j:
                for x in k + v:
                    x[table[b][(H + j) // P], :, (H + j) % P] = x[table[b][(H + i) // P], :, (H + i) % P]
        lens.append(H + len(path))
    return {"seq_lens": torch.tensor(lens, dtype=torch.int32, device=s["table"].device), "k": k, "v": v}
