"""The serving steps around paged decode, one pass each: whole-prompt attention
(`pa_prefill_packed`), attention of a tree of drafted tokens over the paged
cache (`pa_decode_tree`), and moving the accepted tokens' K/V into place
(`pa_compact_tokens`).

`run` makes one pass: with `own` false in plain torch operations, in 32 bits
and rounded once at the end; with `own` true through the library's calls.
Head counts and types are the library's Llama-2-7B (32 / 32, f16) and
Llama-3-70B (64 / 8, bf16) layer shapes and the smaller ones of its tests.
"""
import math

import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases

def _prompt(name, lens, max_len, heads, kv_heads, dim, dtype, fused=True):
    return {"name": name, "op": "prompt", "seqs": lens, "max_len": max_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "fused": fused}


def _tree(name, seqs, max_ctx, nodes, heads, kv_heads, dim, dtype, cache):
    return {"name": name, "op": "tree", "seqs": seqs, "max_ctx": max_ctx, "nodes": nodes,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache}


def _compact(name, layers, seqs, nodes, max_accepted, kv_heads, dim, dtype):
    return {"name": name, "op": "compact", "layers": layers, "seqs": seqs, "nodes": nodes,
            "max_accepted": max_accepted, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def listed():
    return [
        # one chat turn of a few words: the time to the first token is latency
        _prompt("prompt_short", 1, 37, 64, 8, 128, "bf16"),
        # a batch of chat prompts of different lengths, admitted in one step
        _prompt("prompt_ragged", 16, 2100, 64, 8, 128, "bf16"),
        # a few long-ish prompts with full multi-head attention
        _prompt("prompt_mha_f16", 4, 2047, 32, 32, 128, "f16"),
        # a small model (64-wide heads), separate q, k and v tensors
        _prompt("prompt_d64", 8, 1500, 32, 8, 64, "bf16", fused=False),
        # one long document
        _prompt("prompt_long", 1, 16384, 32, 8, 128, "bf16"),
        # one interactive user with a small draft tree: latency
        _tree("tree_one", 1, 777, 8, 64, 8, 128, "bf16", "same"),
        # a serving batch, 16 drafted tokens each: the cache's bytes count
        _tree("tree_batch", 64, 8000, 16, 64, 8, 128, "bf16", "same"),
        # wide trees of 64 nodes over long contexts: the products count
        _tree("tree_wide", 16, 8191, 64, 64, 8, 128, "bf16", "same"),
        # the E4M3 cache of the mixed step, two dozen drafted tokens
        _tree("tree_fp8", 96, 4000, 24, 32, 8, 128, "bf16", "fp8"),
        # multi-head attention with 64-wide heads, f16
        _tree("tree_mha_d64", 24, 2500, 12, 16, 16, 64, "f16", "same"),
        # the accepted path of one user's tree, one layer at a time
        _compact("compact_one", 1, 4, 16, 5, 8, 128, "bf16"),
        # a serving batch's accepted paths, all layers at once
        _compact("compact_layers", 32, 128, 24, 8, 8, 128, "bf16"),
    ]


HEADS = [(64, 8), (32, 32), (32, 8), (16, 4), (8, 1), (28, 4), (24, 8), (12, 2)]
MOST_PROMPT = 32 * 16384 * 16384  # score elements of the largest listed prompt


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "compact"])
    heads, kv_heads = rng.choice(HEADS)
    dim, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f16"])
    if op == "prompt":
        seqs, max_len = _log_int(rng, 1, 48), _log_int(rng, 1, 8192)
        while seqs * heads * max_len * max_len > MOST_PROMPT // 2:
            seqs, max_len = (seqs + 1) // 2, max(1, max_len * 7 // 8)
        c = _prompt("", seqs, max_len, heads, kv_heads, dim, dtype, rng.random() < 0.6)
    elif op == "tree":
        seqs, max_ctx, nodes = _log_int(rng, 1, 96), _log_int(rng, 8, 12000), _log_int(rng, 1, 64)
        while seqs * max_ctx * kv_heads * dim > 64 * 8000 * 8 * 128 or \
                seqs * max_ctx * nodes * heads * dim > 16 * 8191 * 64 * 64 * 128:
            seqs = max(1, seqs * 3 // 4)
            max_ctx = max(8, max_ctx * 7 // 8)
        if heads // kv_heads > 8:
            kv_heads = heads // 8
        c = _tree("", seqs, max_ctx, nodes, heads, kv_heads, dim, dtype,
                  rng.choice(["same", "same", "fp8"]))
    else:
        nodes = _log_int(rng, 2, 64)
        c = _compact("", _log_int(rng, 1, 32), _log_int(rng, 1, 128), nodes,
                     rng.randint(1, min(nodes, 12)), kv_heads, dim, dtype)
        while c["layers"] * c["seqs"] * kv_heads * dim > 32 * 128 * 8 * 128:
            c["layers"] = max(1, c["layers"] // 2)
            c["seqs"] = max(1, c["seqs"] * 3 // 4)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lens(case, seed=0):
    """Lengths that follow from the case alone (its work does not depend on the
    seed): the longest first, the others spread below it, odd ones among them."""
    n, hi = case["seqs"], case["max_len"] if case["op"] == "prompt" else case["max_ctx"]
    lo = 1 if case["op"] == "prompt" else min(hi, case["nodes"])
    out = [hi]
    for i in range(1, n):
        u = (i * 0.6180339887498949) % 1.0  # a low-discrepancy spread
        out.append(max(lo, int(hi * math.exp(-2.5 * u)) | 1) if hi > 1 else 1)
    return [min(x, hi) for x in out]


def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(1000003 * int(seed) + 17)


def _masks(nodes, n_of, cpu):
    """Ancestor masks of random trees in topological order: bit j of [s][i] is
    set where node j is node i or one of its ancestors."""
    out = torch.zeros(len(n_of), nodes, dtype=torch.int64)
    for s, n in enumerate(n_of):
        rows = []
        parents = torch.rand(nodes, generator=cpu).tolist()
        for i in range(n):
            up = 0 if i == 0 else rows[int(i * parents[i] ** 0.5)]
            rows.append(up | (1 << i))
        out[s, :n] = torch.tensor([r - (1 << 64) if r >> 63 else r for r in rows])
    return out


def _tables(ctx, spare, cpu):
    """Shuffled block tables (unused entries -1) and the pool's size."""
    need = [-(-c // BLOCK) for c in ctx]
    total = sum(need) + spare
    order = torch.randperm(total, generator=cpu).to(torch.int32)
    bt = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = order[at:at + k]
        at += k
    return bt, total


def prepare(case, seed):
    dev = torch.device("cuda")
    g, cpu = _gen(seed, dev), _gen(seed, "cpu")
    h, kv, d, dt = case["heads"] if "heads" in case else 0, case["kv_heads"], case["dim"], \
        DTYPES[case["dtype"]]
    st = {"case": case, "scale": d ** -0.5}
    if case["op"] == "prompt":
        lens = _lens(case)
        total = sum(lens)
        if case["fused"]:  # views into the fused projection's output
            qkv = torch.randn(total, h + 2 * kv, d, generator=g, device=dev, dtype=dt)
            q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        else:
            q, k, v = (torch.randn(total, n, d, generator=g, device=dev, dtype=dt)
                       for n in (h, kv, kv))
        q.mul_(2)  # scores with a spread of 2, as trained heads have, not 1
        start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
        # padded positions of the plain form (a program's batch layout)
        pos = torch.full((len(lens), max(lens)), 0, dtype=torch.int64)
        keep = torch.zeros(len(lens), max(lens), dtype=torch.bool)
        at = 0
        for s, n in enumerate(lens):
            pos[s, :n] = torch.arange(at, at + n)
            keep[s, :n] = True
            at += n
        st.update(q=q, k=k, v=v, start=start, pos=pos.to(dev), keep=keep.to(dev),
                  out=torch.empty(total, h, d, device=dev, dtype=dt))
    elif case["op"] == "tree":
        ctx, nodes = _lens(case), case["nodes"]
        n_of = [min(c, max(1, nodes - (s % 4) * (nodes // 8))) for s, c in enumerate(ctx)]
        bt, total = _tables(ctx, len(ctx), cpu)
        shape = (total, kv, BLOCK, d)
        st.update(k_scale=1.0, v_scale=1.0)
        k, v = (torch.randn(shape, generator=g, device=dev, dtype=dt) for _ in range(2))
        if case["cache"] == "fp8":
            st.update(k_scale=0.015625, v_scale=0.0125)
            k, v = ((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    for x, s in ((k, st["k_scale"]), (v, st["v_scale"])))
        q = torch.randn(len(ctx), nodes, h, d, generator=g, device=dev, dtype=dt).mul_(2)
        st.update(q=q, k=k, v=v, tables=bt.to(dev),
                  ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
                  lens=torch.tensor(n_of, dtype=torch.int32, device=dev),
                  masks=_masks(nodes, n_of, cpu).to(dev), out=torch.empty_like(q))
    else:
        nodes, most, S = case["nodes"], case["max_accepted"], case["seqs"]
        ctx = [nodes + 20 + (37 * s) % 61 for s in range(S)]
        bt, total = _tables(ctx, S, cpu)
        pools = torch.randn(case["layers"], 2, total, kv, BLOCK, d, generator=g, device=dev,
                            dtype=dt)
        # accepted nodes, increasing: the drafts' first guesses for a while,
        # then nodes behind the kept ones (so a second pass moves nothing new)
        acc = torch.zeros(S, most, dtype=torch.int32)
        n_acc = torch.randint(1, most + 1, (S,), generator=cpu).to(torch.int32)
        for s in range(S):
            n = int(n_acc[s])
            first = int(torch.randint(0, n + 1, (1,), generator=cpu))
            rest = torch.randperm(nodes - n, generator=cpu)[:n - first].sort().values + n
            first = n - len(rest)
            acc[s, :n] = torch.cat([torch.arange(first), rest]).to(torch.int32)
        st.update(pools=pools, k_pools=pools[:, 0], v_pools=pools[:, 1], tables=bt.to(dev),
                  ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
                  lens=torch.full((S,), nodes, dtype=torch.int32, device=dev),
                  accepted=acc.to(dev), n_accepted=n_acc.to(dev))
    return st


# --------------------------------------------------------------- the passes

def _softmax_rows(x, seen):
    """Masked scores to weights, in place; rows that see nothing get zeros."""
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min_(-3e38)
    x.sub_(top).exp_()
    return x.div_(x.sum(-1, keepdim=True).clamp_min_(1e-38))


def _prompt_plain(st):
    q, k, v, pos, keep = st["q"], st["k"], st["v"], st["pos"], st["keep"]
    S, L = pos.shape
    h, kv, d = q.shape[1], k.shape[1], q.shape[2]
    qp = q[pos].float().view(S, L, kv, h // kv, d).permute(0, 2, 3, 1, 4)
    kp, vp = (x[pos].float().permute(0, 2, 1, 3).unsqueeze(2) for x in (k, v))
    x = torch.matmul(qp * st["scale"], kp.transpose(-1, -2))  # [S, kv, G, L, L]
    at = torch.arange(L, device=q.device)
    w = _softmax_rows(x, at <= at[:, None])
    o = torch.matmul(w, vp).permute(0, 3, 1, 2, 4).reshape(S, L, h, d)
    return o[keep].to(q.dtype)


def _cache_rows(pool, tables, scale):
    x = pool[tables.clamp_min(0).long()]  # [S, blocks, kv, 16, d]
    x = x.view(torch.float8_e4m3fn).float() * scale if x.dtype == torch.uint8 else x.float()
    S, nb, kv, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(S, kv, nb * BLOCK, d)


def _tree_plain(st):
    q, ctx, n = st["q"], st["ctx"].long(), st["lens"].long()
    S, T, h, d = q.shape
    k = _cache_rows(st["k"], st["tables"], st["k_scale"])
    v = _cache_rows(st["v"], st["tables"], st["v_scale"])
    kv, L = k.shape[1], k.shape[2]
    at = torch.arange(L, device=q.device)
    node = at - (ctx - n)[:, None]  # [S, L]: the tree's node at each position
    bit = st["masks"][:, :, None] >> node.clamp(0, 63)[:, None, :] & 1  # [S, T, L]
    live = (torch.arange(T, device=q.device) < n[:, None])[:, :, None]
    seen = ((node < 0)[:, None, :] | (bit == 1)) & (at < ctx[:, None])[:, None, :] & live
    qp = q.float().view(S, T, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(S, kv, -1, d)
    x = torch.matmul(qp * st["scale"], k.transpose(-1, -2)).view(S, kv, h // kv, T, L)
    w = _softmax_rows(x, seen[:, None, None]).view(S, kv, -1, L)
    o = torch.matmul(w, v).view(S, kv, h // kv, T, d).permute(0, 3, 1, 2, 4)
    return o.reshape(S, T, h, d).to(q.dtype)


def _slots(st, node):
    """(block, offset) of tree node `node` [S, n] of every sequence."""
    p = (st["ctx"] - st["lens"])[:, None].long() + node.long()
    return st["tables"].gather(1, p // BLOCK).long(), p % BLOCK


def _compact_plain(st):
    pools, acc, n = st["pools"], st["accepted"], st["n_accepted"]
    i = torch.arange(acc.shape[1], device=acc.device).expand_as(acc)
    used = i < n[:, None]
    sb, so = (x[used] for x in _slots(st, acc))
    db, do = (x[used] for x in _slots(st, i))
    pools[:, :, db, :, do] = pools[:, :, sb, :, so]
    return pools


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        if op == "prompt":
            return _prompt_plain(st)
        return _tree_plain(st) if op == "tree" else _compact_plain(st)
    from pagedattention_paged_kv_pa_b200 import binding as B
    if op == "prompt":
        return B.pa_prefill_packed(st["out"], st["q"], st["k"], st["v"], st["start"],
                                   st["scale"])
    if op == "tree":
        if "workspace" not in st:  # a serving loop keeps it
            st["workspace"] = B.alloc_tree_workspace(st["q"], st["k"])
        return B.pa_decode_tree(st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"],
                                st["masks"], st["scale"], tree_lens=st["lens"],
                                k_scale=st["k_scale"], v_scale=st["v_scale"],
                                workspace=st["workspace"])
    B.pa_compact_tokens(st["k_pools"], st["v_pools"], st["tables"], st["ctx"], st["lens"],
                        st["accepted"], st["n_accepted"])
    return st["pools"]


# ------------------------------------------------------------------- sizes

def work(case):
    kv, d = case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        lens, h = _lens(case), case["heads"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * h + 2 * kv) * d * 2, "flops": 4 * pairs * h * d}
    if case["op"] == "tree":
        ctx, h, t = _lens(case), case["heads"], case["nodes"]
        es = 1 if case["cache"] == "fp8" else 2
        n_of = [min(c, max(1, t - (s % 4) * (t // 8))) for s, c in enumerate(ctx)]
        rows = case["seqs"] * t * h * d * 2
        return {"bytes": sum(ctx) * kv * d * 2 * es + sum(n_of) * h * d * 2 + rows +
                sum(-(-c // BLOCK) * 4 + 8 for c in ctx) + case["seqs"] * t * 8,
                "flops": 4 * sum(c * n for c, n in zip(ctx, n_of)) * h * d}
    # half of a path's nodes on average stay where they are; the moved rows
    # are read once and written once
    moved = case["seqs"] * (case["max_accepted"] + 1) / 4.0
    return {"bytes": case["layers"] * 2 * moved * kv * d * 2 * 2, "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "compact":
        new = st["pools"].double()
        acc, n, ctx = st["accepted"].tolist(), st["n_accepted"].tolist(), st["ctx"].tolist()
        bt = st["tables"].tolist()
        for s in range(case["seqs"]):
            base = ctx[s] - case["nodes"]
            for i in range(n[s]):
                a, b = base + acc[s][i], base + i
                new[:, :, bt[s][b // BLOCK], :, b % BLOCK] = \
                    st["pools"][:, :, bt[s][a // BLOCK], :, a % BLOCK].double()
        return new
    if case["op"] == "prompt":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        G = case["heads"] // case["kv_heads"]
        at = 0
        for n in _lens(case):
            for a in range(0, case["heads"]):
                qs, ks, vs = (x[at:at + n, y].double() for x, y in
                              ((st["q"], a), (st["k"], a // G), (st["v"], a // G)))
                s = (qs @ ks.T * st["scale"]).tril_()
                s += torch.full_like(s, -math.inf).triu_(1) if n > 1 else 0
                out[at:at + n, a] = torch.softmax(s, -1) @ vs
            at += n
        return out
    q, ctx, lens = st["q"], st["ctx"].tolist(), st["lens"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G, bits = case["heads"] // case["kv_heads"], st["masks"].tolist()
    for s, (c, n) in enumerate(zip(ctx, lens)):
        ids = st["tables"][s, :-(-c // BLOCK)].long()

        def rows(pool, scale):
            x = pool[ids].transpose(0, 1).reshape(case["kv_heads"], -1, case["dim"])[:, :c]
            return x.view(torch.float8_e4m3fn).double() * scale if x.dtype == torch.uint8 \
                else x.double()
        k, v = rows(st["k"], st["k_scale"]), rows(st["v"], st["v_scale"])
        hide = torch.zeros(n, c, dtype=torch.float64)
        for i in range(n):
            for j in range(n):
                if not bits[s][i] >> j & 1:
                    hide[i, c - n + j] = -math.inf
        hide = hide.to(q.device)
        for a in range(case["heads"]):
            w = torch.softmax(q[s, :n, a].double() @ k[a // G].T * st["scale"] + hide, -1)
            out[s, :n, a] = w @ v[a // G]
    return out
