"""pa_compact_tokens (moving the accepted tokens' K/V) against plain indexing,
and prompt -> tree -> accept -> decode as a serving loop runs them."""
import pytest
import torch

from tests import plain64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_device):
    from pagedattention_paged_kv_pa_b200 import binding
    return binding


def make(ctx, layers, n_kv, d, dt, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-c // 16) for c in ctx]
    order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    bt = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n]
        at += n
    shape = (layers, 2, sum(need) + 2, n_kv, 16, d)
    x = torch.randint(0, 256, shape + (torch.empty(0, dtype=dt).element_size(),), generator=g,
                      dtype=torch.uint8).view(dt).squeeze(-1).contiguous().to(dev)
    return x, bt


def expected(pools, bt, ctx, lens, acc):
    new = pools.clone()
    for s, a in enumerate(acc):
        for i, node in enumerate(a):
            p, t = ctx[s] - lens[s] + node, ctx[s] - lens[s] + i
            new[:, :, bt[s, t // 16], :, t % 16] = pools[:, :, bt[s, p // 16], :, p % 16]
    return new


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def call(B, pools, bt, ctx, lens, acc, most, as_list=False, none=False, **kw):
    dev = pools.device
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    rows = [list(a) + [-9] * (most - len(a)) for a in acc]
    k, v = pools[:, 0], pools[:, 1]
    if as_list:
        k, v = list(k), list(v)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    B.pa_compact_tokens(k, v, bt.to(dev), t(ctx), None if none else t(lens),
                        t(rows).view(len(acc), most), t([len(a) for a in acc]), dev_err=err, **kw)
    torch.cuda.synchronize()
    return int(err.item())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32, torch.uint8])
@pytest.mark.parametrize("n_kv,d", [(8, 128), (3, 64), (1, 16)])
@pytest.mark.parametrize("layers", [1, 3])
def test_paths(B, cuda_device, dt, n_kv, d, layers):
    ctx = [64, 70, 33, 100, 17, 64, 80]
    lens = [64, 20, 16, 9, 1, 64, 30]
    acc = [[0, 1, 5, 9, 33, 63], list(range(20)), [15], [], [0], list(range(63, 64)),
           [2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 20, 21, 22, 23, 24, 29]]
    pools, bt = make(ctx, layers, n_kv, d, dt, cuda_device, seed=d)
    want = expected(pools, bt, ctx, lens, acc)
    assert call(B, pools, bt, ctx, lens, acc, 20, as_list=layers == 3) == 0
    assert same(pools, want)


def test_every_node_shifted_by_one(B, cuda_device):
    # every row written is the next move's source
    ctx, lens = [100, 64], [64, 64]
    pools, bt = make(ctx, 2, 4, 128, torch.bfloat16, cuda_device)
    acc = [list(range(1, 64)), list(range(1, 64, 2))]
    want = expected(pools, bt, ctx, lens, acc)
    assert call(B, pools, bt, ctx, lens, acc, 63) == 0
    assert same(pools, want)


def test_more_layers_than_one_launch_takes(B, cuda_device):
    ctx, lens, acc = [40, 21], [10, 12], [[3, 7], [1, 2, 9]]
    pools, bt = make(ctx, 131, 2, 64, torch.bfloat16, cuda_device)
    want = expected(pools, bt, ctx, lens, acc)
    assert call(B, pools, bt, ctx, lens, acc, 5) == 0
    assert same(pools, want)


def test_full_trees_without_lens(B, cuda_device):
    ctx, acc = [40, 21], [[3, 7], [1, 2, 9]]
    pools, bt = make(ctx, 1, 2, 64, torch.bfloat16, cuda_device)
    want = expected(pools, bt, ctx, [10, 10], acc)
    assert call(B, pools, bt, ctx, None, acc, 3, none=True, q_len=10) == 0
    assert same(pools, want)


@pytest.mark.parametrize("acc,lens,ctx,flag", [
    ([5, 5], 10, 60, "PA_DEVERR_SLOT"), ([5, 3], 10, 60, "PA_DEVERR_SLOT"),
    ([0, 10], 10, 60, "PA_DEVERR_SLOT"), ([-1, 3], 10, 60, "PA_DEVERR_SLOT"),
    ([2, 3], 65, 80, "PA_DEVERR_QUERY_LOC"), ([2, 3], -1, 60, "PA_DEVERR_QUERY_LOC"),
    ([2, 3], 10, 9, "PA_DEVERR_QUERY_LOC"), ([2, 3], 10, 1000, "PA_DEVERR_BLOCK_ID")])
def test_broken_lists_leave_their_sequence_alone(B, cuda_device, acc, lens, ctx, flag):
    pools, bt = make([80, 60, 45], 2, 2, 64, torch.bfloat16, cuda_device)
    all_acc, all_lens = [acc, [4, 6], [1]], [lens, 10, 12]
    want = expected(pools, bt, [80, 60, 45], [10, 10, 12], [[], [4, 6], [1]])
    err = call(B, pools, bt, [ctx, 60, 45], all_lens, all_acc, 4)
    assert err == getattr(B, flag)
    assert same(pools, want)


def test_bad_block_ids_are_left_out(B, cuda_device):
    ctx, lens, acc = [70, 60], [30, 10], [[2, 25], [4, 6]]
    pools, bt = make(ctx, 2, 2, 64, torch.bfloat16, cuda_device)
    good = bt.clone()
    bt[0, 4] = pools.shape[2]  # positions 64..79: the source of node 25
    want = expected(pools, good, ctx, lens, [[2], [4, 6]])
    assert call(B, pools, bt, ctx, lens, acc, 4) == B.PA_DEVERR_BLOCK_ID
    assert same(pools, want)


def test_captured_and_replayed(B, cuda_device):
    ctx, lens = [64, 70], [20, 20]
    pools, bt = make(ctx, 2, 2, 64, torch.bfloat16, cuda_device)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    a = (bt.to(cuda_device), t(ctx), t(lens), t([[0, 0, 0], [0, 0, 0]]), t([0, 0]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pa_compact_tokens(pools[:, 0], pools[:, 1], *a)
    for acc in ([[1, 2, 3], [5, 9, 19]], [[7], [0, 2]]):
        want = expected(pools, bt, ctx, lens, acc)
        a[3].copy_(t([x + [0] * (3 - len(x)) for x in acc]))
        a[4].copy_(t([len(x) for x in acc]))
        g.replay()
        torch.cuda.synchronize()
        assert same(pools, want)


def test_prompt_tree_accept_decode(B, cuda_device):
    """Two requests through the serving loop: prompts, then rounds of drafting
    a tree, checking it, keeping one path and cutting the rest, and a decode
    step at the end, every attention against the 64-bit form over a plain copy
    of the tokens kept so far."""
    dev, n_q, n_kv, d, layers, dt = cuda_device, 8, 2, 128, 2, torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(1)
    c = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=g, dtype=dt)  # noqa: E731
    scale, blocks, cols = d ** -0.5, 60, 20
    pools = torch.full((layers, 2, blocks, n_kv, 16, d), float("nan"), device=dev, dtype=dt)
    al = B.BlockAllocator(blocks)
    al.set_prefix_caching(True)
    lens = [45, 130]
    ids = [list(range(100 * s, 100 * s + n)) for s, n in enumerate(lens)]
    kept = [[rnd(n, 2, layers, n_kv, d)] for n in lens]  # every token's K/V, plainly

    def table():
        t = torch.full((2, cols), -1, dtype=torch.int32)
        for s in range(2):
            b = al.block_table(s)
            t[s, :len(b)] = torch.tensor(b, dtype=torch.int32)
        return t.to(dev)

    def write(new, slots):  # new [n, 2, layers, n_kv, d]
        sl = torch.tensor(slots, dtype=torch.int64, device=dev)
        for l in range(layers):
            B.pa_reshape_and_cache(pools[l, 0], pools[l, 1], new[:, 0, l].contiguous(),
                                   new[:, 1, l].contiguous(), sl)

    # the prompts
    start = torch.tensor([0, 45, 175], dtype=torch.int32, device=dev)
    kv = torch.cat([k[0] for k in kept])
    for l in range(layers):
        q = rnd(175, n_q, d)
        out = torch.empty_like(q)
        B.pa_prefill_packed(out, q, kv[:, 0, l].contiguous(), kv[:, 1, l].contiguous(), start,
                            scale)
        for s, (a, n) in enumerate(((0, 45), (45, 130))):
            ref, mag = plain64.attend(q[a:a + n], kv[a:a + n, 0, l], kv[a:a + n, 1, l],
                                      plain64.causal(n, dev), scale)
            plain64.check(out[a:a + n], ref, mag, n, 6.0, dt, f"prompt {s} layer {l}")
    slots = []
    for s in range(2):
        st, sl, _ = al.admit(s, ids[s])
        assert st == B.PA_OK
        slots += sl
    write(kv, slots)

    for step in range(6):
        T = [7, 12, 20, 1, 16, 9][step]
        n_of = [T, max(1, T - 4)]
        parents = torch.full((2, T), -1, dtype=torch.int32)
        for s in range(2):
            for i in range(1, n_of[s]):
                parents[s, i] = int(torch.randint(-1, i, (1,), generator=c))
        tl = torch.tensor(n_of, dtype=torch.int32)
        masks = B.tree_masks(parents, tl)
        drafts = [rnd(n, 2, layers, n_kv, d) for n in n_of]
        ctx = []
        for s in range(2):
            ctx.append(al.num_tokens(s) + n_of[s])
            st, sl = al.append(s, n_of[s])
            assert st == B.PA_OK
            write(drafts[s], sl)
        bt, cl = table(), torch.tensor(ctx, dtype=torch.int32, device=dev)
        for l in range(layers):
            q = rnd(2, T, n_q, d)
            out = torch.empty_like(q)
            B.pa_decode_tree(out, q, pools[l, 0], pools[l, 1], bt, cl, masks.to(dev), scale,
                             tree_lens=tl.to(dev))
            for s in range(2):
                all_kv = torch.cat(kept[s] + [drafts[s]])
                P = ctx[s] - n_of[s]
                seen = torch.ones(n_of[s], ctx[s], dtype=torch.bool)
                for j in range(n_of[s]):
                    seen[:, P + j] = (masks[s, :n_of[s]] >> j & 1).bool()
                ref, mag = plain64.attend(q[s, :n_of[s]], all_kv[:, 0, l], all_kv[:, 1, l],
                                          seen.to(dev), scale)
                plain64.check(out[s, :n_of[s]], ref, mag, ctx[s], 6.0, dt, f"step {step}")
        # one leaf's path is accepted
        acc = torch.zeros(2, T, dtype=torch.int32)
        n_acc = torch.zeros(2, dtype=torch.int32)
        for s in range(2):
            i, path = int(torch.randint(0, n_of[s], (1,), generator=c)), []
            while i >= 0:
                path.insert(0, i)
                i = int(parents[s, i])
            acc[s, :len(path)] = torch.tensor(path, dtype=torch.int32)
            n_acc[s] = len(path)
            kept[s].append(drafts[s][path])
        B.pa_compact_tokens(pools[:, 0], pools[:, 1], bt, cl, tl.to(dev), acc.to(dev),
                            n_acc.to(dev))
        for s in range(2):
            n = int(n_acc[s])
            new = [1000 * step + 10 * s + i for i in range(n)]
            ids[s] += new
            assert al.truncate(s, ctx[s] - n_of[s] + n, new) == B.PA_OK
            assert al.num_tokens(s) == len(ids[s])
            assert len(al.block_table(s)) == -(-len(ids[s]) // 16)

    # a decode step over what is left, and the cache row by row
    bt = table()
    cl = torch.tensor([len(x) for x in ids], dtype=torch.int32, device=dev)
    for l in range(layers):
        q = rnd(2, n_q, d)
        out = torch.empty_like(q)
        B.pa_decode(out, q, pools[l, 0], pools[l, 1], bt, cl, scale)
        for s in range(2):
            all_kv, n = torch.cat(kept[s]), len(ids[s])
            rows = torch.stack([pools[l, x][bt[s, :-(-n // 16)].long()].transpose(1, 2)
                                .reshape(-1, n_kv, d)[:n] for x in range(2)], 1)
            assert torch.equal(rows, all_kv[:, :, l])
            ref, mag = plain64.attend(q[s][None], all_kv[:, 0, l], all_kv[:, 1, l],
                                      torch.ones(1, n, dtype=torch.bool, device=dev), scale)
            plain64.check(out[s][None], ref, mag, n, 6.0, dt, "decode")
    # the accepted tokens' full blocks are found again by another request
    st, _, cached = al.admit(7, ids[1] + [1])
    assert st == B.PA_OK and cached == len(ids[1]) // 16 * 16
