"""pa_decode_tree (a tree of drafted tokens over the paged cache) against the
64-bit form."""
import math

import pytest
import torch

from tests import plain64

pytestmark = pytest.mark.gpu

CTX = [0, 1, 3, 15, 16, 17, 64, 90, 127, 128, 129, 200, 255, 256, 400, 1100, 2049]
TYPES = [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
         (torch.float16, True)]


@pytest.fixture(scope="module")
def B(cuda_device):
    from pagedattention_paged_kv_pa_b200 import binding
    return binding


class Case:
    """A batch over a shuffled pool; cache rows that no context holds (spare
    blocks, the end of a last block) hold NaN."""

    def __init__(self, ctx, nodes, n_q, n_kv, d, dt, fp8, dev, lens=None, seed=0, spare=3,
                 masks="tree", extra_cols=2):
        g = torch.Generator(device=dev).manual_seed(seed)
        c = torch.Generator().manual_seed(seed)
        need = [-(-x // 16) for x in ctx]
        total = sum(need) + spare
        order = torch.randperm(total, generator=c)
        self.tables = torch.full((len(ctx), max(max(need), 1) + extra_cols), -1,
                                 dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = order[at:at + n]
            at += n
        used = torch.zeros(total, 16, dtype=torch.bool)
        for s, n in enumerate(ctx):
            for p in range(n):
                used[self.tables[s, p // 16], p % 16] = True
        shape = (total, n_kv, 16, d)
        self.k_scale, self.v_scale = (0.0173, 0.0121) if fp8 else (1.0, 1.0)
        k, v = (torch.randn(shape, device=dev, generator=g, dtype=torch.float32)
                for _ in range(2))
        hole = ~used.to(dev)[:, None, :, None].expand(shape)
        if fp8:
            k, v = ((x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    for x, s in ((k, self.k_scale), (v, self.v_scale)))
            k, v = (x.masked_fill(hole, 0x7f) for x in (k, v))  # E4M3's NaN
        else:
            k, v = (x.to(dt).masked_fill(hole, float("nan")) for x in (k, v))
        self.k, self.v = k.contiguous(), v.contiguous()
        self.q = torch.randn(len(ctx), nodes, n_q, d, device=dev, generator=g).mul_(2).to(dt)
        self.ctx, self.fp8, self.dev = list(ctx), fp8, dev
        self.lens = list(lens) if lens is not None else [nodes] * len(ctx)
        self.has_lens = lens is not None
        m = torch.zeros(len(ctx), nodes, dtype=torch.int64)
        if masks == "tree":
            for s in range(len(ctx)):
                for i in range(self.lens[s]):
                    up = int(torch.randint(-1, i, (1,), generator=c)) if i else -1
                    m[s, i] = (m[s, up] if up >= 0 else 0) | (torch.tensor(1) << i)
        elif masks == "random":  # any bits, also later nodes', also none
            m = torch.randint(-2 ** 63, 2 ** 63 - 1, m.shape, generator=c)
            m[:, ::3] = 0
        elif masks == "all":
            m[:] = -1
        self.masks = m
        self.scale = d ** -0.5

    def args(self):
        to = lambda x: x.to(self.dev)  # noqa: E731
        t = torch.tensor
        return (self.q, self.k, self.v, to(self.tables), to(t(self.ctx, dtype=torch.int32)),
                to(self.masks), self.scale), dict(
                    tree_lens=to(t(self.lens, dtype=torch.int32)) if self.has_lens else None,
                    k_scale=self.k_scale, v_scale=self.v_scale)

    def run(self, B, want_err=0, **kw):
        a, k = self.args()
        out = torch.full_like(self.q, 7.0)
        err = torch.zeros(1, dtype=torch.int32, device=self.dev)
        B.pa_decode_tree(out, *a, **k, dev_err=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == want_err
        return out

    def rows(self, pool, s, scale):
        n = self.ctx[s]
        ids = self.tables[s, :-(-n // 16)].long().to(self.dev)
        x = pool[ids].transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:n]
        return x.view(torch.float8_e4m3fn).double() * scale if self.fp8 else x.double()

    def check(self, out, what, seqs=None):
        T = self.q.shape[1]
        for s in range(len(self.ctx)) if seqs is None else seqs:
            n, c = self.lens[s], self.ctx[s]
            assert (out[s, n:] == 0).all(), f"{what}: rows behind the tree of {s}"
            seen = torch.zeros(T, c, dtype=torch.bool)
            P = c - n
            seen[:, :max(P, 0)] = True
            for j in range(max(0, -P), n):
                seen[:, P + j] = (self.masks[s] >> j & 1).bool()
            seen = seen[:n].to(self.dev)
            k, v = self.rows(self.k, s, self.k_scale), self.rows(self.v, s, self.v_scale)
            if c == 0:
                assert (out[s] == 0).all()
                continue
            ref, mag = plain64.attend(self.q[s, :n], k, v, seen, self.scale)
            empty = ~seen.any(-1)
            assert (out[s, :n][empty] == 0).all(), f"{what}: rows of {s} that see nothing"
            plain64.check(out[s, :n], ref, mag, c, v.abs().max().item(),
                          torch.float16 if self.fp8 else out.dtype, f"{what}, sequence {s}")


@pytest.mark.parametrize("dt,fp8", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8])
@pytest.mark.parametrize("nodes", [1, 6, 16, 33, 64])
def test_grid(B, cuda_device, dt, fp8, d, G, nodes):
    lens = [min(nodes, max(0, nodes - 3 * (i % 3))) for i in range(len(CTX))]
    c = Case(CTX, nodes, 2 * G, 2, d, dt, fp8, cuda_device, lens=lens, seed=G + d + nodes)
    c.check(c.run(B), f"{dt} fp8={fp8} d={d} G={G} nodes={nodes}")


@pytest.mark.parametrize("dt,fp8", TYPES)
@pytest.mark.parametrize("masks", ["random", "all", "none"])
@pytest.mark.parametrize("nodes", [5, 64])
def test_any_mask(B, cuda_device, dt, fp8, masks, nodes):
    # a prefix of zero with an empty mask leaves a row with nothing
    ctx = [nodes, nodes, nodes + 1, 140, 2, 300]
    c = Case(ctx, nodes, 8, 2, 128, dt, fp8, cuda_device, masks=masks, seed=5)
    c.check(c.run(B), f"{masks} {dt} fp8={fp8}")


def test_long_context_few_sequences(B, cuda_device):
    for nodes in (1, 12, 40):
        c = Case([20011, 9], nodes, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=nodes)
        c.check(c.run(B), f"20011 keys, {nodes} nodes")


def test_many_sequences(B, cuda_device):
    ctx = [(97 * i) % 400 for i in range(500)]
    c = Case(ctx, 4, 4, 2, 128, torch.bfloat16, False, cuda_device,
             lens=[i % 5 for i in range(500)], seed=8)
    c.check(c.run(B), "500 sequences")
    c = Case(ctx, 4, 4, 2, 64, torch.bfloat16, True, cuda_device, seed=9)
    c.check(c.run(B), "500 sequences, fp8")


def test_a_chain_is_multi_query_decode(B, cuda_device):
    c = Case([300, 40, 1500], 5, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=10)
    c.masks[:] = torch.tensor([1, 3, 7, 15, 31])
    a, _ = c.args()
    out, multi = c.run(B), torch.empty_like(c.q)
    c.check(out, "chain")
    B.pa_decode_multi(multi, *a[:5], c.scale)
    torch.cuda.synchronize()
    # both are within their roundings of the same values
    assert ((out.float() - multi.float()).abs() <= 2e-3 + 2e-2 * multi.float().abs()).all()


def test_block_order_does_not_matter(B, cuda_device):
    c = Case([513, 2000, 31], 9, 8, 2, 128, torch.bfloat16, False, cuda_device, seed=11)
    a = c.run(B)
    perm = torch.randperm(c.k.shape[0], generator=torch.Generator().manual_seed(1))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm))
    c.k, c.v = c.k[perm.to(c.dev)].contiguous(), c.v[perm.to(c.dev)].contiguous()
    c.tables = torch.where(c.tables >= 0, inv[c.tables.clamp_min(0).long()].to(torch.int32),
                           c.tables)
    assert torch.equal(a, c.run(B))


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_block_ids_are_flagged_and_read_as_zeros(B, cuda_device, fp8):
    c = Case([400, 400, 90], 7, 8, 2, 128, torch.bfloat16, fp8, cuda_device, seed=12)
    c.run(B)
    good = c.tables.clone()
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.tables = good.clone()
        c.tables[1, 3] = bad
        out = c.run(B, want_err=B.PA_DEVERR_BLOCK_ID)
        c.check(out, "neighbours of the bad one", seqs=[0, 2])
        # sequence 1: as if that block held zeros
        z = Case.__new__(Case)
        z.__dict__ = dict(c.__dict__)
        z.tables = good
        z.k, z.v = c.k.clone(), c.v.clone()
        z.k[good[1, 3]] = 0
        z.v[good[1, 3]] = 0
        z.check(out, "zeros", seqs=[1])


def test_lens_and_contexts_out_of_range_are_flagged(B, cuda_device):
    c = Case([60, 60, 60], 4, 8, 2, 128, torch.bfloat16, False, cuda_device, lens=[4, 4, 4],
             seed=13, extra_cols=0)
    c.lens = [4, 9, 4]
    out = c.run(B, want_err=B.PA_DEVERR_QUERY_LOC)
    c.lens = [4, 4, 4]
    c.check(out, "clamped")
    c.ctx = [60, 200, -3]  # beyond the table; negative
    out = c.run(B, want_err=B.PA_DEVERR_BLOCK_ID)
    c.ctx = [60, 64, 0]
    c.check(out, "the ordinary one", seqs=[0])
    assert (out[2] == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_scales(B, cuda_device, scale):
    c = Case([200, 33, 700], 6, 8, 2, 128, torch.bfloat16, False, cuda_device, seed=14)
    c.scale = scale
    c.check(c.run(B), f"scale {scale}")


def staircase(c, unit):
    """Keys and queries for which a row's maximum grows by 9 (in log2 units, more
    than the kernel's lazy limit of 8) again and again: `unit` tiles of 128 keys
    on one level, then `unit` tiles where one key lies 9 above it and the others at
    0.  The 128 weights of 2^-9 that such a jump leaves behind are a fifth of the
    sum, and V is positive on the levels and negative between them, so a wrong
    factor shows.  Levels are whole numbers N / 8, N the sum of a
    key's small whole components, exact in every type and in the fp32 sums (N <
    1,024; N / 8 log2 e within 2^-17, far below what plain64 counts for scores).
    Odd heads get -q, for which the keys fall."""
    d = c.q.shape[-1]
    for s, n in enumerate(c.ctx):
        p = torch.arange(n)
        u = p // (128 * unit)
        spike = (u % 2 == 1) & (p % (128 * unit) == 37 + s)
        N = torch.where(u % 2 == 0, 72 * (u // 2), torch.where(spike, 72 * (u // 2 + 1), 0))
        assert n == 0 or N.max() < 1024
        rows = (N[:, None] // d + (torch.arange(d) < N[:, None] % d)).to(c.dev)
        rows = rows.to(torch.float8_e4m3fn).view(torch.uint8) if c.fp8 else rows.to(c.k.dtype)
        at = c.tables[s, p // 16].long().to(c.dev), slice(None), (p % 16).to(c.dev)
        c.k[at] = rows[:, None]
        neg = (u % 2 == 1)[:, None, None].to(c.dev)
        v = c.v[at]
        c.v[at] = torch.where(neg, v | 0x80, v & 0x7f) if c.fp8 else \
            torch.where(neg, -v.abs(), v.abs())
    c.q[:] = 1.0
    c.q[:, :, 1::2] = -1.0
    c.k_scale = 0.5 if c.fp8 else 1.0
    c.scale = math.log(2.0) / 8 / c.k_scale


@pytest.mark.parametrize("dt,fp8", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,G,unit", [(7, 4, 1), (7, 4, 2), (16, 8, 2), (40, 4, 1), (33, 8, 1),
                                          (64, 8, 2)])
def test_growing_scores_rescale(B, cuda_device, dt, fp8, d, nodes, G, unit):
    # 24 sequences of 3 kv heads: units cut into segments of several tiles, whose
    # maxima differ by tens, contexts that end on different steps of the stairs
    # (most just behind a jump)
    ctx = [unit * 128 * (2 * k + 1) + r for k in (0, 1, 4, 7, 10, 12) for r in (70, 91, 127, -30)]
    c = Case(ctx, nodes, 3 * G, 3, d, dt, fp8, cuda_device, seed=50,
             lens=[max(1, nodes - 5 * (i % 3)) for i in range(24)])
    staircase(c, unit)
    c.check(c.run(B), f"staircase of {unit}, {dt} fp8={fp8} d={d} nodes={nodes} G={G}")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,G", [(6, 4), (16, 8), (40, 4), (64, 8)])
def test_rows_of_very_different_sizes_over_fp8(B, cuda_device, dt, d, nodes, G):
    # over an E4M3 cache a bf16 row is brought into f16's range by a power of two of its
    # own: neighbouring nodes, heads and sequences differ here, and a CTA works on
    # several sequences one after another
    ctx = [(97 * i) % 400 for i in range(300)]
    c = Case(ctx, nodes, 2 * G, 2, d, dt, True, cuda_device, seed=51,
             lens=[(i * 7) % (nodes + 1) for i in range(300)])
    at = [torch.arange(n, device=cuda_device) for n in c.q.shape[:3]]
    e = (7 * at[0][:, None, None] + 5 * at[1][:, None] + 3 * at[2]) % 13
    if dt == torch.bfloat16:
        e = torch.where(e == 11, 40, torch.where(e == 12, 100, e))
    c.q = (c.q.double() * torch.exp2(-e.double())[..., None]).to(dt)
    c.check(c.run(B), f"{dt} d={d} nodes={nodes} G={G}")


def test_captured_and_replayed_with_other_contexts(B, cuda_device):
    c = Case([900, 300, 77], 10, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=15,
             lens=[10, 7, 3])
    a, k = c.args()
    out = torch.zeros_like(c.q)
    ws = B.alloc_tree_workspace(c.q, c.k)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.pa_decode_tree(out, *a, **k, workspace=ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pa_decode_tree(out, *a, **k, workspace=ws)
    for ctx, lens in (([900, 300, 77], [10, 7, 3]), ([500, 299, 12], [1, 10, 0]),
                      ([10, 0, 77], [10, 4, 9])):
        # shorter contexts of the same tables (their cut tails are finite)
        a[4].copy_(torch.tensor(ctx, dtype=torch.int32))
        k["tree_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xff)
        c.ctx, c.lens = ctx, lens
        g.replay()
        torch.cuda.synchronize()
        c.check(out, f"replayed {ctx}")


def test_two_streams_at_once(B, cuda_device):
    cs = [Case([1900, 60 + i, 700], 20, 16, 2, 128, torch.bfloat16, False, cuda_device,
               seed=20 + i) for i in range(2)]
    outs = [torch.zeros_like(c.q) for c in cs]
    ws = [B.alloc_tree_workspace(c.q, c.k) for c in cs]
    args = [c.args() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (a, k), o, w, st in zip(args, outs, ws, streams):
            B.pa_decode_tree(o, *a, **k, workspace=w, stream=st)
    torch.cuda.synchronize()
    for i, (c, o) in enumerate(zip(cs, outs)):
        c.check(o, f"stream {i}")


def test_repeats_are_bit_equal(B, cuda_device):
    c = Case([3000, 1200, 60, 2500], 24, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=30)
    a = c.run(B)
    for _ in range(3):
        assert torch.equal(a, c.run(B))


@pytest.mark.parametrize("dt,fp8", TYPES)
@pytest.mark.parametrize("G", [5, 6])
@pytest.mark.parametrize("nodes", [25, 64])
def test_groups_that_leave_rows_of_a_tile_empty(B, cuda_device, dt, fp8, G, nodes):
    c = Case([nodes, 500, 131], nodes, G, 1, 128, dt, fp8, cuda_device,
             lens=[nodes, nodes - 3, 1], seed=G)
    c.check(c.run(B), f"G={G} nodes={nodes} {dt} fp8={fp8}")


@pytest.mark.parametrize("nodes", [6, 40])
def test_a_bad_key_reaches_only_the_rows_that_see_it(B, cuda_device, nodes):
    c = Case([400, 350], nodes, 8, 2, 128, torch.bfloat16, False, cuda_device, seed=16)
    bad = nodes // 2  # a node of sequence 0
    at = 400 - nodes + bad
    good = c.k.clone()
    c.k[c.tables[0, at // 16].item(), :, at % 16] = float("nan")
    out = c.run(B)
    c.k = good
    sees = (c.masks[0] >> bad & 1).bool().to(c.dev)
    assert sees.any() and torch.isnan(out[0][sees]).all()
    out[0][sees] = 0
    full = c.run(B)
    full[0][sees] = 0
    c.check(out, "the other sequence", seqs=[1])
    assert torch.equal(out[0], full[0])


@pytest.mark.parametrize("nodes", [3, 17, 64])
def test_the_workspace_size_holds(B, cuda_device, nodes):
    c = Case([3000, 1500, 40, 2200], nodes, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=17)
    n = B.pa_decode_tree_workspace_size(4, nodes, 16, 2, 128)
    room = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device=cuda_device)
    out = c.run(B, workspace=room[4096:4096 + n])
    assert (room[:4096] == 0x5a).all() and (room[-4096:] == 0x5a).all()
    c.check(out, f"{nodes} nodes")
    with pytest.raises(B.PAError):
        c.run(B, workspace=room[4096:4096 + n - 16])


def test_captured_graphs_with_a_workspace_each(B, cuda_device):
    cs = [Case([2500, 700], 12, 16, 2, 128, torch.bfloat16, False, cuda_device, seed=40 + i)
          for i in range(2)]
    outs = [torch.zeros_like(c.q) for c in cs]
    ws = [B.alloc_tree_workspace(c.q, c.k) for c in cs]
    args = [c.args() for c in cs]
    graphs = []
    for (a, k), o, w in zip(args, outs, ws):
        B.pa_decode_tree(o, *a, **k, workspace=w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.pa_decode_tree(o, *a, **k, workspace=w)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i, (c, o) in enumerate(zip(cs, outs)):
        c.check(o, f"graph {i}")


@pytest.mark.parametrize("as_int", [False, True])
def test_own_workspace_belongs_to_the_calls_stream(B, cuda_device, as_int, monkeypatch):
    c = Case([1500, 3, 900], 16, 8, 2, 128, torch.bfloat16, False, cuda_device, seed=23)
    a, k = c.args()
    out = torch.full_like(c.q, 7.0)
    made = []
    alloc = B.alloc_tree_workspace

    def recorded(*x):
        w = alloc(*x)
        made.append((w.data_ptr(), w.numel()))
        return w

    monkeypatch.setattr(B, "alloc_tree_workspace", recorded)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    B.pa_decode_tree(out, *a, **k, stream=side.cuda_stream if as_int else side)
    # what the current stream allocates next is not the memory in use there
    other = torch.empty(made[0][1], dtype=torch.uint8, device=cuda_device)
    assert other.data_ptr() != made[0][0]
    other.fill_(0x7f)
    torch.cuda.synchronize()
    c.check(out, "own workspace")
