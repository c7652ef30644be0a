"""pa_prefill_packed (attention over whole prompts) against the 64-bit form."""
import math

import pytest
import torch

from tests import plain64

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 15, 16, 17, 0, 31, 33, 127, 128, 129, 255, 256, 257, 300]


@pytest.fixture(scope="module")
def B(cuda_device):
    from pagedattention_paged_kv_pa_b200 import binding
    return binding


def make(lens, n_q, n_kv, d, dt, dev, fused=True, pad=0, seed=0, fill=float("nan")):
    g = torch.Generator(device=dev).manual_seed(seed)
    total = sum(lens) + pad
    if fused:
        qkv = torch.randn(total, n_q + 2 * n_kv, d, device=dev, generator=g, dtype=dt)
        q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    else:
        q, k, v = (torch.randn(total, n, d, device=dev, generator=g, dtype=dt)
                   for n in (n_q, n_kv, n_kv))
    q.mul_(2)
    if pad:
        for x in (q, k, v):
            x[sum(lens):] = fill
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    return q, k, v, start


def check(out, q, k, v, lens, scale, what, at=0):
    for s, n in enumerate(lens):
        if n:
            r = slice(at, at + n)
            ref, mag = plain64.attend(q[r], k[r], v[r], plain64.causal(n, q.device), scale)
            plain64.check(out[r], ref, mag, n, v[r].abs().max().item(), q.dtype,
                          f"{what}, sequence {s} of {n}")
        at += n


def run(B, q, k, v, start, scale, **kw):
    out = torch.full(q.shape, 7.0, device=q.device, dtype=q.dtype)
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    B.pa_prefill_packed(out, q, k, v, start, scale, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", [(2, 2), (4, 2), (6, 2), (8, 2), (5, 1), (7, 1), (16, 2),
                                      (12, 1), (16, 1)])
def test_ragged_batch(B, cuda_device, dt, d, n_q, n_kv):
    q, k, v, start = make(EDGES, n_q, n_kv, d, dt, cuda_device, seed=d + n_q)
    out, err = run(B, q, k, v, start, d ** -0.5)
    assert err == 0
    check(out, q, k, v, EDGES, d ** -0.5, f"{dt} d={d} {n_q}/{n_kv}")


@pytest.mark.parametrize("n", [1, 5, 16, 64, 128, 129, 511, 512, 513, 1000, 2305])
@pytest.mark.parametrize("n_q,n_kv", [(8, 1), (3, 3)])
def test_one_sequence(B, cuda_device, n, n_q, n_kv):
    q, k, v, start = make([n], n_q, n_kv, 128, torch.bfloat16, cuda_device, seed=n)
    out, err = run(B, q, k, v, start, 128 ** -0.5)
    assert err == 0
    check(out, q, k, v, [n], 128 ** -0.5, f"{n} tokens")


def test_long_prompt(B, cuda_device):
    q, k, v, start = make([9001], 4, 1, 128, torch.bfloat16, cuda_device, seed=3)
    out, err = run(B, q, k, v, start, 128 ** -0.5)
    assert err == 0
    check(out, q, k, v, [9001], 128 ** -0.5, "9001 tokens")


def test_many_sequences(B, cuda_device):
    lens = [(37 * i) % 61 for i in range(700)] + [900]
    q, k, v, start = make(lens, 4, 2, 64, torch.bfloat16, cuda_device, seed=4)
    out, err = run(B, q, k, v, start, 0.125)
    assert err == 0
    check(out, q, k, v, lens, 0.125, "701 sequences")


def test_separate_tensors_match_the_fused_ones(B, cuda_device):
    lens = [40, 200, 3]
    q, k, v, start = make(lens, 8, 2, 128, torch.float16, cuda_device, seed=5)
    a, _ = run(B, q, k, v, start, 0.09)
    b, _ = run(B, q.contiguous(), k.contiguous(), v.contiguous(), start, 0.09)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_padding_rows_are_neither_read_nor_written(B, cuda_device, fill):
    lens = [70, 0, 129, 5]
    q, k, v, start = make(lens, 4, 2, 128, torch.bfloat16, cuda_device, pad=50, seed=6, fill=fill)
    out, err = run(B, q, k, v, start, 0.09)
    assert err == 0
    assert (out[sum(lens):] == 7).all()
    check(out, q, k, v, lens, 0.09, "padded")


def test_rows_before_the_first_sequence_and_neighbours(B, cuda_device):
    # the batch starts at row 9; a neighbour's values that are not finite stay
    # its own
    lens = [60, 77, 200]
    q, k, v, start = make([9] + lens, 4, 2, 64, torch.bfloat16, cuda_device, seed=7)
    for x in (q, k, v):
        x[:9] = float("nan")
        x[9 + 60:9 + 60 + 77] = float("inf")
    out, err = run(B, q, k, v, start[1:].contiguous(), 0.125)
    assert err == 0
    assert (out[:9] == 7).all()
    check(out, q, k, v, [60], 0.125, "before", at=9)
    check(out, q, k, v, [200], 0.125, "behind", at=9 + 137)


@pytest.mark.parametrize("scale", [0.0, -0.09, 1.0])
def test_scales(B, cuda_device, scale):
    lens = [140, 33]
    q, k, v, start = make(lens, 4, 2, 128, torch.bfloat16, cuda_device, seed=8)
    q, k = q / 8, k / 2  # keeps the scores' sums as the tolerance counts them
    out, err = run(B, q, k, v, start, scale)
    assert err == 0
    check(out, q, k, v, lens, scale, f"scale {scale}")


def test_growing_scores_rescale(B, cuda_device):
    # keys whose scores climb by tens from tile to tile: every tile moves the
    # running maximum; the weights of all but the last keys vanish
    n, d = 700, 128
    q, k, v, start = make([n], 2, 1, d, torch.bfloat16, cuda_device, seed=9)
    q[:] = 1.0
    k[:] = (torch.arange(n, device=cuda_device) / 8).floor()[:, None, None] / 16
    out, err = run(B, q, k, v, start, 0.5)
    assert err == 0
    check(out, q, k, v, [n], 0.5, "climbing")
    k[:] = -k
    out, err = run(B, q, k, v, start, 0.5)
    check(out, q, k, v, [n], 0.5, "falling")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", [(2, 1), (3, 3)])
def test_small_steps_rescale(B, cuda_device, dt, d, n_q, n_kv):
    # tiles of 128 keys on one level, then one where a single key lies 9 higher (in
    # log2 units, the lazy limit is 8) and the others at 0: the 128 weights of 2^-9
    # it leaves behind are a fifth of a row's sum, with V of the other sign.  Levels
    # are whole numbers N / 8, N < 1,024 the sum of a key's small whole
    # components, exact in the fp32 sums; odd heads get -q, for which they fall
    lens = [3400, 129, 700, 1500]
    q, k, v, start = make(lens, n_q, n_kv, d, dt, cuda_device, seed=16)
    q[:] = 1.0
    q[:, 1::2] = -1.0
    at = 0
    for n in lens:
        p = torch.arange(n, device=cuda_device)
        u = p // 128
        top = torch.where(p % 128 == 37, 72 * (u // 2 + 1), 0)
        N = torch.where(u % 2 == 0, 72 * (u // 2), top)
        assert N.max() < 1024
        k[at:at + n] = (N[:, None] // d + (torch.arange(d, device=cuda_device)
                                           < N[:, None] % d)).to(dt)[:, None]
        v[at:at + n] = v[at:at + n].abs() * torch.where(u % 2 == 0, 1, -1).to(dt)[:, None, None]
        at += n
    scale = math.log(2.0) / 8
    out, err = run(B, q, k, v, start, scale)
    assert err == 0
    check(out, q, k, v, lens, scale, f"steps of 9, {dt} d={d} {n_q}/{n_kv}")


def test_inconsistent_starts_are_flagged_and_stay_in_bounds(B, cuda_device):
    q, k, v, _ = make([100], 4, 2, 64, torch.bfloat16, cuda_device, seed=10)
    bad = torch.tensor([0, 40, 30, 150], dtype=torch.int32, device=cuda_device)
    out, err = run(B, q, k, v, bad, 0.125)
    assert err == B.PA_DEVERR_QUERY_LOC
    check(out, q, k, v, [30], 0.125, "first of the bad ones")  # rows 30..39 are claimed twice
    bad = torch.tensor([-5, 40], dtype=torch.int32, device=cuda_device)
    out, err = run(B, q, k, v, bad, 0.125)
    assert err == B.PA_DEVERR_QUERY_LOC
    assert (out[40:] == 7).all()


@pytest.mark.parametrize("starts", [
    [-5, 40], [0, 40, 30, 150], [-300, -200, 7], [500, 3], [0, 100] * 40 + [0, 100],
    [20, 10, 60, 50, 200, -1, 80], [0, 10, 5] + [11 + i for i in range(90)],
    [3] * 30 + [2, 50, 49, 48, 47, 77, 500], [i + (37 * i) % 29 - 12 for i in range(96)], [2 ** 31 - 1, -2 ** 31, 60, 40]],
    ids=lambda x: f"{len(x) - 1}_{x[0]}_{x[1]}")
def test_starts_out_of_order_count_as_the_largest_so_far(B, cuda_device, starts):
    # every row has one owner and the sequences are those of the running maximum
    total = 100
    q, k, v, _ = make([total], 16, 1, 64, torch.bfloat16, cuda_device, seed=15)
    at = torch.tensor(starts).clamp(0, total).cummax(0).values
    assert at.tolist() != starts
    out, err = run(B, q, k, v, torch.tensor(starts, dtype=torch.int32, device=cuda_device), 0.125)
    assert err == B.PA_DEVERR_QUERY_LOC
    assert (out[:at[0]] == 7).all() and (out[at[-1]:] == 7).all()
    check(out, q, k, v, at.diff().tolist(), 0.125, f"{starts[:8]}", at=int(at[0]))
    same, err = run(B, q, k, v, at.to(torch.int32).to(cuda_device), 0.125)
    assert err == 0 and torch.equal(out, same)


def test_captured_and_replayed_with_other_lengths(B, cuda_device):
    lens = [50, 300, 17]
    q, k, v, start = make(lens, 8, 2, 128, torch.bfloat16, cuda_device, seed=11)
    out = torch.zeros_like(q.contiguous())
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.pa_prefill_packed(out, q, k, v, start, 0.09)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pa_prefill_packed(out, q, k, v, start, 0.09)
    for new in ([50, 300, 17], [200, 7, 160], [0, 0, 367]):
        start.copy_(torch.tensor([0] + new).cumsum(0).to(torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(out, q, k, v, new, 0.09, f"replayed {new}")


def test_two_streams_at_once(B, cuda_device):
    sets = [make([257 + 50 * i, 90], 8, 2, 128, torch.bfloat16, cuda_device, seed=20 + i)
            for i in range(2)]
    outs = [torch.zeros_like(x[0].contiguous()) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, st in zip(sets, outs, streams):
            B.pa_prefill_packed(o, *x, 0.09, stream=st)
    torch.cuda.synchronize()
    for i, (x, o) in enumerate(zip(sets, outs)):
        check(o, *x[:3], [257 + 50 * i, 90], 0.09, f"stream {i}")


def test_repeats_are_bit_equal(B, cuda_device):
    q, k, v, start = make([700, 33, 400], 8, 2, 128, torch.bfloat16, cuda_device, seed=30)
    a, _ = run(B, q, k, v, start, 0.09)
    for _ in range(3):
        b, _ = run(B, q, k, v, start, 0.09)
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_a_bad_key_reaches_only_the_rows_that_see_it(B, cuda_device, d):
    n, at = 300, 140
    q, k, v, start = make([n], 4, 2, d, torch.bfloat16, cuda_device, seed=12)
    k[at] = float("nan")
    out, err = run(B, q, k, v, start, 0.09)
    assert err == 0
    assert torch.isnan(out[at:]).all()
    ref, mag = plain64.attend(q[:at], k[:at], v[:at], plain64.causal(at, q.device), 0.09)
    plain64.check(out[:at], ref, mag, at, v[:at].abs().max().item(), q.dtype, "before the bad key")


def test_strides_of_different_tensors(B, cuda_device):
    # q, k and v with their own strides, wider than a token
    g = torch.Generator(device=cuda_device).manual_seed(13)
    n, n_q, n_kv, d = 210, 6, 2, 64
    base = [torch.randn(n, w, d, device=cuda_device, generator=g, dtype=torch.float16)
            for w in (n_q + 5, n_kv + 1, n_kv + 9)]
    q, k, v = base[0][:, 2:2 + n_q], base[1][:, 1:], base[2][:, 3:3 + n_kv]
    start = torch.tensor([0, 150, 210], dtype=torch.int32, device=cuda_device)
    out, err = run(B, q, k, v, start, 0.125)
    assert err == 0
    check(out, q, k, v, [150, 60], 0.125, "strided")


def test_nothing_is_written_around_the_output(B, cuda_device):
    lens, n_q, d = [129, 31], 5, 128
    q, k, v, start = make(lens, n_q, 1, d, torch.bfloat16, cuda_device, seed=14)
    room = torch.full((160 * n_q * d + 4096,), 3.0, device=cuda_device, dtype=torch.bfloat16)
    out = room[2048:-2048].view(160, n_q, d)
    B.pa_prefill_packed(out, q, k, v, start, 0.09)
    torch.cuda.synchronize()
    assert (room[:2048] == 3).all() and (room[-2048:] == 3).all()
    check(out, q, k, v, lens, 0.09, "inside a larger buffer")
