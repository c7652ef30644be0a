"""Refusals of pa_prefill_packed, pa_decode_tree and pa_compact_tokens before
any launch, the tree masks, and pa_alloc_truncate (no GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from pagedattention_paged_kv_pa_b200 import build
    build.build()
    from pagedattention_paged_kv_pa_b200 import binding
    return binding


V = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


def _packed(B, **kw):
    a = dict(out=16, q=16, k=16, v=16, qsl=16, scale=0.1, nq=8, nkv=2, d=128, ns=3, total=50,
             qs=1024, ks=256, vs=256, dt=B.PA_BF16)
    a.update(kw)
    return B.lib.pa_prefill_packed(V(a["out"]), V(a["q"]), V(a["k"]), V(a["v"]), V(a["qsl"]),
                                   a["scale"], a["nq"], a["nkv"], a["d"], a["ns"], a["total"],
                                   a["qs"], a["ks"], a["vs"], a["dt"], None, None)


def test_packed_prefill_refusals(B):
    assert _packed(B, d=96) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, dt=B.PA_F32) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, dt=B.PA_FP8_E4M3) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, dt=9) == B.PA_ERR_INVALID_ARG
    assert _packed(B, nq=7) == B.PA_ERR_INVALID_ARG
    assert _packed(B, nkv=0) == B.PA_ERR_INVALID_ARG
    assert _packed(B, total=-1) == B.PA_ERR_INVALID_ARG
    assert _packed(B, ns=-1) == B.PA_ERR_INVALID_ARG
    assert _packed(B, scale=float("nan")) == B.PA_ERR_INVALID_ARG
    for x in ("out", "q", "k", "v", "qsl"):
        assert _packed(B, **{x: None}) == B.PA_ERR_INVALID_ARG
    for x in ("out", "q", "k", "v"):
        assert _packed(B, **{x: 24}) == B.PA_ERR_INVALID_ARG   # misaligned
    assert _packed(B, qs=1023) == B.PA_ERR_INVALID_ARG         # overlapping tokens
    assert _packed(B, ks=248) == B.PA_ERR_INVALID_ARG
    assert _packed(B, vs=260) == B.PA_ERR_INVALID_ARG          # not a multiple of 8
    assert _packed(B, ks=1 << 38) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, ns=65536) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, nq=65536, nkv=1, d=64, qs=1 << 22) == B.PA_ERR_UNSUPPORTED
    assert _packed(B, nq=4096, qs=1 << 19, total=1 << 24) == B.PA_ERR_UNSUPPORTED  # too many items
    assert _packed(B, ns=0, q=None) == B.PA_OK
    assert _packed(B, total=0, q=None) == B.PA_OK


def _tree(B, **kw):
    a = dict(out=16, q=16, k=16, v=16, bt=16, cl=16, m=16, tl=None, scale=0.1, bs=16, nq=8,
             nkv=2, d=128, ns=4, ql=10, mb=40, nb=100, qdt=B.PA_BF16, kvdt=B.PA_BF16, ks=1.0,
             vs=1.0, ws=16, wsb=1 << 40)
    a.update(kw)
    return B.lib.pa_decode_tree(V(a["out"]), V(a["q"]), V(a["k"]), V(a["v"]), V(a["bt"]),
                                V(a["cl"]), V(a["m"]), V(a["tl"]), a["scale"], a["bs"], a["nq"],
                                a["nkv"], a["d"], a["ns"], a["ql"], a["mb"], a["nb"], a["qdt"],
                                a["kvdt"], a["ks"], a["vs"], V(a["ws"]), a["wsb"], None, None)


def test_tree_refusals(B):
    assert _tree(B, ql=0) == B.PA_ERR_INVALID_ARG
    assert _tree(B, ql=65) == B.PA_ERR_INVALID_ARG
    assert _tree(B, d=96) == B.PA_ERR_UNSUPPORTED
    assert _tree(B, bs=32) == B.PA_ERR_UNSUPPORTED
    assert _tree(B, nq=18, nkv=2) == B.PA_ERR_UNSUPPORTED      # group 9
    assert _tree(B, nq=7) == B.PA_ERR_INVALID_ARG
    assert _tree(B, qdt=B.PA_F32, kvdt=B.PA_F32) == B.PA_ERR_UNSUPPORTED
    assert _tree(B, qdt=B.PA_F16, kvdt=B.PA_BF16) == B.PA_ERR_UNSUPPORTED
    assert _tree(B, kvdt=B.PA_FP8_E4M3, vs=0.0) == B.PA_ERR_INVALID_ARG
    assert _tree(B, scale=float("nan")) == B.PA_ERR_INVALID_ARG
    for x in ("out", "q", "k", "v", "bt", "cl", "m"):
        assert _tree(B, **{x: None}) == B.PA_ERR_INVALID_ARG
    for x in ("out", "q", "k", "v"):
        assert _tree(B, **{x: 24}) == B.PA_ERR_INVALID_ARG
    assert _tree(B, m=20) == B.PA_ERR_INVALID_ARG              # masks not 8-byte aligned
    assert _tree(B, nb=1 << 27) == B.PA_ERR_UNSUPPORTED        # pool rows >= 2^31
    assert _tree(B, ns=0, q=None) == B.PA_OK
    need = B.pa_decode_tree_workspace_size(4, 10, 8, 2, 128)
    if need:
        assert _tree(B, wsb=need - 1) == B.PA_ERR_INVALID_ARG
        assert _tree(B, ws=None) == B.PA_ERR_INVALID_ARG
        assert _tree(B, ws=24) == B.PA_ERR_INVALID_ARG


def _compact(B, **kw):
    a = dict(k=[16, 32], v=[48, 64], bt=16, cl=16, tl=16, acc=16, al=16, ns=4, ql=10, ma=5, mb=8,
             nkv=2, d=128, bs=16, nb=100, dt=B.PA_BF16)
    a.update(kw)
    arr = lambda x: (ctypes.c_void_p * len(x))(*x) if x is not None else None  # noqa: E731
    return B.lib.pa_compact_tokens(arr(a["k"]), arr(a["v"]), len(a["k"] or a["v"]), V(a["bt"]),
                                   V(a["cl"]), V(a["tl"]), V(a["acc"]), V(a["al"]), a["ns"],
                                   a["ql"], a["ma"], a["mb"], a["nkv"], a["d"], a["bs"], a["nb"],
                                   a["dt"], None, None)


def test_compact_refusals(B):
    assert _compact(B, bs=8) == B.PA_ERR_UNSUPPORTED
    assert _compact(B, d=4) == B.PA_ERR_UNSUPPORTED            # 8-byte rows
    assert _compact(B, ql=65) == B.PA_ERR_INVALID_ARG
    assert _compact(B, ma=-1) == B.PA_ERR_INVALID_ARG
    assert _compact(B, mb=0) == B.PA_ERR_INVALID_ARG
    assert _compact(B, dt=7) == B.PA_ERR_INVALID_ARG
    assert _compact(B, k=[16, 0]) == B.PA_ERR_INVALID_ARG
    assert _compact(B, v=[16, 40]) == B.PA_ERR_INVALID_ARG     # misaligned
    assert _compact(B, k=None) == B.PA_ERR_INVALID_ARG
    for x in ("bt", "cl", "acc", "al"):
        assert _compact(B, **{x: None}) == B.PA_ERR_INVALID_ARG
    assert _compact(B, ns=0, bt=None) == B.PA_OK
    assert _compact(B, ma=0, bt=None) == B.PA_OK
    assert _compact(B, k=[], v=[]) == B.PA_OK


def test_binding_refusals_on_host_tensors(B):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(B.PAError):  # not on a GPU
        B.pa_prefill_packed(z(4, 8, 64), z(4, 8, 64), z(4, 2, 64), z(4, 2, 64), i(2), 0.1)
    with pytest.raises(B.PAError):
        B.pa_decode_tree(z(1, 4, 8, 64), z(1, 4, 8, 64), z(3, 2, 16, 64), z(3, 2, 16, 64),
                         i(1, 2), i(1), torch.zeros(1, 4, dtype=torch.int64), 0.1)
    with pytest.raises(B.PAError):
        B.pa_compact_tokens([z(3, 2, 16, 64)], [z(3, 2, 16, 64)], i(1, 2), i(1), i(1), i(1, 2),
                            i(1))
    with pytest.raises(B.PAError):  # the layers differ
        B.pa_compact_tokens([z(3, 2, 16, 64), z(4, 2, 16, 64)], [z(3, 2, 16, 64)] * 2, i(1, 2),
                            i(1), i(1), i(1, 2), i(1))


def test_tree_masks(B):
    #        0 -> 1 -> 3, 0 -> 2, 4 beside 0, 5 below 2
    par = torch.tensor([[-1, 0, 0, 1, -1, 2], [-1, -1, 1, 9, 9, 9]], dtype=torch.int32)
    m = B.tree_masks(par, torch.tensor([6, 3]))
    assert m.tolist() == [[1, 3, 5, 11, 16, 37], [1, 2, 6, 0, 0, 0]]
    chain = torch.arange(-1, 63, dtype=torch.int32)[None]
    m = B.tree_masks(chain)
    assert [x & (2 ** 64 - 1) for x in m[0].tolist()] == [2 ** (i + 1) - 1 for i in range(64)]
    for bad in ([[0]], [[-1, 1]], [[-2]], [[-1, 5]]):
        with pytest.raises(B.PAError):
            B.tree_masks(torch.tensor(bad, dtype=torch.int32))
    with pytest.raises(B.PAError):
        B.tree_masks(torch.zeros(1, 65, dtype=torch.int32) - 1)
    with pytest.raises(B.PAError):
        B.tree_masks(par, torch.tensor([6, 7]))
    assert B.tree_masks(torch.zeros(0, 4, dtype=torch.int32)).shape == (0, 4)


def test_truncate_releases_blocks_last_first(B):
    a = B.BlockAllocator(10)
    a.append(1, 70)                      # blocks 0..4
    assert a.truncate(1, 33) == B.PA_OK  # keeps 3
    assert a.block_table(1) == [0, 1, 2]
    assert a.num_tokens(1) == 33
    assert a.free_list() == [5, 6, 7, 8, 9, 4, 3]
    st, slots = a.append(1, 2)           # goes on in the kept block
    assert st == B.PA_OK and slots == [33 + 0, 34]
    assert a.truncate(1, 0) == B.PA_OK and a.block_table(1) == []
    assert a.num_seqs() == 1
    st, slots = a.append(1, 1)
    assert st == B.PA_OK and a.num_tokens(1) == 1


def test_truncate_refusals(B):
    a = B.BlockAllocator(10)
    a.append_tokens(1, list(range(20)))
    for bad in ((2, 3), (1, 21), (1, -1)):
        assert a.truncate(*bad) == B.PA_ERR_INVALID_ARG
    assert a.truncate(1, 2, [1, 2, 3]) == B.PA_ERR_INVALID_ARG   # more ids than tokens
    assert a.truncate(1, 10, [8, 8]) == B.PA_ERR_INVALID_ARG     # differs from a known id
    assert a.num_tokens(1) == 20
    assert a.truncate(1, 10, [8, 9]) == B.PA_OK


def test_truncate_of_a_shared_sequence_keeps_the_others(B):
    a = B.BlockAllocator(10)
    a.append(1, 40)
    a.fork(1, 2)
    assert a.truncate(2, 20) == B.PA_OK
    assert a.block_table(1) == [0, 1, 2] and a.block_table(2) == [0, 1]
    assert [a.refcount(b) for b in range(3)] == [2, 2, 1]
    st, _ = a.append(2, 1)               # its cut block is shared: copy first
    assert st == B.PA_ERR_INVALID_ARG
    st, pairs = a.prepare_write(2)
    assert st == B.PA_OK and pairs == [(1, 3)]


def test_truncate_and_prefix_caching(B):
    a = B.BlockAllocator(12)
    a.set_prefix_caching(True)
    ids = list(range(48))
    a.admit(1, ids)                                   # blocks 0, 1, 2 registered
    assert a.truncate(1, 24) == B.PA_OK               # block 2 cached, block 1 cut
    assert a.cached_list() == [2]
    # the cut block still holds its 16 tokens: another request finds all three
    st, _, n = a.admit(2, ids + [1])
    assert st == B.PA_OK and n == 48 and a.block_table(2)[:3] == [0, 1, 2]
    a.free_seq(2)
    # written again, it is not found any more
    st, _ = a.append_tokens(1, [99])
    assert st == B.PA_OK
    st, _, n = a.admit(3, ids)
    assert st == B.PA_OK and n == 16
    a.free_seq(3)
    # filled with other tokens, it is found under those
    a.append_tokens(1, list(range(200, 207)))
    st, _, n = a.admit(4, ids[:24] + [99] + list(range(200, 207)) + [5])
    assert st == B.PA_OK and n == 32


def test_accepted_ids_bring_prefix_caching_back(B):
    a = B.BlockAllocator(12)
    a.set_prefix_caching(True)
    a.admit(1, list(range(30)))
    a.append(1, 12)                                   # drafts, ids unknown
    assert a.truncate(1, 34, [50, 51, 52, 53]) == B.PA_OK
    full = list(range(30)) + [50, 51]
    st, _, n = a.admit(2, full + [7])
    assert st == B.PA_OK and n == 32
    # a gap in the ids: not known, nothing registered
    a.append(1, 20)
    assert a.truncate(1, 50, list(range(10))) == B.PA_OK
    st, _, n = a.admit(3, full + [52, 53] + list(range(14)) + [1])
    assert st == B.PA_OK and n == 32
    # cut back to the known ones, it registers again from there on
    assert a.truncate(1, 34) == B.PA_OK
    st, _ = a.append_tokens(1, list(range(60, 74)))
    assert st == B.PA_OK
    st, _, n = a.admit(4, full + [52, 53] + list(range(60, 74)) + [1])
    assert st == B.PA_OK and n == 48


def test_overlapping_memory_is_refused(B):
    # out [50][8 x 128] of 102,400 bytes against q, k, v far away
    far = dict(out=1 << 30, q=1 << 31, k=1 << 32, v=1 << 33)
    for x, n in (("q", 50 * 1024 * 2), ("k", 50 * 256 * 2), ("v", 50 * 256 * 2)):
        for at in (1 << 30, (1 << 30) + 102400 - 16, (1 << 30) - n + 16):
            assert _packed(B, **{**far, x: at}) == B.PA_ERR_INVALID_ARG
    # a row of a strided k inside out; its first row ends before out
    assert _packed(B, **{**far, "k": (1 << 30) - 512, "ks": 256 + 8}) == B.PA_ERR_INVALID_ARG
    at = 1 << 30
    for q in (at, at + 4 * 10 * 1024 * 2 - 16, at - 4 * 10 * 1024 * 2 + 16):
        assert _tree(B, out=at, q=q) == B.PA_ERR_INVALID_ARG
    pool = 100 * 2 * 16 * 128 * 2
    apart = [pool * i + 16 for i in range(1, 5)]
    for i in range(4):
        for j in range(4):
            if i != j:
                x = list(apart)
                x[i] = x[j]
                assert _compact(B, k=x[:2], v=x[2:]) == B.PA_ERR_INVALID_ARG
    assert _compact(B, k=apart[:2], v=[apart[2], apart[2] + pool - 16]) == B.PA_ERR_INVALID_ARG
    many = [pool * i + 16 for i in range(1, 201)]
    assert _compact(B, k=many[:100], v=many[100:199] + many[:1]) == B.PA_ERR_INVALID_ARG


def test_timeout_hook_refusals(B):
    for skip, limit in ((-1, 2000), (0, 0), (0, 1_000_001)):
        assert B.lib.pa_test_prefill_packed_timeout(
            *[V(16)] * 5, 0.1, 8, 2, 128, 3, 50, 1024, 256, 256, B.PA_BF16, None, None, skip,
            limit) == B.PA_ERR_INVALID_ARG
        assert B.lib.pa_test_decode_tree_timeout(
            *[V(16)] * 7, None, 0.1, 16, 8, 2, 128, 4, 10, 40, 100, B.PA_BF16, B.PA_BF16, 1.0, 1.0,
            V(16), 1 << 40, None, None, skip, limit) == B.PA_ERR_INVALID_ARG
