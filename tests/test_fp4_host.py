"""Without a GPU: the 4-bit format's definition against brute force, the
refusals of its calls and of the compaction, and the allocator's part."""
import ctypes as C

import numpy as np
import pytest

import oracle
from oracle import fp4
from paged_kv_cache_142_gb300 import _lib as L

BAD, UNSUP, WS = L.PA_ERR_INVALID_ARG, L.PA_ERR_UNSUPPORTED, L.PA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def test_levels_and_ties():
    assert fp4.E4M3[126] == 448 and fp4.E4M3[1] == 2.0 ** -9 and fp4.E4M3[8] == 2.0 ** -6
    assert len(fp4.E4M3) == 127 and (np.diff(fp4.E4M3) > 0).all()
    assert fp4.nearest(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 9]), fp4.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    x = np.random.default_rng(0).uniform(0, 7, 4000)
    d = np.abs(x[:, None] - fp4.E2M1)
    assert (d[np.arange(len(x)), fp4.nearest(x, fp4.E2M1)] == d.min(axis=1)).all()


def test_round_trip_of_values_that_the_format_holds():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, size=(50, 64))
    codes[:, ::16] = 7                                  # a 6 in every group fixes its scale
    codes = np.where(codes == 8, 0, codes).astype(np.uint8)
    scales = rng.integers(1, 127, size=(50, 4)).astype(np.uint8)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    v = fp4.dequantise(packed, scales, 0.25)
    again = fp4.quantise(v, 0.25)
    assert np.array_equal(again[0], packed) and np.array_equal(again[1], scales)
    assert np.array_equal(v.astype(np.float32), v)      # 6 significant bits
    bits = v.astype(np.float32).view(np.uint32)
    assert not (bits & 0xffff).any()                    # exact in bf16


def test_quantisation_error_is_half_a_step():
    x = np.random.default_rng(2).standard_normal((200, 128))
    v = fp4.dequantise(*fp4.quantise(x, 1 / 64), 1 / 64)
    top = np.abs(x.reshape(200, 8, 16)).max(axis=-1, keepdims=True)
    # the widest step is 2 of 6, the scale at most 1/16 off (3 bits), and what passes 6 is cut there
    assert (np.abs(v - x).reshape(200, 8, 16) <= top * (1 / 6) * (1 + 1 / 16) + 1e-12).all()


def test_tile_bytes(lib):
    for bs in (1, 2, 4, 8, 16, 32, 64, 128, 256):
        for d in (64, 128, 256):
            assert lib.pa_fp4_tile_bytes(bs, d) == fp4.tile_bytes(bs, d)
    assert lib.pa_fp4_tile_bytes(12, 128) == 0 and lib.pa_fp4_tile_bytes(16, 96) == 0
    assert lib.pa_fp4_tile_bytes(512, 128) == 0 and lib.pa_fp4_tile_bytes(0, 128) == 0


P = 4096  # an aligned address that no refused call reads


def test_append_and_gather_refusals(lib):
    for fn in (lib.pa_reshape_and_cache_fp4, lib.pa_gather_cache_fp4):
        def call(key=P, dt=1, t=3, slots=P, kc=P, nb=8, bs=16, h=2, d=128, ks=1.0, vs=1.0, status=None):
            return fn(key, P, dt, t, slots, kc, P, nb, bs, h, d, ks, vs, status, None)
        assert call(bs=12) == UNSUP and call(bs=512) == UNSUP and call(d=96) == UNSUP
        assert call(nb=0) == BAD and call(h=0) == BAD and call(t=-1) == BAD and call(bs=-4) == BAD
        assert call(dt=2) == BAD and call(dt=9) == BAD
        for s in (0.0, -1.0, 3.0, 0.1, float("inf"), float("nan"), 2.0 ** 33, 2.0 ** -33):
            assert call(ks=s) == BAD and call(vs=s) == BAD
        assert call(key=None) == BAD and call(slots=None) == BAD and call(kc=None) == BAD
        assert call(key=P + 16) == BAD and call(kc=P + 4) == BAD and call(slots=P + 4) == BAD and call(status=P + 2) == BAD
        assert call(t=0, key=None, slots=None, kc=None) == L.PA_OK


def test_decode_refusals(lib):
    def call(out=P, odt=0, q=P, n=2, h=8, kc=P, nb=8, bs=16, hkv=2, d=128, tab=P, m=4, lens=P, ml=64, scale=1.0,
             ks=1.0, vs=1.0, ws=P, wb=1 << 40):
        return lib.pa_decode_fp4(out, odt, q, n, h, kc, P, nb, bs, hkv, d, tab, m, lens, ml, scale, ks, vs, ws, wb, None)
    assert call(bs=24) == UNSUP and call(d=80) == UNSUP and call(h=6) == UNSUP and call(h=64) == UNSUP
    assert call(h=7) == BAD and call(h=0) == BAD and call(n=-1) == BAD and call(m=0) == BAD and call(ml=-1) == BAD
    assert call(ml=65) == BAD                            # more tokens than the table holds
    assert call(odt=2) == BAD and call(scale=float("nan")) == BAD and call(ks=0.3) == BAD and call(vs=0.0) == BAD
    for name in ("out", "q", "kc", "tab", "lens"):
        assert call(**{name: None}) == BAD
    assert call(q=P + 2) == BAD and call(out=P + 4) == BAD
    assert call(ws=None) == WS and call(ws=P + 4) == WS and call(wb=16) == WS
    assert call(n=0, out=None, ws=None) == L.PA_OK
    assert call(m=1 << 27, ml=(1 << 30) + 1) == UNSUP    # positions are 32-bit numbers
    assert call(scale=1e38, ks=2.0 ** 32) == BAD         # the product is not finite
    size = lib.pa_decode_fp4_workspace_size
    assert size(2, 8, 2, 128, 16, 64) > 0
    assert size(2, 6, 2, 128, 16, 64) == 0 and size(2, 8, 2, 96, 16, 64) == 0 and size(-1, 8, 2, 128, 16, 64) == 0


def test_prefill_refusals(lib):
    def call(out=P, odt=0, q=P, t=10, cu=P, qs=P, n=2, mq=5, ml=64, h=8, kc=P, nb=8, bs=16, hkv=2, d=128, tab=P, m=4,
             scale=1.0, ks=1.0, vs=1.0, status=None, ws=P, wb=1 << 40):
        return lib.pa_prefill_fp4(out, odt, q, t, cu, qs, n, mq, ml, h, kc, P, nb, bs, hkv, d, tab, m, scale, ks, vs,
                                  status, ws, wb, None)
    assert call(d=64) == UNSUP and call(bs=24) == UNSUP and call(h=6) == UNSUP
    assert call(scale=0.0) == BAD and call(scale=-1.0) == BAD and call(scale=float("inf")) == BAD
    assert call(t=-1) == BAD and call(n=-1) == BAD and call(mq=-1) == BAD and call(ml=65) == BAD and call(odt=3) == BAD
    assert call(ks=5.0) == BAD and call(vs=-2.0) == BAD and call(h=7) == BAD
    for name in ("out", "q", "cu", "qs", "kc", "tab"):
        assert call(**{name: None}) == BAD
    assert call(out=P + 16) == BAD and call(q=P + 8) == BAD and call(status=P + 2) == BAD
    assert call(ws=None) == WS and call(wb=8) == WS and call(ws=P + 8) == WS
    assert call(t=0, q=None, ws=None) == L.PA_OK and call(mq=0, q=None) == L.PA_OK
    assert call(m=1 << 27, ml=(1 << 30) + 1) == UNSUP and call(scale=1e38, ks=2.0 ** 32) == BAD
    assert lib.pa_prefill_fp4_workspace_size(2, 8, 2, 64, 16, 5, 64) == 0


def test_compact_refusals(lib):
    def call(kc=P, stride=0, layers=1, nb=8, bs=16, hkv=2, d=128, dt=1, tab=P, m=4, dst=P, keep=P, cu=P, n=2, mk=3,
             status=None):
        return lib.pa_compact_tokens(kc, P, stride, layers, nb, bs, hkv, d, dt, tab, m, dst, keep, cu, n, mk, status,
                                     None)
    assert call(bs=12) == UNSUP and call(d=3) == UNSUP and call(dt=2, d=96) == UNSUP
    assert call(dt=5) == BAD and call(n=-1) == BAD and call(mk=-1) == BAD and call(m=0) == BAD and call(layers=0) == BAD
    assert call(layers=2, stride=8 * 2 * 16 * 128 - 8) == BAD and call(layers=32768, stride=1 << 20) == BAD
    for name in ("kc", "tab", "dst", "keep", "cu"):
        assert call(**{name: None}) == BAD
    assert call(kc=P + 8) == BAD and call(status=P + 1) == BAD
    assert call(n=0, kc=None) == L.PA_OK and call(mk=0, kc=None) == L.PA_OK


def test_checked_compact_refusals(lib):
    def call(kc=P, bs=16, d=128, dt=1, keep=P, num_keep=4, cu=P, n=2, mk=3, status=None):
        return lib.pa_compact_tokens_checked(kc, P, 0, 1, 8, bs, 2, d, dt, P, 4, P, keep, num_keep, cu, n, mk, status, None)
    assert call(num_keep=-1) == BAD and call(num_keep=-5) == BAD
    assert call(bs=12) == UNSUP and call(d=3) == UNSUP and call(dt=5) == BAD and call(n=-1) == BAD and call(mk=-1) == BAD
    assert call(kc=None) == BAD and call(keep=None) == BAD and call(cu=None) == BAD and call(status=P + 1) == BAD
    assert call(n=0, num_keep=0, keep=None) == L.PA_OK and call(mk=0, num_keep=0) == L.PA_OK


def test_copy_accepts_4bit_pools(lib):
    def call(bs=16, d=128, n=1, layers=1, stride=0):
        return lib.pa_copy_blocks_layers(None, None, stride, layers, 8, bs, 2, d, L.PA_DTYPE_FP4, None, n, None)
    assert call(n=0) == L.PA_OK and call() == BAD
    assert call(bs=12, n=0) == UNSUP and call(d=96, n=0) == UNSUP
    need = 8 * 2 * fp4.tile_bytes(16, 128)
    assert call(layers=2, stride=need, n=0) == L.PA_OK and call(layers=2, stride=need - 16, n=0) == BAD
    # a cache of this kind is no argument of the calls that hold full values
    assert lib.pa_reshape_and_cache(None, None, 0, None, None, None, 8, 16, 2, 128, L.PA_DTYPE_FP4, None) == BAD


def test_binding_refuses_wrong_tensors(ops):
    import torch
    c = torch.zeros(4, 2, ops.fp4_tile_bytes(16, 128), dtype=torch.uint8)
    x = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError):
        ops.pa_reshape_and_cache_fp4(x, x, torch.zeros(3, dtype=torch.int64), c, c, 16)  # host tensors
    with pytest.raises(ValueError):
        ops.pa_copy_blocks(c, c, torch.zeros(0, 2, dtype=torch.int64))                    # sizes not given
    with pytest.raises(ops.PAError):
        ops.fp4_tile_bytes(16, 100)


@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
def test_prefill_workspace_never_shrinks_as_the_bound_grows(lib, group):
    """max_q_len is a bound, however loose: every size up to the largest int
    has room for the parts of the longest chunk that the context allows."""
    for hkv in (1, 8):
        for ctx in (1, 100, 4096, 1 << 20):
            bounds = sorted({1, 2, 15, 16, 17, 255, 256, 257, *(1 << e for e in range(9, 31)), ctx, (1 << 31) - 1})
            # a sequence's places, (2 + key tiles) for each tile pair and head, are numbered in 31 bits
            fits = [mq for mq in bounds if (2 + -(-ctx // 128)) * -(-min(mq, ctx) // (256 // group)) * hkv < 1 << 31]
            size = {mq: lib.pa_prefill_fp4_workspace_size(1, group * hkv, hkv, 128, 16, mq, ctx) for mq in bounds}
            assert all(0 < size[a] <= size[b] < 1 << 40 for a, b in zip(fits, fits[1:])), (hkv, ctx, size)
            assert all(size[mq] == 0 for mq in bounds if mq not in fits)
            assert size[(1 << 31) - 1] == size[ctx]


# ---------------------------------------------------------------------------
# allocator
# ---------------------------------------------------------------------------
def test_truncate_frees_the_blocks_behind(ops):
    a = ops.BlockAllocator(16, 4)
    s = a.seq_create()
    a.append_tokens(s, 18)
    table = a.block_table(s)
    a.truncate(s, 9)
    assert a.seq_len(s) == 9 and a.block_table(s) == table[:3] and a.num_free() == 13
    assert a.free_list()[-2:] == table[3:]               # in table order, at the back
    a.truncate(s, 9)
    a.truncate(s, 8)
    assert a.block_table(s) == table[:2]
    assert a.append_slot(s)[0] == a.block_table(s)[2] * 4
    a.truncate(s, 0)
    assert a.num_free() == 16 and a.block_table(s) == []
    for bad in (-1, 1):
        with pytest.raises(ops.PAError):
            a.truncate(s, bad)
    with pytest.raises(ops.PAError):
        a.truncate(99, 0)


def test_truncate_of_a_fork_keeps_the_parents_blocks(ops):
    a = ops.BlockAllocator(16, 4)
    s = a.seq_create()
    a.append_tokens(s, 10)
    table = a.block_table(s)
    c = a.fork(s)
    a.truncate(c, 5)
    assert a.block_table(s) == table and [a.refcount(b) for b in table] == [2, 2, 1]
    slot, src, dst = a.append_slot(c)                    # its last block is shared: copied first
    assert src == table[1] and slot == dst * 4 + 1


def test_make_writable_replaces_shared_blocks_only(ops):
    a = ops.BlockAllocator(8, 4)
    s = a.seq_create()
    a.append_tokens(s, 14)
    table = a.block_table(s)
    assert len(a.make_writable(s, 0, 14)) == 0 and a.block_table(s) == table
    c = a.fork(s)
    pairs = a.make_writable(c, 5, 8)
    assert pairs.tolist() == [[table[1], a.block_table(c)[1]]]
    assert a.block_table(s) == table and a.refcount(table[1]) == 1 and a.refcount(table[0]) == 2
    assert len(a.make_writable(c, 3, 3)) == 0
    pairs = a.make_writable(c, 0, 13)                    # the second one is its own by now
    assert pairs[:, 0].tolist() == [table[0], table[2], table[3]] and a.num_free() == 0
    for lo, hi in ((-1, 2), (3, 2), (0, 15)):
        with pytest.raises(ops.PAError):
            a.make_writable(c, lo, hi)


def test_make_writable_without_room_changes_nothing(ops, lib):
    a = ops.BlockAllocator(5, 4)
    s = a.seq_create()
    a.append_tokens(s, 16)
    c = a.fork(s)
    before = a.snapshot()
    with pytest.raises(ops.AllocatorOOM):
        a.make_writable(c, 0, 16)
    assert a.snapshot() == before
    n = C.c_int32(7)
    buf = (C.c_int64 * 2)()
    assert lib.pa_alloc_make_writable(a._h, c, 0, 8, buf, 1, C.byref(n)) == BAD and n.value == 0
    assert a.snapshot() == before
    assert lib.pa_alloc_make_writable(None, c, 0, 1, buf, 1, C.byref(n)) == BAD
    assert lib.pa_alloc_make_writable(a._h, c, 0, 1, buf, 1, None) == BAD
    assert lib.pa_alloc_truncate(None, 0, 0) == BAD


def test_prefix_keys_follow_truncation_and_rewriting(ops):
    a = ops.BlockAllocator(16, 4)
    a.enable_prefix_cache()
    ids = list(range(100, 118))
    s, cached, _ = a.seq_create_prefix(ids)
    assert cached == 0 and a.num_cached() == 4
    table = a.block_table(s)
    keys = [a.block_key(b) for b in table[:4]]
    a.truncate(s, 10)                                    # block 2 is partly used: its key is gone
    assert a.block_key(table[2]) is None and a.block_key(table[3]) == keys[3] and a.num_cached() == 3
    assert a.free_list()[-2:] == [table[4], table[3]]    # the last block first
    a.append_token_ids(s, ids[10:12])                    # the same tokens again: the same key
    assert a.block_key(table[2]) == oracle.block_key(keys[1], ids[8:12], b"") == keys[2]
    a.truncate(s, 8)
    a.append_token_ids(s, [1, 2, 3, 4])
    t2 = a.block_table(s)[2]
    assert a.block_key(t2) == oracle.block_key(keys[1], [1, 2, 3, 4], b"")
    # rewriting: the keys of the range go, the sequence is no longer keyed
    a.make_writable(s, 5, 9)
    assert a.block_key(table[0]) == keys[0] and a.block_key(table[1]) is None and a.block_key(t2) is None
    a.append_token_ids(s, [9, 9, 9, 9])
    assert a.block_key(a.block_table(s)[3]) is None
    # another request for the first tokens still finds the block that was not touched
    s2, cached, _ = a.seq_create_prefix(ids[:8])
    assert cached == 4 and a.block_table(s2)[0] == table[0]


def _two_holders(ops):
    """Two requests of the same 12 tokens in three shared, keyed blocks; the
    first cut to 10 tokens."""
    a = ops.BlockAllocator(16, 4)
    a.enable_prefix_cache()
    ids = list(range(50, 62))
    s1 = a.seq_create_prefix(ids)[0]
    s2, cached, _ = a.seq_create_prefix(ids)
    table = a.block_table(s1)
    assert cached == 12 and a.block_table(s2) == table and a.num_cached() == 3
    key = a.block_key(table[2])
    a.truncate(s1, 10)
    return a, ids, s1, s2, table, key


def test_truncation_into_a_shared_block_keeps_its_key(ops):
    """Its contents are another sequence's too, and do not change: a third
    request finds all 12 tokens.  A copy for the writer leaves them alone."""
    a, ids, s1, s2, table, key = _two_holders(ops)
    assert a.block_key(table[2]) == key and a.num_cached() == 3
    s3, cached, _ = a.seq_create_prefix(ids)
    assert cached == 12 and a.block_table(s3) == table
    with pytest.raises(ops.PAError):
        a.append_token_ids(s1, [7])                      # the block would have to be copied first
    slot, src, dst = a.append_slot(s1)
    assert src == table[2] and slot == dst * 4 + 2 and a.block_key(dst) is None and a.block_key(table[2]) == key


@pytest.mark.parametrize("how", ["ids", "slot", "slots", "tokens", "writable"])
def test_the_key_goes_with_the_first_write_in_place(ops, how):
    """The other holder leaves: the block is the truncated sequence's own, still
    with its contents, until the sequence writes into it."""
    a, ids, s1, s2, table, key = _two_holders(ops)
    a.free_seq(s2)
    assert a.refcount(table[2]) == 1 and a.block_key(table[2]) == key
    s3, cached, _ = a.seq_create_prefix(ids)
    assert cached == 12
    a.free_seq(s3)
    if how == "ids":
        a.append_token_ids(s1, [7])
    elif how == "slot":
        a.append_slot(s1)
    elif how == "slots":
        assert len(a.append_slots([s1])[1]) == 0
    elif how == "tokens":
        a.append_tokens(s1, 2)
    else:
        assert len(a.make_writable(s1, 9, 10)) == 0
    assert a.block_table(s1)[2] == table[2] and a.block_key(table[2]) is None and a.num_cached() == 2
    assert a.seq_create_prefix(ids)[1] == 8
    if how == "ids":
        a.append_token_ids(s1, [8])                      # full again, with other tokens: keyed for those
        k1 = oracle.block_key(a.block_key(table[1]), ids[8:10] + [7, 8], b"")
        assert a.block_key(table[2]) == k1


def test_a_truncated_holder_that_leaves_last_keeps_the_block_cached(ops):
    a, ids, s1, s2, table, key = _two_holders(ops)
    a.free_seq(s2)
    a.free_seq(s1)
    assert a.num_free() == 16 and a.block_key(table[2]) == key
    s3, cached, _ = a.seq_create_prefix(ids + [1])
    assert cached == 12 and a.block_table(s3)[:3] == table
