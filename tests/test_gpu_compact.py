"""Token compaction: bytes of the whole pool against a plain reordering."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _pool(rng, kind, layers, nb, hkv, bs, d):
    if kind == "fp4":
        return rng.integers(0, 256, size=(layers, nb, hkv, fp4.tile_bytes(bs, d)), dtype=np.uint8)
    e = 4 if kind == "f32" else 2
    return rng.integers(0, 256, size=(layers, nb, hkv, bs, d * e), dtype=np.uint8)


def _rows(c, kind, bs, d):
    """[L, NB, Hkv, bs, bytes] of every token's row (a copy for 4-bit pools)."""
    if kind != "fp4":
        return c
    codes, scales = fp4.rows(c, bs, d)
    return np.concatenate((codes, scales), axis=-1)


def _tensor(c, kind, d):
    t = _dev(c)
    return t if kind == "fp4" else t.view(torch.float32 if kind == "f32" else torch.bfloat16)


def _bytes(t):
    return t.cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp4"])
@pytest.mark.parametrize("layers,hkv,d,bs,counts,starts,span", [
    (1, 2, 128, 16, [5, 0, 40], [3, 0, 11], 60), (3, 8, 64, 4, [7, 1], [0, 9], 9),
    (1, 1, 256, 64, [500, 700], [1, 0], 900), (2, 3, 128, 1, [33], [5], 50), (1, 4, 128, 256, [256, 64], [0, 255], 256),
    (32, 8, 128, 16, [1, 3, 8], [40, 41, 63], 32)])
def test_compaction_moves_exactly_the_kept_tokens(ops, kind, layers, hkv, d, bs, counts, starts, span):
    rng = np.random.default_rng(len(counts) + span)
    need = [-(-(s + span) // bs) for s in starts]
    nb = sum(need) + 2
    perm = rng.permutation(nb)
    tables = np.full((len(counts), max(need)), -3, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    keep = [starts[i] + np.sort(rng.permutation(span)[:c]) for i, c in enumerate(counts)]
    k, v = (_pool(rng, kind, layers, nb, hkv, bs, d) for _ in range(2))
    kt, vt = _tensor(k, kind, d), _tensor(v, kind, d)
    args = (_dev(tables), _dev(np.array(starts, np.int32)), _dev(np.concatenate(keep).astype(np.int32)),
            _dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)), max(counts))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if layers == 1:
        ops.pa_compact_tokens(kt[0], vt[0], *args, block_size=bs, head_dim=d, status=status)
    else:
        ops.pa_compact_tokens(kt, vt, *args, block_size=bs, head_dim=d, status=status)
    assert int(status.item()) == 0
    for before, after in ((k, kt), (v, vt)):
        old = _rows(before, kind, bs, d)
        want = old.copy()
        for i, p in enumerate(keep):
            for j, src in enumerate(p):
                dst = starts[i] + j
                want[:, tables[i, dst // bs], :, dst % bs] = old[:, tables[i, src // bs], :, src % bs]
        assert np.array_equal(_rows(_bytes(after).reshape(before.shape), kind, bs, d), want)


def test_bad_positions_are_reported_and_not_moved(ops):
    rng = np.random.default_rng(2)
    hkv, bs, d, nb = 2, 16, 128, 8
    k = _pool(rng, "bf16", 1, nb, hkv, bs, d)
    tables = _dev(np.arange(8, dtype=np.int32).reshape(4, 2))
    cases = [([5, 5], 0), ([3], 4), ([32], 0), ([-1], 0), ([6, 5], 0)]
    for keep, start in cases:
        kt, vt = _tensor(k, "bf16", d), _tensor(k, "bf16", d)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = len(keep)
        ops.pa_compact_tokens(kt[0], vt[0], tables, _dev(np.array([0, 0, start, 0], np.int32)),
                              _dev(np.array(keep, np.int32)), _dev(np.array([0, 0, 0, n, n], np.int32)), n,
                              status=status)
        assert int(status.item()) == 1, keep
        want = k.copy()
        if n == 2:  # the first is fine, the second is not behind it
            want[0, 4, :, 0] = k[0, 4, :, keep[0]]
        assert np.array_equal(_bytes(kt).reshape(k.shape), want), keep
    # counts outside [0, max_keep], a destination past the table, a table entry outside the pool
    for starts, cu, tab in (([0, 0, 0, 0], [0, 2, 2, 2, 2], None), ([0, 31, 0, 0], [0, 0, 1, 1, 1], "keep 31"),
                            ([0, 0, 0, 0], [0, 0, 0, 0, 1], "table")):
        kt, vt = _tensor(k, "bf16", d), _tensor(k, "bf16", d)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = tables.clone()
        keep = [4, 6]
        if tab == "keep 31":
            starts, keep = [0, 32, 0, 0], [33, 34]
        if tab == "table":
            t[3, 0] = nb
        ops.pa_compact_tokens(kt[0], vt[0], t, _dev(np.array(starts, np.int32)), _dev(np.array(keep, np.int32)),
                              _dev(np.array(cu, np.int32)), 1, status=status)
        assert int(status.item()) == 1
        assert np.array_equal(_bytes(kt).reshape(k.shape), k)


def test_compaction_replayed_from_a_graph(ops):
    rng = np.random.default_rng(4)
    hkv, bs, d, nb = 2, 16, 128, 8
    k = _pool(rng, "fp4", 1, nb, hkv, bs, d)
    kt, vt = _dev(k[0]), _dev(k[0])
    tables, start = _dev(np.arange(8, dtype=np.int32).reshape(1, 8)), _dev(np.array([2], np.int32))
    keep, cu = _dev(np.array([4, 9, 70], np.int32)), _dev(np.array([0, 3], np.int32))
    call = lambda: ops.pa_compact_tokens(kt, vt, tables, start, keep, cu, 3, bs, d)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    assert np.array_equal(_bytes(kt).reshape(k[0].shape), k[0])  # capture runs nothing
    rows = _rows(k, "fp4", bs, d)[0]
    for pos in ([4, 9, 70], [2, 3, 100]):
        keep.copy_(torch.tensor(pos, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = rows.copy()
        for j, p in enumerate(pos):
            want[(2 + j) // bs, :, (2 + j) % bs] = rows[p // bs, :, p % bs]
        rows = want
        assert np.array_equal(_rows(_bytes(kt).reshape(k.shape), "fp4", bs, d)[0], rows)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_ranges_behind_keep_are_reported_and_left_alone(ops, lib, kind):
    """cu_keep that points behind keep, with counts that are small: what lies
    there (memory of the test's own, with positions that could be moved) is
    not taken for a list; the sequences whose lists are whole are compacted."""
    rng = np.random.default_rng(5)
    hkv, bs, d, nb = 2, 16, 128, 8
    k = _pool(rng, kind, 1, nb, hkv, bs, d)
    tables = _dev(np.arange(8, dtype=np.int32).reshape(4, 2))
    wide = _dev(np.array([4, 9, 5, 6, 7, 20, 3, 8], np.int32))
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    #        entries of keep, cu_keep, sequences that move
    cases = [(4, [0, 2, 4, 4, 6], [0, 1]), (4, [0, 2, 5, 6, 8], [0]), (2, [0, 2, 1 << 30, (1 << 30) + 2, 2], [0]),
             (8, [0, 2, 5, 6, 8], [0, 1, 2, 3])]
    for entries, cu, moved in cases:
        kt, vt = _tensor(k, kind, d), _tensor(k, kind, d)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_compact_tokens(kt[0], vt[0], tables, start, wide[:entries], _dev(np.array(cu, np.int32)), 3, bs, d,
                              status=status)
        assert int(status.item()) == (0 if len(moved) == 4 else 1), cu
        want = _rows(k, kind, bs, d).copy()
        for i in moved:
            for j, src in enumerate(wide[cu[i]:cu[i + 1]].tolist()):
                want[:, 2 * i + j // bs, :, j % bs] = _rows(k, kind, bs, d)[:, 2 * i + src // bs, :, src % bs]
        for t in (kt, vt):
            assert np.array_equal(_rows(_bytes(t).reshape(k.shape), kind, bs, d), want), cu
    # without keep's length the call goes by cu_keep[num_seqs]
    kt, vt = _tensor(k, kind, d), _tensor(k, kind, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = _dev(np.array([0, 2, 5, 6, 4], np.int32))
    st = lib.pa_compact_tokens(kt.data_ptr(), vt.data_ptr(), 0, 1, nb, bs, hkv, d, 1 if kind == "bf16" else 2,
                               tables.data_ptr(), 2, start.data_ptr(), wide.data_ptr(), cu.data_ptr(), 4, 3,
                               status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and int(status.item()) == 1
    want = _rows(k, kind, bs, d).copy()
    for j, src in enumerate((4, 9)):
        want[:, 0, :, j] = _rows(k, kind, bs, d)[:, src // bs, :, src % bs]
    assert np.array_equal(_rows(_bytes(kt).reshape(k.shape), kind, bs, d), want)
