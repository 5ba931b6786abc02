"""Eviction by accumulated attention weight on the GPU: the weights, the
selection, and a run of both with decode and compaction."""
import numpy as np
import pytest
import torch

from latent_case import LATENT, ROPE, ROW, bf16, blank_unused, check, dev, dev16, tables_of
from oracle import latent as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def weights_case(rng, lens, bs, W, H, hkv, d, extra=0):
    tables, nb = tables_of(rng, lens, bs, pad=-1)
    k = bf16(rng.standard_normal((nb, hkv, bs, d)))
    q = bf16(rng.standard_normal((len(lens), W, H, d)))
    before = rng.uniform(0, 1, size=(len(lens), max(lens) + extra)).astype(np.float32)
    return tables, k, q, before


def run_weights(ops, before, q, k, tables, lens, bs, scale, ws=None):
    B, W, H, d = q.shape
    hkv, max_len = k.shape[1], max(lens)
    if ws is None:
        ws = ops.make_workspace_weights(B, W, H, hkv, d, bs, max_len)
    w = dev(before)
    ops.pa_accumulate_weights(w, dev16(q), k, dev(tables), dev(np.array(lens, np.int32)), scale, hkv, max_len, ws)
    assert ops.pa_workspace_error(ws) == 0
    return w


@pytest.mark.parametrize("d,hkv,G", [(64, 2, 1), (128, 2, 4), (128, 1, 16), (256, 3, 2), (ROW, 1, 128), (ROW, 1, 16),
                                     (128, 2, 5)])
@pytest.mark.parametrize("W,bs", [(1, 16), (3, 8), (32, 64), (40, 256)])
def test_weights(ops, d, hkv, G, W, bs):
    rng = np.random.default_rng(d + G * W)
    lens = [1, 0, 127, 128, 129, 20, 300]
    tables, k, q, before = weights_case(rng, lens, bs, W, hkv * G, hkv, d, extra=3)
    scale = 1.0 / np.sqrt(d)
    ref, tol = O.weights(before, q.f32, k.f32, tables, lens, scale)
    for fill in (0.0, float("nan")):
        pool = blank_unused(dev16(k), tables, lens, bs, fill, heads=True)
        check(run_weights(ops, before, q, pool, tables, lens, bs, scale), ref, tol, False)


@pytest.mark.parametrize("B,top,W,H,hkv,d,bs", [(1, 9000, 1, 8, 2, 128, 16), (2, 5000, 32, 8, 2, 128, 32),
                                                (100, 200, 1, 8, 8, 64, 8), (1, 4000, 2, 128, 1, ROW, 16)])
def test_weights_lengths(ops, B, top, W, H, hkv, d, bs):
    rng = np.random.default_rng(B + W)
    lens = [int(x) for x in rng.integers(0, top, size=B)]
    lens[-1] = top
    tables, k, q, before = weights_case(rng, lens, bs, W, H, hkv, d)
    ref, tol = O.weights(before, q.f32, k.f32, tables, lens, 0.1)
    a = run_weights(ops, before, q, dev16(k), tables, lens, bs, 0.1)
    check(a, ref, tol, False)
    b = run_weights(ops, before, q, dev16(k), tables, lens, bs, 0.1)
    assert torch.equal(a, b)  # sums in a fixed order


@pytest.mark.parametrize("d,G,W", [(64, 4, 14), (64, 3, 19), (64, 4, 19), (64, 7, 11), (64, 5, 17), (64, 2, 70), (128, 4, 19), (128, 4, 20), (128, 3, 50), (128, 128, 1)])
def test_weights_of_rows_on_both_sides_of_the_second_product(ops, d, G, W):
    """56, 57, 76, 77, 85, 140, 76, 80, 150 and 128 rows of a kv head."""
    rng = np.random.default_rng(d + G * W)
    lens = [260, 0, 3, 128, 75]
    tables, k, q, before = weights_case(rng, lens, 16, W, 2 * G, 2, d)
    check(run_weights(ops, before, q, dev16(k), tables, lens, 16, d ** -0.5),
          *O.weights(before, q.f32, k.f32, tables, lens, d ** -0.5), False)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 4.0])
def test_weights_with_any_softmax_scale(ops, scale):
    rng = np.random.default_rng(4)
    lens = [300, 70]
    tables, k, q, before = weights_case(rng, lens, 16, 2, 8, 2, 128)
    ref, tol = O.weights(before, q.f32, k.f32, tables, lens, scale)
    check(run_weights(ops, before, q, dev16(k), tables, lens, 16, scale), ref, tol, False)


# ------------------------------------------------------------- selection
def run_select(ops, w, start, lens, counts, recent, stride=None, status_is=0):
    S, m = w.shape
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    wide = torch.full((S, (stride or m)), 9.0, device="cuda")
    wide[:, :m] = dev(w)
    keep = torch.full((int(cu[-1]),), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_select_tokens(keep, dev(cu), wide[:, :m], dev(np.array(start, np.int32)), dev(np.array(lens, np.int32)), recent,
                         int(max(lens)), status=status)
    assert int(status.item()) == status_is
    assert (wide[:, m:] == 9.0).all()
    return keep.cpu().numpy(), wide[:, :m].cpu().numpy()


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special"])
@pytest.mark.parametrize("top,recent", [(1, 0), (40, 0), (700, 16), (2500, 64), (5000, 4000), (33000, 1)])
def test_select(ops, kind, top, recent):
    rng = np.random.default_rng(top + recent)
    lens = [top, 0, max(1, top // 2), top]
    start = [0, 0, min(3, top // 2), top // 3]
    spans = [b - a for a, b in zip(start, lens)]
    counts = [spans[0] // 2, 0, spans[2], (spans[3] + 3) // 4]
    w = rng.standard_normal((4, top + 2)).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 2) / 2
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "special":
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.1] = -np.inf
        w[rng.random(w.shape) < 0.1] = -0.0
        w[rng.random(w.shape) < 0.1] = 0.0
    keep, after = O.select(w, start, lens, counts, recent)
    got, moved = run_select(ops, w, start, lens, counts, recent, stride=top + 6)
    assert np.array_equal(got, keep)
    assert np.array_equal(moved.view(np.int32), after.view(np.int32))


@pytest.mark.parametrize("count", [0, 1, 399_999, 400_000])
def test_select_from_more_than_shared_memory_holds(ops, count):
    rng = np.random.default_rng(3)
    n = 400_000
    w = np.round(rng.standard_normal((1, n)) * 4).astype(np.float32)
    keep, after = O.select(w, [0], [n], [count], 0)
    got, moved = run_select(ops, w, [0], [n], [count], 0)
    assert np.array_equal(got, keep) and np.array_equal(moved, after)


def test_select_many_sequences(ops):
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 300, size=500)
    start = lens // 4
    counts = ((lens - start) * 0.3).astype(int)
    w = rng.standard_normal((500, 300)).astype(np.float32)
    keep, after = O.select(w, start, lens, counts, 8)
    got, moved = run_select(ops, w, start, lens, counts, 8)
    assert np.array_equal(got, keep) and np.array_equal(moved, after)


def test_select_reports_what_lies_outside(ops):
    rng = np.random.default_rng(7)
    w = rng.standard_normal((3, 100)).astype(np.float32)
    keep, after = O.select(w[[0, 2]], [0, 5], [100, 90], [10, 20], 2)
    # more kept than there are, a length past the bound, a start below zero
    for start, length, n in ((50, 60, 11), (0, 101, 5), (-1, 50, 5), (60, 50, 0)):
        cu = np.array([0, 10, 10 + n, 30 + n], np.int32)
        got = torch.full((30 + n,), -1, dtype=torch.int32, device="cuda")
        ww, status = dev(w), torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_select_tokens(got, dev(cu), ww, dev(np.array([0, start, 5], np.int32)),
                             dev(np.array([100, length, 90], np.int32)), 2, 100, status=status)
        assert int(status.item()) == 1
        got, ww = got.cpu().numpy(), ww.cpu().numpy()
        assert np.array_equal(np.r_[got[:10], got[10 + n:]], keep) and (got[10:10 + n] == -1).all()
        assert np.array_equal(ww[[0, 2]], after) and np.array_equal(ww[1], w[1])


def test_select_reports_bounds_whose_differences_wrap(ops):
    top, least = 2 ** 31 - 1, -2 ** 31
    w = np.arange(100, dtype=np.float32)[None]
    for cu, start, length in (([0, 1], top, least), ([top, least], 0, 100), ([least, top], 0, 100), ([0, 1], least, 100),
                              ([0, top], 0, 100), ([0, least], 0, 100), ([0, 1], 0, least), ([-1, 0], 0, 100)):
        keep, ww = torch.full((4,), -1, dtype=torch.int32, device="cuda"), dev(w)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_select_tokens(keep, dev(np.array(cu, np.int32)), ww, dev(np.array([start], np.int32)),
                             dev(np.array([length], np.int32)), 0, 100, status=status)
        assert int(status.item()) == 1, (cu, start, length)
        assert (keep == -1).all() and np.array_equal(ww.cpu().numpy(), w)


# ------------------------------------------------- the operators together
def test_eviction_of_a_latent_history(ops):
    """Append, decode, weights, selection, compaction, truncation and the next
    decode over the thinned cache, as a server does them."""
    rng = np.random.default_rng(11)
    bs, H, lens = 16, 16, [300, 77]
    alloc = ops.BlockAllocator(64, bs)
    seqs = [alloc.seq_create() for _ in lens]
    slots = np.concatenate([alloc.append_tokens(s, n) for s, n in zip(seqs, lens)])
    latent, rope = bf16(rng.standard_normal((sum(lens), LATENT))), bf16(rng.standard_normal((sum(lens), ROPE)))
    cache = torch.zeros(64, bs, ROW, dtype=torch.bfloat16, device="cuda")
    ops.pa_reshape_and_cache_latent(dev16(latent), dev16(rope), dev(slots), cache)
    tables, _ = alloc.export_tables(seqs, 20)
    pool = cache.float().cpu().numpy()
    q = bf16(rng.standard_normal((2, 1, H, ROW)) * 0.6)
    d_lens = dev(np.array(lens, np.int32))
    w = torch.zeros(2, 320, device="cuda")
    ws, wd = (make(2, 1, H, *dims, bs, 300) for make, dims in
              ((ops.make_workspace_weights, (1, ROW)), (ops.make_workspace_latent, (LATENT, ROPE))))
    out = torch.zeros(2, 1, H, LATENT, device="cuda")
    ops.pa_decode_latent(out, dev16(q), cache, dev(tables), d_lens, 0.07, 300, wd)
    ops.pa_accumulate_weights(w, dev16(q), cache, dev(tables), d_lens, 0.07, 1, 300, ws)
    check(out, *O.decode(q.f32, pool, tables, lens, 0.07, LATENT), False)
    ref_w, tol = O.weights(np.zeros((2, 320)), q.f32, pool[:, None], tables, lens, 0.07)
    check(w, ref_w, tol, False)
    # half of what lies behind the first four tokens stays, the last eight among it
    first, counts = np.array([4, 4], np.int32), [148, 36]
    cu = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    want, after = O.select(w.cpu().numpy(), first, lens, counts, 8)
    keep = torch.zeros(sum(counts), dtype=torch.int32, device="cuda")
    ops.pa_select_tokens(keep, cu, w, dev(first), d_lens, 8, 300)
    assert np.array_equal(keep.cpu().numpy(), want) and np.array_equal(w.cpu().numpy(), after)
    for s, n in zip(seqs, counts):
        assert len(alloc.make_writable(s, 4, 4 + n)) == 0
    ops.pa_compact_tokens_latent(cache, dev(tables), dev(first), keep, cu, max(counts))
    for s, n in zip(seqs, counts):
        alloc.truncate(s, 4 + n)
    new_tables, new_lens = alloc.export_tables(seqs, 20)
    at = np.split(want, [counts[0]])
    thin = [np.r_[0:4, a] for a in at]
    ops.pa_decode_latent(out, dev16(q), cache, dev(new_tables), dev(new_lens), 0.07, 300, wd)
    for i in range(2):
        x = O.rows(pool, tables[i], lens[i], bs)[thin[i]]
        ref, tol = O.attend(q.f32[i, 0].astype(np.float64), x, x[:, :LATENT], 0.07, np.full(H, len(x)))
        check(out[i, 0], ref, tol, False)
