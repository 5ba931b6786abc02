"""Calls of the latent cache and of eviction that their documentation allows
around the plain ones: captured graphs beside eager calls, other streams, one
workspace for many shapes, pools past 2^31 bytes, long contexts, batches past
one launch, shared blocks, values that are not finite, rows of nobody."""
import numpy as np
import pytest
import torch

from latent_case import HEAD, LATENT, ROPE, ROW, bf16, check, dev, dev16, tables_of
from oracle import latent as O
from test_gpu_latent import decode_case, prefill_case, run_decode, run_prefill
from test_gpu_evict import run_select, run_weights, weights_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def test_one_decode_workspace_for_many_shapes(ops):
    rng = np.random.default_rng(1)
    ws = ops.make_workspace_latent(8, 4, 128, LATENT, ROPE, 8, 4000)
    for lens, bs, H, Q in ([700] * 6, 16, 16, 1), ([3000, 5], 8, 128, 1), ([2500], 32, 40, 3), ([9, 4000], 64, 2, 1), ([700] * 6, 16, 16, 1):
        tables, cache, q = decode_case(rng, lens, bs, H, Q)
        ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
        for dt in (torch.float32, torch.bfloat16):
            check(run_decode(ops, q, dev16(cache), tables, lens, bs, 0.07, dt, ws=ws), ref, tol, dt == torch.bfloat16)


def test_graph_beside_eager_calls(ops):
    """A captured append, decode, weights and prefill, replayed with new inputs
    while eager calls use other workspaces."""
    rng = np.random.default_rng(2)
    lens, bs, H = [300, 64, 1], 16, 20
    tables, cache, q = decode_case(rng, lens, bs, H, 1)
    pool, tab, dl = dev16(cache), dev(tables), dev(np.array(lens, np.int32))
    ws = ops.make_workspace_latent(3, 1, H, LATENT, ROPE, bs, 300)
    ww = ops.make_workspace_weights(3, 1, H, 1, ROW, bs, 300)
    qd, out, w = dev16(q), torch.zeros(3, 1, H, LATENT, device="cuda"), torch.zeros(3, 300, device="cuda")
    _, _, _, _, qp, w_k, w_v = prefill_case(rng, [(0, 3)], bs, 2)
    cu, start = dev(np.array([0, 1, 2, 3], np.int32)), dev(np.array([n - 1 for n in lens], np.int32))
    wp = ops.make_prefill_workspace_latent(3, 2, LATENT, ROPE, HEAD, bs, 1, 300, sum(lens))
    outp, qpd, wk, wv = torch.zeros(3, 2, HEAD, dtype=torch.bfloat16, device="cuda"), dev16(qp), dev16(w_k), dev16(w_v)

    def step():
        ops.pa_decode_latent(out, qd, pool, tab, dl, 0.07, 300, ws)
        ops.pa_accumulate_weights(w, qd, pool, tab, dl, 0.07, 1, 300, ww)
        ops.pa_prefill_latent(outp, qpd, pool, wk, wv, cu, start, tab, 0.07, 1, 300, sum(lens), wp)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        q2, new = bf16(rng.standard_normal(q.shape) * 0.6), bf16(rng.standard_normal(cache.shape))
        qd.copy_(dev16(q2))
        pool.copy_(dev16(new))
        w.zero_()
        g.replay()
        check(run_decode(ops, q2, pool, tables, lens, bs, 0.07), *O.decode(q2.f32, new.f32, tables, lens, 0.07, LATENT), False)
        check(out, *O.decode(q2.f32, new.f32, tables, lens, 0.07, LATENT), False)
        check(w, *O.weights(np.zeros((3, 300)), q2.f32, new.f32[:, None], tables, lens, 0.07), False)
        check(outp, *O.prefill(qp.f32, new.f32, w_k.f32, w_v.f32, np.arange(4), np.array(lens) - 1, tables, 0.07), True)
    assert ops.pa_workspace_error(ws) == 0 and ops.pa_workspace_error(ww) == 0


def test_two_streams_with_their_own_workspaces(ops):
    rng = np.random.default_rng(3)
    cases = []
    for lens, H in (([2000, 30], 128), ([500, 900, 1], 16)):
        tables, cache, q = decode_case(rng, lens, 16, H, 1)
        args = [dev16(q), dev16(cache), dev(tables), dev(np.array(lens, np.int32))]
        ws = ops.make_workspace_latent(len(lens), 1, H, LATENT, ROPE, 16, max(lens))
        ww = ops.make_workspace_weights(len(lens), 1, H, 1, ROW, 16, max(lens))
        cases.append((lens, tables, cache, q, args, ws, ww, torch.zeros(len(lens), 1, H, LATENT, device="cuda"),
                      torch.zeros(len(lens), max(lens), device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for lens, _, _, _, (qd, pool, tab, dl), ws, ww, out, w, stream in cases:
            ops.pa_decode_latent(out, qd, pool, tab, dl, 0.07, max(lens), ws, stream=stream)
            with torch.cuda.stream(stream):
                w.zero_()
                ops.pa_accumulate_weights(w, qd, pool, tab, dl, 0.07, 1, max(lens), ww)
    torch.cuda.synchronize()
    for lens, tables, cache, q, _, _, _, out, w, _ in cases:
        check(out, *O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT), False)
        check(w, *O.weights(np.zeros(w.shape), q.f32, cache.f32[:, None], tables, lens, 0.07), False)


def test_prefills_on_two_streams(ops):
    """Overlapping prefills of different shapes and outputs, an odd number of
    tiles and of heads among them, each with its own workspace."""
    rng = np.random.default_rng(31)
    cases = []
    for chunks, H, dt in (([(0, 300), (40, 129)], 5, torch.bfloat16), ([(700, 20)], 16, torch.bfloat16), ([(128, 130)], 3, torch.float32)):
        _, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, 16, H)
        start = [s for s, _ in chunks]
        most, total = max(s + n for s, n in chunks), sum(s + n for s, n in chunks)
        wp = ops.make_prefill_workspace_latent(len(chunks), H, LATENT, ROPE, HEAD, 16, max(n for _, n in chunks), most, total)
        out = torch.zeros(q.shape[0], H, HEAD, dtype=dt, device="cuda")
        args = [dev16(q), dev16(cache), dev16(w_k), dev16(w_v), dev(np.asarray(cu, np.int32)), dev(np.asarray(start, np.int32)), dev(tables)]
        ref = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.07, two=dt == torch.float32)
        cases.append((out, args, max(n for _, n in chunks), most, total, wp, torch.cuda.Stream(), ref))
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(6):
        for out, args, longest, most, total, wp, stream, _ in cases:
            ops.pa_prefill_latent(out, *args, 0.07, longest, most, total, wp, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for out, *_, ref in cases:
        check(out, *ref, out.dtype == torch.bfloat16)


@pytest.mark.parametrize("chunks,H", [([(4000, 3)], 2), ([(1500, 70), (0, 2)], 3), ([(0, 100)], 1), ([(900, 65), (0, 0), (31, 1)], 5), ([(0, 1)] * 3, 1)])
def test_fp32_prefill_with_split_keys(ops, chunks, H):
    """Few queries: their keys are shared among CTAs, some of which see nothing
    of a row's, and rows of nobody stay."""
    rng = np.random.default_rng(41 + H)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, 16, H, pad=-1)
    start = [s for s, _ in chunks]
    out = run_prefill(ops, q, dev16(cache), w_k, w_v, cu, start, tables, 16, 0.07, max(n for _, n in chunks) + 40, max(lens), sum(lens) + 5)
    check(out, *O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.07, two=True), False)


@pytest.mark.parametrize("H,dt", [(16, torch.float32), (32, torch.bfloat16), (17, torch.float32)])
def test_few_rows_of_many_sequences(ops, H, dt):
    """2048 sequences a launch, where the shared memory is fullest, with items of
    one tile and of several."""
    rng = np.random.default_rng(32 + H)
    lens = [int(x) for x in rng.integers(0, 30, size=2048)]
    lens[5], lens[-1], lens[1000] = 700, 500, 65
    tables, cache, q = decode_case(rng, lens, 16, H, 1)
    ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
    check(run_decode(ops, q, dev16(cache), tables, lens, 16, 0.07, dt), ref, tol, dt == torch.bfloat16)


@pytest.mark.parametrize("lens,H,Q", [([5000], 16, 1), ([5000], 128, 1), ([3000, 0, 7, 2500], 128, 1), ([900] * 15, 16, 1), ([900] * 16, 16, 1),
                                      ([2000] * 5, 128, 1), ([0, 4000], 3, 1), ([3000, 40], 100, 3), ([6000], 1, 300)])
def test_few_long_sequences(ops, lens, H, Q):
    """Items in many parts, beside ones in one."""
    rng = np.random.default_rng(len(lens) + H)
    tables, cache, q = decode_case(rng, lens, 32, H, Q)
    check(run_decode(ops, q, dev16(cache), tables, lens, 32, 0.07), *O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT), False)


def test_pool_past_2_to_the_31_bytes(ops):
    """Blocks at the far end of a pool of more than 2^32 bytes."""
    rng = np.random.default_rng(4)
    bs, n, H = 16, 75, 24
    nb = (1 << 32) // (bs * ROW * 2) + 100
    pool = torch.zeros(nb, bs, ROW, dtype=torch.bfloat16, device="cuda")
    tables = np.array([[nb - 1, 3, nb - 7, nb - 2, nb - 50]], dtype=np.int32)
    rows = bf16(rng.standard_normal((n, ROW)))
    slots = tables[0, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
    d = dev16(rows)
    ops.pa_reshape_and_cache_latent(d[:, :LATENT], d[:, LATENT:], dev(slots), pool)
    small = np.zeros((5, bs, ROW), np.float32)
    small.reshape(-1, ROW)[:n] = rows.f32
    near = np.arange(5, dtype=np.int32)[None]
    q = bf16(rng.standard_normal((1, 2, H, ROW)) * 0.6)
    check(run_decode(ops, q, pool, tables, [n], bs, 0.07), *O.decode(q.f32, small, near, [n], 0.07, LATENT), False)
    before = np.zeros((1, n), np.float32)
    check(run_weights(ops, before, q, pool.unsqueeze(1), tables, [n], bs, 0.07),
          *O.weights(before, q.f32, small[:, None], near, [n], 0.07), False)
    _, _, _, cu, qp, w_k, w_v = prefill_case(rng, [(n - 9, 9)], bs, 3)
    out = run_prefill(ops, qp, pool, w_k, w_v, cu, [n - 9], tables, bs, 0.07, 9, n, n, torch.bfloat16)
    check(out, *O.prefill(qp.f32, small, w_k.f32, w_v.f32, cu, [n - 9], near, 0.07), True)
    ops.pa_copy_blocks_latent(pool, torch.tensor([[nb - 1, nb - 90]], device="cuda"))
    assert torch.equal(pool[nb - 90], pool[nb - 1])
    keep = np.arange(1, n, 2).astype(np.int32)
    ops.pa_compact_tokens_latent(pool, dev(tables), dev(np.zeros(1, np.int32)), dev(keep), dev(np.array([0, len(keep)], np.int32)),
                                 len(keep))
    got = pool[torch.from_numpy(tables[0].astype(np.int64)).cuda()].flatten(0, 1)[: len(keep)].float().cpu().numpy()
    assert np.array_equal(got, rows.f32[keep])


@pytest.mark.parametrize("n", [70_001, 1_000_003])
def test_long_context_finds_single_keys(ops, n):
    """One token of a long context holds nearly all the weight of a query."""
    bs, H = 256, 3
    nb = -(-n // bs)
    g = torch.Generator(device="cuda").manual_seed(5)
    pool = torch.randn(nb, bs, ROW, generator=g, device="cuda").bfloat16() * 0.01
    tables = torch.randperm(nb, generator=g, device="cuda").int()[None]
    flat = pool.view(-1, ROW)
    places = [0, n // 2 + 1, n - 1]
    q = torch.zeros(1, 1, H, ROW, dtype=torch.bfloat16, device="cuda")
    rows = []
    for h, t in enumerate(places):
        slot = int(tables[0, t // bs]) * bs + t % bs
        flat[slot] = 0
        flat[slot, 100 * h] = 8.0
        flat[slot, LATENT + h] = 16.0
        q[0, 0, h, LATENT + h] = 4.0   # 64 against at most a few hundredths: 64 > ln(10^6) + 40
        rows.append(flat[slot].clone())
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = ops.make_workspace_latent(1, 1, H, LATENT, ROPE, bs, n)
    out = torch.zeros(1, 1, H, LATENT, device="cuda")
    ops.pa_decode_latent(out, q, pool, tables, lens, 1.0, n, ws)
    assert ops.pa_workspace_error(ws) == 0
    want = torch.stack(rows)[:, :LATENT].float()
    # the others weigh n e^-64 together; probabilities are held to 2^-16, and the value is 8
    assert float((out[0, 0] - want).abs().max()) < 8 * 2.0 ** -16
    w = torch.zeros(1, n, device="cuda")
    ww = ops.make_workspace_weights(1, 1, H, 1, ROW, bs, n)
    ops.pa_accumulate_weights(w, q, pool, tables, lens, 1.0, 1, n, ww)
    assert ops.pa_workspace_error(ww) == 0
    assert float((w[0, places] - 1).abs().max()) < 1e-5 and float(w.sum()) < 3 + 1e-4
    keep = torch.zeros(3, dtype=torch.int32, device="cuda")
    ops.pa_select_tokens(keep, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), w, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         lens, 0, n)
    assert keep.tolist() == places


def test_batches_past_one_launch(ops):
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 40, size=2500)]
    lens[-1] = 40
    tables, cache, q = decode_case(rng, lens, 8, 2, 1)
    check(run_decode(ops, q, dev16(cache), tables, lens, 8, 0.07), *O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT), False)
    before = rng.uniform(0, 1, size=(2500, 40)).astype(np.float32)
    check(run_weights(ops, before, q, dev16(cache).unsqueeze(1), tables, lens, 8, 0.07),
          *O.weights(before, q.f32, cache.f32[:, None], tables, lens, 0.07), False)


def test_blocks_that_sequences_share(ops):
    """Three sequences over one prefix, one block named twice by a table."""
    rng = np.random.default_rng(7)
    bs, lens = 16, [80, 70, 64]
    tables = np.array([[0, 1, 2, 3, 4], [0, 1, 2, 5, 6], [0, 1, 0, 1, 0]], dtype=np.int32)
    cache, q = bf16(rng.standard_normal((7, bs, ROW))), bf16(rng.standard_normal((3, 1, 16, ROW)) * 0.6)
    check(run_decode(ops, q, dev16(cache), tables, lens, bs, 0.07), *O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT), False)
    before = np.zeros((3, 80), np.float32)
    check(run_weights(ops, before, q, dev16(cache).unsqueeze(1), tables, lens, bs, 0.07),
          *O.weights(before, q.f32, cache.f32[:, None], tables, lens, 0.07), False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Q", [(16, 3), (70, 4)])
def test_decode_rows_that_do_not_see_a_value_that_is_not_finite(ops, bad, H, Q):
    """The newest token holds one: queries before it are right, its own are not finite."""
    rng = np.random.default_rng(8)
    for lens in ([65, 200], [128, 64]):
        tables, cache, q = decode_case(rng, lens, 16, H, Q)
        pool = dev16(cache)
        for i, n in enumerate(lens):
            pool[int(tables[i, (n - 1) // 16]), (n - 1) % 16, 37 + 300 * i] = bad
        ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
        out = run_decode(ops, q, pool, tables, lens, 16, 0.07)
        check(out[:, :-1], ref[:, :-1], tol[:, :-1], False)
        assert not torch.isfinite(out[:, -1]).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_prefill_rows_that_do_not_see_a_value_that_is_not_finite(ops, dt):
    rng = np.random.default_rng(9)
    chunks, bs, H = [(100, 60), (0, 200)], 16, 2
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, bs, H)
    pool = dev16(cache)
    pool[int(tables[0, 130 // bs]), 130 % bs, 5] = float("nan")
    pool[int(tables[1, 150 // bs]), 150 % bs, 200] = float("inf")
    ref, tol = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, [100, 0], tables, 0.07, two=dt == torch.float32)
    out = run_prefill(ops, q, pool, w_k, w_v, cu, [100, 0], tables, bs, 0.07, 200, 200, sum(lens), dt)
    good = np.r_[0:30, 60:210]
    check(out[good], ref[good], tol[good], dt == torch.bfloat16)
    assert torch.isnan(out[30:60]).all() and torch.isnan(out[210:]).all()


def test_weights_of_a_key_that_is_not_finite_stay_with_its_sequence(ops):
    rng = np.random.default_rng(10)
    lens = [200, 150]
    tables, k, q, before = weights_case(rng, lens, 16, 1, 8, 2, 128)
    ref, tol = O.weights(before, q.f32, k.f32, tables, lens, 0.1)
    pool = dev16(k)
    pool[int(tables[0, 3]), 1, 5, 7] = float("nan")
    w = run_weights(ops, before, q, pool, tables, lens, 16, 0.1)
    check(w[1:], ref[1:], tol[1:], False)
    assert torch.isnan(w[0, :200]).all()


def test_rows_behind_the_last_chunk_stay(ops):
    rng = np.random.default_rng(11)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, [(3, 20), (0, 7)], 16, 2)
    more = bf16(np.concatenate([q.f32, rng.standard_normal((5, 2, HEAD + ROPE)).astype(np.float32)]))
    for dt in (torch.float32, torch.bfloat16):
        out = run_prefill(ops, more, dev16(cache), w_k, w_v, cu, [3, 0], tables, 16, 0.07, 20, 23, 30, dt)
        check(out[:27], *O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, [3, 0], tables, 0.07, two=dt == torch.float32),
              dt == torch.bfloat16)
        assert (out[27:] == -7).all()


def test_selected_places_are_what_compaction_takes_for_k_and_v(ops):
    """Weights, selection and compaction over K and V pages, then decode over what is left."""
    rng = np.random.default_rng(12)
    lens, bs, hkv, d = [400, 120], 16, 2, 128
    tables, k, q, before = weights_case(rng, lens, bs, 4, 8, hkv, d)
    v = bf16(rng.standard_normal(k.shape))
    w = run_weights(ops, np.zeros_like(before), q, dev16(k), tables, lens, bs, 0.09)
    counts, first = [100, 57], np.array([8, 0], np.int32)
    keep, after = run_select(ops, w.cpu().numpy(), first, lens, counts, 16)
    kc, vc = dev16(k), dev16(v)
    cu = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_compact_tokens(kc, vc, dev(tables), dev(first), dev(keep), cu, 100, status=status)
    assert int(status.item()) == 0
    for i, part in enumerate(np.split(keep, [counts[0]])):
        held = np.r_[0:first[i], part]
        t = np.arange(len(held))
        for pool, old in ((kc, k), (vc, v)):
            got = pool.float().cpu().numpy()[tables[i, t // bs], :, t % bs]
            assert np.array_equal(got, old.f32[tables[i, held // bs], :, held % bs])


def test_empty_calls(ops):
    e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    i32 = lambda *s: e(*s, dtype=torch.int32)
    cache = e(4, 16, ROW)
    ops.pa_reshape_and_cache_latent(e(0, LATENT), e(0, ROPE), e(0, dtype=torch.int64), cache)
    ops.pa_copy_blocks_latent(cache, e(0, 2, dtype=torch.int64))
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    ops.pa_decode_latent(e(0, 8, LATENT), e(0, 8, ROW), cache, i32(0, 2), i32(0), 0.1, 16, ws)
    ops.pa_prefill_latent(e(0, 2, HEAD), e(0, 2, HEAD + ROPE), cache, e(2, HEAD, LATENT), e(2, HEAD, LATENT), i32(2), i32(1), i32(1, 2),
                          0.1, 4, 16, 16, ws)
    ops.pa_accumulate_weights(e(0, 16, dtype=torch.float32), e(0, 8, ROW), cache, i32(0, 2), i32(0), 0.1, 1, 16, ws)
    ops.pa_select_tokens(i32(0), i32(1), e(0, 16, dtype=torch.float32), i32(0), i32(0), 4, 16)
    # sequences without tokens: zeros, and nothing added
    out = torch.full((3, 8, LATENT), 7.0, device="cuda")
    wd = ops.make_workspace_latent(3, 1, 8, LATENT, ROPE, 16, 16)
    ops.pa_decode_latent(out, e(3, 8, ROW), cache, i32(3, 2), i32(3), 0.1, 16, wd)
    assert (out == 0).all()
    w = torch.ones(3, 16, device="cuda")
    ww = ops.make_workspace_weights(3, 1, 8, 1, ROW, 16, 16)
    ops.pa_accumulate_weights(w, e(3, 8, ROW), cache, i32(3, 2), i32(3), 0.1, 1, 16, ww)
    assert (w == 1).all()
