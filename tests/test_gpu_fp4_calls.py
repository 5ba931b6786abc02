"""Calls of the 4-bit cache that its documentation allows around the plain
ones: one workspace for calls of many shapes, captured graphs beside eager
calls, other streams, pools past 2^31 bytes, batches past one launch, softmax
scales of any sign, rows behind the last chunk."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp4
from fp4_case import attention_bound, bf16, pool
from paged_case import to_device, to_f64
from test_gpu_fp4 import KS, VS, _attention_case, _check, _decode, _dev, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def test_one_workspace_for_many_shapes(ops):
    """Batches, lengths, groups and chunk sizes change from call to call over a
    workspace that was zeroed once."""
    rng = np.random.default_rng(1)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    shapes = [(4, 8, 128, 16, [700] * 6), (1, 2, 64, 8, [3000, 5]), (16, 1, 128, 32, [2500]), (4, 8, 128, 16, [9, 4000]),
              (2, 1, 256, 16, [1900]), (4, 8, 128, 16, [700] * 6)]
    for G, hkv, d, bs, lens in shapes:
        tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
        q = bf16(rng.standard_normal((len(lens), G * hkv, d)))
        ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.1, range(len(lens)), lens)
        _check(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, 0.1, hkv, ws=ws), ref, tol)
        if d != 128:
            continue
        for n in (1, 70):  # the same sequences' last tokens as a chunk, through the same workspace
            n = min(n, min(lens))
            chunks = [(x - n, n) for x in lens]
            qp = bf16(rng.standard_normal((n * len(lens), G * hkv, d)))
            cu = np.arange(0, n * len(lens) + 1, n, dtype=np.int32)
            out = torch.full(qp.shape, float("nan"), device="cuda")
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            ops.pa_prefill_fp4(out, to_device(qp), _dev(kc), _dev(vc), _dev(cu),
                               _dev(np.array([s for s, _ in chunks], np.int32)), _dev(tables), 0.1, hkv, bs, n, max(lens),
                               ws, KS, VS, status=st)
            rows = [(i, s + j + 1) for i, (s, c) in enumerate(chunks) for j in range(c)]
            pick = sorted({0, len(rows) - 1, *rng.integers(0, len(rows), 12).tolist()})
            ref, tol = _reference(qp.f32[pick], tables, kc, vc, bs, d, 0.1, [rows[r][0] for r in pick],
                                  [rows[r][1] for r in pick])
            assert int(st.item()) == 0
            _check(out[torch.tensor(pick, device="cuda")], ref, tol)
    assert ops.pa_workspace_error(ws) == 0


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 3.0])
def test_decode_with_any_softmax_scale(ops, scale):
    rng = np.random.default_rng(2)
    lens, d, bs = [100, 1, 70], 128, 16
    tables, kc, vc = _attention_case(rng, lens, 4, 2, d, bs)
    q = bf16(rng.standard_normal((3, 8, d)))
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, scale, range(3), lens)
    _check(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, scale, 2), ref, tol)


def test_pool_past_2_to_the_31_bytes(ops):
    """Blocks at the far end of pools of more than 2^31 bytes: append, gather,
    decode, prefill, copy and compaction."""
    rng = np.random.default_rng(3)
    hkv, bs, d, G, n = 8, 16, 128, 4, 75
    tile = fp4.tile_bytes(bs, d)
    nb = (1 << 31) // (hkv * tile) + 100
    kc, vc = ops.make_cache_fp4(nb, hkv, bs, d), ops.make_cache_fp4(nb, hkv, bs, d)
    table = np.array([[nb - 1, 3, nb - 7, nb - 2, nb - 50]], dtype=np.int32)
    k, v = (bf16(rng.standard_normal((n, hkv, d))) for _ in range(2))
    pos = np.arange(n)
    slots = table[0, pos // bs].astype(np.int64) * bs + pos % bs
    ops.pa_reshape_and_cache_fp4(to_device(k), to_device(v), _dev(slots), kc, vc, bs, KS, VS)
    K, V = fp4.dequantise(*fp4.quantise(k.f32, KS), KS), fp4.dequantise(*fp4.quantise(v.f32, VS), VS)
    ko, vo = (torch.zeros(n, hkv, d, device="cuda") for _ in range(2))
    ops.pa_gather_cache_fp4(ko, vo, _dev(slots), kc, vc, bs, KS, VS)
    assert np.array_equal(to_f64(ko), K) and np.array_equal(to_f64(vo), V)
    q = bf16(rng.standard_normal((n, G * hkv, d)))
    got = _decode(ops, q[n - 1:], table, [n], kc, vc, bs, 0.1, hkv)
    ref = oracle.contiguous_attention(q.f32[n - 1], K, V, 0.1)
    tol = attention_bound(q.f32[n - 1].astype(np.float64), K, V, 0.1)[:, None]
    _check(got[0], ref, tol)
    ws = ops.make_prefill_workspace_fp4(1, G * hkv, hkv, d, bs, n, n)
    out = torch.zeros(n, G * hkv, d, device="cuda")
    ops.pa_prefill_fp4(out, to_device(q), kc, vc, _dev(np.array([0, n], np.int32)), _dev(np.array([0], np.int32)),
                       _dev(table), 0.1, hkv, bs, n, n, ws, KS, VS)
    _check(out[n - 1], ref, tol)
    ops.pa_copy_blocks(kc, vc, _dev(np.array([[nb - 1, nb - 3]], np.int64)), block_size=bs, head_dim=d)
    table2 = table.copy()
    table2[0, 0] = nb - 3
    _check(_decode(ops, q[n - 1:], table2, [n], kc, vc, bs, 0.1, hkv)[0], ref, tol)
    keep = [9, 20, 40, 70]
    ops.pa_compact_tokens(kc, vc, _dev(table2), _dev(np.array([2], np.int32)), _dev(np.array(keep, np.int32)),
                          _dev(np.array([0, 4], np.int32)), 4, bs, d)
    kept = [0, 1] + keep
    ref = oracle.contiguous_attention(q.f32[0], K[kept], V[kept], 0.1)
    tol = attention_bound(q.f32[0].astype(np.float64), K[kept], V[kept], 0.1)[:, None]
    _check(_decode(ops, q[:1], table2, [6], kc, vc, bs, 0.1, hkv)[0], ref, tol)


def test_prefill_batches_past_one_launch(ops):
    """More sequences than one launch takes, empty ones at both ends and between."""
    rng = np.random.default_rng(4)
    S, hkv, G, bs, d = 5000, 1, 2, 16, 128
    n = rng.integers(0, 3, size=S)
    n[[0, 1, 4095, 4096, 4097, S - 1]] = 0
    start = rng.integers(0, 20, size=S)
    need = -(-(start + n) // bs)
    m = int(need.max())
    nb = 64
    tables = rng.integers(0, nb, size=(S, m)).astype(np.int32)  # sequences share blocks freely: only read
    kc, vc = pool(rng, nb, hkv, bs, d, KS), pool(rng, nb, hkv, bs, d, VS)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = bf16(rng.standard_normal((int(cu[-1]) + 3, G * hkv, d)))
    ws = ops.make_prefill_workspace_fp4(S, G * hkv, hkv, d, bs, 2, 22)
    out = torch.full(q.shape, 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_prefill_fp4(out, to_device(q), _dev(kc), _dev(vc), _dev(cu), _dev(start.astype(np.int32)), _dev(tables), 0.1,
                       hkv, bs, 2, 22, ws, KS, VS, status=st)
    assert int(st.item()) == 0 and bool((out[cu[-1]:] == 5.0).all())  # rows behind the last chunk stay
    rows = [(i, start[i] + j + 1) for i in range(S) for j in range(n[i])]
    pick = sorted({0, len(rows) - 1, *rng.integers(0, len(rows), 300).tolist()})
    ref, tol = _reference(q.f32[pick], tables, kc, vc, bs, d, 0.1, [rows[r][0] for r in pick], [rows[r][1] for r in pick])
    _check(out[torch.tensor(pick, device="cuda")], ref, tol)


def test_two_streams_and_captured_prefill(ops):
    """Decode and prefill at the same time on two streams with workspaces of
    their own; the prefill captured and replayed with other chunk lengths."""
    rng = np.random.default_rng(5)
    lens, G, hkv, bs, d = [900, 40, 333], 4, 8, 16, 128
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    H = G * hkv
    k, v, t = _dev(kc), _dev(vc), _dev(tables)
    q1, q2 = bf16(rng.standard_normal((3, H, d))), bf16(rng.standard_normal((60, H, d)))
    d1, d2, n1 = to_device(q1), to_device(q2), _dev(np.array(lens, np.int32))
    o1, o2 = torch.zeros(3, H, d, device="cuda"), torch.zeros(60, H, d, device="cuda")
    w1 = ops.make_workspace_fp4(3, H, hkv, d, bs, 900)
    w2 = ops.make_prefill_workspace_fp4(3, H, hkv, d, bs, 40, 900)
    chunks = [(860, 40), (35, 5), (318, 15)]
    cu = _dev(np.array([0, 40, 45, 60], np.int32))
    start = _dev(np.array([s for s, _ in chunks], np.int32))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pre = lambda: ops.pa_prefill_fp4(o2, d2, k, v, cu, start, t, 0.1, hkv, bs, 40, 900, w2, KS, VS, status=st)
    dec = lambda: ops.pa_decode_fp4(o1, d1, k, v, t, n1, 0.1, hkv, bs, 900, w1, KS, VS)
    pre()
    dec()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pre()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            dec()
        with torch.cuda.stream(s2):
            g.replay()
    torch.cuda.synchronize()

    def check_prefill(chunks):
        rows = [(i, s + j + 1) for i, (s, c) in enumerate(chunks) for j in range(c)]
        ref, tol = _reference(q2.f32[:len(rows)], tables, kc, vc, bs, d, 0.1, [r[0] for r in rows], [r[1] for r in rows])
        _check(o2[:len(rows)], ref, tol)

    check_prefill(chunks)
    ref, tol = _reference(q1.f32, tables, kc, vc, bs, d, 0.1, range(3), lens)
    _check(o1, ref, tol)
    chunks = [(0, 3), (0, 40), (200, 0)]
    cu.copy_(torch.tensor([0, 3, 43, 43], dtype=torch.int32))
    start.copy_(torch.tensor([0, 0, 200], dtype=torch.int32))
    o2.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    check_prefill(chunks)
    assert int(st.item()) == 0 and bool(torch.isnan(o2[43:]).all())


@pytest.mark.parametrize("ks,vs", [(2.0 ** -32, 2.0 ** 32), (1.0, 1.0), (2.0 ** 10, 2.0 ** -20)])
def test_extreme_global_scales(ops, ks, vs):
    rng = np.random.default_rng(6)
    n, hkv, bs, d, G = 40, 2, 16, 64, 2
    k, v = (rng.standard_normal((n, hkv, d)) * ks * 8).astype(np.float32), (rng.standard_normal((n, hkv, d)) * vs * 8).astype(
        np.float32)
    kc, vc = ops.make_cache_fp4(3, hkv, bs, d), ops.make_cache_fp4(3, hkv, bs, d)
    slots = np.arange(n, dtype=np.int64)
    ops.pa_reshape_and_cache_fp4(_dev(k), _dev(v), _dev(slots), kc, vc, bs, ks, vs)
    K, V = fp4.dequantise(*fp4.quantise(k, ks), ks), fp4.dequantise(*fp4.quantise(v, vs), vs)
    ko, vo = (torch.zeros(n, hkv, d, device="cuda") for _ in range(2))
    ops.pa_gather_cache_fp4(ko, vo, _dev(slots), kc, vc, bs, ks, vs)
    assert np.array_equal(to_f64(ko), K) and np.array_equal(to_f64(vo), V)
    q = bf16(rng.standard_normal((1, G * hkv, d)) / 8)
    scale = 0.25 / ks if ks < 1 else 0.25 / ks
    ws = ops.make_workspace_fp4(1, G * hkv, hkv, d, bs, n)
    out = torch.zeros(1, G * hkv, d, device="cuda")
    ops.pa_decode_fp4(out, to_device(q), kc, vc, _dev(np.array([[0, 1, 2]], np.int32)), _dev(np.array([n], np.int32)),
                      scale, hkv, bs, n, ws, ks, vs)
    ref = oracle.contiguous_attention(q.f32[0], K, V, scale)
    tol = attention_bound(q.f32[0].astype(np.float64), K, V, scale)[:, None]
    _check(out[0], ref, tol)


def test_tables_wider_than_the_lengths(ops):
    """max_context_len is a bound: the tables and it may be far larger than any
    length, and the entries behind a sequence's pages are never read."""
    rng = np.random.default_rng(7)
    lens, d, bs, hkv, G = [33, 0, 129, 16], 128, 16, 2, 4
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    wide = np.full((4, 2048), 1 << 30, dtype=np.int32)
    wide[:, :tables.shape[1]] = np.where(tables < 0, 1 << 30, tables)
    q = bf16(rng.standard_normal((4, G * hkv, d)))
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.1, range(4), lens)
    _check(_decode(ops, q, wide, lens, _dev(kc), _dev(vc), bs, 0.1, hkv, max_len=32768), ref, tol)


def test_refusals_of_the_binding(ops):
    hkv, bs, d, G = 2, 16, 128, 4
    kc, vc = ops.make_cache_fp4(4, hkv, bs, d), ops.make_cache_fp4(4, hkv, bs, d)
    q = torch.zeros(2, G * hkv, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    t, n = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    ws = ops.make_workspace_fp4(2, G * hkv, hkv, d, bs, 32)
    good = dict(out=out, q=q, k_cache=kc, v_cache=vc, block_tables=t, context_lens=n, scale=0.1, num_kv_heads=hkv,
                block_size=bs, max_context_len=32, workspace=ws)
    ops.pa_decode_fp4(**good)
    for change in (dict(q=q.float()), dict(out=out[:1]), dict(out=out.half()), dict(k_cache=kc[:, :1]), dict(block_size=8),
                   dict(num_kv_heads=1), dict(block_tables=t.long()), dict(block_tables=t[:1]), dict(context_lens=n[:1]),
                   dict(context_lens=n.cpu()), dict(workspace=ws.float()), dict(q=q.transpose(0, 1)),
                   dict(k_cache=kc.cpu()), dict(v_cache=kc.to(torch.int8))):
        with pytest.raises(ValueError):
            ops.pa_decode_fp4(**{**good, **change})
    for change in (dict(max_context_len=33), dict(workspace=ws[:300]), dict(k_scale=0.3), dict(scale=float("inf"))):
        with pytest.raises(ops.PAError):
            ops.pa_decode_fp4(**{**good, **change})
    x = torch.zeros(3, hkv, d, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in ((x.half(), x.half(), slots), (x, x[:2], slots), (x, x, slots.int()), (x, x, slots[:2]),
                (x.transpose(0, 1), x.transpose(0, 1), slots[:2])):
        with pytest.raises(ValueError):
            ops.pa_reshape_and_cache_fp4(*bad, kc, vc, bs)
    pad = torch.zeros(3 * hkv * d + 4, device="cuda")[4:].view(3, hkv, d)  # 16-byte aligned only
    with pytest.raises(ops.PAError):
        ops.pa_reshape_and_cache_fp4(pad, x, slots, kc, vc, bs)
    torch.cuda.synchronize()


def test_prefill_nan_reaches_the_rows_that_see_it(ops):
    """NaN groups of keys and of values inside the chunk and before it: rows in
    front of the token are finite, rows behind it are NaN, in all dims for a
    key and in the group's 16 for a value; also where an item is split."""
    rng = np.random.default_rng(8)
    G, hkv, bs, d = 4, 2, 16, 128
    for start, n, at_k, at_v in ((0, 150, 40, 100), (5000, 90, 5050, 5003), (0, 300, 299, 0)):
        tables, kc, vc = _attention_case(rng, [start + n], G, hkv, d, bs)

        def spoil(c, pos, head, group):
            c[tables[0, pos // bs], head, bs * 64 + (pos % bs) * 8 + group] = 0x7f

        spoil(kc, at_k, 0, 3)
        spoil(vc, at_v, 1, 5)
        spoil(vc, at_v, 1, 0)
        q = bf16(rng.standard_normal((n, G * hkv, d)))
        ws = ops.make_prefill_workspace_fp4(1, G * hkv, hkv, d, bs, n, start + n)
        out = torch.zeros(n, G * hkv, d, device="cuda")
        ops.pa_prefill_fp4(out, to_device(q), _dev(kc), _dev(vc), _dev(np.array([0, n], np.int32)),
                           _dev(np.array([start], np.int32)), _dev(tables), 0.1, hkv, bs, n, start + n, ws, KS, VS)
        want = np.zeros(out.shape, dtype=bool)
        rows = np.arange(start, start + n)
        want[rows >= at_k, :G] = True
        for g in (0, 5):
            want[rows >= at_v, G:, 16 * g:16 * g + 16] = True
        got = to_f64(out)
        assert np.array_equal(np.isnan(got), want)
        pick = [r for r in sorted({0, n - 1, n // 2}) if start + r < min(at_k, at_v)]
        if pick:
            ref, tol = _reference(q.f32[pick], tables, kc, vc, bs, d, 0.1, [0] * len(pick), [start + r + 1 for r in pick])
            _check(out[torch.tensor(pick, device="cuda")], ref, tol)


def test_many_short_items(ops):
    """Items of a single step, several hundred for every CTA, NaN values in some."""
    rng = np.random.default_rng(9)
    S, G, hkv, bs, d = 3000, 1, 16, 8, 128
    nb = 40
    tables = rng.integers(0, nb, size=(S, 1)).astype(np.int32)
    kc, vc = pool(rng, nb, hkv, bs, d, KS), pool(rng, nb, hkv, bs, d, VS)
    bad, clean = [3, 17], vc.copy()
    for b in bad:
        vc[b, 5, bs * 64 + 6 * 8 + 2] = 0x7f  # token 6 of the block, head 5, group 2
    n = rng.integers(1, 9, size=S)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = bf16(rng.standard_normal((int(cu[-1]), G * hkv, d)))
    ws = ops.make_prefill_workspace_fp4(S, G * hkv, hkv, d, bs, 8, 8)
    out = torch.zeros(q.shape, device="cuda")
    ops.pa_prefill_fp4(out, to_device(q), _dev(kc), _dev(vc), _dev(cu), _dev(np.zeros(S, np.int32)), _dev(tables), 0.1,
                       hkv, bs, 8, 8, ws, KS, VS)
    got = to_f64(out)
    want = np.zeros(got.shape, dtype=bool)
    for i in range(S):
        if tables[i, 0] in bad and n[i] > 6:
            want[cu[i] + 6:cu[i + 1], 5, 32:48] = True
    assert np.array_equal(np.isnan(got), want)
    rows = [(i, j + 1) for i in range(S) for j in range(n[i])]
    pick = [r for r in sorted({0, len(rows) - 1, *rng.integers(0, len(rows), 200).tolist()}) if not want[r].any()]
    ref, tol = _reference(q.f32[pick], tables, kc, clean, bs, d, 0.1, [rows[r][0] for r in pick],
                          [rows[r][1] for r in pick])
    keep = [k for k, r in enumerate(pick) if tables[rows[r][0], 0] not in bad]
    _check(out[torch.tensor([pick[k] for k in keep], device="cuda")], ref[keep], tol[keep])


def test_contexts_of_millions_of_tokens(ops):
    """Positions around 6 million (their pages repeat, so a key's weight is the
    number of times that a row sees it): decode, and a chunk of several tiles."""
    rng = np.random.default_rng(8)
    nb, bs, d, G, n, start, scale = 64, 256, 128, 16, 40, 6_000_037, 0.1
    period = nb * bs
    kc, vc = pool(rng, nb, 1, bs, d, KS), pool(rng, nb, 1, bs, d, VS)
    order = rng.permutation(nb).astype(np.int32)
    end = start + n
    m = -(-end // bs)
    tables = np.resize(order, (1, m)).astype(np.int32)
    K = oracle.gather_sequence(fp4.values(kc, bs, d, KS), order, period)[:, 0]
    V = oracle.gather_sequence(fp4.values(vc, bs, d, VS), order, period)[:, 0]

    def reference(q, pos):
        s = scale * (q.astype(np.float64) @ K.T)
        count = (pos - np.arange(period)) // period + 1
        w = count * np.exp(s - s.max(axis=1, keepdims=True))
        return (w / w.sum(axis=1, keepdims=True)) @ V

    # attention_bound counts one period's keys.  An accumulator takes those of
    # a CTA's share: at least 100 CTAs share 3 tiles' rows of `end` keys.
    more = 3 * end / 100 * 2.0 ** -23 * float(np.abs(V).max())

    def check(out, q, pos):
        tol = attention_bound(q.astype(np.float64), K[:, None], V[:, None], scale) + more
        _check(out, reference(q, pos), tol[:, None])

    q = bf16(rng.standard_normal((n, G, d)))
    ws = ops.make_prefill_workspace_fp4(1, G, 1, d, bs, n, end)
    out = torch.full(q.shape, float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_prefill_fp4(out, to_device(q), _dev(kc), _dev(vc), _dev(np.array([0, n], np.int32)),
                       _dev(np.array([start], np.int32)), _dev(tables), scale, 1, bs, n, end, ws, KS, VS, status=st)
    assert int(st.item()) == 0
    for t in (0, 15, 16, 31, 32, n - 1):
        check(out[t], q.f32[t], start + t)
    got = _decode(ops, bf16(q.f32[:1]), tables, [end], _dev(kc), _dev(vc), bs, scale, 1)
    check(got[0], q.f32[0], end - 1)


def test_calls_behind_one_another(ops):
    """Each call of a chain reads what the one before it writes, without a
    synchronisation between them; eager, then captured and replayed."""
    rng = np.random.default_rng(9)
    S, n, hkv, bs, d = 8, 600, 4, 16, 128
    m = -(-n // bs)
    tables = rng.permutation(S * m).reshape(S, m).astype(np.int32)
    keep = [np.sort(rng.permutation(n)[:n // 2]) for _ in range(S)]
    t = np.arange(n)
    slots = np.concatenate([tables[i][t // bs].astype(np.int64) * bs + t % bs for i in range(S)])
    kept = np.concatenate([slots[i * n:(i + 1) * n][:n // 2] for i in range(S)])
    rounds = 6
    keys = [bf16(rng.standard_normal((S * n, hkv, d)) * 2.0 ** r) for r in range(rounds)]
    dev = [to_device(x) for x in keys]
    kc, vc = (ops.make_cache_fp4(S * m, hkv, bs, d) for _ in range(2))
    outs = [[torch.zeros((S * n // 2, hkv, d), device="cuda") for _ in range(2)] for _ in range(rounds)]
    args = (_dev(tables), torch.zeros(S, dtype=torch.int32, device="cuda"),
            _dev(np.concatenate(keep).astype(np.int32)), _dev(np.arange(S + 1, dtype=np.int32) * (n // 2)))
    slots_dev, kept_dev = _dev(slots), _dev(kept)

    def chain():
        for r in range(rounds):
            ops.pa_reshape_and_cache_fp4(dev[r], dev[-1 - r], slots_dev, kc, vc, bs)
            ops.pa_compact_tokens(kc, vc, *args, n // 2, bs, d)
            ops.pa_gather_cache_fp4(*outs[r], kept_dev, kc, vc, bs)

    moved = np.concatenate([i * n + keep[i] for i in range(S)])

    def check():
        for r in range(rounds):
            for out, x in zip(outs[r], (keys[r], keys[-1 - r])):
                codes, scales = fp4.quantise(x.f32[moved], 1.0)
                assert np.array_equal(to_f64(out), fp4.dequantise(codes, scales, 1.0))

    chain()
    check()
    for pair in outs:
        for out in pair:
            out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        chain()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check()


@pytest.mark.parametrize("G,hkv,max_q", [(4, 8, 1 << 30), (16, 1, 1 << 28), (8, 2, (1 << 31) - 1), (1, 3, 1 << 29)])
def test_prefill_with_a_loose_bound_of_the_chunks(ops, G, hkv, max_q):
    """max_q_len far above every chunk: the results of the tight bound, from a
    workspace of the size asked for, nothing behind it written."""
    rng = np.random.default_rng(G)
    chunks, bs, d = [(3000, 70), (0, 300), (0, 0), (900, 1)], 16, 128
    lens = [s + c for s, c in chunks]
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    n = [c for _, c in chunks]
    q = to_device(bf16(rng.standard_normal((sum(n), G * hkv, d))))
    cu, start = _dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)), _dev(np.array([s for s, _ in chunks], np.int32))
    kd, vd, td = _dev(kc), _dev(vc), _dev(tables)
    outs = []
    for mq in (max(n), max_q):
        need = ops.make_prefill_workspace_fp4(4, G * hkv, hkv, d, bs, mq, max(lens)).numel()
        room = torch.full((need + (1 << 22),), 0x5a, dtype=torch.uint8, device="cuda")
        room[:need] = 0
        out = torch.full(q.shape, float("nan"), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_prefill_fp4(out, q, kd, vd, cu, start, td, 0.1, hkv, bs, mq, max(lens), room[:need], KS, VS, status=st)
        assert int(st.item()) == 0 and bool((room[need:] == 0x5a).all())
        outs.append(out)
    assert bool(torch.isfinite(outs[0]).all()) and torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("G,hkv,S", [(16, 1, 4000), (8, 3, 3000), (16, 4, 2500)])
def test_items_of_two_tiles_between_items_of_one(ops, G, hkv, S):
    """Chunks that fill two tiles, with NaN values in some, in front of runs of
    chunks that fill one: the notes of the former reach their rows and no
    others, call after call."""
    rng = np.random.default_rng(10 * G + hkv)
    bs, d, nb, tile = 8, 128, 48, 128 // G
    n = rng.integers(1, tile + 1, size=S)
    two = rng.random(S) < 0.15
    n[two] = rng.integers(tile + 1, 2 * tile + 1, size=int(two.sum()))
    m = 2 * tile // bs
    tables = rng.integers(0, nb, size=(S, m)).astype(np.int32)
    kc, vc = pool(rng, nb, hkv, bs, d, KS), pool(rng, nb, hkv, bs, d, VS)
    bad = [3, 17, 30, 31]
    spoilt = {b: (int(rng.integers(0, bs)), int(rng.integers(0, hkv)), int(rng.integers(0, 8))) for b in bad}
    for b, (tok, head, group) in spoilt.items():
        vc[b, head, bs * 64 + tok * 8 + group] = 0x7f
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = bf16(rng.standard_normal((int(cu[-1]), G * hkv, d)))
    want = np.zeros(q.shape, dtype=bool)
    for i in range(S):
        for j in range(m):
            if int(tables[i, j]) in spoilt:
                tok, head, group = spoilt[int(tables[i, j])]
                want[cu[i] + j * bs + tok:cu[i + 1], head * G:(head + 1) * G, 16 * group:16 * group + 16] = True
    rows = [(i, j + 1) for i in range(S) for j in range(n[i])]
    pick = [r for r in sorted({0, len(rows) - 1, *rng.integers(0, len(rows), 150).tolist()}) if not want[r].any()
            and not set(tables[rows[r][0]].tolist()) & set(bad)]
    ref, tol = _reference(q.f32[pick], tables, kc, vc, bs, d, 0.1, [rows[r][0] for r in pick],
                          [rows[r][1] for r in pick])
    ws = ops.make_prefill_workspace_fp4(S, G * hkv, hkv, d, bs, 2 * tile, 2 * tile)
    qd, kd, vd, cd, td = to_device(q), _dev(kc), _dev(vc), _dev(cu), _dev(tables)
    zero = torch.zeros(S, dtype=torch.int32, device="cuda")
    for _ in range(5):
        out = torch.zeros(q.shape, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_prefill_fp4(out, qd, kd, vd, cd, zero, td, 0.1, hkv, bs, 2 * tile, 2 * tile, ws, KS, VS, status=st)
        assert int(st.item()) == 0
        assert np.array_equal(np.isnan(to_f64(out)), want)
        _check(out[torch.tensor(pick, device="cuda")], ref, tol)


def test_single_keys_among_millions(ops):
    """Every query is aligned with one of 60 keys planted among 6 million, so
    its output is that key's value: at the first and last token, around the
    chunk and past 5.9 million among them.  Rows in front of their key do not
    see it, and average the others.

    A planted key's score is 0.1 * 384 = 38.4 and no other key's comes near
    it, so its weight is 1 - rest with a rest that the reference knows.  Then
    the output is off by half a step of the weight's f16, 2^-12, the
    exponential's 2^-21 and a few fp32 roundings (2^-20 together) and the rest's
    own errors (at most 2 of each: as much again) of max |V|.  No other
    addition counts: what came before the key is scaled by exp(-38) when the
    reference is raised to it, and what comes after is 0 in f16."""
    rng = np.random.default_rng(21)
    nb, ns, bs, d, G, n, start, scale = 64, 60, 256, 128, 16, 40, 6_000_037, 0.1
    end = start + n
    m = -(-end // bs)
    kc, vc = pool(rng, nb + ns, 1, bs, d, KS), pool(rng, nb + ns, 1, bs, d, VS)
    # pages: shared ones, and one of its own for every planted key
    last = (end - 1) // bs
    own = np.unique(np.concatenate([[0, 1, start // bs - 1, start // bs, last],
                                    rng.choice(np.arange(5_900_000 // bs, last - 2), 20, replace=False),
                                    rng.choice(np.arange(2, 5_900_000 // bs), 45, replace=False)]))
    own = np.concatenate([own[:2], rng.permutation(own[2:-3])[:ns - 5], own[-3:]])[:ns]
    tables = np.resize(rng.permutation(nb), m).astype(np.int32)
    tables[own] = nb + np.arange(len(own))
    off = rng.integers(0, bs, size=len(own))
    off[own == 0] = 0
    off[own == last] = (end - 1) % bs
    off[own == start // bs] = min(bs - 1, start % bs + n // 2)   # inside the chunk, if its page goes so far
    place = own * bs + off
    u = rng.choice([-1.0, 1.0], size=(len(own), d)).astype(np.float32)
    val = rng.choice([-1.5, 1.5], size=(len(own), d)).astype(np.float32)
    slots = (nb + np.arange(len(own), dtype=np.int64)) * bs + off
    fp4.reshape_and_cache((3 * u)[:, None], kc, slots, bs, KS)
    fp4.reshape_and_cache(val[:, None], vc, slots, bs, VS)
    K, V = (fp4.values(c, bs, d, s)[:, 0].reshape(-1, d) for c, s in ((kc, KS), (vc, VS)))
    assert np.array_equal(K[slots], 3 * u) and np.array_equal(V[slots], val)
    uses = [np.flatnonzero(tables == b) for b in range(nb + ns)]   # the pages of every block, ascending
    vmax = float(np.abs(V).max())

    def reference(target, pos):
        """The outputs of queries u[target] [H] at position pos, and their bounds."""
        count = np.zeros((nb + ns, bs))
        for b, pages in enumerate(uses):
            whole = np.searchsorted(pages, (pos + 1) // bs)        # pages that end before pos
            count[b] = whole
            if whole < len(pages) and pages[whole] == (pos + 1) // bs:
                count[b, :(pos + 1) % bs] += 1
        count = count.reshape(-1)
        assert count.sum() == pos + 1
        s = scale * (u[target].astype(np.float64) @ K.T)
        s[:, count == 0] = -np.inf
        w = count * np.exp(s - s.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        seen = place[target] <= pos
        rest = 1 - w[np.arange(len(target)), slots[target]]
        assert (rest[seen] < 1e-6).all()
        tight = vmax * (2.0 ** -12 + 2.0 ** -20 + 2 * rest)
        # without the planted key: fp32 sums over a CTA's share of the keys, of which 100 CTAs or more have 3 tiles' rows
        ds = (d + 4) * 2.0 ** -23 * scale * float(np.abs(K).sum(axis=1).max())  # a score's, as in attention_bound
        loose = vmax * (2 * ds + 2.0 ** -21 + 2.0 ** -12 + 3 * end / 100 * 2.0 ** -23)
        return w @ V, np.where(seen, tight, loose), seen

    def check(out, target, pos):
        ref, tol, seen = reference(target, pos)
        # the bounds tell the outputs from zeros, from other keys' and from the key left out or let in
        assert (np.abs(ref[seen]) > 1.4).all() and (tol < 0.1).all() and (np.abs(ref[~seen]) < 1.0).all()
        for a, b in ((a, b) for a in range(len(target)) for b in range(a) if target[a] != target[b] and seen[a] and seen[b]):
            assert np.abs(ref[a] - ref[b]).max() > 2.5
        _check(out, ref, tol[:, None])
        return int(seen.sum()), int((~seen).sum())

    kd, vd = _dev(kc), _dev(vc)
    # single tokens: four sequences over the same pages
    lens = [end, end - 1, 5_900_003, start]
    target = np.resize(rng.permutation(len(own)), (4, G))
    target[0, :2] = [int(np.argmax(place)), int(np.argmin(place))]
    got = _decode(ops, bf16(u[target]), np.tile(tables, (4, 1)), lens, kd, vd, bs, scale, 1)
    for i in range(4):
        check(got[i], target[i], lens[i] - 1)
    # a chunk: every planted key is some row's, those inside the chunk several rows'
    target = np.resize(rng.permutation(len(own)), (n, G))
    inside = np.flatnonzero(place >= start)
    target[:, :len(inside)] = inside
    ws = ops.make_prefill_workspace_fp4(1, G, 1, d, bs, n, end)
    out = torch.full((n, G, d), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_prefill_fp4(out, to_device(bf16(u[target])), kd, vd, _dev(np.array([0, n], np.int32)),
                       _dev(np.array([start], np.int32)), _dev(tables[None]), scale, 1, bs, n, end, ws, KS, VS, status=st)
    assert int(st.item()) == 0
    done = [check(out[t], target[t], start + t) for t in range(n)]
    assert len(inside) >= 1 and sum(b for _, b in done) >= n // 2 and sum(a for a, _ in done) > 400
