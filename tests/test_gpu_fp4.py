"""The 4-bit cache on the GPU against its float64 definition: the bytes that
the append writes, the values read back, attention of single tokens and of
chunks, block copies, and all of them in a row."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp4
from fp4_case import attention_bound, bf16, pool
from paged_case import bf16_half_ulp, to_device, to_f64

pytestmark = pytest.mark.gpu
KS, VS = 0.0625, 0.03125


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------
def _special_rows(rng, t, hkv, d):
    """Normal rows, among them zeros, tiny and huge groups, exact halfway cases
    of both roundings, negative zeros, infinities and NaN."""
    x = (rng.standard_normal((t, hkv, d)) * 0.5).astype(np.float32)
    flat = x.reshape(-1, 16)
    r = rng.permutation(len(flat))
    flat[r[0]] = 0
    flat[r[1]] = -0.0
    flat[r[2]] = 1e-30
    flat[r[3]] = 3e38
    flat[r[4], 3] = np.inf
    flat[r[5], 7] = np.nan
    flat[r[6]] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * KS
    flat[r[7]] = np.float32(6 * 17 / 16 * KS)          # a / 6 halfway between 1 and 1.125
    flat[r[8]] = np.float32(6 * 19 / 16 * KS)
    flat[r[9]] = np.nextafter(np.float32(6 * 17 / 16 * KS), np.float32(0))
    flat[r[10]] = np.float32(6 * 2.0 ** -10 * KS)      # halfway between 0 and the smallest scale
    flat[r[11]] = np.float32(6 * 3 * 2.0 ** -10 * KS)
    flat[r[12], 0] = -np.inf
    flat[r[13]] = np.float32(1e-42)
    return x


@pytest.mark.parametrize("d,bs,hkv,t", [(128, 16, 8, 37), (64, 1, 2, 21), (256, 256, 1, 300), (128, 8, 3, 1),
                                        (64, 2, 4, 50), (128, 1, 2, 33)])
@pytest.mark.parametrize("src", ["f32", "bf16"])
def test_append_and_gather(ops, d, bs, hkv, t, src):
    rng = np.random.default_rng(d + bs + t)
    x = _special_rows(rng, t, hkv, d) if t * hkv * d >= 16 * 16 else rng.standard_normal((t, hkv, d))
    y = rng.standard_normal((t, hkv, d)) * 3
    with np.errstate(over="ignore", invalid="ignore"):
        if src == "bf16":
            kx, vx = bf16(x), bf16(y)
            key, value, kf, vf = to_device(kx), to_device(vx), kx.f32, vx.f32
        else:
            kf, vf = np.asarray(x, np.float32), np.asarray(y, np.float32)
            key, value = _dev(kf), _dev(vf)
    nb = -(-t // bs) + 2
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    if t > 4:
        slots[[1, 4]] = -1
    garbage = pool(rng, nb, hkv, bs, d, KS, garbage=True)
    ref_k, ref_v = garbage.copy(), garbage.copy()
    kc, vc = _dev(garbage), _dev(garbage)
    ops.pa_reshape_and_cache_fp4(key, value, _dev(slots), kc, vc, bs, KS, VS)
    with np.errstate(all="ignore"):
        fp4.reshape_and_cache(kf, ref_k, slots, bs, KS)
        fp4.reshape_and_cache(vf, ref_v, slots, bs, VS)
    assert np.array_equal(kc.cpu().numpy(), ref_k)
    assert np.array_equal(vc.cpu().numpy(), ref_v)
    for dt in (torch.float32, torch.bfloat16):
        ko = torch.full((t, hkv, d), 7.0, dtype=dt, device="cuda")
        vo = torch.full_like(ko, 7.0)
        ops.pa_gather_cache_fp4(ko, vo, _dev(slots), kc, vc, bs, KS, VS)
        for got, ref, gs in ((ko, ref_k, KS), (vo, ref_v, VS)):
            want = fp4.values(ref, bs, d, gs)[slots // bs, :, slots % bs]
            want[slots < 0] = 7.0
            assert np.array_equal(to_f64(got), want, equal_nan=True)


def test_slots_past_the_pool_are_reported(ops):
    rng = np.random.default_rng(3)
    nb, hkv, bs, d = 4, 2, 16, 128
    cache = pool(rng, nb, hkv, bs, d, 1.0)
    kc, vc = _dev(cache), _dev(cache)
    x = torch.randn(3, hkv, d, device="cuda")
    slots = _dev(np.array([-1, nb * bs, 5], dtype=np.int64))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_reshape_and_cache_fp4(x, x, slots, kc, vc, bs, status=status)
    assert int(status.item()) == 1
    ref = cache.copy()
    fp4.reshape_and_cache(x.cpu().numpy(), ref, [-1, -1, 5], bs, 1.0)
    assert np.array_equal(kc.cpu().numpy(), ref)
    status.zero_()
    out = torch.full_like(x, 7.0)
    ops.pa_gather_cache_fp4(out, torch.empty_like(out), slots, kc, vc, bs, status=status)
    assert int(status.item()) == 1 and bool((out[:2] == 7.0).all()) and bool((out[2] != 7.0).any())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attention_case(rng, lens, G, hkv, d, bs, sigma=0.5, spare=3):
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    maxb = max(max(need), 1)
    tables = np.full((len(lens), maxb), -7, dtype=np.int32)  # unused entries are never read
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    kc = pool(rng, nb, hkv, bs, d, KS, sigma)
    vc = pool(rng, nb, hkv, bs, d, VS, sigma)
    # rows behind a sequence's last token hold anything
    for i, n in enumerate(lens):
        if n % bs:
            blk, off = tables[i, n // bs], n % bs
            for c in (kc, vc):
                codes, scales = fp4.rows(c[blk:blk + 1].copy(), bs, d)
                codes[:, :, off:] = rng.integers(0, 256, size=codes[:, :, off:].shape, dtype=np.uint8)
                scales[:, :, off:] = rng.choice([0x7f, 0xff, 0x7e, 0x00], size=scales[:, :, off:].shape)
                c[blk, :, :bs * d // 2] = codes.reshape(hkv, -1)
                c[blk, :, bs * d // 2:bs * d * 9 // 16] = scales.reshape(hkv, -1)
    return tables, kc, vc


def _reference(q, tables, kc, vc, bs, d, scale, row_seq, row_len):
    kf, vf = fp4.values(kc, bs, d, KS), fp4.values(vc, bs, d, VS)
    ref = np.zeros(q.shape)
    tol = np.zeros(q.shape[:2])
    for r, (i, n) in enumerate(zip(row_seq, row_len)):
        K = oracle.gather_sequence(kf, tables[i], n)
        V = oracle.gather_sequence(vf, tables[i], n)
        ref[r] = oracle.contiguous_attention(q[r], K, V, scale)
        tol[r] = attention_bound(q[r].astype(np.float64), K, V, scale)
    return ref, tol[:, :, None]


def _check(out, ref, tol):
    got = to_f64(out)
    if out.dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(np.abs(ref) + tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-30))))


def _decode(ops, q, tables, lens, kc, vc, bs, scale, hkv, out_dtype=torch.float32, max_len=None, ws=None):
    B, H, d = q.shape
    max_len = max(int(max(lens)), 0) if max_len is None else max_len
    own = ws is None
    if own:
        ws = ops.make_workspace_fp4(B, H, hkv, d, bs, max_len)
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    ops.pa_decode_fp4(out, to_device(q), kc, vc, _dev(tables), _dev(np.asarray(lens, np.int32)), scale, hkv, bs,
                      max_len, ws, KS, VS)
    torch.cuda.synchronize()
    if own:
        assert ops.pa_workspace_error(ws) == 0
    return out


LENS = [1, 0, 17, 16, 15, 33, 64, 65, 300, 129, 31, 2]


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 8), (256, 32), (128, 1), (128, 4), (64, 256), (256, 64), (128, 128),
                                  (64, 1), (256, 2)])
def test_decode_matches_definition(ops, G, d, bs):
    rng = np.random.default_rng(1000 * G + d + bs)
    hkv = 2 if G < 16 else 1
    tables, kc, vc = _attention_case(rng, LENS, G, hkv, d, bs)
    q = bf16(rng.standard_normal((len(LENS), G * hkv, d)))
    scale = float(np.float32(1 / np.sqrt(d)))
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, scale, range(len(LENS)), LENS)
    for dt in (torch.float32, torch.bfloat16):
        _check(_decode(ops, q, tables, LENS, _dev(kc), _dev(vc), bs, scale, hkv, dt), ref, tol)


@pytest.mark.parametrize("G,hkv,d,bs,lens", [
    (4, 8, 128, 16, [5000]), (8, 1, 128, 32, [20011]), (1, 32, 128, 16, [1500, 3]), (16, 2, 64, 64, [9001, 1]),
    (4, 2, 256, 16, [4097, 4096, 0, 1])])
def test_decode_long_contexts(ops, G, hkv, d, bs, lens):
    rng = np.random.default_rng(sum(lens))
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    q = bf16(rng.standard_normal((len(lens), G * hkv, d)))
    scale = float(np.float32(1 / np.sqrt(d)))
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, scale, range(len(lens)), lens)
    a = _decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, scale, hkv)
    _check(a, ref, tol)
    b = _decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, scale, hkv)
    assert torch.equal(a, b)  # the order of the sums is fixed


def test_decode_many_sequences(ops):
    """More sequences than one pass of the CTAs over their lengths."""
    rng = np.random.default_rng(77)
    lens = rng.integers(0, 40, size=1500).tolist()
    tables, kc, vc = _attention_case(rng, lens, 2, 1, 64, 8)
    q = bf16(rng.standard_normal((len(lens), 2, 64)))
    ref, tol = _reference(q.f32, tables, kc, vc, 8, 64, 0.125, range(len(lens)), lens)
    _check(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), 8, 0.125, 1), ref, tol)


def test_decode_peaked_and_large_scores(ops):
    """Scores that grow along the keys by far more than the exponential's
    range, queries of very different magnitudes, a zero query."""
    rng = np.random.default_rng(5)
    lens, d, bs = [700, 90], 128, 16
    tables, kc, vc = _attention_case(rng, lens, 4, 1, d, bs, sigma=4.0)
    q = rng.standard_normal((2, 4, d)) * np.array([1e-3, 1.0, 30.0, 0.0])[None, :, None]
    q[1, 0] *= 1e-30
    q[1, 2] *= 1e4
    q = bf16(q)
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.3, range(2), lens)
    _check(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, 0.3, 1), ref, tol)


def test_decode_nan_tokens_reach_their_sequence_only(ops):
    rng = np.random.default_rng(6)
    lens, d, bs = [50, 50, 50], 128, 16
    tables, kc, vc = _attention_case(rng, lens, 2, 2, d, bs)
    kc[tables[0, 1], 0, bs * 64 + 3 * 8 + 2] = 0x7f       # sequence 0, kv head 0: a key group
    vc[tables[2, 0], 1, bs * 64 + 5 * 8 + 7] = 0x7f       # sequence 2, kv head 1: a value group
    q = bf16(rng.standard_normal((3, 4, d)))
    got = to_f64(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, 0.1, 2))
    assert np.isnan(got[0, :2]).all() and np.isfinite(got[0, 2:]).all() and np.isfinite(got[1]).all()
    assert np.isfinite(got[2, :2]).all() and np.isnan(got[2, 2:, 112:]).all() and np.isfinite(got[2, 2:, :112]).all()


def test_decode_reports_bad_tables_and_lengths(ops):
    rng = np.random.default_rng(8)
    lens, d, bs = [40, 20], 128, 16
    tables, kc, vc = _attention_case(rng, lens, 4, 2, d, bs)
    q = bf16(rng.standard_normal((2, 8, d)))
    ws = ops.make_workspace_fp4(2, 8, 2, d, bs, 40)
    bad = tables.copy()
    bad[1, 1] = kc.shape[0]
    _decode(ops, q, bad, lens, _dev(kc), _dev(vc), bs, 0.1, 2, max_len=40, ws=ws)
    assert ops.pa_workspace_error(ws) == 1
    _decode(ops, q, tables, [41, -3], _dev(kc), _dev(vc), bs, 0.1, 2, max_len=40, ws=ws)
    assert ops.pa_workspace_error(ws) == 1
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.1, range(2), lens)
    _check(_decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, 0.1, 2, max_len=40, ws=ws), ref, tol)
    assert ops.pa_workspace_error(ws) == 0  # the workspace is as before


def test_decode_graph_replay_and_streams(ops):
    """A captured decode replayed with new lengths, on another stream, between
    eager calls that have a workspace of their own."""
    rng = np.random.default_rng(9)
    lens, d, bs, hkv, G = [900, 33, 64, 257], 128, 16, 8, 4
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    q = bf16(rng.standard_normal((4, G * hkv, d)))
    args = dict(kc=_dev(kc), vc=_dev(vc), t=_dev(tables), q=to_device(q))
    n = _dev(np.asarray(lens, np.int32))
    out = torch.empty(4, G * hkv, d, device="cuda")
    ws = ops.make_workspace_fp4(4, G * hkv, hkv, d, bs, 900)
    call = lambda: ops.pa_decode_fp4(out, args["q"], args["kc"], args["vc"], args["t"], n, 0.1, hkv, bs, 900, ws, KS, VS)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for cut in ([900, 33, 64, 257], [1, 0, 64, 100], [500, 33, 2, 256]):
        n.copy_(torch.tensor(cut, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        eager = _decode(ops, q, tables, cut, args["kc"], args["vc"], bs, 0.1, hkv, max_len=900)
        torch.cuda.synchronize()
        ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.1, range(4), cut)
        _check(out, ref, tol)
        assert torch.equal(out, eager)
    assert ops.pa_workspace_error(ws) == 0


CHUNKS = [(0, 1), (0, 7), (0, 33), (0, 130), (100, 20), (250, 64), (17, 200), (30, 0), (0, 300), (511, 1)]


def _prefill(ops, q, tables, chunks, kc, vc, bs, scale, hkv, out_dtype=torch.float32, max_len=None):
    n = [c for _, c in chunks]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    start = np.array([s for s, _ in chunks], dtype=np.int32)
    T, H, d = q.shape
    max_len = max([s + c for s, c in chunks if c] + [0]) if max_len is None else max_len
    ws = ops.make_prefill_workspace_fp4(len(chunks), H, hkv, d, bs, max(n), max_len)
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_prefill_fp4(out, to_device(q), kc, vc, _dev(cu), _dev(start), _dev(tables), scale, hkv, bs, max(n), max_len,
                       ws, KS, VS, status=status)
    torch.cuda.synchronize()
    return out, int(status.item())


def _prefill_check(ops, chunks, G, hkv, bs, seed, dtypes=(torch.float32, torch.bfloat16), sigma=0.5):
    rng = np.random.default_rng(seed)
    d = 128
    tables, kc, vc = _attention_case(rng, [s + c for s, c in chunks], G, hkv, d, bs, sigma)
    total = sum(c for _, c in chunks)
    q = bf16(rng.standard_normal((total, G * hkv, d)))
    scale = float(np.float32(1 / np.sqrt(d)))
    rows = [(i, s + j + 1) for i, (s, c) in enumerate(chunks) for j in range(c)]
    pick = range(total) if total <= 800 else sorted({0, total - 1, *rng.integers(0, total, size=200).tolist()})
    ref, tol = _reference(q.f32[list(pick)], tables, kc, vc, bs, d, scale, [rows[r][0] for r in pick],
                          [rows[r][1] for r in pick])
    for dt in dtypes:
        out, st = _prefill(ops, q, tables, chunks, _dev(kc), _dev(vc), bs, scale, hkv, dt)
        assert st == 0 and bool(torch.isfinite(out).all())
        _check(out[torch.tensor(list(pick), device="cuda")], ref, tol)


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("bs", [16, 1, 8, 64, 256])
def test_prefill_matches_definition(ops, G, bs):
    _prefill_check(ops, CHUNKS, G, 2 if G < 8 else 1, bs, 10 * G + bs)


@pytest.mark.parametrize("G,hkv,chunks", [(4, 1, [(6000, 3)]), (4, 2, [(3000, 70), (10, 5)]), (1, 8, [(0, 600)]),
                                          (8, 2, [(2047, 130)] * 3), (2, 2, [(5000, 1), (0, 1), (4999, 2)])])
def test_prefill_long_histories(ops, G, hkv, chunks):
    _prefill_check(ops, chunks, G, hkv, 16, sum(s for s, _ in chunks))


def test_prefill_bad_chunks_are_reported(ops):
    rng = np.random.default_rng(12)
    d, bs, hkv, G = 128, 16, 2, 4
    tables, kc, vc = _attention_case(rng, [40, 10], G, hkv, d, bs)
    q = bf16(rng.standard_normal((50, G * hkv, d)))
    out, st = _prefill(ops, q, tables, [(0, 40), (tables.shape[1] * bs, 10)], _dev(kc), _dev(vc), bs, 0.1, hkv,
                       max_len=40)
    assert st == 1 and bool(torch.isnan(out[40:]).all())
    ref, tol = _reference(q.f32[:40], tables, kc, vc, bs, d, 0.1, [0] * 40, range(1, 41))
    _check(out[:40], ref, tol)
    bad = tables.copy()
    bad[0, 1] = -1
    _, st = _prefill(ops, q, bad, [(0, 40), (0, 10)], _dev(kc), _dev(vc), bs, 0.1, hkv)
    assert st == 1


def test_prefill_last_token_equals_decode(ops):
    rng = np.random.default_rng(13)
    d, bs, hkv, G = 128, 16, 2, 4
    lens = [300, 17, 1]
    tables, kc, vc = _attention_case(rng, lens, G, hkv, d, bs)
    q = bf16(rng.standard_normal((3, G * hkv, d)))
    a = _decode(ops, q, tables, lens, _dev(kc), _dev(vc), bs, 0.1, hkv)
    b, st = _prefill(ops, q, tables, [(n - 1, 1) for n in lens], _dev(kc), _dev(vc), bs, 0.1, hkv)
    ref, tol = _reference(q.f32, tables, kc, vc, bs, d, 0.1, range(3), lens)
    _check(a, ref, tol)
    _check(b, ref, tol)
    assert st == 0


# ---------------------------------------------------------------------------
# copies, and a run of the calls as a server makes them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layers", [None, 3])
def test_copy_blocks_of_a_4bit_pool(ops, layers):
    rng = np.random.default_rng(14)
    nb, hkv, bs, d = 12, 2, 16, 64
    shape = (nb, hkv, fp4.tile_bytes(bs, d)) if layers is None else (layers, nb, hkv, fp4.tile_bytes(bs, d))
    k, v = (rng.integers(0, 256, size=shape, dtype=np.uint8) for _ in range(2))
    pairs = np.array([[0, 5], [0, 6], [3, 9]], dtype=np.int64)
    kc, vc = _dev(k), _dev(v)
    if layers is None:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_copy_blocks(kc, vc, _dev(pairs), status=status, block_size=bs, head_dim=d)
        assert int(status.item()) == 0
        for c in (k, v):
            c[pairs[:, 1]] = c[pairs[:, 0]]
    else:
        ops.pa_copy_blocks_layers(kc, vc, _dev(pairs), block_size=bs, head_dim=d)
        for c in (k, v):
            c[:, pairs[:, 1]] = c[:, pairs[:, 0]]
    assert np.array_equal(kc.cpu().numpy(), k) and np.array_equal(vc.cpu().numpy(), v)


def test_serving_run(ops):
    """Prompt, generation, a fork with copy-on-write, drafted tokens of which
    some are rejected from the middle, compaction, truncation, and generation
    again; each step's attention against a plain list of the tokens."""
    rng = np.random.default_rng(15)
    d, bs, hkv, G, nb = 128, 16, 2, 4, 64
    H = G * hkv
    a = ops.BlockAllocator(nb, bs, rng.permutation(nb).astype(np.int32))
    kc, vc = ops.make_cache_fp4(nb, hkv, bs, d), ops.make_cache_fp4(nb, hkv, bs, d)
    hist = {}

    def stored(x, gs):
        return fp4.dequantise(*fp4.quantise(x, gs), gs)

    def write(seq_of, slots):
        k, v = bf16(rng.standard_normal((len(slots), hkv, d))), bf16(rng.standard_normal((len(slots), hkv, d)))
        ops.pa_reshape_and_cache_fp4(to_device(k), to_device(v), _dev(np.asarray(slots, np.int64)), kc, vc, bs, KS, VS)
        for r, s in enumerate(seq_of):
            hist[s].append((stored(k.f32[r], KS), stored(v.f32[r], VS)))

    def check(seqs):
        tables, lens = a.export_tables(seqs, 16)
        assert lens.tolist() == [len(hist[s]) for s in seqs]
        q = bf16(rng.standard_normal((len(seqs), H, d)))
        got = _decode(ops, q, tables, lens, kc, vc, bs, 0.1, hkv)
        for r, s in enumerate(seqs):
            K, V = (np.stack([t[e] for t in hist[s]]) for e in (0, 1))
            ref = oracle.contiguous_attention(q.f32[r], K, V, 0.1)
            tol = attention_bound(q.f32[r].astype(np.float64), K, V, 0.1)[:, None]
            assert (np.abs(to_f64(got[r]) - ref) <= tol).all()

    seqs = []
    for n in (37, 5, 80):
        s = a.seq_create()
        hist[s] = []
        write([s] * n, a.append_tokens(s, n))
        seqs.append(s)
    check(seqs)
    child = a.fork(seqs[0])
    hist[child] = list(hist[seqs[0]])
    seqs.append(child)
    for _ in range(3):
        slots, pairs = a.append_slots(seqs)
        ops.pa_copy_blocks(kc, vc, _dev(pairs), block_size=bs, head_dim=d)
        write(seqs, slots)
    check(seqs)
    # 9 drafted tokens each, of which positions base + {1, 4, 5} are accepted
    base = {s: len(hist[s]) for s in seqs}
    for s in seqs:
        write([s] * 9, a.append_tokens(s, 9))
    keep = [[base[s] + j for j in (1, 4, 5)] for s in seqs]
    pairs = [a.make_writable(s, base[s], base[s] + 3) for s in seqs]
    assert sum(len(p) for p in pairs) == 0  # nobody shares the drafts' blocks
    tables, _ = a.export_tables(seqs, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_compact_tokens(kc, vc, _dev(tables), _dev(np.array([base[s] for s in seqs], np.int32)),
                          _dev(np.concatenate(keep).astype(np.int32)),
                          _dev(np.arange(0, 3 * len(seqs) + 1, 3, dtype=np.int32)), 3, bs, d, status=status)
    assert int(status.item()) == 0
    for s, k in zip(seqs, keep):
        hist[s] = hist[s][:base[s]] + [hist[s][p] for p in k]
        a.truncate(s, base[s] + 3)
    check(seqs)
    # half of a shared history evicted: the child's blocks are copied first
    drop = [p for p in range(2, len(hist[child])) if p % 2]
    pairs = a.make_writable(child, 2, 2 + len(drop))
    assert len(pairs) >= 1
    ops.pa_copy_blocks(kc, vc, _dev(pairs), block_size=bs, head_dim=d)
    tables, _ = a.export_tables([child], 16)
    ops.pa_compact_tokens(kc, vc, _dev(tables), _dev(np.array([2], np.int32)), _dev(np.array(drop, np.int32)),
                          _dev(np.array([0, len(drop)], np.int32)), len(drop), bs, d)
    hist[child] = hist[child][:2] + [hist[child][p] for p in drop]
    a.truncate(child, len(hist[child]))
    slots, pairs = a.append_slots(seqs)
    ops.pa_copy_blocks(kc, vc, _dev(pairs), block_size=bs, head_dim=d)
    write(seqs, slots)
    check(seqs)
