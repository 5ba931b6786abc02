"""The latent cache on the GPU: append, copies, compaction, absorbed decode and
expanded prefill against the 64-bit definitions."""
import numpy as np
import pytest
import torch

from latent_case import HEAD, LATENT, ROPE, ROW, bf16, blank_unused, check, dev, dev16, tables_of
from oracle import latent as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,bs,dl,dr,joint", [(1, 16, 512, 64, True), (37, 1, 512, 64, False), (300, 16, 512, 64, True),
                                              (70, 256, 64, 8, True), (33, 8, 1024, 128, False)])
def test_append(ops, t, bs, dl, dr, joint, dtype):
    g = torch.Generator(device="cuda").manual_seed(t)
    wide = torch.randn(t, dl + dr + 16, generator=g, device="cuda").to(dtype)
    latent, rope = wide[:, :dl], wide[:, dl:dl + dr]
    if not joint:
        latent, rope = latent.contiguous(), rope.contiguous()
    nb = -(-t // bs) + 3
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:t]
    if t > 5:
        slots[3], slots[4] = -1, nb * bs  # padding, and past the pool
    cache = torch.full((nb, bs, dl + dr), -3.0, dtype=dtype, device="cuda")
    ref = cache.cpu().float().numpy()
    O.append(latent.cpu().float().numpy(), rope.cpu().float().numpy(), slots.cpu().numpy(), ref)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_reshape_and_cache_latent(latent, rope, slots, cache, status=status)
    assert np.array_equal(cache.cpu().float().numpy(), ref)
    assert int(status.item()) == (1 if t > 5 else 0)


# ------------------------------------------------- block copy, compaction
@pytest.mark.parametrize("layers", [None, 1, 3])
def test_block_copy(ops, layers):
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (9, 16, ROW) if layers is None else (layers, 9, 16, ROW)
    cache = torch.randn(shape, generator=g, device="cuda").bfloat16()
    ref = cache.clone()
    c = ref if layers is None else ref.transpose(0, 1)
    c[7], c[2] = c[1].clone(), c[0].clone()
    pairs = torch.tensor([[1, 7], [0, 2], [20, 3]], device="cuda")
    ops.pa_copy_blocks_latent(cache, pairs)  # a pair outside the pool is skipped
    assert torch.equal(cache, ref)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_copy_blocks_latent(cache, torch.tensor([[1, 3], [4, 3]], device="cuda"), status=status)
    assert int(status.item()) == 1 and torch.equal(cache, ref)


@pytest.mark.parametrize("layers,dtype", [(None, torch.bfloat16), (4, torch.bfloat16), (3, torch.float32)])
def test_compaction(ops, layers, dtype):
    rng = np.random.default_rng(2)
    lens, bs = [700, 90, 33], 16
    tables, nb = tables_of(rng, lens, bs)
    g = torch.Generator(device="cuda").manual_seed(3)
    shape = (nb, bs, ROW) if layers is None else (layers, nb, bs, ROW)
    cache = torch.randn(shape, generator=g, device="cuda").to(dtype)
    start = np.array([4, 0, 33], dtype=np.int32)
    keep = [np.sort(4 + rng.permutation(696)[:300]), np.arange(1, 90, 2), np.zeros(0)]
    cu = np.concatenate([[0], np.cumsum([len(k) for k in keep])]).astype(np.int32)
    ref = cache.clone()
    c, r = (x if layers is None else x.transpose(0, 1).transpose(1, 2) for x in (cache, ref))
    old = c.clone()
    for i, k in enumerate(keep):
        for j, s in enumerate(k.astype(int)):
            d = int(start[i]) + j
            r[int(tables[i, d // bs]), d % bs] = old[int(tables[i, s // bs]), s % bs]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_compact_tokens_latent(cache, dev(tables), dev(start), dev(np.concatenate(keep).astype(np.int32)), dev(cu), 300,
                                 status=status)
    assert int(status.item()) == 0 and torch.equal(cache, ref)


# ---------------------------------------------------------------- decode
def decode_case(rng, lens, bs, H, Q, pad=0, sigma=1.0):
    tables, nb = tables_of(rng, lens, bs, pad=pad)
    cache = bf16(rng.standard_normal((nb, bs, ROW)) * sigma)
    q = bf16(rng.standard_normal((len(lens), Q, H, ROW)) * 0.6)
    return tables, cache, q


def run_decode(ops, q, cache, tables, lens, bs, scale, out_dtype=torch.float32, ws=None, max_len=None):
    B, Q, H, _ = q.shape
    max_len = max(lens) if max_len is None else max_len
    if ws is None:
        ws = ops.make_workspace_latent(B, Q, H, LATENT, ROPE, bs, max_len)
    out = torch.full((B, Q, H, LATENT), float("nan"), dtype=out_dtype, device="cuda")
    ops.pa_decode_latent(out, dev16(q), cache, dev(tables), dev(np.array(lens, np.int32)), scale, max_len, ws)
    assert ops.pa_workspace_error(ws) == 0
    return out


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 256])
@pytest.mark.parametrize("H,Q", [(1, 1), (16, 1), (128, 1), (5, 3), (40, 1), (96, 2), (3, 50)])
def test_decode(ops, H, Q, bs):
    rng = np.random.default_rng(H * 100 + Q + bs)
    lens = [1, 0, 63, 64, 65, 17, 200, 129]
    tables, cache, q = decode_case(rng, lens, bs, H, Q, pad=-1)
    exact = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT, O.TWO)
    rounded = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
    for fill in (0.0, float("nan"), float("inf")):
        pool = blank_unused(dev16(cache), tables, lens, bs, fill)
        check(run_decode(ops, q, pool, tables, lens, bs, 0.07), *exact, False)
        check(run_decode(ops, q, pool, tables, lens, bs, 0.07, torch.bfloat16), *rounded, True)


@pytest.mark.parametrize("B,H,top,bs", [(1, 16, 9000, 16), (1, 128, 5000, 32), (3, 128, 3000, 16), (90, 16, 400, 16),
                                        (200, 7, 150, 8), (2, 64, 20000, 64)])
def test_decode_lengths(ops, B, H, top, bs):
    """Long contexts cut into parts, batches of more sequences than the GPU has CTAs."""
    rng = np.random.default_rng(B + H)
    lens = [int(x) for x in rng.integers(0, top, size=B)]
    lens[-1] = top
    tables, cache, q = decode_case(rng, lens, bs, H, 1)
    for dt, dp in ((torch.float32, O.TWO), (torch.bfloat16, O.BF16)):
        ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT, dp)
        check(run_decode(ops, q, dev16(cache), tables, lens, bs, 0.07, dt), ref, tol, dt == torch.bfloat16)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 2.0])
def test_decode_with_any_softmax_scale(ops, scale):
    rng = np.random.default_rng(7)
    lens = [300, 1, 70]
    tables, cache, q = decode_case(rng, lens, 16, 20, 2)
    ref, tol = O.decode(q.f32, cache.f32, tables, lens, scale, LATENT)
    check(run_decode(ops, q, dev16(cache), tables, lens, 16, scale), ref, tol, False)


def test_decode_maxima_that_rise_late(ops):
    """Scores that grow along the context by more than any slack, for some rows only."""
    rng = np.random.default_rng(8)
    lens, bs, H = [1000, 640], 16, 70
    tables, cache, q = decode_case(rng, lens, bs, H, 1, sigma=0.2)
    x = cache.f32.copy()
    u = rng.standard_normal(ROW).astype(np.float32)
    for i, n in enumerate(lens):
        for t in range(n):
            x[tables[i, t // bs], t % bs] += u * (t // 100) * 0.5
    cache = bf16(x)
    qq = q.f32.copy()
    qq[:, :, ::3] = u * rng.uniform(0.5, 1.5, size=(2, 1, len(range(0, H, 3)), 1))
    q = bf16(qq)
    ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
    check(run_decode(ops, q, dev16(cache), tables, lens, bs, 0.07), ref, tol, False)


def test_decode_reports_what_lies_outside(ops):
    """A table entry outside the pool and a length past the bound are reported, other sequences are right."""
    rng = np.random.default_rng(9)
    lens, bs = [100, 100, 64], 16
    tables, cache, q = decode_case(rng, lens, bs, 16, 1)
    ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT)
    for entry in (-5, 1 << 30):
        bad = tables.copy()
        bad[1, 3] = entry
        ws = ops.make_workspace_latent(3, 1, 16, LATENT, ROPE, bs, 100)
        out = torch.zeros(3, 16, LATENT, device="cuda")
        ops.pa_decode_latent(out, dev16(q)[:, 0].contiguous(), dev16(cache), dev(bad), dev(np.array(lens, np.int32)), 0.07,
                             100, ws)
        assert ops.pa_workspace_error(ws) == 1
        check(out[[0, 2]], ref[[0, 2], 0], tol[[0, 2], 0], False)
    for n in (-1, 101, 2 ** 31 - 1):
        ws = ops.make_workspace_latent(3, 1, 16, LATENT, ROPE, bs, 100)
        ops.pa_decode_latent(out, dev16(q)[:, 0].contiguous(), dev16(cache), dev(tables),
                             dev(np.array([100, n, 64], np.int32)), 0.07, 100, ws)
        assert ops.pa_workspace_error(ws) == 1
        check(out[[0, 2]], ref[[0, 2], 0], tol[[0, 2], 0], False)


# --------------------------------------------------------------- prefill
def prefill_case(rng, chunks, bs, H, pad=0):
    lens = [s + n if n else 0 for s, n in chunks]
    tables, nb = tables_of(rng, lens, bs, pad=pad)
    cache = bf16(rng.standard_normal((nb, bs, ROW)))
    cu = np.concatenate([[0], np.cumsum([n for _, n in chunks])]).astype(np.int32)
    q = bf16(rng.standard_normal((int(cu[-1]), H, HEAD + ROPE)))
    w_k, w_v = (bf16(rng.standard_normal((H, HEAD, LATENT)) / np.sqrt(LATENT)) for _ in range(2))
    return lens, tables, cache, cu, q, w_k, w_v


def run_prefill(ops, q, pool, w_k, w_v, cu, start, tables, bs, scale, max_q, max_len, total, out_dtype=torch.float32,
                ws=None, status_is=0):
    S, H = len(start), q.shape[1]
    if ws is None:
        ws = ops.make_prefill_workspace_latent(S, H, LATENT, ROPE, HEAD, bs, max_q, max_len, total)
        ws.fill_(255)  # NaN wherever it is read as it is
    out = torch.full((q.shape[0], H, HEAD), -7.0, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.pa_prefill_latent(out, dev16(q), pool, dev16(w_k), dev16(w_v), dev(cu), dev(np.array(start, np.int32)), dev(tables),
                          scale, max_q, max_len, total, ws, status=status)
    assert int(status.item()) == status_is
    return out


@pytest.mark.parametrize("chunks,H,bs", [
    ([(0, 1)], 1, 16), ([(0, 5), (7, 0), (100, 30)], 3, 16), ([(0, 129), (200, 64)], 2, 8), ([(511, 1), (0, 128), (1, 256)], 4, 32),
    ([(0, 300)], 5, 256), ([(130, 257), (3, 1), (0, 2)], 2, 64), ([(1000, 17)], 16, 128), ([(0, 700), (300, 513)], 6, 16),
    ([(5, 3)] * 30, 2, 16), ([(5000, 40)], 1, 32)])
def test_prefill(ops, chunks, H, bs):
    rng = np.random.default_rng(len(chunks) * 10 + H)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, bs, H, pad=-1)
    start = [s for s, _ in chunks]
    exact = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.072, two=True)
    rounded = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.072)
    args = (cu, start, tables, bs, 0.072, max(n for _, n in chunks), max(lens), sum(lens))
    for fill in (0.0, float("nan")):
        pool = blank_unused(dev16(cache), tables, lens, bs, fill)
        check(run_prefill(ops, q, pool, w_k, w_v, *args), *exact, False)
        check(run_prefill(ops, q, pool, w_k, w_v, *args, out_dtype=torch.bfloat16), *rounded, True)


def test_prefill_reports_what_lies_outside(ops):
    rng = np.random.default_rng(5)
    chunks, bs = [(20, 40), (0, 30), (64, 64)], 16
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, bs, 2)
    start = [s for s, _ in chunks]
    ref, tol = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.072, two=True)
    pool, total = dev16(cache), sum(lens)
    rest = np.r_[0:40, 70:134]
    # a chunk that starts below zero, ends behind max_context_len, is longer than max_q_len
    for bad, max_q, max_len in ((-1, 64, 128), (99, 64, 128)):
        s = [20, bad, 64]
        out = run_prefill(ops, q, pool, w_k, w_v, cu, s, tables, bs, 0.072, max_q, max_len, total, status_is=1)
        check(out[rest], ref[rest], tol[rest], False)
        assert (out[40:70] == -7).all()
    out = run_prefill(ops, q, pool, w_k, w_v, cu, start, tables, bs, 0.072, 63, 128, total, status_is=1)
    check(out[:70], ref[:70], tol[:70], False)
    assert (out[70:] == -7).all()
    # contexts that do not fit total_context: the chunks before them are computed
    out = run_prefill(ops, q, pool, w_k, w_v, cu, start, tables, bs, 0.072, 64, 128, 90, status_is=1)
    check(out[:70], ref[:70], tol[:70], False)
    assert (out[70:] == -7).all()
    bad = tables.copy()
    bad[1, 1] = 1 << 29
    out = run_prefill(ops, q, pool, w_k, w_v, cu, start, bad, bs, 0.072, 64, 128, total, status_is=1)
    check(out[rest], ref[rest], tol[rest], False)
