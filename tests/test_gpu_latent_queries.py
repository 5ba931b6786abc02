"""Query rows that are not finite, or that nobody has, over the latent cache (and in
the weights): every other row is what the 64-bit definition gives."""
import numpy as np
import pytest
import torch

from latent_case import LATENT, ROW, check, dev16
from oracle import latent as O
from test_gpu_evict import run_weights, weights_case
from test_gpu_latent import decode_case, prefill_case, run_decode, run_prefill

pytestmark = pytest.mark.gpu

DTYPES = ((torch.float32, O.TWO), (torch.bfloat16, O.BF16))


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


class Rows:
    """What run_decode takes as queries, with some rows replaced on the way to the GPU."""

    def __init__(self, q, where, value):
        x = q.f32.copy()
        x.reshape(len(x), -1, ROW)[:, where] = value
        self.bits = type(q).from_f32(x, "bf16").bits
        self.shape = q.bits.shape


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e38])
@pytest.mark.parametrize("H,Q", [(16, 2), (5, 3), (1, 30), (70, 4), (128, 3), (3, 50), (40, 2)])
def test_rows_beside_a_query_that_is_not_finite(ops, H, Q, value):
    """The first row of every 128 holds it (1e38: its fp32 scores overflow); tokens
    that only the later queries see keep their values for them."""
    rng = np.random.default_rng(H + Q)
    lens = [1, 2, 65, 64, 200, 130, Q, 0]
    tables, cache, q = decode_case(rng, lens, 16, H, Q)
    where = np.arange(0, H * Q, 128)
    others = np.setdiff1d(np.arange(H * Q), where)
    for dt, dp in DTYPES:
        ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT, dp)
        out = run_decode(ops, Rows(q, where, value), dev16(cache), tables, lens, 16, 0.07, dt)
        flat = [x.reshape(len(lens), H * Q, LATENT)[:, others] for x in (out, ref, tol)]
        check(*flat, dt == torch.bfloat16)


@pytest.mark.parametrize("H,Q", [(16, 2), (2, 16), (128, 3), (20, 7)])
def test_queries_before_the_first_token_may_hold_anything(ops, H, Q):
    """Contexts shorter than the query's tokens: rows at positions below zero are
    zeros whatever their queries hold, and the others are right."""
    rng = np.random.default_rng(H * Q)
    for n in range(1, Q):
        lens = [n, Q, n]
        tables, cache, q = decode_case(rng, lens, 8, H, Q)
        x = q.f32.copy()
        for i in (0, 2):
            x[i, : Q - n] = np.nan
        for dt, dp in DTYPES:
            ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT, dp)
            assert (ref[0, : Q - n] == 0).all() and (tol[0, : Q - n] == 0).all()
            bad = type(q).from_f32(x, "bf16")
            check(run_decode(ops, bad, dev16(cache), tables, lens, 8, 0.07, dt), ref, tol, dt == torch.bfloat16)


@pytest.mark.parametrize("H,Q", [(16, 2), (4, 8), (70, 4)])
def test_values_and_queries_that_are_not_finite_together(ops, H, Q):
    """A value of the newest token and the first row's query: the queries before the
    newest are right but for that row."""
    rng = np.random.default_rng(H)
    lens = [65, 200, 64]
    tables, cache, q = decode_case(rng, lens, 16, H, Q)
    for bad in (float("nan"), float("inf")):
        pool = dev16(cache)
        for i, n in enumerate(lens):
            pool[int(tables[i, (n - 1) // 16]), (n - 1) % 16, 37 + 150 * i] = bad
        for dt, dp in DTYPES:
            ref, tol = O.decode(q.f32, cache.f32, tables, lens, 0.07, LATENT, dp)
            out = run_decode(ops, Rows(q, [0], float("nan")), pool, tables, lens, 16, 0.07, dt)
            assert torch.isnan(out[:, 0, 0]).all()
            keep = lambda x: x[:, :-1].reshape(3, -1, LATENT)[:, 1:]
            check(*(keep(x) for x in (out, ref, tol)), dt == torch.bfloat16)
            assert not torch.isfinite(out[:, -1]).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prefill_beside_a_query_that_is_not_finite(ops, value, dt):
    rng = np.random.default_rng(21)
    chunks, H = [(100, 200), (0, 130), (900, 3)], 3
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, 16, H)
    start = [s for s, _ in chunks]
    x = q.f32.copy()
    bad = [(0, 0), (130, 2), (200, 1), (331, 0)]
    for t, h in bad:
        x[t, h] = value
    ref, tol = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.07, f32=dt == torch.float32)
    out = run_prefill(ops, type(q).from_f32(x, "bf16"), dev16(cache), w_k, w_v, cu, start, tables, 16, 0.07, 200, max(lens), sum(lens), dt)
    keep = np.ones(x.shape[:2], bool)
    for t, h in bad:
        assert torch.isnan(out[t, h]).all()
        keep[t, h] = False
    check(out[torch.from_numpy(keep).cuda()], ref[keep], tol[keep], dt == torch.bfloat16)


@pytest.mark.parametrize("W,H,hkv,d", [(1, 8, 2, 128), (40, 8, 2, 64), (3, 16, 1, ROW), (12, 4, 2, 256), (30, 8, 2, 128)])
def test_weights_beside_queries_before_the_first_token(ops, W, H, hkv, d):
    """Rows at positions below zero add nothing, whatever their queries hold."""
    rng = np.random.default_rng(W)
    lens = [max(1, W // 2), 300, 0, 1]
    tables, k, q, before = weights_case(rng, lens, 16, W, H, hkv, d)
    x = q.f32.copy()
    for i, n in enumerate(lens):
        x[i, : max(0, W - n)] = np.nan
    ref, tol = O.weights(before, q.f32, k.f32, tables, lens, 0.1)
    check(run_weights(ops, before, type(q).from_f32(x, "bf16"), dev16(k), tables, lens, 16, 0.1), ref, tol, False)
