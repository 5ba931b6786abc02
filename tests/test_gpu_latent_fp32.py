"""fp32 outputs of the latent cache at the bounds that they promise: prefill with
keys, values and probabilities in fp32, decode with probabilities to 2^-16; and
calls that repeat themselves bit by bit.

The bounds of random inputs are wide, since they allow every sum its worst case
(a score's errors alone may come to a percent).  So there are inputs of which all
sums are exact, too: one product or two a score, key and value, and values that
hand single probabilities out.  What is left then is counted in units of 2^-24."""
import numpy as np
import pytest
import torch

from latent_case import LATENT, ROPE, ROW, bf16, blank_unused, check, dev16
from oracle import latent as O
from test_gpu_latent import decode_case, prefill_case, run_decode, run_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


# ---------------------------------------------------------------- prefill
@pytest.mark.parametrize("chunks,H,bs", [
    ([(0, 1)], 1, 16), ([(0, 5), (7, 0), (100, 30)], 3, 16), ([(0, 129), (200, 64)], 2, 8), ([(511, 1), (0, 128), (1, 256)], 4, 32),
    ([(0, 300)], 5, 256), ([(130, 257), (3, 1), (0, 2)], 2, 64), ([(1000, 17)], 16, 128), ([(0, 700), (300, 513)], 6, 16),
    ([(5, 3)] * 30, 2, 16), ([(5000, 40)], 1, 32),
    # few queries: their keys are shared among CTAs
    ([(4000, 3)], 2, 16), ([(1500, 70), (0, 2)], 3, 16), ([(900, 65), (0, 0), (31, 1)], 5, 8), ([(0, 1)] * 3, 1, 16),
    # one more query tile than is split
    ([(2000, 64)], 76, 16), ([(2000, 65)], 76, 16)])
def test_prefill_keeps_fp32(ops, chunks, H, bs):
    rng = np.random.default_rng(len(chunks) * 10 + H)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, bs, H, pad=-1)
    start = [s for s, _ in chunks]
    ref = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, start, tables, 0.072, f32=True)
    for fill in (0.0, float("nan")):
        pool = blank_unused(dev16(cache), tables, lens, bs, fill)
        check(run_prefill(ops, q, pool, w_k, w_v, cu, start, tables, bs, 0.072, max(n for _, n in chunks), max(lens), sum(lens)),
              *ref, False)


@pytest.mark.parametrize("scale", [1e-30, 0.02, 1.0])
def test_prefill_keeps_fp32_at_any_scale(ops, scale):
    rng = np.random.default_rng(3)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, [(100, 70), (0, 33)], 16, 4)
    ref = O.prefill(q.f32, cache.f32, w_k.f32, w_v.f32, cu, [100, 0], tables, scale, f32=True)
    check(run_prefill(ops, q, dev16(cache), w_k, w_v, cu, [100, 0], tables, 16, scale, 70, 170, sum(lens)), *ref, False)


# ---------------------------------------------------------------- decode
def check_decode(ops, q, cache, tables, lens, bs, scale, ws=None):
    ref = O.decode(q.f32, cache.f32, tables, lens, scale, LATENT, O.TWO)
    check(run_decode(ops, q, dev16(cache), tables, lens, bs, scale, ws=ws), *ref, False)


@pytest.mark.parametrize("lens,H,Q", [([5000], 16, 1), ([5000], 128, 1), ([3000, 0, 7, 2500], 128, 1), ([900] * 15, 16, 1), ([900] * 16, 16, 1),
                                      ([2000] * 5, 128, 1), ([0, 4000], 3, 1), ([3000, 40], 100, 3), ([6000], 1, 300), ([2500], 40, 5)])
def test_decode_of_items_in_many_parts(ops, lens, H, Q):
    rng = np.random.default_rng(len(lens) + H)
    check_decode(ops, *decode_case_q(rng, lens, 32, H, Q), lens, 32, 0.07)


def decode_case_q(rng, lens, bs, H, Q):
    tables, cache, q = decode_case(rng, lens, bs, H, Q)
    return q, cache, tables


@pytest.mark.parametrize("H,bs,B", [(16, 16, 2048), (17, 16, 2048), (2, 8, 2500)])
def test_decode_of_many_short_sequences(ops, H, bs, B):
    rng = np.random.default_rng(32 + H)
    lens = [int(x) for x in rng.integers(0, 30, size=B)]
    lens[5], lens[-1], lens[1000] = 700, 500, 65
    check_decode(ops, *decode_case_q(rng, lens, bs, H, 1), lens, bs, 0.07)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 2.0])
def test_decode_at_any_scale(ops, scale):
    rng = np.random.default_rng(7)
    lens = [300, 1, 70]
    for H, Q in ((20, 2), (16, 1), (128, 1)):
        check_decode(ops, *decode_case_q(rng, lens, 16, H, Q), lens, 16, scale)


def test_one_workspace_in_turns(ops):
    rng = np.random.default_rng(1)
    ws = ops.make_workspace_latent(8, 4, 128, LATENT, ROPE, 8, 4000)
    for lens, bs, H, Q in ([700] * 6, 16, 16, 1), ([3000, 5], 8, 128, 1), ([2500], 32, 40, 3), ([9, 4000], 64, 2, 1), ([700] * 6, 16, 16, 1):
        check_decode(ops, *decode_case_q(rng, lens, bs, H, Q), lens, bs, 0.07, ws=ws)


@pytest.mark.parametrize("H,Q", [(70, 1), (16, 1), (24, 5), (128, 2)])
def test_decode_with_maxima_that_rise_late(ops, H, Q):
    """Outputs are put on a new reference again and again, of some rows only, and parts of items weigh differently."""
    rng = np.random.default_rng(8)
    lens, bs = [1000, 640, 4000], 16
    tables, cache, q = decode_case(rng, lens, bs, H, Q, sigma=0.2)
    x, qq = cache.f32.copy(), q.f32.copy()
    u = rng.standard_normal(ROW).astype(np.float32)
    for i, n in enumerate(lens):
        t = np.arange(n)
        x[tables[i, t // bs], t % bs] += u[None] * (t // 100)[:, None] * 0.5
    qq[:, :, ::3] = u * rng.uniform(0.5, 1.5, size=(len(lens), Q, len(range(0, H, 3)), 1))
    check_decode(ops, bf16(qq), bf16(x), tables, lens, bs, 0.01)


# ---------------------------------------------------------- exact sums
HALF = 2.0 ** -24  # a rounding to fp32
# exp2 of the two kinds (2 units of 2^-23 by CUDA's tables); the quotient by the sum, and its product
EXP2, QUOTIENT = 4 * HALF, 2 * HALF


def argument(top):
    """Of scores up to top: the scale in the base of 2, a product with it and the
    difference from the reference, each up to 2 top log2 e, as a share of the exponential."""
    return 3 * HALF * 2 * top


def probabilities(s):
    e = np.exp(s - s.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def near(got, want, rel):
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= rel * want).all(), f"off by {np.nanmax(off / np.maximum(want, 1e-300)) / HALF:.1f} x 2^-24, allowed {rel / HALF:.1f}"


def weights_of_24_bits(rng, shape):
    """Three columns [..., 3] of bf16 values whose sum, with any signs, has 24 bits and is exact in fp32 on the way."""
    return np.stack([1 + rng.integers(0, 127, shape) / 128, 2.0 ** -15 * rng.integers(1, 256, shape),
                     2.0 ** -23 * rng.integers(1, 256, shape)], -1)


def two_parts(x):
    hi = bf16(x).f32.astype(np.float64)
    return hi + bf16(x - hi).f32


def test_prefill_values_hold_fp32(ops):
    """One token is its value, which has more bits than two bf16 parts."""
    rng = np.random.default_rng(31)
    H, n = 5, 40
    w_k, w_v = (np.zeros((H, 128, LATENT), np.float32) for _ in range(2))
    w_v[:, :, :3] = weights_of_24_bits(rng, (H, 128))
    c = np.zeros((n, ROW), np.float32)
    c[:, :3] = rng.choice([-1, 1], (n, 3))
    cu = np.arange(n + 1, dtype=np.int32)
    q = bf16(rng.standard_normal((n, H, 192)))
    out = run_prefill(ops, q, dev16(bf16(c[:, None])).repeat(1, 8, 1), bf16(w_k), bf16(w_v), cu, [0] * n,
                      np.arange(n, dtype=np.int32)[:, None], 8, 0.07, 1, 1, n)
    want = np.einsum("tl,hdl->thd", c[:, :3].astype(np.float64), w_v[:, :, :3].astype(np.float64))
    assert np.array_equal(want, want.astype(np.float32)) and (np.abs(two_parts(want) - want) > 2.0 ** -19).any()
    assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("by_key", [False, True])
def test_prefill_probabilities_and_keys_hold_fp32(ops, by_key):
    """Eight tokens whose values hand their probabilities out, scores by the position
    part (up to 1) or by a key of 24 bits (from 4 to 8)."""
    rng = np.random.default_rng(32)
    H, T, S = 64, 8, 6
    w_k, w_v = (np.zeros((H, 128, LATENT), np.float32) for _ in range(2))
    w_v[:, np.arange(T), 3 + np.arange(T)] = 1
    w_k[:, 5, :3] = weights_of_24_bits(rng, H)
    c = np.zeros((S, T, ROW), np.float32)
    c[:, np.arange(T), 3 + np.arange(T)] = 1
    c[:, :, 0], c[:, :, 1:3] = 1, rng.choice([-1, 1], (S, T, 2))
    c[:, :, LATENT + 7] = rng.uniform(-1, 1, (S, T))
    cache, q = bf16(c), np.zeros((S, H, 192), np.float32)
    if by_key:
        q[:, :, 5] = 4
    else:
        q[:, :, 128 + 7] = rng.uniform(-1, 1, (S, H))
    q = bf16(q)
    out = run_prefill(ops, q, dev16(cache), bf16(w_k), bf16(w_v), np.arange(S + 1, dtype=np.int32), [T - 1] * S,
                      np.arange(S, dtype=np.int32)[:, None], 8, 1.0, 1, T, S * T)
    x = cache.f32.astype(np.float64)
    k = np.einsum("stl,hl->sht", x[:, :, :3], w_k[:, 5, :3].astype(np.float64))
    s = 4 * k if by_key else q.f32[:, :, None, 135] * x[:, None, :, LATENT + 7]
    top = 8 if by_key else 1
    rel = 2 * (argument(top) + EXP2 + T * HALF) + QUOTIENT
    # what two bf16 parts of the keys, or of the probabilities, leave would be seen
    e = np.exp(s - s.max(-1, keepdims=True))
    lost = np.abs(probabilities(4 * two_parts(k)) / probabilities(s) - 1) if by_key else np.abs(two_parts(e) / e - 1)
    assert lost.max() > 2 * rel
    near(out[:, :, :T], probabilities(s), rel)
    assert (out[:, :, T:] == 0).all()


@pytest.mark.parametrize("lens,H,Q", [([9, 64, 300], 16, 1), ([3000], 16, 1), ([200, 3000], 128, 1), ([700, 5, 1500], 20, 4),
                                      ([2000], 3, 40), ([500] * 40, 32, 1), ([4000, 90], 64, 3)])
def test_decode_probabilities_hold_16_bits(ops, lens, H, Q):
    """512 tokens of each context hand their probabilities out; scores up to 16 rise for
    some heads along the context and fall for others, past the slack of the references."""
    rng = np.random.default_rng(H + Q)
    bs = 16
    tables, cache, q = decode_case(rng, lens, bs, H, Q)
    x, y = np.zeros_like(cache.f32), np.zeros_like(q.f32)
    r = LATENT + 11
    chosen = []
    for i, n in enumerate(lens):
        t = np.arange(n)
        x[tables[i, t // bs], t % bs, r] = 8 * t / n - 4 + rng.uniform(-0.5, 0.5, n)
        pick = np.sort(rng.permutation(n)[:LATENT])
        chosen.append(pick)
        x[tables[i, pick // bs], pick % bs, np.arange(len(pick))] = 1
    y[..., r] = rng.choice([-3.5, 3.5, 1.25, 0.25, -1], y.shape[:-1])
    cache, q = bf16(x), bf16(y)
    out = run_decode(ops, q, dev16(cache), tables, lens, bs, 1.0)
    for i, n in enumerate(lens):
        t = np.arange(n)
        s = q.f32[i, ..., r, None].astype(np.float64) * cache.f32[tables[i, t // bs], t % bs, r]
        for j in range(Q):
            seen = max(0, n - Q + 1 + j)
            want = np.zeros((H, n))
            if seen:
                want[:, :seen] = probabilities(s[j][:, :seen])
            rel = O.TWO + 2 * (argument(16) + EXP2 + (n + 64) * HALF) + QUOTIENT
            assert rel < 2.0 ** -10
            near(out[i, j][:, : len(chosen[i])], want[:, chosen[i]], rel)
            assert (out[i, j][:, len(chosen[i]):] == 0).all()


# ------------------------------------------------------------- repetition
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_calls_repeat_themselves(ops, dt):
    rng = np.random.default_rng(12)
    for lens, H, Q in (([700, 30, 2000], 16, 1), ([1500, 900], 128, 1), ([4000], 20, 4)):
        tables, cache, q = decode_case(rng, lens, 16, H, Q)
        first = run_decode(ops, q, dev16(cache), tables, lens, 16, 0.07, dt)
        for _ in range(3):
            assert torch.equal(run_decode(ops, q, dev16(cache), tables, lens, 16, 0.07, dt), first)
    for chunks, H in (([(900, 200), (0, 300)], 20), ([(3000, 5)], 2)):
        lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, 16, H)
        call = lambda: run_prefill(ops, q, dev16(cache), w_k, w_v, cu, [s for s, _ in chunks], tables, 16, 0.07,
                                   max(n for _, n in chunks), max(lens), sum(lens), dt)
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)
