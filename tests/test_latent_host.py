"""The latent cache and eviction without a GPU: the 64-bit definitions against
closed forms, and the refusals of every call."""
import ctypes as C

import numpy as np
import pytest

from oracle import latent as O

P = 0x10000  # stands for a device pointer; never reached


# ------------------------------------------------------------ definitions
def test_decode_of_one_token_is_its_latent_row():
    rng = np.random.default_rng(0)
    cache = rng.standard_normal((3, 4, 12))
    q = rng.standard_normal((1, 1, 2, 12))
    out, _ = O.decode(q, cache, np.array([[2]]), [1], 0.3, 8)
    assert np.allclose(out[0, 0], cache[2, 0, :8])


def test_expanded_form_equals_absorbed_form():
    """Projecting the query and the output instead of every row is the same sum."""
    rng = np.random.default_rng(1)
    L, R, D, H, n = 16, 4, 8, 3, 11
    cache, q = rng.standard_normal((6, 4, L + R)), rng.standard_normal((1, H, D + R))
    w_k, w_v = rng.standard_normal((H, D, L)), rng.standard_normal((H, D, L))
    tables = np.array([[5, 1, 3]])
    x = O.rows(cache, tables[0], n, 4)
    absorbed = np.concatenate([np.einsum("hd,hdl->hl", q[0, :, :D], w_k), q[0, :, D:]], 1)
    out, _ = O.decode(absorbed[None, None], cache, tables, [n], 0.3, L)
    want = np.einsum("hl,hdl->hd", out[0, 0], w_v)
    for h in range(H):
        k = np.concatenate([x[:, :L] @ w_k[h].T, x[:, L:]], 1)
        got, _ = O.attend(q[:, h], k, x[:, :L] @ w_v[h].T, 0.3, [n])
        assert np.allclose(got[0], want[h])
    # and the prefill definition is this up to the rounding of keys and values to
    # bf16: a value x moves by at most 2^-8 |x|, and attend's bound carries that
    # through (it holds for any keys and values within dk and dv of these)
    got, _ = O.prefill(q, cache, w_k, w_v, np.array([0, 1]), np.array([n - 1]), tables, 0.3)
    for h in range(H):
        k, v = np.concatenate([x[:, :L] @ w_k[h].T, x[:, L:]], 1), x[:, :L] @ w_v[h].T
        _, allowed = O.attend(q[:, h], k, v, 0.3, [n], np.abs(k) * O.BF16, np.abs(v) * O.BF16)
        assert (np.abs(got[0, h] - want[h]) <= allowed[0]).all()


def test_to_bf16_is_nearest_even():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -30, -3.14159, 0.0])
    want = [1.0, 1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -3.140625, 0.0]
    assert O.to_bf16(x).tolist() == want


def test_weights_of_a_window_sum_to_its_rows():
    rng = np.random.default_rng(2)
    k = rng.standard_normal((9, 2, 4, 8))
    q = rng.standard_normal((2, 3, 4, 8))
    tables = np.array([[1, 2, 3], [4, 5, 6]])
    after, _ = O.weights(np.zeros((2, 12)), q, k, tables, [9, 2], 0.5)
    assert np.isclose(after[0].sum(), 12) and (after[0, 9:] == 0).all()
    assert np.isclose(after[1].sum(), 8)  # its first query has no position
    # the newest token is seen by the last query alone
    assert after[0, 8] <= 4


def test_select_definition():
    w = np.array([[9, 0, 3, 3, 1, 3, 0, 2]], dtype=np.float32)
    keep, after = O.select(w, [1], [7], [3], 1)
    assert keep.tolist() == [2, 3, 6] and after.tolist() == [[9, 3, 3, 0, 0, 0, 0, 2]]
    w[0, 3] = np.nan
    assert O.select(w, [0], [8], [8], 0)[0].tolist() == list(range(8))
    assert O.select(w, [2], [5], [2], 0)[0].tolist() == [2, 4]


# --------------------------------------------------------------- refusals
def codes():
    from paged_kv_cache_142_gb300 import _lib as L
    return L.PA_OK, L.PA_ERR_INVALID_ARG, L.PA_ERR_UNSUPPORTED, L.PA_ERR_WORKSPACE


def test_append_refusals(lib):
    OK, BAD, UNSUPPORTED, _ = codes()

    def call(latent=P, ls=576, rope=P, rs=576, t=3, slots=P, cache=P, nb=8, bs=16, dl=512, dr=64, dt=1, status=None):
        return lib.pa_reshape_and_cache_latent(latent, ls, rope, rs, t, slots, cache, nb, bs, dl, dr, dt, status, None)

    for name in ("latent", "rope", "slots", "cache"):
        assert call(**{name: None}) == BAD
    for name in ("latent", "rope", "cache"):
        assert call(**{name: P + 8}) == BAD
    assert call(slots=P + 4) == BAD and call(status=P + 2) == BAD
    assert call(nb=0) == BAD and call(bs=0) == BAD and call(dl=0) == BAD and call(dr=0) == BAD and call(t=-1) == BAD
    assert call(dt=2) == BAD and call(ls=511) == BAD and call(rs=63) == BAD and call(ls=577) == BAD and call(rs=-64) == BAD
    assert call(bs=12) == UNSUPPORTED and call(bs=512) == UNSUPPORTED
    assert call(dl=511) == UNSUPPORTED and call(dr=4) == UNSUPPORTED and call(dl=4096) == UNSUPPORTED
    assert call(t=0, latent=None, rope=None, cache=None, slots=None) == OK


def test_copy_and_compaction_refusals(lib):
    OK, BAD, UNSUPPORTED, _ = codes()

    def copy(cache=P, stride=0, layers=1, nb=8, bs=16, dl=512, dr=64, dt=1, pairs=P, n=2, status=None):
        return lib.pa_copy_blocks_latent(cache, stride, layers, nb, bs, dl, dr, dt, pairs, n, status, None)

    assert copy(cache=None) == BAD and copy(pairs=None) == BAD and copy(cache=P + 8) == BAD and copy(n=-1) == BAD
    assert copy(layers=0) == BAD and copy(layers=32768) == BAD and copy(layers=2, stride=8 * 16 * 576 - 8) == BAD
    assert copy(layers=2, stride=8 * 16 * 576 + 4) == BAD and copy(dt=2) == BAD and copy(bs=3) == UNSUPPORTED
    assert copy(n=0, cache=None) == OK

    def compact(cache=P, stride=0, layers=1, nb=8, bs=16, dl=512, dr=64, dt=1, tab=P, m=4, start=P, keep=P, nk=4, cu=P, n=2,
                mk=3, status=None):
        return lib.pa_compact_tokens_latent(cache, stride, layers, nb, bs, dl, dr, dt, tab, m, start, keep, nk, cu, n, mk,
                                            status, None)

    for name in ("cache", "tab", "start", "keep", "cu"):
        assert compact(**{name: None}) == BAD
    assert compact(m=0) == BAD and compact(nk=-1) == BAD and compact(n=-1) == BAD and compact(mk=-1) == BAD
    assert compact(layers=2, stride=16) == BAD and compact(dl=500) == UNSUPPORTED
    assert compact(n=0, cache=None) == OK and compact(mk=0, cache=None) == OK


def test_decode_refusals(lib):
    OK, BAD, UNSUPPORTED, WS = codes()

    def call(out=P, odt=0, q=P, n=2, ql=1, h=16, cache=P, nb=8, bs=16, dl=512, dr=64, tab=P, m=4, lens=P, ml=64, scale=0.1,
             ws=P, wb=1 << 40):
        return lib.pa_decode_latent(out, odt, q, n, ql, h, cache, nb, bs, dl, dr, tab, m, lens, ml, scale, ws, wb, None)

    for name in ("out", "q", "cache", "tab", "lens"):
        assert call(**{name: None}) == BAD
    assert call(out=P + 16) == BAD and call(q=P + 8) == BAD and call(cache=P + 8) == BAD and call(tab=P + 2) == BAD
    assert call(odt=2) == BAD and call(n=-1) == BAD and call(ql=0) == BAD and call(h=0) == BAD and call(nb=0) == BAD
    assert call(ml=65) == BAD and call(ml=-1) == BAD and call(m=0) == BAD
    for s in (float("nan"), float("inf"), 3e38):
        assert call(scale=s) == BAD
    assert call(h=129) == UNSUPPORTED and call(dl=256) == UNSUPPORTED and call(dr=128) == UNSUPPORTED
    assert call(bs=4, m=16) == UNSUPPORTED and call(bs=24) == UNSUPPORTED and call(bs=512) == UNSUPPORTED
    assert call(m=1 << 28, ml=(1 << 30) + 1) == UNSUPPORTED and call(n=1 << 24, ql=2, h=128) == UNSUPPORTED
    assert call(ws=None) == WS and call(ws=P + 64) == WS and call(wb=8) == WS
    assert call(n=0, out=None, ws=None) == OK
    size = lib.pa_decode_latent_workspace_size
    assert size(2, 1, 16, 512, 64, 16, 64) >= 256 and size(2, 1, 16, 512, 64, 4, 64) == 0 and size(2, 1, 0, 512, 64, 16, 64) == 0


def test_prefill_refusals(lib):
    OK, BAD, UNSUPPORTED, WS = codes()

    def call(out=P, odt=0, q=P, t=5, cu=P, start=P, n=2, mq=4, ml=64, total=128, h=16, cache=P, nb=8, bs=16, dl=512, dr=64,
             wk=P, wv=P, d=128, tab=P, m=4, scale=0.1, status=None, ws=P, wb=1 << 40):
        return lib.pa_prefill_latent(out, odt, q, t, cu, start, n, mq, ml, total, h, cache, nb, bs, dl, dr, wk, wv, d, tab,
                                     m, scale, status, ws, wb, None)

    for name in ("out", "q", "cu", "start", "cache", "wk", "wv", "tab"):
        assert call(**{name: None}) == BAD
    assert call(out=P + 16) == BAD and call(q=P + 8) == BAD and call(wk=P + 8) == BAD and call(status=P + 1) == BAD
    assert call(t=-1) == BAD and call(n=-1) == BAD and call(mq=-1) == BAD and call(total=-1) == BAD and call(ml=65) == BAD
    for s in (float("nan"), float("inf"), 0.0, -1.0):
        assert call(scale=s) == BAD
    assert call(d=64) == UNSUPPORTED and call(h=65536) == UNSUPPORTED and call(dl=256) == UNSUPPORTED
    assert call(bs=4, m=16) == UNSUPPORTED and call(total=1 << 31) == UNSUPPORTED
    assert call(ws=None) == WS and call(ws=P + 64) == WS and call(wb=8) == WS
    assert call(t=0, q=None) == OK and call(n=0, q=None) == OK and call(mq=0, q=None) == OK


def test_weights_and_selection_refusals(lib):
    OK, BAD, UNSUPPORTED, WS = codes()

    def call(w=P, stride=64, q=P, n=2, win=1, h=16, k=P, nb=8, bs=16, hkv=4, d=128, tab=P, m=4, lens=P, ml=64, scale=0.1,
             ws=P, wb=1 << 40):
        return lib.pa_accumulate_weights(w, stride, q, n, win, h, k, nb, bs, hkv, d, tab, m, lens, ml, scale, ws, wb, None)

    for name in ("w", "q", "k", "tab", "lens"):
        assert call(**{name: None}) == BAD
    assert call(w=P + 2) == BAD and call(q=P + 8) == BAD and call(k=P + 8) == BAD
    assert call(stride=63) == BAD and call(n=-1) == BAD and call(win=0) == BAD and call(h=15) == BAD and call(ml=65) == BAD
    assert call(scale=float("nan")) == BAD
    assert call(d=96) == UNSUPPORTED and call(bs=4, m=16) == UNSUPPORTED and call(h=516) == UNSUPPORTED
    assert call(n=65536) == UNSUPPORTED
    assert call(ws=None) == WS and call(ws=P + 64) == WS and call(wb=8) == WS
    assert call(n=0, w=None) == OK and call(ml=0, w=None) == OK

    def select(keep=P, nk=4, cu=P, w=P, stride=64, start=P, lens=P, n=2, recent=0, ml=64, status=None):
        return lib.pa_select_tokens(keep, nk, cu, w, stride, start, lens, n, recent, ml, status, None)

    for name in ("keep", "cu", "w", "start", "lens"):
        assert select(**{name: None}) == BAD
    assert select(nk=-1) == BAD and select(recent=-1) == BAD and select(n=-1) == BAD and select(ml=-1) == BAD
    assert select(stride=63) == BAD and select(status=P + 2) == BAD and select(ml=(1 << 30) + 1, stride=1 << 31) == UNSUPPORTED
    assert select(n=0, w=None) == OK and select(ml=0, w=None) == OK


def test_binding_refusals(lib):
    import torch
    from paged_kv_cache_142_gb300 import ops
    b = torch.bfloat16
    cache = torch.zeros(4, 16, 576, dtype=b)
    with pytest.raises(ValueError):
        ops.pa_reshape_and_cache_latent(torch.zeros(3, 512), torch.zeros(3, 64), torch.zeros(3, dtype=torch.int64), cache)
    with pytest.raises(ValueError):
        ops.pa_reshape_and_cache_latent(torch.zeros(3, 512, dtype=b), torch.zeros(2, 64, dtype=b),
                                        torch.zeros(3, dtype=torch.int64), cache)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.pa_decode_latent(torch.zeros(2, 16, 512), torch.zeros(2, 16, 575, dtype=b), cache, i32(2, 4), i32(2), 0.1, 64, ws)
    with pytest.raises(ValueError):
        ops.pa_decode_latent(torch.zeros(2, 16, 576), torch.zeros(2, 16, 576, dtype=b), cache, i32(2, 4), i32(2), 0.1, 64, ws)
    with pytest.raises(ValueError):
        ops.pa_prefill_latent(torch.zeros(5, 2, 128), torch.zeros(5, 2, 192, dtype=b), cache, torch.zeros(3, 128, 512, dtype=b),
                              torch.zeros(3, 128, 512, dtype=b), i32(3), i32(2), i32(2, 4), 0.1, 4, 64, 128, ws)
    with pytest.raises(ValueError):
        ops.pa_accumulate_weights(torch.zeros(2, 63), torch.zeros(2, 16, 576, dtype=b), cache, i32(2, 4), i32(2), 0.1, 1, 64, ws)
    with pytest.raises(ops.PAError):
        ops.make_workspace_latent(2, 1, 129, 512, 64, 16, 64)
