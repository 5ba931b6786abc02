"""What the calls report where their bounds leave nothing to do."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("width", [0, 4])
@pytest.mark.parametrize("cu,start,lens,bad", [
    ((0, 1), (0,), (0,), True), ((0, 0), (0,), (3,), True), ((0, 1), (0,), (3,), True), ((0, 0), (1,), (1,), True),
    ((0, 0), (0,), (0,), False), ((0, 0, 0), (0, 0), (0, 0), False), ((0, 0, 1), (0, 0), (0, 0), True)])
def test_selection_bounded_by_no_tokens(ops, cu, start, lens, bad, width):
    keep, status = torch.full((2,), -1, dtype=torch.int32, device="cuda"), new_status()
    w = torch.full((len(lens), width), 5.0, device="cuda")
    ops.pa_select_tokens(keep, ints(*cu), w, ints(*start), ints(*lens), 1, 0, status=status)
    assert int(status.item()) == int(bad)
    assert (keep == -1).all() and (w == 5).all()
    ops.pa_select_tokens(keep, ints(*cu), w, ints(*start), ints(*lens), 1, 0)  # nobody to tell
    assert (keep == -1).all() and (w == 5).all()


@pytest.mark.parametrize("width", [0, 4])
@pytest.mark.parametrize("window,heads,d", [(1, 8, 128), (40, 8, 64), (2, 4, 576), (3, 2, 256)])
def test_weights_bounded_by_no_tokens(ops, window, heads, d, width):
    hkv = 1 if d == 576 else 2
    q = torch.randn(3, window, heads, d, device="cuda").bfloat16()
    cache = torch.randn(4, hkv, 16, d, device="cuda").bfloat16()
    tables = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    w = torch.full((3, width), 5.0, device="cuda")
    for lens, error in (((0, 0, 0), 0), ((0, 1, 0), 1), ((0, 0, -1), 1), ((2 ** 31 - 1, 0, 0), 1)):
        ws = ops.make_workspace_weights(3, window, heads, hkv, d, 16, 0)
        ops.pa_accumulate_weights(w, q, cache, tables, ints(*lens), 0.1, hkv, 0, ws)
        assert ops.pa_workspace_error(ws) == error
        assert (w == 5).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,longest,cu,bad", [
    (0, 4, (0, 3), True), (0, 4, (0, 0), False), (5, 0, (0, 5), True), (5, 0, (0, 0), False), (0, 0, (0, 0, 1, 1), True),
    (0, 4, (0, -1), True), (5, 4, (0, 5), True), (5, 0, (5, 5), False)])
def test_prefill_bounded_by_no_queries(ops, tokens, longest, cu, bad, dt):
    S, H = len(cu) - 1, 2
    e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    out = torch.full((tokens, H, 128), -7.0, dtype=dt, device="cuda")
    ws = ops.make_prefill_workspace_latent(S, H, 512, 64, 128, 16, longest, 16, 16)
    tables, start = torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    args = (out, e(tokens, H, 192), e(4, 16, 576), e(H, 128, 512), e(H, 128, 512), ints(*cu), start, tables, 0.1, longest, 16, 16, ws)
    status = new_status()
    ops.pa_prefill_latent(*args, status=status)
    assert int(status.item()) == int(bad)
    assert (out == -7).all()
    ops.pa_prefill_latent(*args)  # nobody to tell
    assert (out == -7).all()


@pytest.mark.parametrize("latent", [True, False])
@pytest.mark.parametrize("entries,most,cu,bad", [(0, 5, (0, 2), True), (0, 5, (0, 0), False), (4, 0, (0, 2), True),
                                                 (4, 0, (0, 0, 0), False), (4, 0, (0, 0, -1), True)])
def test_compaction_bounded_by_no_tokens(ops, entries, most, cu, bad, latent):
    S = len(cu) - 1
    shape = (4, 16, 576) if latent else (4, 2, 16, 64)
    cache = torch.randn(shape, device="cuda").bfloat16()
    before = cache.clone()
    tables = torch.tensor([[0, 1]] * S, dtype=torch.int32, device="cuda")
    keep, start = torch.arange(entries, dtype=torch.int32, device="cuda") + 3, torch.zeros(S, dtype=torch.int32, device="cuda")
    args = (tables, start, keep, ints(*cu), most)
    call = (lambda **kw: ops.pa_compact_tokens_latent(cache, *args, **kw)) if latent else (
        lambda **kw: ops.pa_compact_tokens(cache, cache, *args, **kw))
    status = new_status()
    call(status=status)
    assert int(status.item()) == int(bad)
    call()  # nobody to tell
    assert torch.equal(cache, before)
