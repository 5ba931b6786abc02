"""The latent cache's and eviction's bounded waits: one that runs out is reported,
every role ends, and the next call is right.

The library's test hook has the warps that take scores or results first wait, with
a short limit, for an event that never comes.  Nothing traps; the other roles run
out their own limits of 2 s, some of them one behind the other."""
import time

import numpy as np
import pytest
import torch

from latent_case import HEAD, LATENT, ROPE, ROW, dev, dev16
from test_gpu_evict import weights_case
from test_gpu_latent import decode_case, prefill_case

pytestmark = pytest.mark.gpu

TIMEOUT = 6  # PA_ERR_DEVICE_TIMEOUT


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


def stalled(lib, call):
    """What call() gives while the hook is on."""
    lib.pa_test_stall_decode(100_000)
    try:
        t0 = time.perf_counter()
        result = call()
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 30
    finally:
        lib.pa_test_stall_decode(0)
    return result


@pytest.mark.parametrize("lens,H,Q,dt", [([2000, 30, 0, 700], 16, 1, torch.bfloat16), ([900], 32, 1, torch.float32),
                                         ([3000, 64], 128, 1, torch.bfloat16), ([500, 700], 70, 3, torch.float32)])
def test_expired_wait_of_the_latent_decode(ops, lib, lens, H, Q, dt):
    rng = np.random.default_rng(H)
    tables, cache, q = decode_case(rng, lens, 16, H, Q)
    args = [dev16(q), dev16(cache), dev(tables), dev(np.array(lens, np.int32))]
    ws = ops.make_workspace_latent(len(lens), Q, H, LATENT, ROPE, 16, max(lens))

    def decode():
        out = torch.full((len(lens), Q, H, LATENT), float("nan"), dtype=dt, device="cuda")
        ops.pa_decode_latent(out, *args, 0.07, max(lens), ws)
        return out, ops.pa_workspace_error(ws)

    before, status = decode()
    assert status == 0
    assert stalled(lib, decode)[1] == TIMEOUT
    ops.pa_workspace_init(ws)
    again, status = decode()
    assert status == 0 and torch.equal(again, before)


@pytest.mark.parametrize("lens,W,H,hkv,d", [([3000, 100, 0], 1, 32, 8, 128), ([2000, 900], 32, 8, 2, 64),
                                            ([1500, 40], 1, 128, 1, ROW)])
def test_expired_wait_of_the_weights(ops, lib, lens, W, H, hkv, d):
    rng = np.random.default_rng(d)
    tables, k, q, base = weights_case(rng, lens, 16, W, H, hkv, d)
    args = [dev16(q), dev16(k), dev(tables), dev(np.array(lens, np.int32))]
    ws = ops.make_workspace_weights(len(lens), W, H, hkv, d, 16, max(lens))

    def weights():
        w = dev(base)
        ops.pa_accumulate_weights(w, *args, 0.1, hkv, max(lens), ws)
        return w, ops.pa_workspace_error(ws)

    before, status = weights()
    assert status == 0
    assert stalled(lib, weights)[1] == TIMEOUT
    ops.pa_workspace_init(ws)
    again, status = weights()
    assert status == 0 and torch.equal(again, before)


@pytest.mark.parametrize("chunks,H,dt", [([(200, 300), (0, 700)], 12, torch.bfloat16), ([(1500, 20)], 3, torch.bfloat16),
                                         ([(100, 90), (700, 3)], 5, torch.float32)])
def test_expired_wait_of_the_latent_prefill(ops, lib, chunks, H, dt):
    rng = np.random.default_rng(H)
    lens, tables, cache, cu, q, w_k, w_v = prefill_case(rng, chunks, 16, H)
    longest = max(n for _, n in chunks)
    args = [dev16(q), dev16(cache), dev16(w_k), dev16(w_v), dev(cu), dev(np.array([s for s, _ in chunks], np.int32)), dev(tables)]
    ws = ops.make_prefill_workspace_latent(len(chunks), H, LATENT, ROPE, HEAD, 16, longest, max(lens), sum(lens))
    ws.zero_()

    def prefill():
        out = torch.full((q.shape[0], H, HEAD), -7.0, dtype=dt, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.pa_prefill_latent(out, *args, 0.07, longest, max(lens), sum(lens), ws, status=status)
        return out, int(status.item())

    before, status = prefill()
    assert status == 0
    assert stalled(lib, prefill)[1] == TIMEOUT
    again, status = prefill()
    assert status == 0 and torch.equal(again, before)
