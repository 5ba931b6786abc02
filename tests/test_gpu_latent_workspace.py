"""One workspace of the largest call for calls of every smaller shape, in any order."""
import numpy as np
import pytest
import torch

from latent_case import ROW, check, dev16
from oracle import latent as O
from test_gpu_evict import run_weights, weights_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(lib):
    import importlib
    return importlib.import_module("paged_kv_cache_142_gb300.ops")


@pytest.mark.parametrize("d,hkv,G,top", [(128, 2, 4, 3000), (64, 1, 8, 2000), (256, 2, 2, 900), (ROW, 1, 16, 1500)])
def test_one_weights_workspace_for_many_shapes(ops, d, hkv, G, top):
    """Sized for the longest window and context, used for shorter ones in between (steps
    behind a prompt), the windows on both sides of where scores are formed again."""
    rng = np.random.default_rng(d)
    widest = 40
    ws = ops.make_workspace_weights(4, widest, hkv * G, hkv, d, 16, top)
    again = 56 // G
    for W, lens in ((widest, [top, 5, 0, 700]), (1, [top, 1]), (again, [600, top, 9, 64]), (again + 1, [64, 33]),
                    (2, [top // 2] * 4), (widest, [300] * 3), (again, [top])):
        tables, k, q, before = weights_case(rng, lens, 16, W, hkv * G, hkv, d)
        check(run_weights(ops, before, q, dev16(k), tables, lens, 16, d ** -0.5, ws=ws),
              *O.weights(before, q.f32, k.f32, tables, lens, d ** -0.5), False)
