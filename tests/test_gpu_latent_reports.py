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
