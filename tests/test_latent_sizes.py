"""Workspaces of the latent cache and of eviction grow with every argument, so
that one made for the largest call serves the smaller ones (no GPU needed)."""
import random

import pytest


def grows(size, draw, argument):
    """size(*a) <= size(*b) where b is a with one argument larger (0: refused, as is everything above)."""
    rng = random.Random(argument)
    pairs = 0
    for _ in range(4000):
        a = draw(rng)
        b = list(a)
        b[argument] = draw(rng)[argument]
        a[argument], b[argument] = sorted((a[argument], b[argument]))
        small, large = size(*a), size(*b)
        if large:
            assert 0 < small <= large, (a, b, small, large)
            pairs += a != b
    assert pairs > 1000


def log(rng, top):
    return min(top, int(2 ** rng.uniform(0, top.bit_length())))


@pytest.mark.parametrize("argument", [0, 1, 2, 3, 5])  # sequences, window, group, kv heads, context
@pytest.mark.parametrize("d", [64, 128, 256, 576])
def test_weights_workspace_grows(lib, d, argument):
    def size(n, window, group, hkv, bs, most):
        return lib.pa_accumulate_weights_workspace_size(n, window, group * hkv, hkv, d, bs, most)

    grows(size, lambda r: [log(r, 4096), log(r, 300), log(r, 128), 1 if d == 576 and argument != 3 else log(r, 32), 16,
                           log(r, 1 << 20)], argument)


@pytest.mark.parametrize("argument", [0, 1, 2, 4])
def test_decode_workspace_grows(lib, argument):
    def size(n, q_len, heads, bs, most):
        return lib.pa_decode_latent_workspace_size(n, q_len, heads, 512, 64, bs, most)

    grows(size, lambda r: [log(r, 4096), log(r, 300), log(r, 128), 16, log(r, 1 << 20)], argument)


@pytest.mark.parametrize("argument", [0, 1, 2, 3, 4])
def test_prefill_workspace_grows(lib, argument):
    def size(n, heads, longest, most, total):
        return lib.pa_prefill_latent_workspace_size(n, heads, 512, 64, 128, 16, longest, most, total)

    grows(size, lambda r: [log(r, 1024), log(r, 128), log(r, 4096), log(r, 1 << 16), log(r, 1 << 18)], argument)


def test_a_prompt_windows_workspace_serves_the_steps_behind_it(lib):
    """A window of 14 under one of 15, which stores no scores; 8192 tokens under 16384, of which fewer sequences fit a launch."""
    size = lib.pa_accumulate_weights_workspace_size
    assert size(8, 14, 32, 8, 128, 16, 16384) <= size(8, 15, 32, 8, 128, 16, 16384) <= size(8, 32, 32, 8, 128, 16, 16384)
    assert size(4, 32, 128, 1, 576, 16, 8192) <= size(4, 32, 128, 1, 576, 16, 16384)
    assert size(8, 1, 32, 8, 128, 16, 16384) <= size(8, 32, 32, 8, 128, 16, 16384)
    # and no launch's room is more than half a gigabyte, or one sequence's
    for window in (1, 14, 15, 32, 300):
        assert size(4096, window, 32, 8, 128, 16, 16384) < (512 << 20) + 4096
