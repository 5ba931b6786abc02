"""Test helpers of the latent cache and of eviction: pools, tables and calls."""
import numpy as np
import torch

from paged_kv_cache_142_gb300 import workloads as W

LATENT, ROPE, HEAD = 512, 64, 128
ROW = LATENT + ROPE


def bf16(x):
    return W.Values.from_f32(np.asarray(x, dtype=np.float32), "bf16")


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def dev16(v):
    """Values.bits of a bf16 array as a CUDA bf16 tensor."""
    return torch.from_numpy(np.ascontiguousarray(v.bits)).view(torch.bfloat16).cuda()


def tables_of(rng, lens, bs, spare=3, pad=0):
    """Shuffled tables int32 [B, M] (``pad`` behind a sequence's pages) and the pool's block count."""
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + spare
    order = rng.permutation(nb)
    t = np.full((len(lens), max(1, max(need))), pad, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, nb


def blank_unused(cache, tables, lens, bs, fill, heads=False):
    """A copy of the pool in which every row that no sequence uses holds ``fill``."""
    used = np.zeros((cache.shape[0], bs), dtype=bool)
    for i, n in enumerate(lens):
        t = np.arange(int(n))
        used[tables[i, t // bs], t % bs] = True
    out = cache.clone()
    hide = ~torch.from_numpy(used).to(cache.device)
    if heads:
        out.transpose(1, 2)[hide] = fill
    else:
        out[hide] = fill
    return out


def check(out, ref, tol, bf16_out):
    got = out.double().cpu().numpy()
    assert got.shape == ref.shape
    limit = tol + (2.0 ** -8 if bf16_out else 2.0 ** -24) * (np.abs(ref) + tol) + 1e-30
    bad = ~(np.abs(got - ref) <= limit)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, the first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} instead of {ref[bad][0]}, allowed {limit[bad][0]}")
