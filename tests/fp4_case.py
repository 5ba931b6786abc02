"""Test helpers of the 4-bit cache: pools of quantised random values, and the
error bounds of attention over them."""
import numpy as np

from oracle import fp4
from paged_kv_cache_142_gb300 import workloads as W


def bf16(x):
    return W.Values.from_f32(np.asarray(x, dtype=np.float32), "bf16")


def pool(rng, nb, hkv, bs, d, gscale, sigma=0.5, garbage=False):
    """A pool [NB, Hkv, tile] of quantised normal values; ``garbage``: random
    bytes instead (any code, any scale, NaN among them)."""
    if garbage:
        return rng.integers(0, 256, size=(nb, hkv, fp4.tile_bytes(bs, d)), dtype=np.uint8)
    out = np.zeros((nb, hkv, fp4.tile_bytes(bs, d)), dtype=np.uint8)
    codes, scales = fp4.quantise(bf16(rng.standard_normal((nb, hkv, bs, d)) * sigma).f32, gscale)
    n = bs * d // 2
    out[..., :n] = codes.reshape(nb, hkv, -1)
    out[..., n:n + bs * d // 16] = scales.reshape(nb, hkv, -1)
    return out


def attention_bound(q, K, V, scale):
    """Largest error of one row's output in fp32, per head, for q [H, D] and
    K, V [T, Hkv, D]:

      score   |ds| <= (D + 4) 2^-23 scale sum_d |q_d K_d|: D exact products
              summed in fp32 by tensor cores (an addition is off by at most one
              unit, 2^-23, where it is cut instead of rounded), the scaling and
              the subtraction of the reference
      weight  a relative 2 ds from the score in numerator and sum, 2^-21 from
              the exponential, and half a step of the weight's f16, 2^-12
      sum     (T + 64) 2^-23 for fp32 additions of weights and outputs, merging
              included
    all times max |V| over the row's keys."""
    H, D = q.shape
    T, Hkv, _ = K.shape
    if T == 0:
        return np.zeros(H)
    G = H // Hkv
    out = np.empty(H)
    for h in range(H):
        k, v = np.abs(K[:, h // G]), np.abs(V[:, h // G])
        ds = (D + 4) * 2.0 ** -23 * abs(scale) * float((k @ np.abs(q[h])).max())
        out[h] = float(v.max()) * (2 * ds + 2.0 ** -21 + 2.0 ** -12 + (T + 64) * 2.0 ** -23)
    return out
