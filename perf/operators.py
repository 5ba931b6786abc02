"""Measured cases of the 4-bit paged KV cache and of page compaction.

Four operators, each in its plain torch form (``own`` false) and as the
library's calls (``own`` true), on the same state:

  append   pa_reshape_and_cache_fp4, then pa_gather_cache_fp4 of the same
           slots: a step's or a prompt's K/V quantised into the pages, and
           read back as the values the pages hold
  decode   pa_decode_fp4: one query per sequence over its pages
  prefill  pa_prefill_fp4: a chunk of queries per sequence, causal
  compact  pa_compact_tokens: the kept tokens of each sequence moved to the
           front of its pages (bf16 pools: every layer of the pool; 4-bit
           pools: then read back as values)

The 4-bit format: a row of head_dim values is cut into groups of 16.  With
a = the group's largest magnitude / global scale (a power of two), the
group's scale is s = a / 6 rounded to e4m3 (nearest, ties to even, at most
448), and a value x is stored as x / global scale / s rounded to e2m1
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; nearest, ties to the even code).  A
(block, kv head) tile holds block_size rows of head_dim / 2 code bytes (even
element in the low nibble), then block_size rows of head_dim / 16 scale
bytes, padded to 16 bytes.
"""
import math

import numpy as np
import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one generation step of a 256-sequence batch: latency counts
        _append("append step 256", 256, 8, 128, 16, "bf16", pad=0),
        # fp32 model, head_dim 64, an odd token count with padded slots
        _append("append fp32 odd", 4097, 4, 64, 16, "f32", pad=5),
        # the prompts of a 16 x 2048 prefill: bandwidth counts
        _append("append prompts", 32768, 8, 128, 16, "bf16", pad=0),
        # a single short request: launch and load latency
        _decode("decode one short", "uniform", 1, 17, 17, 32, 8, 128, 16),
        # the batch-256 GQA step, lognormal lengths
        _decode("decode gqa b256", "lognormal", 256, 16, 4096, 32, 8, 128, 16),
        # multi-head attention (every query head its own K/V), some rows empty
        _decode("decode mha b64", "uniform", 64, 0, 2048, 32, 32, 128, 16),
        # long contexts, few sequences: work split over the tokens
        _decode("decode long 8x32768", "uniform", 8, 32768, 32768, 64, 8, 128, 32),
        # a few drafted tokens per sequence checked against their history
        _prefill("prefill drafts", 16, 3, 9, 300, 1500, 32, 8, 16),
        # next piece of a long prompt: a short chunk over a long history
        _prefill("prefill chunk", 2, 200, 512, 8000, 16000, 32, 8, 16),
        # whole prompts
        _prefill("prefill 16x2048", 16, 2048, 2048, 0, 0, 32, 8, 16),
        # accepted draft tokens moved behind the committed ones, every layer
        _compact("compact accepted", "bf16", 32, 64, 40, 80, 1, 8, 32, 8, 128, 16),
        # half of a long history dropped, 4-bit pages
        _compact("compact evicted", "fp4", 1, 16, 1, 64, 1900, 2100, 4096, 8, 128, 16),
    ]


def _append(name, tokens, hkv, d, bs, src, pad, lens_seed=1):
    return dict(name=name, op="append", tokens=tokens, hkv=hkv, d=d, bs=bs, src=src, pad=pad, lens_seed=lens_seed)


def _decode(name, kind, seqs, lo, hi, h, hkv, d, bs, lens_seed=1):
    return dict(name=name, op="decode", kind=kind, seqs=seqs, lo=lo, hi=hi, h=h, hkv=hkv, d=d, bs=bs,
                lens_seed=lens_seed)


def _prefill(name, seqs, qlo, qhi, slo, shi, h, hkv, bs, lens_seed=1):
    return dict(name=name, op="prefill", seqs=seqs, qlo=qlo, qhi=qhi, slo=slo, shi=shi, h=h, hkv=hkv, d=128, bs=bs,
                lens_seed=lens_seed)


def _compact(name, dtype, layers, seqs, slo, shi, klo, khi, span, hkv, d, bs, lens_seed=1):
    """Sequence i keeps klo..khi of the span tokens behind its first slo..shi."""
    return dict(name=name, op="compact", dtype=dtype, layers=layers, seqs=seqs, slo=slo, shi=shi, klo=klo, khi=khi,
                span=span, hkv=hkv, d=d, bs=bs, lens_seed=lens_seed)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "compact"])
    seed = rng.randrange(2, 1 << 30)
    if op == "append":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        tokens = _log(rng, 1, 32768 * 8 * 128 // (hkv * d) if hkv * d > 1024 else 32768)
        c = _append("", tokens, hkv, d, rng.choice([1, 8, 16, 32, 128]), rng.choice(["bf16", "f32"]),
                    rng.randrange(0, 1 + min(9, tokens // 4)), seed)
    elif op == "decode":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        seqs = _log(rng, 1, 256)
        most = max(64, min(32768, 250_000 // seqs))  # tokens of the batch: no more than the listed ones
        hi = _log(rng, 33, most)
        c = _decode("", rng.choice(["uniform", "lognormal"]), seqs, rng.choice([0, 1, hi // 2]), hi,
                    hkv * rng.choice([1, 2, 4, 8, 16]), hkv, d, rng.choice([4, 8, 16, 32, 64, 256]), seed)
    elif op == "prefill":
        hkv, seqs = rng.choice([1, 2, 4, 8]), _log(rng, 1, 16)
        qhi, shi = _log(rng, 2, 1500), rng.choice([0, _log(rng, 2, 8000)])
        c = _prefill("", seqs, rng.choice([0, 1, qhi // 2]), qhi, shi // 3, shi, hkv * rng.choice([1, 2, 4]), hkv,
                     rng.choice([8, 16, 32, 128]), seed)
    else:
        dtype, seqs, hkv = rng.choice(["bf16", "f32", "fp4"]), _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        span = _log(rng, 4, 60_000 // seqs)
        khi = rng.randrange(1, span + 1)
        c = _compact("", dtype, 1 if dtype == "fp4" else rng.choice([1, 3]), seqs, 0, _log(rng, 1, 100),
                     rng.randrange(0, khi + 1), khi, span, hkv, rng.choice([64, 128]),
                     rng.choice([4, 8, 16, 64]), seed)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes of a case (from its own numbers alone)
# ---------------------------------------------------------------------------
def _sizes(case):
    r = np.random.Generator(np.random.PCG64(case["lens_seed"]))
    op = case["op"]
    if op == "append":
        return None
    n = case["seqs"]
    if op == "decode":
        if case["kind"] == "lognormal":
            mid = 800.0 if case["hi"] >= 4096 else max(1.0, case["hi"] / 4)
            lens = np.clip(np.rint(np.exp(math.log(mid) + 0.5 * r.standard_normal(n))), max(case["lo"], 1), case["hi"])
        else:
            lens = r.integers(case["lo"], case["hi"], size=n, endpoint=True)
            lens[-1] = case["hi"]
        return lens.astype(np.int64)
    if op == "prefill":
        q = r.integers(case["qlo"], case["qhi"], size=n, endpoint=True)
        q[-1] = case["qhi"]
        return q.astype(np.int64), r.integers(case["slo"], case["shi"], size=n, endpoint=True).astype(np.int64)
    start = r.integers(case["slo"], case["shi"], size=n, endpoint=True).astype(np.int64)
    count = r.integers(case["klo"], case["khi"], size=n, endpoint=True).astype(np.int64)
    count[0] = max(count[0], 1)
    keep = [start[i] + np.sort(r.permutation(case["span"])[:count[i]]) for i in range(n)]
    return start, count, np.concatenate(keep).astype(np.int64)


def _tile_bytes(bs, d):
    return (bs * d * 9 // 16 + 15) // 16 * 16


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    row = hkv * d * 9 / 16  # one token's K or V in 4 bits
    if op == "append":
        e = 4 if case["src"] == "f32" else 2
        t = case["tokens"] - case["pad"]
        # key and value read, the pages written, the values read back written
        return {"bytes": 2 * t * (hkv * d * e + row + hkv * d * e) + 8 * case["tokens"], "flops": 0}
    if op == "decode":
        lens = _sizes(case)
        pages = int((-(-lens // case["bs"])).sum())
        io = 2 * case["seqs"] * case["h"] * d * 2
        return {"bytes": 2 * int(lens.sum()) * row + io + 4 * pages + 4 * case["seqs"],
                "flops": 4.0 * int(lens.sum()) * case["h"] * d}
    if op == "prefill":
        q, start = _sizes(case)
        keys = (q * start + q * (q + 1) // 2).sum()
        seen = np.where(q > 0, q + start, 0).sum()
        return {"bytes": 2 * int(seen) * row + 2 * int(q.sum()) * case["h"] * d * 2, "flops": 4.0 * int(keys) * case["h"] * d}
    start, count, keep = _sizes(case)
    moved = int(count.sum())
    if case["dtype"] == "fp4":
        return {"bytes": 2 * moved * (2 * row + hkv * d * 2) + 4 * moved, "flops": 0}
    e = 4 if case["dtype"] == "f32" else 2
    return {"bytes": 2 * moved * 2 * hkv * d * e * case["layers"] + 4 * moved, "flops": 0}


# ---------------------------------------------------------------------------
# the format, in elementary operations
# ---------------------------------------------------------------------------
def _quantise(x, gscale):
    """fp32 [..., D] -> code bytes [..., D/2], scale bytes [..., D/16] (uint8).
    Divisions of values of few bits: fp32 decides every border exactly."""
    g = (x.float() / gscale).reshape(*x.shape[:-1], -1, 16)
    a = g.abs().amax(-1) / 6.0
    # e4m3, to nearest even: 3 bits below the leading one, steps of 2^-9 at the bottom
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(min=-6).float() - 3)
    s = (torch.round(a / step) * step).clamp(max=448.0)
    m = (g.abs() / s.unsqueeze(-1)).clamp(max=6.0)
    m = torch.where(s.unsqueeze(-1) > 0, m, torch.zeros_like(m))
    # e2m1: steps of 0.5 below 2, of 1 below 4, of 2 below 6
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = torch.round(m / step) * step
    code = (2 * m).to(torch.uint8)                        # 0 1 2 3 4 6 8 12
    code = code - (code > 4).to(torch.uint8) - (code > 6).to(torch.uint8) - 3 * (code > 8).to(torch.uint8)  # 0 .. 7
    code = code | ((g < 0) & (code > 0)).to(torch.uint8) << 3
    code = code.reshape(*x.shape)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    return codes, s.to(torch.float8_e4m3fn).view(torch.uint8)


def _rows(cache, bs, d):
    """A pool's code bytes [NB, Hkv, bs, D/2] and scale bytes [NB, Hkv, bs, D/16], as views."""
    nb, hkv, _ = cache.shape
    c, s = cache[..., : bs * d // 2], cache[..., bs * d // 2: bs * d * 9 // 16]
    return c.unflatten(-1, (bs, d // 2)), s.unflatten(-1, (bs, d // 16))


def _values(codes, scales, gscale):
    """The fp32 values that code and scale bytes stand for."""
    t = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = torch.stack((t[(codes & 15).int()], t[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * gscale
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _write(cache, slots, x, bs, gscale):
    codes, scales = _quantise(x, gscale)
    c, s = _rows(cache, bs, x.shape[-1])
    ok = slots >= 0
    b, o = slots[ok] // bs, slots[ok] % bs
    c[b, :, o] = codes[ok]
    s[b, :, o] = scales[ok]


def _read(out, cache, slots, bs, gscale):
    c, s = _rows(cache, bs, out.shape[-1])
    ok = slots >= 0
    b, o = slots[ok] // bs, slots[ok] % bs
    out[ok] = _values(c[b, :, o], s[b, :, o], gscale).to(out.dtype)


def _pages(cache, tables, bs, d, gscale):
    """[B, Hkv, pages * bs, D] fp32 of every sequence's pages."""
    c, s = _rows(cache, bs, d)
    v = _values(c[tables], s[tables], gscale)  # [B, M, Hkv, bs, D]
    return v.transpose(1, 2).flatten(2, 3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
K_SCALE, V_SCALE = 0.0625, 0.03125


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, t, hkv, d):
    """Keys with a few strong channels, as trained models have them."""
    return (_normal(g, t, hkv, d) * torch.exp(0.5 * _normal(g, 1, hkv, d))).bfloat16()


def _tables(g, lens, bs, spare=1.2):
    """Shuffled block tables [B, M] (0 past a sequence's pages) and the pool's block count."""
    need = -(-lens // bs)
    nb = int(math.ceil(need.sum() * spare)) + 1
    perm = torch.randperm(nb, generator=g, device="cuda")
    need_t = torch.from_numpy(need).cuda()
    m = max(1, int(need.max()))
    first = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(m, device="cuda")
    at = first[:, None] + col
    t = torch.where(col < need_t[:, None], perm[at.clamp(max=nb - 1)], torch.zeros_like(at))
    return t.int(), nb


def _token_slots(tables, lens, bs):
    """Slots of every token, sequence after sequence."""
    lens_t = torch.from_numpy(lens).cuda()
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens_t)
    pos = torch.arange(int(lens.sum()), device="cuda") - (torch.cumsum(lens_t, 0) - lens_t)[seq]
    return tables[seq, pos // bs].long() * bs + pos % bs


def _pool(g, case, lens):
    bs, d, hkv = case["bs"], case["d"], case["hkv"]
    tables, nb = _tables(g, lens, bs)
    slots = _token_slots(tables, lens, bs)
    kc = torch.zeros(nb, hkv, _tile_bytes(bs, d), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    t = int(lens.sum())
    _write(kc, slots, _keys(g, t, hkv, d), bs, K_SCALE)
    _write(vc, slots, (_normal(g, t, hkv, d) * 0.5).bfloat16(), bs, V_SCALE)
    return tables, kc, vc


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, bs, d, hkv = case["op"], case["bs"], case["d"], case["hkv"]
    st = dict(case)
    if op == "append":
        t = case["tokens"]
        dt = torch.float32 if case["src"] == "f32" else torch.bfloat16
        nb = -(-t // bs) + 3
        st["slots"] = torch.randperm(nb * bs, generator=g, device="cuda")[:t]
        if t > bs:  # a prompt's tokens fill whole pages, in shuffled order of the pages
            st["slots"] = (torch.randperm(nb, generator=g, device="cuda")[:, None] * bs
                           + torch.arange(bs, device="cuda")).flatten()[:t].contiguous()
        if case["pad"]:
            st["slots"][torch.randperm(t, generator=g, device="cuda")[: case["pad"]]] = -1
        st["key"] = (_normal(g, t, hkv, d) * torch.exp(0.5 * _normal(g, 1, hkv, d))).to(dt)
        st["value"] = (_normal(g, t, hkv, d) * 0.5).to(dt)
        st["kc"] = torch.zeros(nb, hkv, _tile_bytes(bs, d), dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros_like(st["kc"])
        st["key_out"], st["value_out"] = torch.zeros_like(st["key"]), torch.zeros_like(st["value"])
        return st
    st["scale"] = float(np.float32(1.0 / math.sqrt(d)))
    if op == "decode":
        lens = _sizes(case)
        st["tables"], st["kc"], st["vc"] = _pool(g, case, lens)
        st["lens"] = torch.from_numpy(lens).int().cuda()
        st["max_len"] = int(lens.max())
        st["q"] = _normal(g, case["seqs"], case["h"], d).bfloat16()
        st["out"] = torch.zeros_like(st["q"])
        return st
    if op == "prefill":
        q, start = _sizes(case)
        st["tables"], st["kc"], st["vc"] = _pool(g, case, q + start)
        cu = np.concatenate([[0], np.cumsum(q)])
        st["cu"] = torch.from_numpy(cu).int().cuda()
        st["start"] = torch.from_numpy(start).int().cuda()
        st["max_q"], st["max_len"] = int(q.max()), int((q + start).max())
        st["q"] = _normal(g, int(q.sum()), case["h"], d).bfloat16()
        st["out"] = torch.zeros_like(st["q"])
        return st
    start, count, keep = _sizes(case)
    lens = start + case["span"]
    st["start"] = torch.from_numpy(start).int().cuda()
    st["keep"] = torch.from_numpy(keep).int().cuda()
    st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(count)])).int().cuda()
    st["max_keep"] = int(count.max())
    if case["dtype"] == "fp4":
        st["tables"], st["kc"], st["vc"] = _pool(g, case, lens)
        st["slots"] = _token_slots(st["tables"], start + count, bs)  # what is left, to be read back
        st["key_out"] = torch.zeros(int((start + count).sum()), hkv, d, dtype=torch.bfloat16, device="cuda")
        st["value_out"] = torch.zeros_like(st["key_out"])
        return st
    st["tables"], nb = _tables(g, lens, bs, 1.0)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    st["kc"] = torch.empty(case["layers"], nb, hkv, bs, d, dtype=dt, device="cuda").normal_(generator=g)
    st["vc"] = torch.empty_like(st["kc"]).normal_(generator=g)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill,
            "compact": _plain_compact}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_142_gb300 import ops

    op, bs, d, hkv = st["op"], st["bs"], st["d"], st["hkv"]
    if op == "append":
        ops.pa_reshape_and_cache_fp4(st["key"], st["value"], st["slots"], st["kc"], st["vc"], bs, K_SCALE, V_SCALE)
        ops.pa_gather_cache_fp4(st["key_out"], st["value_out"], st["slots"], st["kc"], st["vc"], bs, K_SCALE, V_SCALE)
        return {"key": st["key_out"], "value": st["value_out"]}
    if op == "decode":
        if "ws" not in st:  # kept with the state, as a program keeps it from step to step
            st["ws"] = ops.make_workspace_fp4(st["seqs"], st["h"], hkv, d, bs, st["max_len"])
        ops.pa_decode_fp4(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["lens"], st["scale"], hkv, bs,
                          st["max_len"], st["ws"], K_SCALE, V_SCALE)
        return {"out": st["out"]}
    if op == "prefill":
        if "ws" not in st:
            st["ws"] = ops.make_prefill_workspace_fp4(st["seqs"], st["h"], hkv, d, bs, st["max_q"], st["max_len"])
        ops.pa_prefill_fp4(st["out"], st["q"], st["kc"], st["vc"], st["cu"], st["start"], st["tables"], st["scale"],
                           hkv, bs, st["max_q"], st["max_len"], st["ws"], K_SCALE, V_SCALE)
        return {"out": st["out"]}
    if st["dtype"] == "fp4":
        ops.pa_compact_tokens(st["kc"], st["vc"], st["tables"], st["start"], st["keep"], st["cu"], st["max_keep"],
                              block_size=bs, head_dim=d)
        ops.pa_gather_cache_fp4(st["key_out"], st["value_out"], st["slots"], st["kc"], st["vc"], bs, K_SCALE, V_SCALE)
        return {"key": st["key_out"], "value": st["value_out"]}
    ops.pa_compact_tokens(st["kc"], st["vc"], st["tables"], st["start"], st["keep"], st["cu"], st["max_keep"])
    return {"key": st["kc"], "value": st["vc"]}


def _plain_append(st):
    for_k = (st["key"], st["kc"], st["key_out"], K_SCALE)
    for_v = (st["value"], st["vc"], st["value_out"], V_SCALE)
    _write(for_k[1], st["slots"], for_k[0], st["bs"], for_k[3])
    _write(for_v[1], st["slots"], for_v[0], st["bs"], for_v[3])
    _read(for_k[2], for_k[1], st["slots"], st["bs"], for_k[3])
    _read(for_v[2], for_v[1], st["slots"], st["bs"], for_v[3])
    return {"key": st["key_out"], "value": st["value_out"]}


def _softmax_values(s, mask, v):
    """sum_t softmax_t(s) v_t over the masked-in t (0 where none is)."""
    s = s.masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(st):
    bs, d, hkv = st["bs"], st["d"], st["hkv"]
    k = _pages(st["kc"], st["tables"], bs, d, K_SCALE)
    v = _pages(st["vc"], st["tables"], bs, d, V_SCALE)
    q = st["q"].float().unflatten(1, (hkv, -1)) * st["scale"]
    mask = torch.arange(k.shape[2], device="cuda") < st["lens"][:, None, None, None]
    o = _softmax_values(q @ k.transpose(-1, -2), mask, v)
    return {"out": o.flatten(1, 2).to(st["out"].dtype)}


def _plain_prefill(st):
    bs, d, hkv = st["bs"], st["d"], st["hkv"]
    k = _pages(st["kc"], st["tables"], bs, d, K_SCALE)
    v = _pages(st["vc"], st["tables"], bs, d, V_SCALE)
    n, mq, t = st["seqs"], st["max_q"], st["q"].shape[0]
    j = torch.arange(mq, device="cuda")
    have = j < (st["cu"][1:] - st["cu"][:-1])[:, None]                    # [S, Q]
    row = (st["cu"][:-1, None] + j).clamp(max=t - 1)
    q = st["q"][row].float().unflatten(2, (hkv, -1)) * st["scale"]        # [S, Q, Hkv, G, D]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                            # [S, Hkv, G * Q, D]
    pos = st["start"][:, None] + j
    seen = torch.arange(k.shape[2], device="cuda") <= pos[:, :, None]     # [S, Q, T]
    g = q.shape[2] // mq
    mask = seen[:, None, None].expand(n, 1, g, mq, -1).flatten(2, 3)
    o = _softmax_values(q @ k.transpose(-1, -2), mask, v)
    o = o.unflatten(2, (g, mq)).permute(0, 3, 1, 2, 4).flatten(2, 3)      # [S, Q, H, D]
    out = torch.zeros_like(st["q"])
    out[row[have]] = o[have].to(out.dtype)
    return {"out": out}


def _plain_compact(st):
    bs = st["bs"]
    count = (st["cu"][1:] - st["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(st["seqs"], device="cuda"), count)
    dst = st["start"][seq].long() + torch.arange(len(seq), device="cuda") - st["cu"][seq]
    src = st["keep"].long()
    sb, so = st["tables"][seq, src // bs].long(), src % bs
    db, do = st["tables"][seq, dst // bs].long(), dst % bs
    if st["dtype"] == "fp4":
        kc, ks = _rows(st["kc"], bs, st["d"])
        vc, vs = _rows(st["vc"], bs, st["d"])
        kc[db, :, do], ks[db, :, do], vc[db, :, do], vs[db, :, do] = (
            kc[sb, :, so], ks[sb, :, so], vc[sb, :, so], vs[sb, :, so])
        _read(st["key_out"], st["kc"], st["slots"], bs, K_SCALE)
        _read(st["value_out"], st["vc"], st["slots"], bs, V_SCALE)
        return {"key": st["key_out"], "value": st["value_out"]}
    st["kc"][:, db, :, do], st["vc"][:, db, :, do] = st["kc"][:, sb, :, so], st["vc"][:, sb, :, so]
    return {"key": st["kc"], "value": st["vc"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3():
    """Every finite value of e4m3 that is not negative, ascending: its index is its byte."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(x, levels):
    """Index of the level nearest to x >= 0; halfway, the even index."""
    mid = (levels[1:] + levels[:-1]) / 2
    up = torch.searchsorted(mid, x.contiguous(), right=True)   # a tie counts as above
    tie = x == mid[(up - 1).clamp(min=0)]
    return torch.where(tie & (up % 2 == 1), up - 1, up)


def _stored64(x, gscale):
    """The values that x becomes by being stored, by search among the levels."""
    lev, sc = torch.tensor(LEVELS, dtype=torch.float64, device="cuda"), _e4m3()
    y = x.double().reshape(-1, 16) / gscale
    s = sc[_nearest(y.abs().max(dim=1).values / 6, sc)][:, None]
    m = lev[_nearest(torch.where(s > 0, y.abs() / s, torch.zeros_like(y)), lev)]
    return (torch.sign(y) * m * s * gscale).reshape(x.shape)


def _held64(cache, slots, bs, d, gscale):
    """[n, Hkv, D] double of the tokens in `slots`, byte by byte."""
    lev, sc = torch.tensor(LEVELS, dtype=torch.float64, device="cuda"), _e4m3()
    half = d // 2
    rows = slots % bs
    byte = cache[slots // bs]                                             # [n, Hkv, tile]
    hkv = byte.shape[1]
    e = torch.arange(d, device="cuda")
    at = (rows[:, None] * half + e // 2)[:, None].expand(-1, hkv, -1)
    nib = (byte.gather(2, at).int() >> (4 * (e % 2)).int()) & 15
    at = (bs * half + rows[:, None] * (d // 16) + e // 16)[:, None].expand(-1, hkv, -1)
    s = sc[byte.gather(2, at).long()]
    return lev[(nib & 7).long()] * (1 - 2 * (nib >> 3)).double() * s * gscale


def _attend64(q, k, v, scale, first):
    """q [Q, H, D] at positions first + 0.., k and v [T, Hkv, D]: causal attention."""
    n, h, d = q.shape
    hkv = k.shape[1]
    out = torch.zeros(n, h, d, dtype=torch.float64, device="cuda")
    if k.shape[0] == 0 or n == 0:
        return out
    keys = torch.arange(k.shape[0], device="cuda")
    pos = first + torch.arange(n, device="cuda")
    for j in range(h):
        s = scale * (q[:, j].double() @ k[:, j // (h // hkv)].T)
        s[keys[None] > pos[:, None]] = -math.inf
        out[:, j] = torch.softmax(s, 1) @ v[:, j // (h // hkv)]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, bs, d = case["op"], case["bs"], case["d"]
    if op == "append":
        ok = (st["slots"] >= 0)[:, None, None]
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        return {"key": torch.where(ok, _stored64(st["key"], K_SCALE), zero),
                "value": torch.where(ok, _stored64(st["value"], V_SCALE), zero)}
    if op == "compact":
        start, count, keep = _sizes(case)
        cu = np.concatenate([[0], np.cumsum(count)])
        tables = st["tables"].cpu().numpy().astype(np.int64)
        if case["dtype"] == "fp4":
            kept = [np.concatenate([np.arange(start[i]), keep[cu[i]:cu[i + 1]]]) for i in range(case["seqs"])]
            slots = np.concatenate([tables[i, p // bs] * bs + p % bs for i, p in enumerate(kept)])
            slots = torch.from_numpy(slots).cuda()
            return {"key": _held64(st["kc"], slots, bs, d, K_SCALE), "value": _held64(st["vc"], slots, bs, d, V_SCALE)}
        old = {"key": st["kc"], "value": st["vc"]}
        new = {n: x.clone() for n, x in old.items()}
        for i in range(case["seqs"]):
            src = keep[cu[i]:cu[i + 1]]
            dst = start[i] + np.arange(len(src))
            for n in old:
                new[n][:, tables[i, dst // bs], :, dst % bs] = old[n][:, tables[i, src // bs], :, src % bs]
        return {n: x.double() for n, x in new.items()}
    if op == "decode":
        lens = _sizes(case)
        q_len, first = np.ones_like(lens), lens - 1
    else:
        q_len, first = _sizes(case)
        lens = first + q_len
    cu = np.concatenate([[0], np.cumsum(q_len)])
    tables = st["tables"].cpu().numpy().astype(np.int64)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        t = np.arange(lens[i] if q_len[i] else 0)
        slots = torch.from_numpy(tables[i, t // bs] * bs + t % bs).cuda()
        k, v = _held64(st["kc"], slots, bs, d, K_SCALE), _held64(st["vc"], slots, bs, d, V_SCALE)
        out[cu[i]:cu[i + 1]] = _attend64(st["q"][cu[i]:cu[i + 1]], k, v, st["scale"], int(first[i]))
    return {"out": out}
