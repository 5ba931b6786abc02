"""Measured cases of the latent paged cache and of eviction by attention weight.

Five operators, each in its plain torch form (``own`` false) and as the
library's calls (``own`` true), on the same state:

  append   pa_reshape_and_cache_latent: a step's or a prompt's latent vectors
           and position keys written into the pages of a latent cache
  decode   pa_decode_latent: a few query tokens per sequence, every head over
           the one latent row of each token (absorbed form)
  prefill  pa_prefill_latent: a chunk of queries per sequence, causal, over
           keys and values expanded from the latent rows (expanded form)
  weights  pa_accumulate_weights: the probabilities that a window of queries
           gives each cached token, summed over queries and heads and added to
           the token's running weight (K pages or latent pages)
  select   pa_select_tokens: the tokens with the largest weights (and the most
           recent ones) that stay in the cache, as the position lists that the
           token compaction takes, with the weights moved along

A latent row has ``latent`` + ``rope`` values: the vector that every head's key
and value derive from, and the key part that carries the position.

  absorbed   s[h,t] = scale q[h] . row[t],   out[h] = sum_t softmax(s)[t] row[t][:latent]
  expanded   k[h,t] = (w_k[h] row[t][:latent], row[t][latent:]),  v[h,t] = w_v[h] row[t][:latent]
  weights    weight[t] += sum over queries and heads of softmax_t(scale q . k[t])
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, HEAD = 512, 64, 128  # latent and position parts of a row; a head's key (without position) and value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one generation step of a 256-sequence batch, the rows being slices
        # of one projection's output: latency counts
        _append("append step 256", 256, 16, "bf16", True, 0),
        # the prompts of a 16 x 2048 prefill: bandwidth counts
        _append("append prompts", 32768, 16, "bf16", False, 7),
        # a single short request: launch and load latency
        _decode("decode one short", "uniform", 1, 17, 17, 1, 16, 16),
        # the batch-256 step, lognormal lengths, a tensor-parallel share of the heads
        _decode("decode 16 heads b256", "lognormal", 256, 16, 4096, 1, 16, 16),
        # every head on one GPU, some rows empty: products and bytes in balance
        _decode("decode 128 heads b64", "uniform", 64, 0, 4096, 1, 128, 32),
        # next piece of a long prompt: a short chunk over a long history
        _prefill("prefill chunk", 2, 200, 512, 8000, 16000, 32, 16),
        # whole prompts
        _prefill("prefill 4x2048", 4, 2048, 2048, 0, 0, 128, 16),
        # weights kept up to date in every step of the batch-256 GQA decode
        _weights("weights step b256", "lognormal", 256, 16, 4096, 1, 32, 8, 128, 16),
        # a window of the prompt's last queries over long histories
        _weights("weights window", "uniform", 4, 9000, 16384, 32, 32, 8, 128, 16),
        # every head's step over latent pages
        _weights("weights latent", "uniform", 16, 1, 4096, 1, 128, 1, LATENT + ROPE, 32),
        # half of short histories dropped: latency counts
        _select("select short", 32, 4, 150, 700, 0.5, 16),
        # long histories cut down to a small budget
        _select("select long", 8, 4, 20000, 32768, 0.125, 64),
    ]


def _append(name, tokens, bs, dtype, joint, pad, lens_seed=1):
    """joint: latent and position rows are slices of one [tokens, latent + rope] tensor."""
    return dict(name=name, op="append", tokens=tokens, bs=bs, dtype=dtype, joint=joint, pad=pad, lens_seed=lens_seed)


def _decode(name, kind, seqs, lo, hi, qlen, h, bs, out="bf16", lens_seed=1):
    return dict(name=name, op="decode", kind=kind, seqs=seqs, lo=lo, hi=hi, qlen=qlen, h=h, bs=bs, out=out,
                lens_seed=lens_seed)


def _prefill(name, seqs, qlo, qhi, slo, shi, h, bs, out="bf16", lens_seed=1):
    return dict(name=name, op="prefill", seqs=seqs, qlo=qlo, qhi=qhi, slo=slo, shi=shi, h=h, bs=bs, out=out,
                lens_seed=lens_seed)


def _weights(name, kind, seqs, lo, hi, qlen, h, hkv, d, bs, lens_seed=1):
    return dict(name=name, op="weights", kind=kind, seqs=seqs, lo=lo, hi=hi, qlen=qlen, h=h, hkv=hkv, d=d, bs=bs,
                lens_seed=lens_seed)


def _select(name, seqs, first, lo, hi, share, recent, lens_seed=1):
    """Of lo..hi tokens a sequence, `share` of those behind the first ones stay."""
    return dict(name=name, op="select", seqs=seqs, first=first, lo=lo, hi=hi, share=share, recent=recent,
                lens_seed=lens_seed)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "weights", "select"])
    seed = rng.randrange(2, 1 << 30)
    if op == "append":
        tokens = _log(rng, 1, 32768)
        c = _append("", tokens, rng.choice([1, 8, 16, 32, 128]), rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                    rng.randrange(0, 1 + min(9, tokens // 4)), seed)
    elif op == "decode":
        seqs, h = _log(rng, 1, 256), rng.choice([1, 5, 8, 16, 32, 40, 64, 96, 128])
        hi = _log(rng, 33, max(64, min(32768, 250_000 // seqs)))
        c = _decode("", rng.choice(["uniform", "lognormal"]), seqs, rng.choice([0, 1, hi // 2]), hi,
                    rng.choice([1, 1, 1, 2, 3, 5]), h, rng.choice([8, 16, 32, 64, 128]), rng.choice(["bf16", "f32"]), seed)
    elif op == "prefill":
        seqs, h = _log(rng, 1, 8), rng.choice([1, 3, 8, 16, 32])
        qhi, shi = _log(rng, 2, 1500), rng.choice([0, _log(rng, 2, 8000)])
        c = _prefill("", seqs, rng.choice([0, 1, qhi // 2]), qhi, shi // 3, shi, h, rng.choice([8, 16, 32, 128]),
                     rng.choice(["bf16", "f32"]), seed)
    elif op == "weights":
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 33, max(64, min(32768, 250_000 // seqs)))
        if rng.random() < 0.4:
            hkv, d, group = 1, LATENT + ROPE, rng.choice([1, 16, 40, 128])
        else:
            hkv, d, group = rng.choice([1, 2, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8])
        c = _weights("", rng.choice(["uniform", "lognormal"]), seqs, rng.choice([0, 1, hi // 2]), hi,
                     rng.choice([1, 1, 3, 8, 32] if seqs <= 16 else [1, 1, 2]), hkv * group, hkv, d,
                     rng.choice([8, 16, 32, 64, 256]), seed)
    else:
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 2, max(64, min(131072, 400_000 // seqs)))
        first = rng.choice([0, 1, 4])
        c = _select("", seqs, first, max(first, hi // 3), max(first, hi), round(rng.uniform(0.02, 1.0), 3),
                    rng.choice([0, 1, 16, 64]), seed)
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
    if op in ("decode", "weights"):
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
    lens = r.integers(case["lo"], case["hi"], size=n, endpoint=True).astype(np.int64)
    count = np.rint((lens - case["first"]) * case["share"]).astype(np.int64)
    if count.sum() == 0:
        lens[0] = max(lens[0], case["first"] + 1)
        count[0] = 1
    return lens, count


def work(case):
    op = case["op"]
    if op == "append":
        e = 4 if case["dtype"] == "f32" else 2
        t = case["tokens"] - case["pad"]
        return {"bytes": 2 * t * (LATENT + ROPE) * e + 8 * case["tokens"], "flops": 0}
    row = LATENT + ROPE
    if op == "decode":
        lens, q = _sizes(case), case["qlen"]
        io = case["seqs"] * q * case["h"] * (2 * row + LATENT * (4 if case["out"] == "f32" else 2))
        keys = sum(np.maximum(lens - q + 1 + j, 0).sum() for j in range(q))
        return {"bytes": int(lens.sum()) * row * 2 + io + 4 * int((-(-lens // case["bs"])).sum()) + 4 * case["seqs"],
                "flops": 2.0 * int(keys) * case["h"] * (row + LATENT)}
    if op == "prefill":
        q, start = _sizes(case)
        h = case["h"]
        keys = int((q * start + q * (q + 1) // 2).sum())
        seen = int(np.where(q > 0, q + start, 0).sum())
        io = int(q.sum()) * h * ((HEAD + ROPE) * 2 + HEAD * (4 if case["out"] == "f32" else 2))
        return {"bytes": seen * row * 2 + io + 2 * h * HEAD * LATENT * 2,
                "flops": 2.0 * keys * h * (2 * HEAD + ROPE) + 2.0 * seen * h * 2 * HEAD * LATENT}
    if op == "weights":
        lens, w = _sizes(case), case["qlen"]
        keys = sum(np.maximum(lens - w + 1 + j, 0).sum() for j in range(w))
        return {"bytes": int(lens.sum()) * (case["hkv"] * case["d"] * 2 + 8) + case["seqs"] * w * case["h"] * case["d"] * 2
                + 4 * int((-(-lens // case["bs"])).sum()) + 4 * case["seqs"],
                "flops": 2.0 * int(keys) * case["h"] * case["d"]}
    lens, count = _sizes(case)
    # weights read and (moved or cleared) written, positions written
    return {"bytes": 8 * int((lens - case["first"]).sum()) + 4 * int(count.sum()) + 12 * case["seqs"], "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


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


def _latent_pool(g, nb, bs):
    """A pool of latent rows: a normalised vector with a few strong channels, then a position key."""
    gain = torch.cat([torch.exp(0.5 * _normal(g, LATENT)), torch.ones(ROPE, device="cuda")])
    return (_normal(g, nb, bs, LATENT + ROPE) * gain).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op == "append":
        t, bs = case["tokens"], case["bs"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        nb = -(-t // bs) + 3
        if t > bs:  # a prompt's tokens fill whole pages, in shuffled order of the pages
            st["slots"] = (torch.randperm(nb, generator=g, device="cuda")[:, None] * bs
                           + torch.arange(bs, device="cuda")).flatten()[:t].contiguous()
        else:
            st["slots"] = torch.randperm(nb * bs, generator=g, device="cuda")[:t]
        if case["pad"]:
            st["slots"][torch.randperm(t, generator=g, device="cuda")[: case["pad"]]] = -1
        rows = _normal(g, t, LATENT + ROPE).to(dt)
        st["latent"], st["rope"] = rows[:, :LATENT], rows[:, LATENT:]
        if not case["joint"]:
            st["latent"], st["rope"] = st["latent"].contiguous(), st["rope"].contiguous()
        st["cache"] = torch.zeros(nb, bs, LATENT + ROPE, dtype=dt, device="cuda")
        return st
    if op == "select":
        lens, count = _sizes(case)
        m = int(lens.max()) + 5
        # a few tokens hold most of the weight; many have none at all, so that ties occur
        w = torch.exp(2.0 * _normal(g, case["seqs"], m))
        st["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.3, torch.zeros_like(w), w)
        st["lens"] = torch.from_numpy(lens).int().cuda()
        st["start"] = torch.full((case["seqs"],), case["first"], dtype=torch.int32, device="cuda")
        st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(count)])).int().cuda()
        st["keep"] = torch.zeros(int(count.sum()), dtype=torch.int32, device="cuda")
        st["max_len"] = int(lens.max())
        return st
    bs = case["bs"]
    if op == "prefill":
        q, start = _sizes(case)
        st["tables"], nb = _tables(g, q + start, bs)
        st["cache"] = _latent_pool(g, nb, bs)
        st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q)])).int().cuda()
        st["start"] = torch.from_numpy(start).int().cuda()
        st["max_q"], st["max_len"], st["total"] = int(q.max()), int((q + start).max()), int((q + start).sum())
        h = case["h"]
        st["q"] = _normal(g, int(q.sum()), h, HEAD + ROPE).bfloat16()
        st["w_k"] = (_normal(g, h, HEAD, LATENT) / math.sqrt(LATENT)).bfloat16()
        st["w_v"] = (_normal(g, h, HEAD, LATENT) / math.sqrt(LATENT)).bfloat16()
        st["out"] = torch.zeros(int(q.sum()), h, HEAD, dtype=_dtype(case["out"]), device="cuda")
        st["scale"] = float(np.float32(1.0 / math.sqrt(HEAD + ROPE)))
        return st
    lens = _sizes(case)
    st["tables"], nb = _tables(g, lens, bs)
    st["lens"] = torch.from_numpy(lens).int().cuda()
    st["max_len"] = int(lens.max())
    n, w, h = case["seqs"], case["qlen"], case["h"]
    if op == "decode":
        st["cache"] = _latent_pool(g, nb, bs)
        # queries after the absorbed projection: of the size that scale expects of a head's own query
        st["q"] = (_normal(g, n, w, h, LATENT + ROPE) * math.sqrt((HEAD + ROPE) / (LATENT + ROPE))).bfloat16()
        st["out"] = torch.zeros(n, w, h, LATENT, dtype=_dtype(case["out"]), device="cuda")
        st["scale"] = float(np.float32(1.0 / math.sqrt(HEAD + ROPE)))
        return st
    hkv, d = case["hkv"], case["d"]
    if d == LATENT + ROPE:
        st["cache"] = _latent_pool(g, nb, bs).unsqueeze(1)
    else:
        st["cache"] = (_normal(g, nb, hkv, bs, d) * torch.exp(0.5 * _normal(g, 1, hkv, 1, d))).bfloat16()
    st["q"] = _normal(g, n, w, h, d).bfloat16()
    st["weights"] = torch.rand(n, st["max_len"] + 3, generator=g, device="cuda")
    st["scale"] = float(np.float32(1.0 / math.sqrt(d)))
    return st


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill,
            "weights": _plain_weights, "select": _plain_select}[st["op"]](st)


def _run_own(st):
    from paged_kv_cache_142_gb300 import ops

    op = st["op"]
    if op == "append":
        ops.pa_reshape_and_cache_latent(st["latent"], st["rope"], st["slots"], st["cache"])
        return {"cache": st["cache"]}
    if op == "decode":
        if "ws" not in st:  # kept with the state, as a program keeps it from step to step
            st["ws"] = ops.make_workspace_latent(st["seqs"], st["qlen"], st["h"], LATENT, ROPE, st["bs"], st["max_len"])
        ops.pa_decode_latent(st["out"], st["q"], st["cache"], st["tables"], st["lens"], st["scale"], st["max_len"],
                             st["ws"])
        return {"out": st["out"]}
    if op == "prefill":
        if "ws" not in st:
            st["ws"] = ops.make_prefill_workspace_latent(st["seqs"], st["h"], LATENT, ROPE, HEAD, st["bs"], st["max_q"],
                                                         st["max_len"], st["total"])
        ops.pa_prefill_latent(st["out"], st["q"], st["cache"], st["w_k"], st["w_v"], st["cu"], st["start"], st["tables"],
                              st["scale"], st["max_q"], st["max_len"], st["total"], st["ws"])
        return {"out": st["out"]}
    if op == "weights":
        if "ws" not in st:
            st["ws"] = ops.make_workspace_weights(st["seqs"], st["qlen"], st["h"], st["hkv"], st["d"], st["bs"],
                                                  st["max_len"])
        ops.pa_accumulate_weights(st["weights"], st["q"], st["cache"], st["tables"], st["lens"], st["scale"], st["hkv"],
                                  st["max_len"], st["ws"])
        return {"weights": st["weights"]}
    ops.pa_select_tokens(st["keep"], st["cu"], st["weights"], st["start"], st["lens"], st["recent"], st["max_len"])
    return {"keep": st["keep"], "weights": st["weights"]}


def _plain_append(st):
    ok = st["slots"] >= 0
    slots = st["slots"][ok]
    flat = st["cache"].view(-1, LATENT + ROPE)
    flat[slots, :LATENT] = st["latent"][ok]
    flat[slots, LATENT:] = st["rope"][ok]
    return {"cache": st["cache"]}


def _softmax(s, mask):
    """Probabilities over the masked-in last dimension (0 where none is)."""
    s = s.masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _seen(st, qlen, tokens):
    """[B, qlen, tokens]: query j of a sequence is its token len - qlen + j."""
    pos = st["lens"][:, None] - qlen + torch.arange(qlen, device="cuda")
    return torch.arange(tokens, device="cuda") <= pos[:, :, None]


def _plain_decode(st):
    rows = st["cache"][st["tables"]].flatten(1, 2).float()                      # [B, T, latent + rope]
    q = st["q"].float().flatten(1, 2) * st["scale"]                             # [B, Q * H, latent + rope]
    mask = _seen(st, st["qlen"], rows.shape[1]).repeat_interleave(st["h"], 1)
    o = _softmax(q @ rows.transpose(-1, -2), mask) @ rows[..., :LATENT]
    return {"out": o.unflatten(1, (st["qlen"], st["h"])).to(st["out"].dtype)}


def _plain_prefill(st):
    n, mq, t = st["seqs"], st["max_q"], st["q"].shape[0]
    rows = st["cache"][st["tables"]].flatten(1, 2).float()                      # [S, T, latent + rope]
    c = rows[:, None, :, :LATENT]
    k = c @ st["w_k"].float().transpose(-1, -2)                                 # [S, H, T, head]
    v = c @ st["w_v"].float().transpose(-1, -2)
    k = torch.cat([k, rows[:, None, :, LATENT:].expand(-1, st["h"], -1, -1)], -1)
    j = torch.arange(mq, device="cuda")
    have = j < (st["cu"][1:] - st["cu"][:-1])[:, None]                          # [S, Q]
    row = (st["cu"][:-1, None] + j).clamp(max=max(t - 1, 0))
    q = st["q"][row].float().transpose(1, 2) * st["scale"]                      # [S, H, Q, head + rope]
    seen = torch.arange(k.shape[2], device="cuda") <= (st["start"][:, None] + j)[:, :, None]
    o = (_softmax(q @ k.transpose(-1, -2), seen[:, None]) @ v).transpose(1, 2)  # [S, Q, H, head]
    out = torch.zeros_like(st["out"])
    out[row[have]] = o[have].to(out.dtype)
    return {"out": out}


def _plain_weights(st):
    hkv, w, h = st["hkv"], st["qlen"], st["h"]
    k = st["cache"][st["tables"]].transpose(1, 2).flatten(2, 3).float()         # [B, Hkv, T, D]
    k = k[:, :, : st["max_len"]]
    q = st["q"].float().unflatten(2, (hkv, -1)) * st["scale"]                   # [B, W, Hkv, G, D]
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                                  # [B, Hkv, W * G, D]
    mask = _seen(st, w, k.shape[2]).repeat_interleave(h // hkv, 1)
    p = _softmax(q @ k.transpose(-1, -2), mask[:, None])
    st["weights"][:, : st["max_len"]] += p.sum((1, 2))
    return {"weights": st["weights"]}


def _plain_select(st):
    w = st["weights"]
    pos = torch.arange(w.shape[1], device="cuda")[None]
    first, lens = st["start"][:, None], st["lens"][:, None]
    count = (st["cu"][1:] - st["cu"][:-1])[:, None]
    inside = (pos >= first) & (pos < lens)
    key = torch.where(inside, w, torch.full_like(w, -math.inf))
    key = torch.where(inside & (pos >= lens - count.clamp(max=st["recent"])), torch.full_like(w, math.inf), key)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    chosen = torch.zeros_like(order).scatter_(1, order, (pos < count).long().expand_as(order))  # by rank
    places = torch.sort(torch.where(chosen > 0, pos, w.shape[1]), 1).values                     # ascending positions
    total = st["keep"].shape[0]
    seq = torch.repeat_interleave(torch.arange(st["seqs"], device="cuda"), count[:, 0], output_size=total)
    j = torch.arange(total, device="cuda") - st["cu"][seq]
    src = places[seq, j]
    moved = torch.where(inside, torch.zeros_like(w), w)
    moved[seq, st["start"][seq] + j] = w[seq, src]
    w.copy_(moved)
    st["keep"].copy_(src)
    return {"keep": st["keep"], "weights": w}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _rows64(cache, table, n, bs):
    """[n, Hkv, D] double: the first n tokens of the pages [NB, Hkv, bs, D] that a table names."""
    t = torch.arange(n, device="cuda")
    return cache[table[t // bs].long(), :, t % bs].double()


def _softmax64(s, limit):
    """softmax of s [rows, T] over the first limit[row] columns; rows without any are zero."""
    s = s.masked_fill(torch.arange(s.shape[1], device="cuda")[None] >= limit[:, None], -math.inf)
    return torch.nan_to_num(torch.softmax(s, 1))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        cache = st["cache"].double()
        slots = st["slots"].tolist()
        have = [i for i, s in enumerate(slots) if s >= 0]
        at = torch.tensor([slots[i] for i in have], dtype=torch.int64, device="cuda")
        rows = torch.cat([st["latent"], st["rope"]], 1).double()
        cache[at // case["bs"], at % case["bs"]] = rows[torch.tensor(have, dtype=torch.int64, device="cuda")]
        return {"cache": cache}
    if op == "select":
        lens, count = _sizes(case)
        w = st["weights"].double().cpu().numpy()
        keep = []
        for i in range(case["seqs"]):
            a, b, n = case["first"], int(lens[i]), int(count[i])
            late = min(case["recent"], n)
            old = w[i, a:b - late]
            best = np.lexsort((np.arange(len(old)), -old))[: n - late]
            pick = np.concatenate([a + np.sort(best), np.arange(b - late, b)]).astype(np.int64)
            row = w[i].copy()
            row[a:b] = 0
            row[a:a + n] = w[i, pick]
            w[i] = row
            keep.append(pick)
        return {"keep": torch.from_numpy(np.concatenate(keep)).int().cuda(), "weights": torch.from_numpy(w).cuda()}
    bs, scale = case["bs"], st["scale"]
    if op == "prefill":
        if work(case)["flops"] > 8e12:
            return None
        q_len, first = _sizes(case)
        cu = np.concatenate([[0], np.cumsum(q_len)])
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["seqs"]):
            n, a = int(q_len[i]), int(first[i])
            if n == 0:
                continue
            x = _rows64(st["cache"].unsqueeze(1), st["tables"][i], a + n, bs)[:, 0]
            limit = a + 1 + torch.arange(n, device="cuda")
            for h in range(case["h"]):
                q = st["q"][cu[i]:cu[i + 1], h].double()
                s = q[:, :HEAD] @ (x[:, :LATENT] @ st["w_k"][h].double().T).T + q[:, HEAD:] @ x[:, LATENT:].T
                out[cu[i]:cu[i + 1], h] = _softmax64(scale * s, limit) @ (x[:, :LATENT] @ st["w_v"][h].double().T)
        return {"out": out}
    lens, w, h = _sizes(case), case["qlen"], case["h"]
    if op == "decode":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["seqs"]):
            n = int(lens[i])
            if n == 0:
                continue
            x = _rows64(st["cache"].unsqueeze(1), st["tables"][i], n, bs)[:, 0]
            for j in range(w):
                s = scale * (st["q"][i, j].double() @ x.T)
                limit = torch.full((h,), n - w + 1 + j, device="cuda")
                out[i, j] = _softmax64(s, limit) @ x[:, :LATENT]
        return {"out": out}
    total = st["weights"].double()
    group = h // case["hkv"]
    for i in range(case["seqs"]):
        n = int(lens[i])
        if n == 0:
            continue
        k = _rows64(st["cache"], st["tables"][i], n, bs)
        for j in range(w):
            limit = torch.full((group,), n - w + 1 + j, device="cuda")
            for a in range(case["hkv"]):
                s = scale * (st["q"][i, j, a * group:(a + 1) * group].double() @ k[:, a].T)
                total[i, :n] += _softmax64(s, limit).sum(0)
    return {"weights": total}
