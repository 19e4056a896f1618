"""Work of the operators of a target step whose cache is held in 4 bits: the
append that normalises, rotates (in halves or interleaved pairs) and rounds
rows into it, the attention that reads it, and the tables of the next step
(lengths, row starts, pages, slots) built on the GPU from what was accepted
and what is asked for.

A 4-bit head row goes in blocks of 16 elements: one e4m3 scale a block, one
e2m1 code an element (even elements in a byte's low half).

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program has in
hand before the call, ``run()`` one pass: the plain form in elementary torch
operations, or the library's calls where ``own`` is true.  ``exact()`` is the
definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one sequence: the smallest step, all latency
        {"name": "append4-decode-1", "op": "append", "n_seq": 1, "rows_lo": 1, "rows_hi": 1, "extra_lo": 776,
         "extra_hi": 776, "prefix": 0, "hq": 32, "hkv": 4, "d": 128, "rot": 128, "inter": False, "page": 64,
         "layout": "hnd", "in": "bf16", "dtype": "bf16", "norm": True, "yarn": False, "fused_qkv": True,
         "values": False, "shape_seed": 1},
        # 32 sequences verifying drafts of ragged length behind a shared prompt: interleaved pairs of half the head,
        # YaRN, f32 projections; the rounded rows are wanted as well
        {"name": "append4-verify-32", "op": "append", "n_seq": 32, "rows_lo": 1, "rows_hi": 17, "extra_lo": 0,
         "extra_hi": 3000, "prefix": 16383, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "inter": True, "page": 16,
         "layout": "nhd", "in": "f32", "dtype": "bf16", "norm": True, "yarn": True, "fused_qkv": False,
         "values": True, "shape_seed": 2},
        # prompts entering the cache: eight ragged prompts, normed heads, f16
        {"name": "append4-prompts-8", "op": "append", "n_seq": 8, "rows_lo": 1001, "rows_hi": 8191, "extra_lo": 0,
         "extra_hi": 0, "prefix": 0, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "page": 64,
         "layout": "hnd", "in": "f16", "dtype": "f16", "norm": True, "yarn": False, "fused_qkv": True,
         "values": False, "shape_seed": 3},
        # one new token of one short sequence: latency of the attention
        {"name": "attend4-decode-1", "op": "attend", "n_seq": 1, "rows_lo": 1, "rows_hi": 1, "extra_lo": 776,
         "extra_hi": 776, "prefix": 0, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "hnd", "dtype": "bf16",
         "causal": True, "shape_seed": 4},
        # a small model's ragged verification behind a short shared prompt; odd group, small pages, f16
        {"name": "attend4-ragged-8", "op": "attend", "n_seq": 8, "rows_lo": 1, "rows_hi": 17, "extra_lo": 0,
         "extra_hi": 300, "prefix": 2053, "hq": 12, "hkv": 4, "d": 64, "page": 16, "layout": "nhd", "dtype": "f16",
         "causal": True, "shape_seed": 5},
        # one long document being decoded with drafts of 15 tokens: split over the keys
        {"name": "attend4-long-1", "op": "attend", "n_seq": 1, "rows_lo": 16, "rows_hi": 16, "extra_lo": 131000,
         "extra_hi": 131000, "prefix": 0, "hq": 32, "hkv": 8, "d": 128, "page": 64, "layout": "hnd",
         "dtype": "bf16", "causal": True, "shape_seed": 6},
        # 64 long conversations decoding token by token, what a small cache is for: its bytes bound it
        {"name": "attend4-decode-64", "op": "attend", "n_seq": 64, "rows_lo": 1, "rows_hi": 1, "extra_lo": 1023,
         "extra_hi": 32767, "prefix": 4096, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "hnd",
         "dtype": "bf16", "causal": True, "shape_seed": 7},
        # 32 sequences verifying blocks of 16 behind a long shared prompt: matrix products bound it
        {"name": "attend4-verify-32", "op": "attend", "n_seq": 32, "rows_lo": 16, "rows_hi": 16, "extra_lo": 100,
         "extra_hi": 1024, "prefix": 16384, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "nhd",
         "dtype": "bf16", "causal": True, "shape_seed": 8},
        # three pieces of long prompts over what came before them
        {"name": "attend4-prompts-3", "op": "attend", "n_seq": 3, "rows_lo": 700, "rows_hi": 1500, "extra_lo": 0,
         "extra_hi": 8000, "prefix": 0, "hq": 32, "hkv": 8, "d": 128, "page": 64, "layout": "hnd", "dtype": "f16",
         "causal": True, "shape_seed": 9},
        # the next token of a few sequences: latency of the tables
        {"name": "next-decode-8", "op": "next", "n_seq": 8, "page": 64, "prefix": 0, "len_lo": 1, "len_hi": 2000,
         "prev_lo": 1, "prev_hi": 1, "rows_lo": 1, "rows_hi": 1, "verified": False, "done": 0.0, "short": False,
         "shape_seed": 10},
        # a batch whose drafts of 15 were verified: lengths shrink by the rejected and grow by the next block; some end
        {"name": "next-verify-256", "op": "next", "n_seq": 256, "page": 16, "prefix": 1000, "len_lo": 16,
         "len_hi": 5000, "prev_lo": 16, "prev_hi": 16, "rows_lo": 16, "rows_hi": 16, "verified": True, "done": 0.05,
         "short": False, "shape_seed": 11},
        # a full server: finished sequences give way to prompts, the pool runs out before all of them are in
        {"name": "next-batch-4000", "op": "next", "n_seq": 4000, "page": 16, "prefix": 0, "len_lo": 0,
         "len_hi": 3000, "prev_lo": 0, "prev_hi": 17, "rows_lo": 0, "rows_hi": 150, "verified": True, "done": 0.02,
         "short": True, "shape_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "next"])
    if op == "next":
        while True:
            prev = rng.choice([0, 1, 5, 16, 17])
            c = {"op": op, "n_seq": _log(rng, 1, 4096), "page": rng.choice([16, 32, 64, 128, 256]),
                 "prefix": rng.choice([0, _log(rng, 1, 32768)]), "len_lo": prev, "len_hi": prev + _log(rng, 1, 20000),
                 "prev_lo": rng.choice([0, prev]), "prev_hi": prev, "rows_lo": rng.choice([0, 1]),
                 "rows_hi": rng.choice([1, 1, 5, 16, 17, _log(rng, 20, 3000)]), "verified": rng.random() < 0.6,
                 "done": rng.choice([0.0, 0.1, 0.5]), "short": rng.random() < 0.3,
                 "shape_seed": rng.randint(1, 10 ** 9)}
            if c["n_seq"] * c["rows_hi"] <= 600000 and c["n_seq"] * c["len_hi"] <= 12000000:
                return c
    hkv = rng.choice([1, 2, 4, 8])
    while True:
        c = {"op": op, "n_seq": _log(rng, 1, 64), "rows_lo": rng.choice([0, 1, 1, 1]),
             "rows_hi": rng.choice([1, 1, 5, 16, 17, 33]), "extra_lo": 0, "extra_hi": _log(rng, 1, 32768),
             "prefix": rng.choice([0, _log(rng, 1, 32768)]), "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "hkv": hkv,
             "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "layout": rng.choice(["nhd", "hnd"]),
             "dtype": rng.choice(["bf16", "bf16", "f16"]), "shape_seed": rng.randint(1, 10 ** 9)}
        if op == "attend":
            c["causal"] = rng.random() < 0.85
            if rng.random() < 0.2:     # pieces of prompts
                c.update(n_seq=rng.randint(1, 4), rows_hi=_log(rng, 100, 1500), extra_hi=_log(rng, 1, 8000), prefix=0)
        else:
            c.update(rot=rng.choice([0, c["d"], c["d"], c["d"] // 2, c["d"] // 4]), inter=rng.random() < 0.5,
                     norm=rng.random() < 0.6, yarn=rng.random() < 0.3, fused_qkv=rng.random() < 0.5,
                     values=rng.random() < 0.4)
            c["in"] = rng.choice([c["dtype"], c["dtype"], "f32"])
            if rng.random() < 0.4:     # a prompt's rows rather than a step's
                c.update(n_seq=rng.randint(1, 8), rows_hi=_log(rng, 100, 6000), extra_hi=1)
        w = work(c)
        if sum(_shape(c)[0]) > 0 and w["flops"] <= 2.5e11 and w["bytes"] <= 6e8 and _cache_rows(c) * hkv <= 4.5e6:
            return c


def _shape(c):
    """Rows of the step and own cached keys (these rows included) of every sequence."""
    r = random.Random(c["shape_seed"])
    rows = [r.randint(c["rows_lo"], c["rows_hi"]) for _ in range(c["n_seq"])]
    return rows, [t + r.randint(c["extra_lo"], c["extra_hi"]) for t in rows]


def _cache_rows(c):
    return sum(_shape(c)[1]) + c["prefix"]


def _next_shape(c):
    """Lengths, rows of the step before, accepted drafts, finished ones and rows asked for, of every sequence."""
    r = random.Random(c["shape_seed"])
    prev = [r.randint(c["prev_lo"], c["prev_hi"]) for _ in range(c["n_seq"])]
    old = [max(t, r.randint(c["len_lo"], c["len_hi"])) for t in prev]
    acc = [r.randint(0, max(t - 1, 0)) for t in prev]
    done = [r.random() < c["done"] for _ in prev]
    rows = [r.randint(c["rows_lo"], c["rows_hi"]) for _ in prev]
    return old, prev, acc, done, rows


def _next_pool(c):
    """(pages of a sequence's table, pages in all, pages free before the step)."""
    old, prev, acc, done, rows = _next_shape(c)
    cols = max(-(-(n + t) // c["page"]) for n, t in zip(old, rows)) + 1
    held = sum(-(-n // c["page"]) for n in old)
    grow = sum(-(-t // c["page"]) + 1 for t in rows)
    free = grow // 8 if c["short"] else grow
    return cols, held + free + 5, free


def work(c):
    if c["op"] == "next":
        old, prev, acc, done, rows = _next_shape(c)
        moved = sum(max(0, -(-(n + t) // c["page"]) - -(-n // c["page"])) for n, t in zip(old, rows))
        return {"bytes": c["n_seq"] * 24 + sum(rows) * 16 + moved * 8, "flops": c["n_seq"] * 8 + sum(rows) * 4}
    rows, kv = _shape(c)
    R, d = sum(rows), c["d"]
    if c["op"] == "append":
        ei = 4 if c["in"] == "f32" else 2
        heads = c["hq"] + 2 * c["hkv"]
        out = R * (c["hq"] * d * 2 + 2 * c["hkv"] * (d // 2 + d // 16 + (2 * d if c["values"] else 0)))
        return {"bytes": R * heads * d * ei + out, "flops": R * heads * d * 8}
    keys = sum(kv) + (c["prefix"] if R else 0)
    pairs = 0
    for t, n in zip(rows, kv):
        pairs += t * (c["prefix"] + n) - (t * (t - 1) // 2 if c["causal"] else 0)
    return {"bytes": R * c["hq"] * (d * 4 + 4) + keys * c["hkv"] * 2 * (d // 2 + d // 16),
            "flops": 4 * pairs * c["hq"] * d}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def prepare(case, seed):
    return (_prepare_next if case["op"] == "next" else _prepare_step)(case, seed)


def _prepare_step(c, seed):
    g = _gen(seed)
    rows, kv = _shape(c)
    R, page, d, hq, hkv, dt = sum(rows), c["page"], c["d"], c["hq"], c["hkv"], _T[c["dtype"]]
    n_own = [-(-n // page) for n in kv]
    n_pre = -(-c["prefix"] // page)
    n_pages = sum(n_own) + n_pre + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).cpu().tolist()
    pre, order = order[:n_pre], order[n_pre:]
    cols = max(n_own + [1])
    table = torch.zeros(len(kv), cols, dtype=torch.int32)
    for i, n in enumerate(n_own):
        table[i, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    starts = [0]
    for t in rows:
        starts.append(starts[-1] + t)
    s = {"case": c, "rows": rows, "kv": kv, "starts": starts, "pre": torch.tensor(pre, dtype=torch.int32, device=DEV),
         "table": table.to(DEV), "row_start": torch.tensor(starts, dtype=torch.int32, device=DEV),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV)}
    # caches that were written before: codes and scales of normal rows
    for name in ("k", "v"):
        codes = torch.empty(n_pages, hkv, page, d // 2, dtype=torch.uint8, device=DEV)
        scales = torch.empty(n_pages, hkv, page, d // 16, dtype=torch.uint8, device=DEV)
        for p in range(0, n_pages, 2048):
            shape = (min(2048, n_pages - p), hkv, page, d)
            mag, neg, sc = _round4(_randn(g, *shape))
            code = mag | neg << 3
            codes[p:p + 2048] = code[..., ::2] | code[..., 1::2] << 4
            scales[p:p + 2048] = sc.float().to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scale"] = scales.transpose(1, 2).view(torch.float8_e4m3fn)
        # seen as [n_pages, page, heads, bytes] whichever way they lie
        s[name + "_cache"] = codes.transpose(1, 2) if c["layout"] == "hnd" else codes.transpose(1, 2).contiguous()
    if c["op"] == "append":
        ti = _T[c["in"]]
        if c["fused_qkv"]:     # one projection's rows hold q, k and v side by side
            x = _randn(g, R, (hq + 2 * hkv) * d, dtype=ti)
            q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
        else:
            q, k, v = (_randn(g, R, h * d, dtype=ti) for h in (hq, hkv, hkv))
        s.update(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)),
                 q_gain=None, k_gain=None)
        if c["norm"]:
            s.update(q_gain=1 + 0.1 * _randn(g, d), k_gain=1 + 0.1 * _randn(g, d))
        s["inv_freq"], s["mscale"] = _frequencies(c)
    else:
        # what lies behind a sequence's last key was never written
        for i, n in enumerate(kv):
            if n % page:
                p = int(table[i, n // page])
                for name in ("k", "v"):
                    s[name + "_scale"].view(torch.uint8)[p, n % page:] = 0x7F
        s["q"] = _randn(g, R, hq, d, dtype=dt)
    if own:
        from speculative_decoding_block_ingest_gb300 import target
        s["cache"] = target.PagedCache4(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], dtype=dt)
        s["step"] = target.Step(s["row_start"], s["kv_len"], s["table"], prefix_pages=s["pre"],
                                prefix_len=c["prefix"])
        if c["op"] == "append" and c["rot"]:
            yarn = {"yarn_factor": 32.0, "yarn_original_max_pos": 8192} if c["yarn"] else {}
            s["rope"] = target.Rope(c["rot"], theta=1e6, interleaved=c["inter"], **yarn)
    return s


def _prepare_next(c, seed):
    g = _gen(seed)
    old, prev, acc, done, rows = _next_shape(c)
    cols, n_pages, n_free = _next_pool(c)
    # the smallest integers of the seed: which pages are whose
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    have = torch.tensor([-(-n // c["page"]) for n in old], device=DEV)
    col = torch.arange(cols, device=DEV)
    held = col[None] < have[:, None]
    table = torch.full((c["n_seq"], cols), -1, dtype=torch.int32, device=DEV)
    table[held] = order[n_free:n_free + int(have.sum())]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[:n_free] = order[:n_free]
    start = [0]
    for t in prev:
        start.append(start[-1] + t)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    # what verification and the end of sequences say differs from step to step
    shift = int(torch.randint(0, 1 << 30, (1,), generator=g, device=DEV))
    acc = [(a + shift) % max(t, 1) for a, t in zip(acc, prev)]
    s = {"case": c, "cols": cols, "kv_len": ints(old), "row_start": ints(start), "table": table, "free": free,
         "n_free": ints([n_free]), "rows": ints(rows), "accepted": ints(acc) if c["verified"] else None,
         "keep": ints([0 if x else -1 for x in done]) if c["done"] else None, "n_rows": sum(rows)}
    n = s["n_rows"]
    s["slots"] = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    s["positions"], s["seqs"] = (torch.full((n,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    if own:
        from speculative_decoding_block_ingest_gb300 import target
        s["pool"] = target.PagePool(s["free"], s["n_free"], s["table"], s["kv_len"], s["row_start"],
                                    page_size=c["page"], prefix_len=c["prefix"])
        # the plan of a step goes beside the lengths it starts from
        s["next"] = s["pool"].beside()
    return s


def _frequencies(c):
    """Inverse frequencies [rot / 2] in 64 bits and the factor on cos and sin."""
    rot = c["rot"]
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    inv = 1e6 ** (-2 * j / max(rot, 1))
    if not c["yarn"] or not rot:
        return inv, 1.0
    factor, orig, fast, slow = 32.0, 8192, 32.0, 1.0
    lo, hi = (rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(1e6)) for turns in (fast, slow))
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return inv * (1 - ramp + ramp / factor), 0.1 * math.log(factor) + 1


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from speculative_decoding_block_ingest_gb300 import target
        if op == "append":
            c, values = s["case"], {}
            if c["values"]:
                values = {n + "_values": torch.empty(s["k"].shape, dtype=s["cache"].dtype, device=DEV) for n in "kv"}
            q = target.append(s["cache"], s["step"], s["q"], s["k"], s["v"], rope=s.get("rope"), q_gain=s["q_gain"],
                              k_gain=s["k_gain"], **values)
            return _appended(s, q, values.get("k_values"), values.get("v_values"))
        if op == "attend":
            return target.attention(s["cache"], s["step"], s["q"], causal=s["case"]["causal"])
        target.next_step(s["pool"], s["rows"], n_accepted=s["accepted"], keep=s["keep"], out=s["next"],
                         slots=s["slots"], positions=s["positions"], sequences=s["seqs"])
        return _planned(s, s["next"].kv_len, s["next"].row_start, s["next"].n_free)
    return {"append": _plain_append, "attend": _plain_attend, "next": _plain_next}[op](s)


def _appended(s, q, kv, vv):
    out = {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if kv is not None:
        out.update(k_values=kv, v_values=vv)
    return out


def _planned(s, kv_len, row_start, n_free):
    return {"kv_len": kv_len, "row_start": row_start, "n_free": n_free, "table": s["table"], "free": s["free"],
            "slots": s["slots"], "positions": s["positions"], "seqs": s["seqs"]}


def _round4(x):
    """Rows rounded to 4 bits: code magnitudes 0..7, signs (both uint8) and the scales, as the values they stand for."""
    b = x.unflatten(-1, (-1, 16))
    top = b.abs().amax(dim=-1)
    # e4m3: 4 significant bits down to 2^-6, then steps of 2^-9; ties to even
    a = (top / 6).clamp(max=448)
    e = torch.frexp(a)[1].clamp(min=-5) - 4
    step = ((e.long() + 1023) << 52).view(torch.float64).to(x.dtype)     # 2^e by its bits: pow() is not exact
    sc = (torch.round(a / step) * step).clamp(max=448)
    fine = torch.isfinite(top)
    sc = torch.where(fine, sc, float("nan"))
    t, u = b.abs(), sc[..., None]
    # ties go to the even code
    mag = ((t > 0.25 * u).to(torch.uint8) + (t >= 0.75 * u) + (t > 1.25 * u) + (t >= 1.75 * u) + (t > 2.5 * u)
           + (t >= 3.5 * u) + (t > 5 * u))
    some = (fine & (sc > 0))[..., None]
    neg = torch.signbit(b) & fine[..., None]
    return torch.where(some, mag, 0).flatten(-2), neg.to(torch.uint8).flatten(-2), sc


def _plain_append(s):
    c = s["case"]
    R, dt, half = s["q"].shape[0], _T[c["dtype"]], c["rot"] // 2
    # which sequence, own index and position each row has
    row = torch.arange(R, device=DEV, dtype=torch.int32)
    seq = (row[:, None] >= s["row_start"][None, 1:]).sum(dim=1)
    idx = s["kv_len"][seq] - s["row_start"][seq + 1] + row
    page, at = s["table"][seq, (idx // c["page"]).long()].long(), (idx % c["page"]).long()
    ang = (c["prefix"] + idx).double()[:, None] * s["inv_freq"]
    cos, sin = ((f(ang) * s["mscale"])[:, None] for f in (torch.cos, torch.sin))

    def head(x, gain):
        # 64 bits: rounding to 4 bits has its borders everywhere
        x = x.double()
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * gain
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        if c["inter"]:
            a, b = r[..., ::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, rest], dim=-1)

    values = []
    lut = torch.tensor(_E2M1, dtype=torch.float32, device=DEV)
    for name, x in (("k", head(s["k"], s["k_gain"])), ("v", s["v"].double())):
        mag, neg, sc = _round4(x)
        code = mag | neg << 3
        s[name + "_cache"][page, at] = code[..., ::2] | code[..., 1::2] << 4
        s[name + "_scale"].view(torch.uint8)[page, at] = sc.float().to(torch.float8_e4m3fn).view(torch.uint8)
        if c["values"]:
            y = (lut[mag.long()] * (1 - 2 * neg.float())).unflatten(-1, (-1, 16)) * sc.float()[..., None]
            values.append(y.flatten(-2).to(dt))
    return _appended(s, head(s["q"], s["q_gain"]).to(dt), *(values or [None, None]))


def _plain_attend(s):
    c = s["case"]
    hkv, hq, d, P, page = c["hkv"], c["hq"], c["d"], c["prefix"], c["page"]
    n, R, G = len(s["kv"]), s["q"].shape[0], c["hq"] // c["hkv"]
    T, N = max(s["rows"]), max(s["kv"])
    # the pages of [prefix ; own keys] of every sequence, padded to the longest
    j = torch.arange(P + N, device=DEV)
    own_j = (j - P).clamp(min=0)
    pages, at = s["table"][:, own_j // page], torch.where(j < P, j, own_j) % page
    if P:
        pages = torch.where(j < P, s["pre"][j.clamp(max=P - 1) // page], pages)
    kv_len, t_len = s["kv_len"][:, None], (s["row_start"][1:] - s["row_start"][:-1])[:, None]
    there = j[None] < P + kv_len                                              # [n, keys]
    pages = torch.where(there, pages, 0).long()
    lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float32, device=DEV)

    def rows(name):
        x = s[name + "_cache"][pages, at]                                     # [n, keys, hkv, d / 2]
        x = torch.stack([lut[(x & 15).long()], lut[(x >> 4).long()]], dim=-1).flatten(-2)
        x = (x.unflatten(-1, (-1, 16)) * s[name + "_scale"].view(torch.uint8)[pages, at].view(torch.float8_e4m3fn)
             .float()[..., None]).flatten(-2)
        return torch.where(there[..., None, None], x, 0)

    k, v = rows("k").permute(0, 2, 3, 1), rows("v").transpose(1, 2)           # [n, hkv, d, keys], [n, hkv, keys, d]
    # the rows of every sequence, padded to the most
    t = torch.arange(T, device=DEV)
    at_row = (s["row_start"][:-1, None] + t).clamp(max=R - 1).long()          # [n, T]
    q = s["q"][at_row].float().unflatten(2, (hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    sc = torch.matmul(q, k) * d ** -0.5                                       # [n, hkv, T * G, keys]
    seen = there[:, None]
    if c["causal"]:
        seen = seen & (j <= (P + kv_len - t_len + t)[..., None])              # [n, T, keys]
    sc = torch.where(seen.expand(n, T, P + N).repeat_interleave(G, dim=1)[:, None], sc, float("-inf"))
    m = sc.amax(dim=-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    real = t[None] < t_len
    o = o.unflatten(2, (T, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)           # [n, T, hq, d]
    lse = (m + torch.log(l)).squeeze(-1).unflatten(2, (T, G)).transpose(1, 2).flatten(2, 3)
    return o[real].to(s["q"].dtype), lse[real]


def _plain_next(s):
    """Lengths that stand (what is kept of a sequence, or the step's first row and its accepted drafts), the rows asked
    for while pages and buffer last, in order; pages no longer needed go on the free stack, the last one first, and
    those needed come off it."""
    c = s["case"]
    page, cols, cap = c["page"], s["cols"], s["n_rows"]
    old, start, want = (s[x].long() for x in ("kv_len", "row_start", "rows"))
    kept = old
    if s["accepted"] is not None:
        T, acc = start[1:] - start[:-1], s["accepted"].long()
        kept = torch.where(acc >= 0, old - T + torch.minimum(T, acc + 1), old)
    if s["keep"] is not None:
        keep = s["keep"].long()
        kept = torch.where(keep >= 0, torch.minimum(keep, old), kept)

    def pages(n):
        return (n + page - 1) // page

    have, want = pages(old), want.clamp(min=0)
    want = torch.where(pages(kept + want) <= cols, want, 0)
    need = pages(kept + want) - have
    room = s["n_free"].long() + (-need).clamp(min=0).sum()
    granted = (need.clamp(min=0).cumsum(0) <= room) & (want.cumsum(0) <= cap)
    new = kept + torch.where(granted, want, 0)
    need = pages(new) - have
    take, give = need.clamp(min=0), (-need).clamp(min=0)
    row_start = torch.cat([torch.zeros_like(start[:1]), (new - kept).cumsum(0)])
    # pages given back, the last first, then the ones taken off the top
    col = torch.arange(cols, device=DEV)[None]
    old_pages = (col >= pages(new)[:, None]) & (col < have[:, None])
    n_give, n_free = give.sum(), s["n_free"].long()
    stack = torch.arange(s["free"].shape[0], device=DEV)
    from_give = (n_free + n_give - 1 - stack).clamp(min=0)     # rank among the given in ascending order
    given = torch.cat([s["table"][old_pages], s["free"][:1]])
    s["free"][:] = torch.where((stack >= n_free) & (stack < n_free + n_give),
                               given[from_give.clamp(max=given.shape[0] - 1)], s["free"])
    new_pages = (col < pages(new)[:, None]) & (col >= have[:, None])
    rank = (take.cumsum(0) - take)[:, None] + col - have[:, None]
    s["table"][:] = torch.where(new_pages, s["free"][(n_free + n_give - 1 - rank).clamp(0, stack.shape[0] - 1)],
                                s["table"])
    # what the stack holds behind its new end is of no account: as it was before the step
    r = torch.arange(cap, device=DEV)
    seq = torch.searchsorted(row_start[1:], r, right=True).clamp(max=old.shape[0] - 1)
    live = r < row_start[-1]
    idx = kept[seq] + r - row_start[seq]
    slot = s["table"][seq, torch.where(live, idx // page, 0)].long() * page + idx % page
    for name, x in (("slots", slot), ("positions", c["prefix"] + idx), ("seqs", seq)):
        s[name][:] = torch.where(live, x.to(s[name].dtype), s[name])
    return _planned(s, new.to(torch.int32), row_start.to(torch.int32), (n_free + n_give - take.sum()).to(torch.int32))


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "next": _exact_next}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    inv, ms = _frequencies(c)
    dev_table = s["table"].cpu().tolist()
    pos, pages, at = [], [], []
    for t, n, tab in zip(s["rows"], s["kv"], dev_table):
        for i in range(n - t, n):
            pos.append(c["prefix"] + i)
            pages.append(tab[i // c["page"]])
            at.append(i % c["page"])
    # the rotation as a product of complex numbers
    turn = torch.polar(torch.full((len(pos), 1, c["rot"] // 2), ms, dtype=torch.float64, device=DEV),
                       (torch.tensor(pos, dtype=torch.float64, device=DEV)[:, None] * inv)[:, None])

    def head(x, gain):
        x = x.double()
        if gain is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
        h = c["rot"] // 2
        y = x[..., :2 * h].unflatten(-1, (h, 2) if c["inter"] else (2, h))
        if not c["inter"]:
            y = y.transpose(-1, -2)
        z = torch.view_as_real(torch.complex(y[..., 0].contiguous(), y[..., 1].contiguous()) * turn)
        if not c["inter"]:
            z = z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., 2 * h:]], dim=-1)

    at = (torch.tensor(pages, device=DEV), torch.tensor(at, device=DEV))
    out = {"q": head(s["q"], s["q_gain"])}
    # every positive value of the two formats, and the nearest one with ties to the even code
    e4m3 = [m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    tables = [torch.tensor(x, dtype=torch.float64, device=DEV) for x in (e4m3, _E2M1)]

    def nearest(x, values):
        mid = (values[1:] + values[:-1]) / 2
        below, upto = torch.searchsorted(mid, x), torch.searchsorted(mid, x, right=True)
        return torch.where(below == upto, below, below + below % 2)

    for name, x in (("k", head(s["k"], s["k_gain"])), ("v", s["v"].double())):
        b = x.unflatten(-1, (-1, 16))
        top = b.abs().amax(-1)
        code = nearest((top / 6).contiguous(), tables[0])
        sc = tables[0][code]
        el = nearest((b.abs() / torch.where(sc == 0, math.inf, sc)[..., None]).contiguous(), tables[1])
        nib = (el + 8 * torch.signbit(b)).flatten(-2).to(torch.uint8)
        codes, scales = s[name + "_cache"].clone(), s[name + "_scale"].to(torch.float64)
        codes[at] = nib[..., 0::2] + 16 * nib[..., 1::2]
        scales[at] = sc
        out[name], out[name + "_scale"] = codes, scales
        if c["values"]:
            sign = 1 - 2 * torch.signbit(b).double()
            out[name + "_values"] = (tables[1][el] * sign * sc[..., None]).flatten(-2)
    order = ("q", "k", "v", "k_scale", "v_scale", "k_values", "v_values")
    return {k: out[k] for k in order if k in out}


def _exact_attend(s):
    c = s["case"]
    G, P, page, d = c["hq"] // c["hkv"], c["prefix"], c["page"], c["d"]
    R = s["q"].shape[0]
    out = torch.zeros(R, c["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((R, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    # what a byte stands for
    two = torch.tensor([[math.copysign(_E2M1[n & 7], -1 if n & 8 else 1) for n in (b & 15, b >> 4)]
                        for b in range(256)], dtype=torch.float64, device=DEV)

    def rows(name, p, at, h):
        sc = s[name + "_scale"].view(torch.uint8)[p, at, h].view(torch.float8_e4m3fn).double()
        return two[s[name + "_cache"][p, at, h].long()].flatten(-2) * sc.repeat_interleave(16, dim=-1)

    for h in range(c["hkv"]):
        heads = slice(h * G, (h + 1) * G)
        for i, (t, n) in enumerate(zip(s["rows"], s["kv"])):
            r = slice(s["starts"][i], s["starts"][i] + t)
            if t == 0 or P + n == 0:
                continue
            parts = []          # (keys, values) of the prefix and of the sequence's own rows
            for pages, m in ((s["pre"], P), (s["table"][i], n)):
                j = torch.arange(m, device=DEV)
                p = pages[j // page].long() if m else j
                parts.append((rows("k", p, j % page, h), rows("v", p, j % page, h)))
            k, v = torch.cat([a for a, _ in parts]), torch.cat([b for _, b in parts])
            sc = torch.einsum("tgd,kd->tgk", s["q"][r, heads].double(), k) / math.sqrt(d)
            if c["causal"]:
                tri = torch.ones(t, P + n, dtype=torch.bool, device=DEV).tril(P + n - t)
                sc = sc.masked_fill(~tri[:, None], -math.inf)
            z = torch.logsumexp(sc, dim=-1)
            lse[r, heads] = z
            out[r, heads] = torch.einsum("tgk,kd->tgd", (sc - z[..., None]).exp().nan_to_num(0.0), v)
    return out, lse


def _exact_next(s):
    """The same with a stack, one sequence after the other."""
    c = s["case"]
    page, cols, cap = c["page"], s["cols"], s["n_rows"]
    old, start, rows = (s[x].tolist() for x in ("kv_len", "row_start", "rows"))
    acc = s["accepted"].tolist() if s["accepted"] is not None else [-1] * len(old)
    keep = s["keep"].tolist() if s["keep"] is not None else [-1] * len(old)
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    n_free = int(s["n_free"])

    def pages(n):
        return -(-n // page)

    kept = []
    for i, n in enumerate(old):
        t = start[i + 1] - start[i]
        kept.append(min(keep[i], n) if keep[i] >= 0 else n - t + min(t, acc[i] + 1) if acc[i] >= 0 else n)
    want = [t if t > 0 and pages(k + t) <= cols else 0 for k, t in zip(kept, rows)]
    room = n_free + sum(max(0, pages(n) - pages(k + t)) for n, k, t in zip(old, kept, want))
    given, taken, used = [], 0, 0
    for i, t in enumerate(want):
        taken += max(0, pages(kept[i] + t) - pages(old[i]))
        used += t
        given.append(t if taken <= room and used <= cap else 0)
    new = [k + t for k, t in zip(kept, given)]
    top = n_free
    for i in reversed(range(len(old))):
        for col in reversed(range(pages(new[i]), pages(old[i]))):
            free[top] = table[i, col]
            top += 1
    slots, positions, seqs = (s[x].cpu().numpy().copy() for x in ("slots", "positions", "seqs"))
    row_start = [0]
    for i, t in enumerate(given):
        for col in range(pages(old[i]), pages(new[i])):
            top -= 1
            table[i, col] = free[top]
        j = np.arange(kept[i], new[i])
        r = slice(row_start[-1], row_start[-1] + t)
        slots[r] = table[i, j // page].astype(np.int64) * page + j % page
        positions[r], seqs[r] = c["prefix"] + j, i
        row_start.append(row_start[-1] + t)
    return {"kv_len": np.array(new, np.int32), "row_start": np.array(row_start, np.int32),
            "n_free": np.array([top], np.int32), "table": table, "free": free, "slots": slots,
            "positions": positions, "seqs": seqs}
