"""Work of the operators a target model runs beside the drafter in one
speculative step: appending the step's keys and values to its paged cache
(head norms and RoPE on the way), attention of the step's rows over that cache
with a prefix all sequences share, and verification of the drafted tokens.

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


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one sequence: the smallest step, all latency
        {"name": "append-decode-1", "op": "append", "n_seq": 1, "rows_lo": 1, "rows_hi": 1, "extra_lo": 776,
         "extra_hi": 776, "prefix": 0, "hq": 32, "hkv": 4, "d": 128, "rot": 128, "page": 64, "layout": "nhd",
         "in": "bf16", "dtype": "bf16", "norm": True, "yarn": False, "fused_qkv": True, "shape_seed": 1},
        # 32 sequences verifying drafts of ragged length behind a shared prompt; YaRN; f32 projections
        {"name": "append-verify-32", "op": "append", "n_seq": 32, "rows_lo": 1, "rows_hi": 17, "extra_lo": 0,
         "extra_hi": 3000, "prefix": 16383, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "page": 16, "layout": "hnd",
         "in": "f32", "dtype": "bf16", "norm": True, "yarn": True, "fused_qkv": False, "shape_seed": 2},
        # prompts entering the cache: eight ragged prompts of 32 thousand rows in all, f16, half the head rotated
        {"name": "append-prompts-8", "op": "append", "n_seq": 8, "rows_lo": 1001, "rows_hi": 8191, "extra_lo": 0,
         "extra_hi": 0, "prefix": 0, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "page": 64, "layout": "nhd",
         "in": "f16", "dtype": "f16", "norm": False, "yarn": False, "fused_qkv": True, "shape_seed": 3},
        # one new token of one short sequence: latency of the attention
        {"name": "attend-decode-1", "op": "attend", "n_seq": 1, "rows_lo": 1, "rows_hi": 1, "extra_lo": 776,
         "extra_hi": 776, "prefix": 0, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "nhd", "dtype": "bf16",
         "causal": True, "shape_seed": 4},
        # a small model's ragged verification behind a short shared prompt; odd group, small pages, f16
        {"name": "attend-ragged-8", "op": "attend", "n_seq": 8, "rows_lo": 1, "rows_hi": 17, "extra_lo": 0,
         "extra_hi": 300, "prefix": 2053, "hq": 12, "hkv": 4, "d": 64, "page": 16, "layout": "hnd", "dtype": "f16",
         "causal": True, "shape_seed": 5},
        # one long document being decoded with drafts of 15 tokens: split over the keys
        {"name": "attend-long-1", "op": "attend", "n_seq": 1, "rows_lo": 16, "rows_hi": 16, "extra_lo": 131000,
         "extra_hi": 131000, "prefix": 0, "hq": 32, "hkv": 8, "d": 128, "page": 64, "layout": "nhd",
         "dtype": "bf16", "causal": True, "shape_seed": 6},
        # 64 conversations decoding token by token behind a shared prompt: the cache's bytes bound it
        {"name": "attend-decode-64", "op": "attend", "n_seq": 64, "rows_lo": 1, "rows_hi": 1, "extra_lo": 1023,
         "extra_hi": 16383, "prefix": 4096, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "nhd",
         "dtype": "bf16", "causal": True, "shape_seed": 7},
        # 32 sequences verifying blocks of 16 behind a long shared prompt: matrix products bound it
        {"name": "attend-verify-32", "op": "attend", "n_seq": 32, "rows_lo": 16, "rows_hi": 16, "extra_lo": 100,
         "extra_hi": 1024, "prefix": 16384, "hq": 32, "hkv": 4, "d": 128, "page": 64, "layout": "nhd",
         "dtype": "bf16", "causal": True, "shape_seed": 8},
        # the block this library drafts greedily (15 tokens after the anchor), verified for one sequence
        {"name": "verify-greedy-1", "op": "verify", "n_seq": 1, "k": 15, "vocab": 32768, "dtype": "f32",
         "draft_probs": False, "ragged": False},
        # sampled drafts of ragged length over a vocabulary whose rows start on no 16-byte boundary
        {"name": "verify-sampled-32", "op": "verify", "n_seq": 32, "k": 15, "vocab": 100003, "dtype": "f32",
         "draft_probs": True, "ragged": True},
        # probabilities kept in 16 bits
        {"name": "verify-bf16-64", "op": "verify", "n_seq": 64, "k": 7, "vocab": 131072, "dtype": "bf16",
         "draft_probs": True, "ragged": False},
        # a large batch over a large vocabulary: bytes bound it
        {"name": "verify-batch-256", "op": "verify", "n_seq": 256, "k": 7, "vocab": 262144, "dtype": "f32",
         "draft_probs": True, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "verify"])
    if op == "verify":
        while True:
            c = {"op": op, "n_seq": _log(rng, 1, 256), "k": rng.randint(1, 16), "vocab": _log(rng, 1000, 262144),
                 "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "draft_probs": rng.random() < 0.6,
                 "ragged": rng.random() < 0.5}
            if c["n_seq"] * (c["k"] + 1) * c["vocab"] <= 256 * 8 * 262144 and work(c)["bytes"] <= 5e8:
                return c
    hkv = rng.choice([1, 2, 4, 8])
    while True:
        c = {"op": op, "n_seq": _log(rng, 1, 64), "rows_lo": rng.choice([0, 1, 1, 1]),
             "rows_hi": rng.choice([1, 1, 5, 16, 17, 33]), "extra_lo": 0, "extra_hi": _log(rng, 1, 16384),
             "prefix": rng.choice([0, _log(rng, 1, 32768)]), "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "hkv": hkv,
             "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "layout": rng.choice(["nhd", "hnd"]),
             "dtype": rng.choice(["bf16", "bf16", "f16"]), "shape_seed": rng.randint(1, 10 ** 9)}
        if op == "attend":
            c["causal"] = rng.random() < 0.85
        else:
            c.update(rot=rng.choice([c["d"], c["d"], c["d"] // 2]), norm=rng.random() < 0.6, yarn=rng.random() < 0.3,
                     fused_qkv=rng.random() < 0.5)
            c["in"] = rng.choice([c["dtype"], c["dtype"], "f32"])
            if rng.random() < 0.4:     # a prompt's rows rather than a step's
                c.update(n_seq=rng.randint(1, 8), rows_hi=_log(rng, 100, 6000), extra_hi=1)
        w = work(c)
        if sum(_shape(c)[0]) > 0 and w["flops"] <= 3e11 and w["bytes"] <= 1.2e9 and _cache_rows(c) * hkv <= 4e6:
            return c


def _shape(c):
    """Rows of the step and own cached keys (these rows included) of every sequence."""
    r = random.Random(c["shape_seed"])
    rows = [r.randint(c["rows_lo"], c["rows_hi"]) for _ in range(c["n_seq"])]
    return rows, [t + r.randint(c["extra_lo"], c["extra_hi"]) for t in rows]


def _cache_rows(c):
    return sum(_shape(c)[1]) + c["prefix"]


def work(c):
    if c["op"] == "verify":
        e = 4 if c["dtype"] == "f32" else 2
        # one target row (and one draft row) of every sequence, the drafts and their probabilities and numbers
        rows = c["n_seq"] * c["vocab"] * (2 if c["draft_probs"] else 1)
        return {"bytes": rows * e + c["n_seq"] * (c["k"] * (8 + 2 * e) + (c["k"] + 1) * 4 + 12), "flops": 3 * rows}
    rows, kv = _shape(c)
    R = sum(rows)
    if c["op"] == "append":
        ei = 4 if c["in"] == "f32" else 2
        heads = c["hq"] + 2 * c["hkv"]
        return {"bytes": R * heads * c["d"] * (ei + 2), "flops": R * (c["hq"] + c["hkv"]) * c["d"] * 8}
    keys = sum(kv) + (c["prefix"] if R else 0)
    pairs = 0
    for t, n in zip(rows, kv):
        pairs += t * (c["prefix"] + n) - (t * (t - 1) // 2 if c["causal"] else 0)
    return {"bytes": R * c["hq"] * (c["d"] * 4 + 4) + keys * c["hkv"] * c["d"] * 4,
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def prepare(case, seed):
    return (_prepare_verify if case["op"] == "verify" else _prepare_step)(case, seed)


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
    shape = (n_pages, page, hkv, d) if c["layout"] == "nhd" else (n_pages, hkv, page, d)
    caches = []
    for _ in range(2):
        t = _randn(g, *shape, dtype=dt)
        caches.append(t if c["layout"] == "nhd" else t.transpose(1, 2))
    starts = [0]
    for t in rows:
        starts.append(starts[-1] + t)
    s = {"case": c, "rows": rows, "kv": kv, "starts": starts, "pre": torch.tensor(pre, dtype=torch.int32, device=DEV),
         "table": table.to(DEV), "row_start": torch.tensor(starts, dtype=torch.int32, device=DEV),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV), "k_cache": caches[0], "v_cache": caches[1]}
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
                s["k_cache"][p, n % page:] = float("nan")
                s["v_cache"][p, n % page:] = float("nan")
        s["q"] = _randn(g, R, hq, d, dtype=dt)
    if own:
        from speculative_decoding_block_ingest_gb300 import target
        s["cache"] = target.PagedCache(s["k_cache"], s["v_cache"])
        s["step"] = target.Step(s["row_start"], s["kv_len"], s["table"], prefix_pages=s["pre"],
                                prefix_len=c["prefix"])
        if c["op"] == "append":
            s["rope"] = (target.Rope(c["rot"], theta=1e6, yarn_factor=32.0, yarn_original_max_pos=8192)
                         if c["yarn"] else target.Rope(c["rot"], theta=1e6))
    return s


def _prepare_verify(c, seed):
    g = _gen(seed)
    n, k, V, dt = c["n_seq"], c["k"], c["vocab"], _T[c["dtype"]]
    tp = torch.empty(n, k + 1, V, dtype=dt, device=DEV)
    dp = torch.empty(n, k, V, dtype=dt, device=DEV) if c["draft_probs"] else None
    tok = torch.empty(n, k, dtype=torch.int32, device=DEV)
    for i in range(n):   # a drafter that agrees with the target for the most part
        z = _randn(g, k + 1, V)
        tp[i] = torch.softmax(3 * z, dim=1).to(dt)
        y = 0.98 * z[:k] + 0.2 * _randn(g, k, V)
        if c["draft_probs"]:
            q = torch.softmax(3 * y, dim=1)
            dp[i] = q.to(dt)
            tok[i] = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
        else:
            tok[i] = y.argmax(dim=1).to(torch.int32)
    nd = None
    if c["ragged"]:
        nd = torch.randint(0, k + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    return {"case": c, "draft": tok, "target_probs": tp, "draft_probs": dp, "n_draft": nd,
            "u_accept": torch.rand(n, k, generator=g, device=DEV), "u_token": torch.rand(n, generator=g, device=DEV)}


def _frequencies(c):
    """Inverse frequencies [rot / 2] in 64 bits and the factor on cos and sin."""
    rot = c["rot"]
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    inv = 1e6 ** (-2 * j / rot)
    if not c["yarn"]:
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
            q = target.append(s["cache"], s["step"], s["q"], s["k"], s["v"], rope=s["rope"], q_gain=s["q_gain"],
                              k_gain=s["k_gain"])
            return q, s["k_cache"], s["v_cache"]
        if op == "attend":
            return target.attention(s["cache"], s["step"], s["q"], causal=s["case"]["causal"])
        return target.verify_tokens(s["draft"], s["target_probs"], s["u_accept"], s["u_token"],
                                    draft_probs=s["draft_probs"], n_draft=s["n_draft"])
    return {"append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[op](s)


def _plain_append(s):
    c = s["case"]
    R, dt, half = s["q"].shape[0], _T[c["dtype"]], c["rot"] // 2
    # which sequence, own index and position each row has
    row = torch.arange(R, device=DEV, dtype=torch.int32)
    seq = (row[:, None] >= s["row_start"][None, 1:]).sum(dim=1)
    idx = s["kv_len"][seq] - s["row_start"][seq + 1] + row
    page, at = s["table"][seq, (idx // c["page"]).long()].long(), (idx % c["page"]).long()
    # angles of far positions need 64 bits
    ang = (c["prefix"] + idx).double()[:, None] * s["inv_freq"]
    cos, sin = ((f(ang) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))

    def head(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * gain
        a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1).to(dt)

    s["k_cache"][page, at] = head(s["k"], s["k_gain"])
    s["v_cache"][page, at] = s["v"].float().to(dt)
    return head(s["q"], s["q_gain"]), s["k_cache"], s["v_cache"]


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
    k = s["k_cache"][pages, at].float().permute(0, 2, 3, 1)                   # [n, hkv, d, keys]
    v = torch.where(there[..., None, None], s["v_cache"][pages, at], 0).float().transpose(1, 2)
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


def _plain_verify(s):
    """Draft j is taken while u_j q_j(x_j) < p_j(x_j); the token behind the last taken one comes from the positive
    part of p - q there (from p where all were taken, or nothing is left of p - q), by the first index whose
    cumulative sum passes u times the total.  64 bits: sums over the vocabulary are compared with a number."""
    draft, tp, dp, nd = s["draft"], s["target_probs"], s["draft_probs"], s["n_draft"]
    n, k = draft.shape
    if nd is None:
        nd = torch.full((n,), k, dtype=torch.int32, device=DEV)
    p = tp[:, :k].gather(2, draft.long()[..., None])[..., 0].double()
    q = 1.0 if dp is None else dp.gather(2, draft.long()[..., None])[..., 0].double()
    j = torch.arange(k, device=DEV)[None]
    take = (s["u_accept"].double() * q < p) & (j < nd[:, None])
    acc = torch.cumprod(take.to(torch.int32), dim=1).sum(dim=1).to(torch.int32)
    i = torch.arange(n, device=DEV)
    w = tp[i, acc.long()].double()
    jr = acc.clamp(max=k - 1).long()
    x = draft[i, jr].long()
    if dp is None:
        r = w.clone()
        r[i, x] = 0
    else:
        r = (w - dp[i, jr].double()).clamp(min=0)
    rejected = (acc < nd) & (r.sum(dim=1) > 0)
    w = torch.where(rejected[:, None], r, w)
    cum = torch.cumsum(w, dim=1)
    tok = (cum > s["u_token"].double()[:, None] * cum[:, -1:]).int().argmax(dim=1).to(torch.int32)
    col = torch.arange(k + 1, device=DEV)[None]
    pad = torch.cat([draft, draft[:, :1]], dim=1)
    tokens = torch.where(col < acc[:, None], pad, torch.where(col == acc[:, None], tok[:, None], -1))
    return tokens.to(torch.int32), acc


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    inv, ms = _frequencies(c)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    pos, pages, at = [], [], []
    for t, n, tab in zip(s["rows"], s["kv"], s["table"].cpu().tolist()):
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
        z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
        return torch.cat([z.real, z.imag, x[..., 2 * h:]], dim=-1)

    at = (torch.tensor(pages, device=DEV), torch.tensor(at, device=DEV))
    kc[at], vc[at] = head(s["k"], s["k_gain"]), s["v"].double()
    return head(s["q"], s["q_gain"]), kc, vc


def _exact_attend(s):
    c = s["case"]
    G, P, page, d = c["hq"] // c["hkv"], c["prefix"], c["page"], c["d"]
    R = s["q"].shape[0]
    out = torch.zeros(R, c["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((R, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    k_all, v_all = s["k_cache"], s["v_cache"]
    for h in range(c["hkv"]):
        heads = slice(h * G, (h + 1) * G)
        for i, (t, n) in enumerate(zip(s["rows"], s["kv"])):
            rows = slice(s["starts"][i], s["starts"][i] + t)
            parts = []          # (keys, values) of the prefix and of the sequence's own rows
            for pages, m in ((s["pre"], P), (s["table"][i], n)):
                j = torch.arange(m, device=DEV)
                p = pages[j // page].long() if m else j
                parts.append((k_all[p, j % page, h].double(), v_all[p, j % page, h].double()))
            k, v = torch.cat([a for a, _ in parts]), torch.cat([b for _, b in parts])
            if t == 0 or P + n == 0:
                continue
            sc = torch.einsum("tgd,kd->tgk", s["q"][rows, heads].double(), k) / math.sqrt(d)
            if c["causal"]:
                tri = torch.ones(t, P + n, dtype=torch.bool, device=DEV).tril(P + n - t)
                sc = sc.masked_fill(~tri[:, None], -math.inf)
            z = torch.logsumexp(sc, dim=-1)
            lse[rows, heads] = z
            out[rows, heads] = torch.einsum("tgk,kd->tgd", (sc - z[..., None]).exp().nan_to_num(0.0), v)
    return out, lse


def _exact_verify(s):
    draft = s["draft"].cpu().numpy()
    n, k = draft.shape
    nd = [k] * n if s["n_draft"] is None else s["n_draft"].tolist()
    ua, ut = s["u_accept"].double().cpu().numpy(), s["u_token"].double().cpu().numpy()

    def row(x, i, j):
        return x[i, j].double().cpu().numpy()

    tokens, taken = np.full((n, k + 1), -1, dtype=np.int32), np.zeros(n, dtype=np.int32)
    for i in range(n):
        j = 0
        while j < nd[i]:
            x = draft[i, j]
            q = 1.0 if s["draft_probs"] is None else float(s["draft_probs"][i, j, x])
            if not ua[i, j] * q < float(s["target_probs"][i, j, x]):
                break
            tokens[i, j] = x
            j += 1
        p = row(s["target_probs"], i, j)
        if j < nd[i]:
            if s["draft_probs"] is None:
                r = p.copy()
                r[draft[i, j]] = 0
            else:
                r = np.maximum(p - row(s["draft_probs"], i, j), 0)
            p = r if r.sum() > 0 else p
        cum = np.cumsum(p)
        tokens[i, j] = np.searchsorted(cum, ut[i] * cum[-1], side="right")
        taken[i] = j
    return torch.from_numpy(tokens), torch.from_numpy(taken)
