"""Speculative steps as a program runs them: the drafter's block and greedy
tokens, the target's rows appended to its paged cache, attention behind a
shared prompt, verification, and the next step over what was accepted."""
import dataclasses

import numpy as np
import pytest
import torch

import _target_ref as R
from speculative_decoding_block_ingest_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DRAFTER = dataclasses.replace(synth.TINY_F32, weight_dtype="bf16", kv_dtype="bf16", hidden=512, n_heads=8,
                              n_kv_heads=2, head_dim=128, intermediate=1024, n_taps=2)
N, BLOCK, PREFIX, PAGE, HQ, HKV, D, V = 3, 16, 37, 16, 8, 2, 64, 1024
EPS = 1e-6


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


class Target:
    """One attention layer between an embedding and an lm_head."""

    def __init__(self, T):
        self.T = T
        g = torch.Generator().manual_seed(1)
        H = DRAFTER.hidden
        bf = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16).to(DEV)
        self.embed, self.qkv = bf(V, H) * 16, bf((HQ + 2 * HKV) * D, H)
        self.out, self.head = bf(H, HQ * D), bf(V, H) * 4
        self.gain = (1 + 0.1 * torch.randn(2, D, generator=g)).to(DEV)
        pool = lambda: torch.full((64, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.cache = T.PagedCache(pool(), pool())
        self.rope = T.Rope(D, 1e4)
        order = torch.randperm(64, generator=g).to(torch.int32)
        self.pre, self.table = order[:3].to(DEV), order[4:4 + N * 8].view(N, 8).to(DEV)
        self.kv_len = i32([0] * N)

    def rows(self, tokens, row_start, kv_len, table, pre_len):
        """q, k, v of a step's tokens through the cache; attention's result, probabilities."""
        x = self.embed[tokens.long()]
        q, k, v = (t.unflatten(1, (-1, D)) for t in (x @ self.qkv.T).split([HQ * D, HKV * D, HKV * D], 1))
        step = self.T.Step(row_start, kv_len, table, self.pre, pre_len)
        q = self.T.append(self.cache, step, q, k, v, rope=self.rope, q_gain=self.gain[0], k_gain=self.gain[1], eps=EPS)
        o, lse = self.T.attention(self.cache, step, q)
        logits = (x + o.flatten(1) @ self.out.T) @ self.head.T
        return q, k, v, o, lse, torch.softmax(logits.float(), -1)

    def keys(self, tokens, first):
        """Cached K and V rows of a token sequence at positions first, first + 1, ... in 64 bits, and K's tolerance."""
        x = self.embed[torch.as_tensor(tokens, device=DEV).long()]
        _, k, v = (t.unflatten(1, (-1, D)) for t in (x @ self.qkv.T).split([HQ * D, HKV * D, HKV * D], 1))
        inv, _ = R.rope_freqs(D, 1e4)
        want, size = R.head_rows(k, self.gain[1], EPS, range(first, first + len(tokens)), inv, 1.0)
        return want, v.double().cpu().numpy(), R.EPS[torch.bfloat16] * np.abs(want) + 1e-6 * size


def test_speculative_steps():
    from speculative_decoding_block_ingest_gb300 import dflash, target as T
    tgt = Target(T)
    g = torch.Generator().manual_seed(3)
    prompt = torch.randint(0, V, (PREFIX,), generator=g)
    # the shared prompt enters the prefix pages as the own rows of one sequence
    tgt.rows(prompt.to(DEV), i32([0, PREFIX]), i32([PREFIX]), tgt.pre[None], 0)

    dr = dflash.Drafter(DRAFTER, synth.make_weights(DRAFTER), max_seqs=N, max_pages=32, max_seq_len=512, max_batch=N,
                        max_ingest_rows=128, device=DEV)
    for i in range(N):
        dr.ingest([i], [PREFIX], list(range(PREFIX)), synth.taps_rows(DRAFTER, i, 0, PREFIX).to(DEV))
    packed, vocab = dr.pack_lm_head(tgt.head)
    anchor = torch.randint(0, V, (N,), generator=g).to(torch.int32).to(DEV)
    sequences = [[] for _ in range(N)]           # own tokens whose keys are in the cache
    row_start = i32([BLOCK * i for i in range(N + 1)])

    for turn in range(3):
        # draft: block rows start from the anchor's embedding
        noise = tgt.embed[anchor.long()].float()[:, None].repeat(1, BLOCK, 1)
        noise[:, 1:] += torch.randn(N, BLOCK - 1, DRAFTER.hidden, generator=g).to(DEV)
        pos = [PREFIX + len(s) + j for s in sequences for j in range(BLOCK)]
        block = dr.draft_tokens(dr.forward_round(list(range(N)), pos, noise), packed, vocab)
        draft = block[:, 1:]
        # verify: the anchor and the drafts go through the target
        tgt.kv_len += BLOCK
        tokens = torch.cat([anchor[:, None], draft], 1)
        q, k, v, o, lse, probs = tgt.rows(tokens.flatten(), row_start, tgt.kv_len, tgt.table, PREFIX)
        ua, ut = torch.rand(N, BLOCK - 1, generator=g).to(DEV), torch.rand(N, generator=g).to(DEV)
        probs = probs.unflatten(0, (N, BLOCK))
        if turn == 1:      # a target that agrees with some drafts
            probs[:, :5].scatter_(2, draft[:, :5, None].long(), 1.0)
        got, accepted = T.verify_tokens(draft, probs, ua, ut)
        torch.cuda.synchronize()
        dr.device_status()

        # the cache holds the prompt and every sequence's tokens, in place
        own = [s + tokens[i].tolist() for i, s in enumerate(sequences)]
        lens = [len(s) for s in own]
        assert lens == tgt.kv_len.tolist()
        table, pre = tgt.table.cpu(), tgt.pre.cpu()
        for pages, toks, first in [(pre, prompt.tolist(), 0)] + [(table[i], own[i], PREFIX) for i in range(N)]:
            wk, wv, tol = tgt.keys(toks, first)
            j = torch.arange(len(toks))
            gk, gv = (c[pages[j // PAGE].long().to(DEV), (j % PAGE).to(DEV)].double().cpu().numpy()
                      for c in (tgt.cache.k, tgt.cache.v))
            assert np.all(np.abs(gk - wk) <= tol) and np.array_equal(gv, wv)
        wo, to, wl, tl = R.attend_step(q, tgt.cache.k, tgt.cache.v, row_start.tolist(), lens, table, pre, PREFIX, PAGE,
                                       causal=True, scale=D ** -0.5)
        assert np.all(np.abs(o.double().cpu().numpy() - wo) <= to)
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= tl)
        wt, wa = R.verify(draft, probs, ua, ut)
        assert np.array_equal(got.cpu().numpy(), wt) and np.array_equal(accepted.cpu().numpy(), wa)
        if turn == 1:
            assert accepted.min() >= 5

        # accepted rows stay, on the device alone: the next step's rows replace the rest
        tgt.kv_len -= BLOCK - 1 - accepted
        anchor = got[torch.arange(N, device=DEV), accepted.long()]
        for i in range(N):
            a = int(accepted[i])
            sequences[i] = own[i][:lens[i] - (BLOCK - 1 - a)]
            at = PREFIX + len(sequences[i]) - a - 1
            dr.ingest([i], [a + 1], list(range(at, at + a + 1)), synth.taps_rows(DRAFTER, i, at, a + 1).to(DEV))
    dr.close()


def test_operators_in_one_graph():
    """Append, attention and verification captured together: the replay equals the eager calls."""
    from speculative_decoding_block_ingest_gb300 import target as T
    tgt = Target(T)
    g = torch.Generator().manual_seed(5)
    prompt = torch.randint(0, V, (PREFIX,), generator=g)
    tgt.rows(prompt.to(DEV), i32([0, PREFIX]), i32([PREFIX]), tgt.pre[None], 0)
    tokens = torch.randint(0, V, (N, BLOCK), generator=g).to(torch.int32).to(DEV)
    row_start = i32([BLOCK * i for i in range(N + 1)])
    ua, ut = torch.rand(N, BLOCK - 1, generator=g).to(DEV), torch.rand(N, generator=g).to(DEV)
    tgt.kv_len += BLOCK

    def step():
        p = tgt.rows(tokens.flatten(), row_start, tgt.kv_len, tgt.table, PREFIX)[-1].unflatten(0, (N, BLOCK))
        return T.verify_tokens(tokens[:, 1:], p, ua, ut)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for seed in range(3):
        gg = torch.Generator().manual_seed(seed)
        tokens.copy_(torch.randint(0, V, (N, BLOCK), generator=gg).to(torch.int32))
        ua.copy_(torch.rand(N, BLOCK - 1, generator=gg))
        tgt.kv_len.copy_(i32([BLOCK, BLOCK + 2 * seed, BLOCK + 60]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
