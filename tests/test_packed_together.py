"""Speculative steps over a 4-bit cache without the host: the next step's tables
from the accepted counts, append, attention and verification in one graph."""
import numpy as np
import pytest
import torch

import _packed_ref as P
import _target_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N, BLOCK, PREFIX, PAGE, HQ, HKV, D, V, H = 5, 6, 37, 16, 8, 2, 64, 512, 256


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


class Server:
    """One attention layer between an embedding and an lm_head, drafts from a table, pages from a pool."""

    def __init__(self, T, n_pages=40):
        self.T = T
        g = torch.Generator().manual_seed(1)
        bf = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16).to(DEV)
        self.embed, self.qkv = bf(V, H) * 16, bf((HQ + 2 * HKV) * D, H)
        self.out, self.head = bf(H, HQ * D), bf(V, H) * 4
        self.gain = (1 + 0.1 * torch.randn(2, D, generator=g)).to(DEV)
        self.rope = T.Rope(D, 1e4, interleaved=True)
        n_pre = -(-PREFIX // PAGE)
        self.cache = T.PagedCache4.zeros(n_pages, PAGE, HKV, D, DEV)
        self.pool = T.PagePool.empty(n_pages, PAGE, N, 8, DEV, reserved=n_pre, prefix_len=PREFIX,
                                     prefix_pages=torch.arange(n_pre, dtype=torch.int32, device=DEV))
        prompt = torch.randint(0, V, (PREFIX,), generator=g).to(DEV)
        self.layer(prompt, T.Step(i32([0, PREFIX]), i32([PREFIX]), self.pool.prefix_pages[None]), None)
        self.anchor = torch.randint(0, V, (N,), generator=g).to(DEV)
        self.next_token = torch.randint(0, V, (V,), generator=g).to(DEV)   # what the drafter thinks
        self.accepted = i32([-1] * N)
        self.rows = i32([BLOCK] * N)
        self.slots = torch.zeros(N * BLOCK, dtype=torch.int64, device=DEV)
        self.positions, self.sequences = (torch.zeros(N * BLOCK, dtype=torch.int32, device=DEV) for _ in range(2))
        self.ua = torch.rand(N, BLOCK - 1, generator=g).to(DEV)
        self.ut = torch.rand(N, generator=g).to(DEV)

    def layer(self, tokens, step, positions):
        x = self.embed[tokens.long()]
        q, k, v = (t.unflatten(1, (-1, D)) for t in (x @ self.qkv.T).split([HQ * D, HKV * D, HKV * D], 1))
        q = self.T.append(self.cache, step, q, k, v, rope=self.rope, q_gain=self.gain[0], k_gain=self.gain[1],
                          positions=positions)
        o, lse = self.T.attention(self.cache, step, q)
        return q, o, lse, (x + o.flatten(1) @ self.out.T) @ self.head.T

    def turn(self):
        """One step, on the device alone."""
        pool = self.T.next_step(self.pool, self.rows, n_accepted=self.accepted, slots=self.slots,
                                positions=self.positions, sequences=self.sequences)
        draft = [self.next_token[self.anchor]]
        for _ in range(BLOCK - 2):
            draft.append(self.next_token[draft[-1]])
        draft = torch.stack(draft, 1)
        tokens = torch.cat([self.anchor[:, None], draft], 1).flatten()
        q, o, lse, logits = self.layer(tokens, pool.step, self.positions)
        probs = torch.softmax(logits.float(), -1).unflatten(0, (N, BLOCK))
        probs[:, :3].scatter_(2, draft[:, :3, None], 1.0)          # a target that agrees with some drafts
        got, accepted = self.T.verify_tokens(draft.to(torch.int32), probs, self.ua, self.ut)
        self.accepted.copy_(accepted)
        self.anchor.copy_(got.gather(1, accepted[:, None].long())[:, 0])
        return q, o, lse, got, accepted


def state(s):
    return [x.clone() for x in (s.pool.kv_len, s.pool.row_start, s.pool.n_free, s.pool.block_table, s.accepted, s.anchor,
                                s.slots, *s.cache.tensors[:2])]


def test_steps_against_64_bits():
    from speculative_decoding_block_ingest_gb300 import target as T
    s = Server(T)
    last = None
    for turn in range(4):
        before = s.accepted.tolist()
        q, o, lse, got, accepted = s.turn()
        kv = s.pool.kv_len.tolist()
        want = [BLOCK] * N if turn == 0 else [n + 1 + a for n, a in zip(last, before)]
        assert kv == want and s.pool.row_start.tolist() == [BLOCK * i for i in range(N + 1)]
        last = kv
        # rows' places and positions are the table's
        table = s.pool.block_table.cpu()
        for r in range(N * BLOCK):
            i, own = r // BLOCK, kv[r // BLOCK] - BLOCK + r % BLOCK
            assert int(s.sequences[r]) == i and int(s.positions[r]) == PREFIX + own
            assert int(s.slots[r]) == int(table[i, own // PAGE]) * PAGE + own % PAGE
        k64, v64 = (P.values(c.cpu().numpy(), sc.view(torch.uint8).cpu().numpy())
                    for c, sc in ((s.cache.k, s.cache.k_scale), (s.cache.v, s.cache.v_scale)))
        wo, to, wl, tl = P.attend_step(q, k64, v64, s.pool.row_start.tolist(), kv, table, s.pool.prefix_pages.cpu(), PREFIX,
                                       PAGE, causal=True, scale=D ** -0.5)
        assert np.all(np.abs(o.double().cpu().numpy() - wo) <= to)
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= tl)
        assert int(accepted.min()) >= 3


def test_the_loop_in_one_graph():
    """Replays of one captured turn go on from each other as eager turns do, bit for bit."""
    from speculative_decoding_block_ingest_gb300 import target as T
    eager, replayed = Server(T), Server(T)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        replayed.turn()          # the first turn, and warm-up
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = replayed.turn()
    eager.turn()
    for _ in range(6):
        want = eager.turn()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(state(eager), state(replayed)):
            assert torch.equal(a, b)
        for a, b in zip(want, out):
            assert torch.equal(a, b)


def test_the_pool_runs_out():
    """Sequences at the end get no rows; nothing of theirs changes."""
    from speculative_decoding_block_ingest_gb300 import target as T
    s = Server(T, n_pages=3 + 7)
    for _ in range(12):          # at least four keys a turn and sequence: 7 pages hold 112
        before = s.pool.kv_len.tolist()
        s.turn()
        kv, given = s.pool.kv_len.tolist(), s.pool.row_start.diff().tolist()
        if 0 in given:
            break
    assert BLOCK in given and 0 in given and given == sorted(given, reverse=True)
    assert all(n <= m for n, m, t in zip(kv, before, given) if t == 0)      # (less what was rejected)
    used = [p for i, n in enumerate(kv) for p in s.pool.block_table[i, :-(-n // PAGE)].tolist()]
    free = s.pool.free[:int(s.pool.n_free)].tolist()
    assert sorted(used + free) == list(range(3, 10))
