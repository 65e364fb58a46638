"""Seeded cases of loopvq_decode_attn_shared and their oracle."""

import math

import numpy as np
import torch

import sub_bit_vq_b200 as L
from oracle import loopvq_oracle as O

from _cases import random_codebooks
from _guard import Guarded, status_word, workspace


class SharedCase:
    """`groups`: (sequences, shared tokens) of each group; `own`: quantised
    tokens of each sequence past the shared ones (negative: the sequence stops
    that many tokens before the end of the shared prefix; None: no tokens at
    all; a float f: int(f) window tokens only). Sequences behind the groups
    (len(own) > sum of sizes) share nothing."""

    def __init__(self, shape, groups, own, *, loop_step=1, seed=0, q_scale=1.0, copy_pages=True, first=0,
                 spare=3):
        self.shape, self.groups, self.own = shape, groups, own
        s = shape
        self.B, self.t = len(own), loop_step
        self.gamma, self.tau = divmod(loop_step, s.loop_group)
        r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        J, Pg = s.J, s.page_tokens
        self.starts = [first]                             # sequences before the first group share nothing
        for n, _ in groups:
            self.starts.append(self.starts[-1] + n)
        self.group_of = [-1] * self.B
        for i in range(len(groups)):
            for b in range(self.starts[i], self.starts[i + 1]):
                self.group_of[b] = i
        self.S = [groups[i][1] if i >= 0 else 0 for i in self.group_of]
        self.n_vq, self.seq_lens = [], []
        for b, o in enumerate(own):
            n = max(0, self.S[b] + o) if isinstance(o, int) else 0
            self.n_vq.append(n)
            self.seq_lens.append(0 if o is None else int(o) if isinstance(o, float) else s.window + n)
        # page tables: whole shared pages in common; the page a prefix ends in is
        # the first sequence's, or a copy of its shared slots
        rows, used = [], 0
        common = {}
        for b in range(self.B):
            i, n = self.group_of[b], max(self.n_vq[b], self.S[b] if self.group_of[b] >= 0 and b == self.starts[self.group_of[b]] else 0)
            need = -(-n // Pg)
            shared_pages = (self.S[b] // Pg) if i >= 0 else 0
            if i not in common and i >= 0:
                common[i] = list(range(used, used + shared_pages))
                used += shared_pages
            row = (common[i] if i >= 0 else [])[:need]
            extra = need - len(row)
            row = row + list(range(used, used + extra))
            used += extra
            rows.append(row)
        self.n_pages = used + spare
        perm = r.permutation(self.n_pages)
        self.max_pages = max(1, max(len(x) for x in rows))
        self.bt = np.zeros((self.B, self.max_pages), dtype=np.int32)
        for b, row in enumerate(rows):
            self.bt[b, :len(row)] = perm[row] if row else []
        self.pool = r.integers(0, 256, (1, s.n_kv_heads, s.G, self.n_pages, 2, Pg * J), dtype=np.uint8)
        if copy_pages:
            for i, (size, shared) in enumerate(groups):
                lead = self.starts[i]
                for b in range(lead + 1, lead + size):
                    n = min(shared, self.n_vq[b])
                    for h in range(s.n_kv_heads):
                        for kv in range(2):
                            p = self.pool[0, h, self.gamma]
                            idx = O.unpack_sequence(p, n, J, self.bt[lead], Pg, kv)
                            O.pack_sequence(p, idx, self.bt[b], Pg, kv)
        self.cb = random_codebooks(s, 1, seed + 7)
        self.q = (torch.randn(self.B, s.n_q_heads, s.head_dim, generator=g) * q_scale).to(torch.bfloat16)
        self.win = [torch.randn(self.B, s.n_kv_heads, s.window, s.head_dim, generator=g).to(torch.bfloat16)
                    for _ in range(2)]
        self.max_group = max([n for n, _ in groups] + [0])
        self.max_shared = max([n for _, n in groups] + [0])
        self.max_own = max([n - min(n, S) for n, S in zip(self.n_vq, self.S)] + [0])
        self.sm_scale = 1.0 / math.sqrt(s.head_dim)

    def config(self):
        s = self.shape
        return L.LoopVQConfig(n_layers=1, n_kv_heads=s.n_kv_heads, n_q_heads=s.n_q_heads, head_dim=s.head_dim,
                              n_loops=s.n_loops, loop_group=s.loop_group, chan_group=s.chan_group,
                              n_pages=self.n_pages, max_batch=self.B, max_pages_per_seq=self.max_pages,
                              prefix_tokens=s.prefix, recent_tokens=s.recent, page_tokens=s.page_tokens)

    def device(self, dev="cuda"):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)
        return dict(q=self.q.to(dev), pool=torch.from_numpy(self.pool).to(dev), codebooks=self.cb.to(dev),
                    block_table=i32(self.bt), seq_lens=i32(self.seq_lens), group_starts=i32(self.starts),
                    shared_lens=i32([n for _, n in self.groups]), win_k=self.win[0].to(dev),
                    win_v=self.win[1].to(dev))

    def workspace_bytes(self):
        return L.loopvq_decode_shared_workspace_bytes(self.config(), self.B, len(self.groups), self.max_group,
                                                      self.max_shared, self.max_own)

    def run_gpu(self, out_dtype=torch.bfloat16, status=0, dev_inputs=None, bounds=None, lse=True):
        s = self.shape
        d = self.device() if dev_inputs is None else dev_inputs
        out = Guarded((self.B, s.n_q_heads, s.head_dim), out_dtype, fill=float("nan"))
        ls = Guarded((self.B, s.n_q_heads), torch.float32, fill=float("nan"))
        mg, ms, mo = bounds or (self.max_group, self.max_shared, self.max_own)
        ws = workspace(L.loopvq_decode_shared_workspace_bytes(self.config(), self.B, len(self.groups), mg, ms, mo))
        L.loopvq_decode_attn_shared(self.config(), 0, self.t, **d, out=out.t, workspace=ws.t, max_group=mg,
                                    max_shared_len=ms, max_own_len=mo, lse=ls.t if lse else None,
                                    sm_scale=self.sm_scale)
        for buf, what in ((out, "output"), (ls, "lse"), (ws, "workspace")):
            buf.check(what)
        assert status_word(ws) == status, f"status {status_word(ws)}"
        return out.t.float().cpu().numpy(), ls.t.cpu().numpy()

    def oracle(self, b, hq):
        """(out, lse, sum of p |v| per channel, largest scaled sum of |q k|)."""
        s = self.shape
        h = hq // (s.n_q_heads // s.n_kv_heads)
        N, n = self.seq_lens[b], self.n_vq[b]
        if N == 0:
            return np.zeros(s.head_dim), -math.inf, np.zeros(s.head_dim), 0.0
        nw = min(N, s.window)
        K, V = [], []
        for kv, dst in ((0, K), (1, V)):
            idx = O.unpack_sequence(self.pool[0, h, self.gamma], n, s.J, self.bt[b], s.page_tokens, kv)
            dst.append(self.win[kv][b, h, :nw].double().numpy())
            dst.append(O.dequant_ref(idx, self.cb[0, h, self.gamma, kv].double().numpy(), self.tau))
        K, V = np.concatenate(K), np.concatenate(V)
        q = self.q[b, hq].double().numpy()
        out, lse = O.attn_ref(q, K, V, self.sm_scale)
        p = O.softmax_weights_ref(q, K, self.sm_scale)
        return out, lse, p @ np.abs(V), float(np.max(np.abs(K) @ np.abs(q)) * self.sm_scale)


def check_shared(case, out, lse, pairs=None):
    """bf16 outputs against the oracle.

    Quantised keys and values enter the tensor cores as fp16 codewords, softmax
    weights as fp16 too; products and sums are float32. With S the largest
    scaled sum of |q k| over a row's tokens, a score is off by at most
    d = S (2^-11 + 140 * 2^-24) (half a step of a codeword; 128 float32
    additions and the scaling), so a weight is off by a factor within e^(+-2d)
    of the softmax, and by half a step more (2^-11) for its own rounding; a
    value codeword by 2^-11. Weights below fp16's normal range (2^-20 of the
    largest) add at most 2^-31 of the largest weight each: below 2^-16 in sum for
    32K tokens. The fast exponential is within 2^-21. With A = sum p |v|:
        |out - ref| <= A (2d' + 2^-10 + 2^-15) + 2^-8 (|ref| + that),
    d' = e^(2d) - 1 over 2, and |lse - ref| <= d + 2^-19 + lse's own float32
    step."""
    s = case.shape
    if pairs is None:
        pairs = [(b, h) for b in range(case.B) for h in range(s.n_q_heads)]
    worst = 0.0
    for b, h in pairs:
        ref, lref, A, S = case.oracle(b, h)
        o = out[b, h].astype(np.float64)
        if case.seq_lens[b] == 0:
            assert np.all(o == 0) and lse[b, h] == -np.inf
            continue
        dx = S * (2.0 ** -11 + 140 * 2.0 ** -24)
        e = A * (math.expm1(2 * dx) + 2.0 ** -10 + 2.0 ** -15)
        tol = e + 2.0 ** -8 * (np.abs(ref) + e)
        err = np.abs(o - ref)
        assert np.all(err <= tol), (b, h, float(np.max(err - tol)), float(np.max(err)))
        worst = max(worst, float(np.max(err / tol)))
        assert abs(float(lse[b, h]) - lref) <= dx + 2.0 ** -19 + 2.0 ** -23 * abs(lref), (b, h, float(lse[b, h]), lref)
    return worst
