"""Whole decode steps: a prompt and then several steps of append, attention at
every loop step, and encoding of what was staged, from a pool that holds no
index yet.

Every token is made of codewords (bf16 values), one per channel group and loop
group, and the rotation turns by quarter turns, so a token's index, its place in
a window and its value after the pool are all the same known numbers: the oracle
is plain attention over all tokens of a sequence, and an index that is read
before it is written shows as a wrong output.
"""

import numpy as np
import pytest
import torch

import sub_bit_vq_b200 as L
from oracle import loopvq_oracle as O

from _shared_cases import check_shared

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, D, C, J, T, G_LOOPS, PAGE = 16, 128, 4, 32, 4, 2, 64
W, R = 72, 64


def quarter_turns(n):
    """Rotation table [n][D]: cosines, then sines, of whole quarter turns."""
    k = (np.arange(n)[:, None] * (1 + np.arange(D // 2)) + np.arange(D // 2) // 3) % 4
    cos, sin = np.array([1, 0, -1, 0])[k], np.array([0, 1, 0, -1])[k]
    return np.concatenate([cos, sin], 1).astype(np.float32)


class Run:
    """B sequences with the same prompt of n0 tokens; tokens[t][kv] and q[t] hold
    every token of every sequence ahead of time, [B][positions][H][D]."""

    def __init__(self, n0, most, B=4, seed=0):
        r = np.random.default_rng(seed)
        self.B, self.n0 = B, n0
        self.rope = quarter_turns(most)
        self.cb = torch.from_numpy(r.standard_normal((1, H, T // G_LOOPS, 2, G_LOOPS, J, 256, C))).to(BF).float()
        cb = self.cb.numpy()
        h, j = np.arange(H)[:, None], np.arange(J)
        self.tokens = [[None, None] for _ in range(T)]    # after the rotation
        for gamma in range(T // G_LOOPS):
            for kv in range(2):
                code = r.integers(0, 256, (B, most, H, J))
                code[:, :n0] = code[:1, :n0]              # the prompt is the same
                for tau in range(G_LOOPS):
                    self.tokens[gamma * G_LOOPS + tau][kv] = cb[0][h, gamma, kv, tau, j, code].reshape(B, most, H, D)
        self.q = [r.standard_normal((B, most, H, D)).astype(np.float32) for _ in range(T)]
        pages = -(-most // PAGE)
        full = (n0 - W) // PAGE                           # whole pages of the prompt are shared
        table = np.zeros((B, pages), np.int32)
        table[:, :full] = np.arange(full)
        table[:, full:] = full + np.arange(B * (pages - full)).reshape(B, -1)
        self.n_pages = int(table.max()) + 1
        self.cfg = L.LoopVQConfig(n_layers=1, n_kv_heads=H, n_q_heads=H, head_dim=D, n_loops=T, loop_group=G_LOOPS,
                                  chan_group=C, n_pages=self.n_pages, max_batch=B, max_pages_per_seq=pages)
        dev = "cuda"
        self.bt = torch.from_numpy(table).to(dev)
        self.pool = torch.full((1, H, T // G_LOOPS, self.n_pages, 2, PAGE * J), 0xff, dtype=torch.uint8, device=dev)
        self.cbd, self.roped = self.cb.to(dev), torch.from_numpy(self.rope).to(dev)
        self.win = [[torch.full((B, H, W, D), float("nan"), dtype=BF, device=dev) for _ in range(2)] for _ in range(T)]
        self.lens = [0] * B

    def unturned(self, x, p):
        """The input whose rotation at positions p is x."""
        cos, sin = self.rope[p][:, None, :D // 2], self.rope[p][:, None, D // 2:]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([a * cos + b * sin, b * cos - a * sin], -1)

    def step(self, counts, ahead, attend):
        """Appends counts[b] tokens, attends at every loop step, encodes."""
        dev, B = "cuda", self.B
        old, self.lens = self.lens, [x + n for x, n in zip(self.lens, counts)]
        starts = np.concatenate([[0], np.cumsum(counts)])
        n = int(starts[-1])
        rows = [(b, p) for b in range(B) for p in range(old[b], self.lens[b])]
        bs, ps = np.array([b for b, _ in rows]), np.array([p for _, p in rows])
        ev = torch.zeros(1, T // G_LOOPS, 2, G_LOOPS, n, H, D, dtype=BF, device=dev)
        slots = torch.zeros(n, dtype=torch.int64, device=dev)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        ts = torch.tensor(starts, dtype=torch.int32, device=dev)
        put = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(BF).to(dev)
        for t in range(T):
            k = put(self.unturned(self.tokens[t][0][bs, ps], ps))
            v, q = put(self.tokens[t][1][bs, ps]), put(self.q[t][bs, ps])
            q_out = torch.empty_like(q)
            L.loopvq_append(self.cfg, 0, t, q, k, v, self.roped, lens, *self.win[t], q_out, ev, token_starts=ts,
                            block_table=self.bt, slot_mapping=slots if t == 0 else None, stage_ahead=ahead)
            if attend:
                self.attend(t, q_out[ts[1:].long() - 1].contiguous(), lens)
        if n <= 64:
            L.loopvq_encode_evict(self.cfg, ev, self.cbd, slots, self.pool)
        else:
            for gamma in range(T // G_LOOPS):
                for kv in range(2):
                    L.loopvq_encode(self.cfg, 0, gamma, kv, ev[0, gamma, kv], None, self.cbd, slots, self.pool)

    def attend(self, t, q, lens):
        out = torch.empty(self.B, H, D, dtype=torch.float32, device="cuda")
        lse = torch.empty(self.B, H, dtype=torch.float32, device="cuda")
        most, S = max(self.lens), self.n0 - W
        ws = torch.zeros(L.loopvq_decode_workspace_bytes(self.cfg, self.B, most), dtype=torch.uint8, device="cuda")
        L.loopvq_decode_attn(self.cfg, 0, t, q, self.pool, self.cbd, self.bt, lens, *self.win[t], out, ws, most, lse=lse)
        own = max(self.lens) - W - S
        out2 = torch.empty(self.B, H, D, dtype=BF, device="cuda")
        lse2 = torch.empty_like(lse)
        ws2 = torch.zeros(L.loopvq_decode_shared_workspace_bytes(self.cfg, self.B, 1, self.B, S, own), dtype=torch.uint8,
                          device="cuda")
        L.loopvq_decode_attn_shared(self.cfg, 0, t, q, self.pool, self.cbd, self.bt, lens,
                                    torch.tensor([0, self.B], dtype=torch.int32, device="cuda"),
                                    torch.tensor([S], dtype=torch.int32, device="cuda"), *self.win[t], out2, ws2, self.B, S,
                                    own, lse=lse2)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32)) == 0 and int(ws2[:4].view(torch.int32)) == 0
        self.t, self.seq_lens, self.qh = t, self.lens, q.double().cpu().numpy()
        out, lse = out.cpu().numpy(), lse.cpu().numpy()
        for b in range(self.B):
            for h in range(H):
                ref, lref, _, _ = self.oracle(b, h)
                assert np.max(np.abs(out[b, h] - ref)) <= 1e-4 * np.max(np.abs(ref)), (t, b, h)
                assert abs(lse[b, h] - lref) <= 1e-4
        check_shared(self, out2.float().cpu().numpy(), lse2.cpu().numpy())

    shape = type("S", (), {"n_q_heads": H})

    def oracle(self, b, h):
        K, V = (self.tokens[self.t][kv][b, :self.lens[b], h].astype(np.float64) for kv in range(2))
        q, sm = self.qh[b, h], D ** -0.5
        out, lse = O.attn_ref(q, K, V, sm)
        return out, lse, O.softmax_weights_ref(q, K, sm) @ np.abs(V), float(np.max(np.abs(K) @ np.abs(q)) * sm)


STEPS = {
    "one_token": (1, [[1, 1, 1, 1]] * 5),
    "one_token_some_wait": (1, [[1, 0, 1, 1], [1, 1, 0, 1], [0, 1, 1, 1], [1, 1, 1, 0]]),
    "up_to_three": (3, [[3, 1, 2, 1], [1, 3, 0, 3], [2, 2, 3, 1], [3, 3, 1, 0]]),
    "a_whole_window_ahead": (64, [[1, 40, 64, 3], [2, 1, 1, 64]]),
}


@pytest.mark.parametrize("name", list(STEPS))
def test_steps_attend_to_written_indices_only(name):
    ahead, steps = STEPS[name]
    # 189 quantised prompt tokens: the steps cross the page end at 192
    run = Run(W + 189, W + 189 + max(sum(s[b] for s in steps) for b in range(4)) + 64, seed=len(name))
    run.step([run.n0] * 4, ahead, attend=False)
    for counts in steps:
        run.step(counts, ahead, attend=True)
    assert L.loopvq_encode_status() == 0


def test_a_long_prompt_in_chunks_and_then_steps():
    # the prompt in three pieces, one longer than the window, each encoded before the next
    run = Run(W + 189, W + 189 + 70, seed=5)
    for n in (100, 7, run.n0 - 107):
        run.step([n] * 4, 1, attend=False)
    for _ in range(2):
        run.step([1, 1, 1, 1], 1, attend=True)
