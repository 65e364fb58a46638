"""GPU parity of loopvq_append with the token-by-token oracle.

Tolerances. Copied values (v, channels past rot_dim, evicted old tokens) are
exact. A rotated value y = a c - b s is computed in float32 (two products and a
sum, each off by at most 2^-24 relative: |error| <= 2^-23 (|a c| + |b s|) to
first order, doubled here for the second-order terms) and rounded once to bf16
(half a step: 2^-8 relative).
"""

import numpy as np
import pytest
import torch

import sub_bit_vq_b200 as L
from oracle import loopvq_oracle as O
from sub_bit_vq_b200 import binding as B

from _guard import Guarded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rope_table(n, rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(n)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()


class Case:
    """Windows of `lens` cached tokens, then counts[b] new ones per sequence."""

    def __init__(self, *, old, counts, Hq=4, Hkv=2, d=128, c=4, rot=128, inter=False, P=8, R=64, page=64, T=4,
                 g=2, n_layers=2, layer=1, loop=3, fused=True, tail=0, one=False, gap=0, seed=0, with_q=True,
                 table=None):
        r = torch.Generator().manual_seed(seed)
        self.old, self.counts, self.B = old, counts, len(old)
        self.Hq, self.Hkv, self.d, self.rot, self.inter, self.P, self.R = Hq, Hkv, d, rot, inter, P, R
        self.total = [o + n for o, n in zip(old, counts)]
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.n = starts[-1] + tail                        # rows behind the last sequence
        self.page, self.layer, self.loop, self.one, self.g, self.T, self.L = page, layer, loop, one, g, T, n_layers
        self.pages = max(1, -(-max(self.total + [1]) // page))
        self.cfg = L.LoopVQConfig(n_layers=n_layers, n_kv_heads=Hkv, n_q_heads=Hq, head_dim=d, n_loops=T,
                                  loop_group=g, chan_group=c, n_pages=self.B * self.pages + 2,
                                  max_batch=self.B, max_pages_per_seq=self.pages, prefix_tokens=P,
                                  recent_tokens=R, page_tokens=page)
        self.bt = torch.randperm(self.cfg.n_pages, generator=r)[:self.B * self.pages].view(self.B, -1).int()
        width = (Hq + 2 * Hkv) * d + gap
        x = torch.randn(self.n, width, generator=r).to(BF)
        if fused:
            self.q = x[:, :Hq * d].view(self.n, Hq, d)
            self.k = x[:, Hq * d:(Hq + Hkv) * d].view(self.n, Hkv, d)
            self.v = x[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].view(self.n, Hkv, d)
        else:
            self.q, self.k, self.v = (torch.randn(self.n, h, d, generator=r).to(BF) for h in (Hq, Hkv, Hkv))
        if not with_q:
            self.q = None
        self.win = [torch.randn(self.B, Hkv, P + R, d, generator=r).to(BF) for _ in range(2)]
        self.rope = None if rot == 0 else rope_table(max(self.total + [1]), rot) if table is None else table

    def run(self, stream=None, skip=()):
        dev = "cuda"
        out = dict(q=Guarded((self.n, self.Hq, self.d), BF, fill=7.0) if self.q is not None else None,
                   ev=Guarded((self.L, self.T // self.g, 2, self.g, self.n, self.Hkv, self.d), BF, fill=5.0),
                   slots=Guarded((self.n,), torch.int64, fill=-9),
                   wk=Guarded(self.win[0].shape, BF), wv=Guarded(self.win[1].shape, BF))
        out["wk"].t.copy_(self.win[0])
        out["wv"].t.copy_(self.win[1])
        base = None
        if self.q is not None and self.q.stride(0) != self.Hq * self.d:   # one fused buffer on the device
            base = self.q._base.to(dev)
            q, k, v = (torch.as_strided(base, t.shape, t.stride(), t.storage_offset()) for t in (self.q, self.k, self.v))
        else:
            q, k, v = (t.to(dev) if t is not None else None for t in (self.q, self.k, self.v))
        sl = [0 if b in skip else t for b, t in enumerate(self.total)]
        args = (self.cfg, self.layer, self.loop, q, k, v, self.rope.to(dev) if self.rope is not None else None,
                torch.tensor(sl, dtype=torch.int32, device=dev), out["wk"].t, out["wv"].t,
                out["q"].t if out["q"] else None, out["ev"].t)
        kw = dict(token_starts=None if self.one else torch.tensor(self.starts, dtype=torch.int32, device=dev),
                  interleaved=self.inter, block_table=self.bt.to(dev), slot_mapping=out["slots"].t)
        self.args = (args, kw)
        L.loopvq_encode_status(clear=True)
        torch.cuda.synchronize()
        L.loopvq_append(*args, stream=stream, **kw)
        torch.cuda.synchronize()
        for name, buf in out.items():
            if buf is not None:
                buf.check(name)
        assert L.loopvq_encode_status() == 0
        return out

    def check(self, out, skip=()):
        rope = self.rope.double().numpy() if self.rope is not None else None
        half = self.rot // 2
        f8 = lambda t: t.double().cpu().numpy()

        def turned(x, p):                                 # value and tolerance
            if rope is None:
                return x, np.zeros_like(x)
            cos, sin = rope[p, :half], rope[p, half:]
            y = O.rotate_ref(x, cos, sin, self.inter)
            size = O.rotate_ref(np.abs(x), np.abs(cos), -np.abs(sin), self.inter)   # |a c| + |b s| of the first
            other = O.rotate_ref(np.abs(x), np.abs(cos), np.abs(sin), self.inter)   # ... of the second entry
            f = 2.0 ** -22 * np.maximum(np.abs(size), np.abs(other))
            tol = np.zeros_like(y)
            tol[..., :self.rot] = (f + 2.0 ** -8 * (np.abs(y) + f))[..., :self.rot]
            return y, tol

        gamma, tau = divmod(self.loop, self.g)
        ev = out["ev"].t
        for a, (src, name) in enumerate(((self.k, "wk"), (self.v, "wv"))):
            want_w = f8(self.win[a])
            tol_w = np.zeros_like(want_w)
            want_e = np.full((self.n, self.Hkv, self.d), 5.0)
            tol_e = np.zeros_like(want_e)
            want_s = np.full(self.n, -1)
            for b in range(self.B):
                if b in skip:
                    continue
                rows = range(self.starts[b], self.starts[b + 1])
                val = [turned(f8(src[r]), self.total[b] - len(rows) + i) if a == 0 else
                       (f8(src[r]), np.zeros((self.Hkv, self.d))) for i, r in enumerate(rows)]
                if not val:
                    continue
                gone = O.append_sequence_ref(want_w[b], np.stack([x for x, _ in val]), self.total[b], self.P, self.R)
                gone_t = O.append_sequence_ref(tol_w[b], np.stack([t for _, t in val]), self.total[b], self.P, self.R)
                for i, (pos, x) in gone.items():
                    r = rows[i]
                    want_e[r], tol_e[r] = x, gone_t[i][1]
                    v = pos - self.P
                    want_s[r] = int(self.bt[b, v // self.page]) * self.page + v % self.page
            assert np.all(np.abs(f8(out[name].t) - want_w) <= tol_w), name
            assert np.all(np.abs(f8(ev[self.layer, gamma, a, tau]) - want_e) <= tol_e), "evicted"
            np.testing.assert_array_equal(out["slots"].t.cpu().numpy(), want_s)
        others = ev.clone()
        others[self.layer, gamma, :, tau] = 5.0
        assert bool((others == 5.0).all()), "another slice of the staging buffer was written"
        if self.q is not None:
            got = f8(out["q"].t)
            want, tol = np.full(got.shape, 7.0), np.zeros(got.shape)
            for b in range(self.B):
                if b not in skip:
                    for i, r in enumerate(range(self.starts[b], self.starts[b + 1])):
                        want[r], tol[r] = turned(f8(self.q[r]), self.old[b] + i)
            assert np.all(np.abs(got - want) <= tol), "q"


CASES = {
    "one_token_each": dict(old=[0, 1, 7, 8, 71, 72, 73, 500, 1000], counts=[1] * 9, one=True),
    "one_token_starts": dict(old=[40, 90, 3], counts=[1, 1, 1]),
    "drafts": dict(old=[300, 71, 0, 66, 135], counts=[5, 3, 8, 7, 1]),
    "around_the_ring": dict(old=[0, 100, 100, 100, 100], counts=[63, 63, 64, 65, 130]),
    "prompts": dict(old=[0, 0, 0, 0, 0, 0], counts=[1, 8, 9, 72, 73, 333]),
    "chunks_on_old": dict(old=[5, 8, 50, 400], counts=[200, 129, 77, 64]),
    "empty_sequences": dict(old=[10, 100, 0, 7], counts=[0, 3, 0, 2]),
    "rows_behind": dict(old=[90, 10], counts=[4, 70], tail=13),
    "interleaved": dict(old=[0, 90, 200], counts=[20, 66, 1], inter=True),
    "half_rotated": dict(old=[0, 90], counts=[20, 66], rot=64),
    "half_interleaved_d96": dict(old=[0, 90], counts=[20, 66], d=96, c=8, rot=48, inter=True, page=96),
    "d96": dict(old=[0, 90, 77], counts=[20, 66, 100], d=96, c=8, rot=96, page=96),
    "narrow_rot": dict(old=[0, 90], counts=[20, 66], rot=20),
    "narrow_interleaved": dict(old=[0, 90], counts=[20, 66], rot=36, inter=True),
    "d24": dict(old=[0, 90], counts=[20, 66], d=24, c=2, rot=24, page=96),
    "d64": dict(old=[3, 90, 128], counts=[1, 1, 1], d=64, rot=64, one=True, Hq=1, Hkv=1),
    "d256": dict(old=[3, 90], counts=[70, 2], d=256, c=8, rot=256),
    "no_rotation_no_q": dict(old=[300, 71, 0], counts=[5, 3, 80], rot=0, with_q=False, fused=False),
    "many_heads": dict(old=[300] * 3, counts=[1] * 3, Hq=40, Hkv=40, one=True),
    "gap_between_tokens": dict(old=[300, 20], counts=[9, 100], gap=72),
    "no_prefix": dict(old=[0, 100], counts=[70, 3], P=0),
    "no_ring": dict(old=[0, 100, 7], counts=[20, 3, 2], R=0),
    "no_window": dict(old=[0, 100], counts=[20, 3], P=0, R=0),
    "ring_of_one": dict(old=[0, 100], counts=[20, 3], P=2, R=1),
    "many_sequences": dict(old=[(37 * i) % 300 for i in range(300)], counts=[(7 * i) % 4 for i in range(300)], Hq=2, Hkv=1,
                           d=64, rot=64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_append_matches_the_oracle(name):
    c = Case(seed=len(name), **CASES[name])
    c.check(c.run())


def test_padded_rows_of_a_batch_write_nothing():
    c = Case(old=[300, 90, 10, 500], counts=[1] * 4, one=True)
    c.check(c.run(skip=(1, 3)), skip=(1, 3))
    c = Case(old=[300, 90, 10], counts=[3, 70, 20])
    c.check(c.run(skip=(1,)), skip=(1,))


def test_infinities_and_nan_stay_where_they_are():
    c = Case(old=[100, 90], counts=[2, 70], fused=False)
    c.k[0, 0, 3] = float("nan")
    c.k[3, 1, 70] = float("inf")
    c.v[1, 1, 0] = float("-inf")
    out = c.run()
    k = out["wk"].t
    bad = ~torch.isfinite(k)
    assert bad.sum() == 2                                  # each spoils its pair only
    assert bool(torch.isnan(k[0, 0, 8 + (100 - 8) % 64, [3, 67]]).all())
    # row 3 is token 91 of sequence 1, which token 155 (row 67) pushes out again
    ev = ~torch.isfinite(out["ev"].t[1, 1, 0, 1])
    assert ev.sum() == 2 and bool(ev[67, 1, [70, 6]].all())
    assert int((~torch.isfinite(out["wv"].t)).sum()) == 1
    assert bool(torch.isfinite(out["q"].t).all())


def test_q_in_place():
    c = Case(old=[100, 90], counts=[2, 70], fused=False)
    want = c.run()["q"].t.clone()
    (args, kw) = c.args
    args = list(args)
    args[10] = args[3]
    L.loopvq_append(*args, **kw)
    assert torch.equal(args[3], want)


def test_bad_positions_and_pages_are_skipped_and_flagged():
    c = Case(old=[100, 90], counts=[3, 2])
    c.rope = c.rope[:101]                                  # the first sequence reaches past the table
    with pytest.raises(AssertionError):
        c.run()
    assert L.loopvq_encode_status(clear=True) == B.LOOPVQ_ENCODE_STATUS_BAD_POSITION
    c = Case(old=[100, 90], counts=[3, 2])
    c.total[1] = 1                                         # shorter than its two rows
    with pytest.raises(AssertionError):
        c.run()
    assert L.loopvq_encode_status(clear=True) == B.LOOPVQ_ENCODE_STATUS_BAD_POSITION
    c = Case(old=[200, 100], counts=[1, 1], one=True)
    c.bt[0, 2] = c.cfg.n_pages                             # v = 200 - 72 = 128: page 2
    c.bt[1, 0] = -1                                        # v = 28: page 0
    with pytest.raises(AssertionError):
        c.run()
    assert L.loopvq_encode_status(clear=True) == B.LOOPVQ_ENCODE_STATUS_BAD_SLOT
    assert c.args[1]["slot_mapping"].tolist() == [-1, -1]
    assert L.loopvq_encode_status() == 0


def test_starts_outside_the_rows_stay_inside_the_buffers():
    c = Case(old=[100, 90, 50], counts=[3, 2, 4])
    c.starts = [-5, 3, 200, 1]                             # clipped; rows 0..2 belong to sequence 0 (8 rows: too many)
    c.total = [3, 6, 0]
    out = c.run()
    assert out["slots"].t.tolist() == [-1] * 9             # short sequences push nothing out


def test_other_stream_and_graph_replay():
    c = Case(old=[300, 71, 0], counts=[5, 3, 80], seed=3)
    want = c.run()
    s = torch.cuda.Stream()
    got = c.run(stream=s)
    for k in want:
        assert torch.equal(want[k].t, got[k].t), k
    (args, kw) = c.args
    with torch.cuda.stream(s):
        L.loopvq_append(*args, **kw)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.loopvq_append(*args, **kw)
    args[8].copy_(c.win[0])
    args[9].copy_(c.win[1])
    args[11].fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[8], want["wk"].t) and torch.equal(args[11], want["ev"].t)
    args[7].add_(64)                                       # the graph reads the lengths on the device
    args[8].copy_(c.win[0])
    args[9].copy_(c.win[1])
    long = rope_table(600, 128).cuda()
    assert args[6].shape[0] < 600 and long.shape[1] == 128
    with pytest.raises(AssertionError):
        g.replay()
        assert L.loopvq_encode_status(clear=True) == 0
    L.loopvq_encode_status(clear=True)


def test_append_then_roll_back_restores_the_windows():
    c = Case(old=[300, 200, 261], counts=[5, 3, 1], layer=0, n_layers=1, g=4, loop=2)
    out = c.run()
    (args, kw) = c.args
    ev = out["ev"].t[0, 0, :, 2]
    back = torch.zeros_like(out["ev"].t)
    L.loopvq_append(c.cfg, 0, 2, None, ev[0], ev[1], None, args[7] - 64, args[8], args[9], None, back,
                    token_starts=kw["token_starts"])
    torch.cuda.synchronize()
    assert torch.equal(out["wk"].t.cpu(), c.win[0]) and torch.equal(out["wv"].t.cpu(), c.win[1])


def test_staged_rows_feed_the_encoder():
    # append at every loop step of a group, then encode_evict: the pool holds the
    # oracle's indices of the evicted tokens at the slots append gave
    c = Case(old=[300, 90], counts=[1, 1], one=True, n_layers=1, layer=0, g=4, T=4, loop=0)
    gen = torch.Generator().manual_seed(9)
    J = 32
    cb = torch.randn(1, c.Hkv, 1, 2, 4, J, 256, 4, generator=gen)
    pool = torch.zeros(L.loopvq_cache_layout(c.cfg)["pool_bytes"], dtype=torch.uint8, device="cuda")
    ev = torch.zeros(1, 1, 2, 4, 2, c.Hkv, c.d, dtype=BF, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    c.run()
    (args, kw) = c.args
    kw["slot_mapping"] = slots
    for t in range(4):
        wins = [torch.randn(2, c.Hkv, 72, c.d, generator=gen).to(BF).cuda() for _ in range(2)]
        a = list(args)
        a[2], a[8], a[9], a[11] = t, wins[0], wins[1], ev
        L.loopvq_append(*a, **kw)
    L.loopvq_encode_evict(c.cfg, ev, cb.cuda(), slots, pool)
    torch.cuda.synchronize()
    plane = pool.cpu().numpy().reshape(c.Hkv, c.cfg.n_pages, 2, c.page * J)
    for kv in range(2):
        ref, dist = O.encode_group_ref(ev[0, 0, kv].double().cpu().numpy(), cb[0, :, 0, kv].double().numpy())
        for n in range(2):
            s = int(slots[n])
            off = O.plane_offsets(np.array([s % c.page]), J)[0]
            for h in range(c.Hkv):
                got = plane[h, s // c.page, kv, off]
                assert (got == ref[n, h]).mean() > 0.96


@pytest.mark.parametrize("ahead", [1, 3, 63, 64])
@pytest.mark.parametrize("name", list(CASES))
def test_staging_ahead_matches_the_oracle(name, ahead, monkeypatch):
    c = Case(seed=len(name), **CASES[name])
    ahead = min(ahead, c.R)
    call, ref = L.loopvq_append, O.append_sequence_ref
    monkeypatch.setattr(L, "loopvq_append", lambda *a, **kw: call(*a, stage_ahead=ahead, **kw))
    monkeypatch.setattr(O, "append_sequence_ref", lambda *a: ref(*a, ahead=ahead))
    c.check(c.run())


def test_staging_ahead_of_a_chunk_by_chunk_prompt_stages_every_token_once():
    # whatever the pieces, the staged rows are the tokens P, P + 1, .. in order
    r = torch.Generator().manual_seed(2)
    k = torch.randn(1, 400, 2, 128, generator=r).to(BF)
    pieces = [1, 5, 70, 64, 3, 1, 1, 130, 63, 62]
    for ahead in (0, 1, 5, 64):
        cfg = L.LoopVQConfig(n_layers=1, n_kv_heads=2, n_q_heads=2, head_dim=128, n_loops=1, loop_group=1, chan_group=4,
                             n_pages=8, max_batch=1, max_pages_per_seq=8)
        win = [torch.zeros(1, 2, 72, 128, dtype=BF, device="cuda") for _ in range(2)]
        bt = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
        done, slot = [], []
        N = 0
        for n in pieces:
            rows = k[0, N:N + n].cuda()
            N += n
            ev = torch.full((1, 1, 2, 1, n, 2, 128), float("nan"), dtype=BF, device="cuda")
            sl = torch.zeros(n, dtype=torch.int64, device="cuda")
            i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
            L.loopvq_append(cfg, 0, 0, None, rows, rows, None, i32([N]), *win, None, ev, token_starts=i32([0, n]),
                            block_table=bt, slot_mapping=sl, stage_ahead=ahead)
            keep = sl >= 0
            assert torch.equal(ev[0, 0, 0, 0][keep], ev[0, 0, 1, 0][keep])
            assert bool(torch.isnan(ev[0, 0, 0, 0][~keep]).all())          # rows without a staged token
            done.append(ev[0, 0, 0, 0][keep])
            slot += sl[keep].tolist()
        m = N - 8 - 64 + ahead
        assert slot == list(range(m))
        assert torch.equal(torch.cat(done).cpu(), k[0, 8:8 + m])


MANY = {   # eight rows per block: at least 16384 blocks of 128 units
    "wide": dict(old=[300, 0, 71, 9], counts=[500, 400, 201, 0], d=256, c=8, rot=256, Hq=40, Hkv=40, tail=13),
    "wide_half_interleaved_gqa": dict(old=[0, 90, 1000], counts=[1300, 66, 1400], d=128, rot=64, inter=True, Hq=64, Hkv=16, tail=3),
    "narrow_interleaved": dict(old=[0, 90], counts=[400, 333], d=96, c=8, rot=36, inter=True, page=96, Hq=40, Hkv=40),
    "narrow": dict(old=[65, 0, 8], counts=[700, 68, 601], rot=20, Hq=16, Hkv=16, tail=9),
    "not_rotated_keys_only": dict(old=[0, 90], counts=[1300, 800], rot=0, with_q=False, fused=False, Hq=60, Hkv=60),
}


@pytest.mark.parametrize("ahead", [0, 1, 5])
@pytest.mark.parametrize("name", list(MANY))
def test_many_rows_match_the_oracle(name, ahead, monkeypatch):
    kw = MANY[name]
    c = Case(seed=len(name), n_layers=1, layer=0, T=2, g=2, loop=1, **kw)
    units = -(-c.d // (16 if c.rot % 16 == 0 else 4))
    assert c.n * -(-((c.Hq if c.q is not None else 0) + 2 * c.Hkv) * units // 128) >= 16384
    call, ref = L.loopvq_append, O.append_sequence_ref
    monkeypatch.setattr(L, "loopvq_append", lambda *a, **kw: call(*a, stage_ahead=ahead, **kw))
    monkeypatch.setattr(O, "append_sequence_ref", lambda *a: ref(*a, ahead=ahead))
    c.check(c.run())


def run_flagged(c, flag, monkeypatch):
    """c.run() of a call that has to set exactly this status (and to stay inside its
    buffers, which run checks first)."""
    read = L.loopvq_encode_status
    with monkeypatch.context() as m:
        m.setattr(L, "loopvq_encode_status", lambda clear=False: read(clear) ^ (0 if clear else flag))
        out = c.run()
    assert read(clear=True) == flag
    return out


def test_a_sequence_at_a_bad_position_writes_nothing(monkeypatch):
    c = Case(old=[100, 90, 20], counts=[3, 2, 70])
    c.rope = c.rope[:101]                                  # the first one reaches past the table
    c.check(run_flagged(c, B.LOOPVQ_ENCODE_STATUS_BAD_POSITION, monkeypatch), skip=(0,))
    c = Case(old=[100, 90, 20], counts=[3, 2, 70])
    c.total[1] = 1                                         # shorter than its two rows
    c.check(run_flagged(c, B.LOOPVQ_ENCODE_STATUS_BAD_POSITION, monkeypatch), skip=(1,))


def test_a_bad_page_costs_the_slot_only(monkeypatch):
    kw = dict(old=[200, 100, 300], counts=[1, 1, 1], one=True, seed=4)
    good, bad = Case(**kw), Case(**kw)
    bad.bt[0, 2] = bad.cfg.n_pages                         # v = 200 - 72 = 128: page 2
    bad.bt[1, 0] = -1                                      # v = 28: page 0
    out = run_flagged(bad, B.LOOPVQ_ENCODE_STATUS_BAD_SLOT, monkeypatch)
    want = good.run()
    good.check(want)
    for k in ("q", "wk", "wv", "ev"):
        assert torch.equal(out[k].t, want[k].t), k
    assert out["slots"].t.tolist() == [-1, -1, int(want["slots"].t[2])]


def test_a_replayed_graph_reads_the_lengths_of_the_replay():
    c = Case(old=[364, 135, 64], counts=[5, 3, 80], seed=3)
    out = c.run()
    c.check(out)
    (args, kw) = c.args
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.loopvq_append(*args, **kw)
    c.old, c.total = [o - 64 for o in c.old], [t - 64 for t in c.total]
    args[7].sub_(64)
    for buf, first in ((args[8], c.win[0]), (args[9], c.win[1])):
        buf.copy_(first)
    args[10].fill_(7.0)
    args[11].fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    for name, buf in out.items():
        buf.check(name)
    c.check(out)
    assert L.loopvq_encode_status() == 0


def test_two_appends_at_once_on_two_streams():
    cases = [Case(old=[300, 71, 0], counts=[5, 3, 80], seed=3), Case(old=[1, 2, 500, 90], counts=[100, 1, 7, 66], seed=6)]
    outs = [c.run() for c in cases]
    want = [{k: b.t.clone() for k, b in o.items()} for o in outs]
    streams = [torch.cuda.Stream() for _ in cases]
    for c, o in zip(cases, outs):
        (args, kw) = c.args
        args[8].copy_(c.win[0])
        args[9].copy_(c.win[1])
        args[11].fill_(5.0)
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        (args, kw) = c.args
        L.loopvq_append(*args, stream=s, **kw)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for k in w:
            assert torch.equal(o[k].t, w[k]), k


def test_the_c_call_without_staging_ahead_is_the_same_call():
    c = Case(old=[300, 71, 0], counts=[5, 3, 80], seed=3)
    out = c.run()
    want = {k: b.t.clone() for k, b in out.items()}
    (args, kw) = c.args
    _, layer, loop, q, k, v, rope, lens, wk, wv, qo, ev = args
    wk.copy_(c.win[0])
    wv.copy_(c.win[1])
    qo.fill_(7.0)
    ev.fill_(5.0)
    p = lambda t: t.data_ptr()
    st = B.library().loopvq_append(c.cfg.c_ref(), layer, loop, c.B, c.n, p(q), q.stride(0), p(k), k.stride(0), p(v),
                                   v.stride(0), p(rope), *rope.shape, 0, p(kw["token_starts"]), p(lens), p(kw["block_table"]),
                                   p(wk), p(wv), p(qo), p(ev), p(kw["slot_mapping"]), torch.cuda.current_stream().cuda_stream)
    assert st == B.LOOPVQ_OK
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(out[name].t, want[name]), name
