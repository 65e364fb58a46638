"""Host-side tests of loopvq_append: refusals before any launch, the
binding's checks, and the window oracle that the GPU tests use."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import sub_bit_vq_b200 as L
from oracle import loopvq_oracle as O
from sub_bit_vq_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E, U = B.LOOPVQ_ERR_INVALID_ARG, B.LOOPVQ_ERR_UNSUPPORTED


def _cfg(**kw):
    base = dict(n_layers=2, n_kv_heads=3, n_q_heads=6, head_dim=128, n_loops=8, loop_group=4,
                chan_group=4, n_pages=10, max_batch=4, max_pages_per_seq=5)
    base.update(kw)
    return L.LoopVQConfig(**base)


def _raw(cfg=None, **over):
    # fake, aligned, never dereferenced addresses
    a = dict(layer=0, loop=0, batch=2, n=2, q=0x1000, qs=768, k=0x2000, ks=384, v=0x3000, vs=384,
             rope=0x4000, pos=100, rot=128, inter=0, starts=None, sl=0x5000, bt=0x6000, wk=0x7000,
             wv=0x8000, qo=0x9000, ev=0xA000, slots=0xB000)
    a.update(over)
    return B.library().loopvq_append(ctypes.byref((cfg or _cfg()).c_struct()), *a.values(), None)


@pytest.mark.parametrize("over", [
    dict(layer=2), dict(layer=-1), dict(loop=8), dict(loop=-1), dict(batch=0), dict(batch=5, n=5), dict(n=-1),
    dict(n=3),                                   # one token per sequence needs n == batch
    dict(k=None), dict(v=None), dict(sl=None), dict(ev=None), dict(wk=None), dict(wv=None),
    dict(q=None), dict(qo=None), dict(bt=None),
    dict(rope=None), dict(rot=0), dict(pos=0), dict(pos=-1), dict(rot=-4), dict(rot=132), dict(rot=127),
    dict(qs=4), dict(ks=-8), dict(vs=12),
    dict(q=0x1008), dict(k=0x2002), dict(v=0x3008), dict(rope=0x4004), dict(starts=0xC002), dict(sl=0x5002),
    dict(bt=0x6002), dict(wk=0x7008), dict(wv=0x8008), dict(qo=0x9004), dict(ev=0xA008), dict(slots=0xB004),
])
def test_rejects_before_launch(over):
    assert _raw(**over) == E


def test_odd_pair_counts_are_unsupported_and_no_tokens_are_no_work():
    assert _raw(rot=126) == U
    assert _raw(n=0, q=None, k=None, v=None, sl=None, ev=None, wk=None, wv=None, qo=None) == B.LOOPVQ_OK
    assert _raw(n=0, layer=2) == E               # the shape arguments are checked all the same


def test_binding_checks_shapes_types_and_device():
    cfg = _cfg()
    n, b = 2, 2

    def call(**over):
        a = dict(q=torch.zeros(n, 6, 128, dtype=torch.bfloat16), k=torch.zeros(n, 3, 128, dtype=torch.bfloat16),
                 v=torch.zeros(n, 3, 128, dtype=torch.bfloat16), rope=torch.zeros(9, 128),
                 seq_lens=torch.ones(b, dtype=torch.int32),
                 win_k=torch.zeros(b, 3, 72, 128, dtype=torch.bfloat16),
                 win_v=torch.zeros(b, 3, 72, 128, dtype=torch.bfloat16),
                 q_out=torch.zeros(n, 6, 128, dtype=torch.bfloat16),
                 evicted=torch.zeros(2, 2, 2, 4, n, 3, 128, dtype=torch.bfloat16), token_starts=None,
                 block_table=torch.zeros(b, 5, dtype=torch.int32), slot_mapping=torch.zeros(n, dtype=torch.int64))
        a.update(over)
        L.loopvq_append(cfg, 0, 0, **a)

    with pytest.raises(ValueError, match="CUDA device"):
        call()
    bf = torch.bfloat16
    for over in (dict(q=torch.zeros(n, 6, 128)), dict(k=torch.zeros(n, 3, 128))):
        with pytest.raises(TypeError):
            call(**over)
    for over in (dict(q=torch.zeros(n, 5, 128, dtype=bf)), dict(q=torch.zeros(3, 6, 128, dtype=bf)),
                 dict(v=torch.zeros(3, 3, 128, dtype=bf)), dict(k=torch.zeros(n, 128, 3, dtype=bf).transpose(1, 2)),
                 dict(q_out=None), dict(q_out=torch.zeros(n, 6, 64, dtype=bf)),
                 dict(win_k=torch.zeros(b, 3, 71, 128, dtype=bf)), dict(win_v=torch.zeros(b, 3, 72, 128)),
                 dict(evicted=torch.zeros(2, 2, 2, 4, n, 3, 64, dtype=bf)),
                 dict(rope=torch.zeros(9, 128, dtype=torch.float64)), dict(rope=torch.zeros(9, 256)[:, ::2]),
                 dict(seq_lens=torch.ones(b, dtype=torch.int64)),
                 dict(token_starts=torch.zeros(b, dtype=torch.int32)),
                 dict(slot_mapping=torch.zeros(n, dtype=torch.int32)), dict(block_table=None),
                 dict(block_table=torch.zeros(b, 4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call(**over)


def test_status_bit_matches_the_header():
    text = open(os.path.join(ROOT, "include", "loopvq.h")).read()
    m = re.search(r"LOOPVQ_ENCODE_STATUS_BAD_POSITION\s*=\s*(\d+)", text)
    assert int(m.group(1)) == B.LOOPVQ_ENCODE_STATUS_BAD_POSITION == L.LOOPVQ_ENCODE_STATUS_BAD_POSITION


@pytest.mark.parametrize("P,R", [(8, 64), (0, 5), (3, 1), (4, 0)])
def test_window_oracle_keeps_prefix_and_recent_tokens(P, R):
    # token t holds the value t; appended in uneven pieces, the window must hold
    # exactly the first P and the last R tokens and every other one must have
    # come out once, in order
    win = np.full((1, P + R, 1), -1.0)
    out, N = [], 0
    for n in (1, 2, 70, 3, 200, 1, 64):
        toks = np.arange(N, N + n, dtype=float).reshape(n, 1, 1)
        N += n
        for i, (pos, val) in sorted(O.append_sequence_ref(win, toks, N, P, R).items()):
            assert val[0, 0] == pos == N - n + i - R
            out.append(pos)
        held = sorted(int(x) for x in win[0, :, 0] if x >= 0)
        assert held == list(range(min(N, P))) + list(range(max(P, N - R), N))
        assert out == list(range(P, max(P, N - R)))


def test_rotation_oracle_is_a_rotation():
    r = np.random.default_rng(0)
    x = r.standard_normal((3, 12))
    ang = r.uniform(0, 6, 4)
    for inter in (False, True):
        y = O.rotate_ref(x, np.cos(ang), np.sin(ang), inter)
        back = O.rotate_ref(y, np.cos(ang), -np.sin(ang), inter)
        np.testing.assert_allclose(back, x, atol=1e-14)
        np.testing.assert_array_equal(y[:, 8:], x[:, 8:])
        np.testing.assert_allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1), rtol=1e-14)
        # a pair as a complex number times e^(i angle)
        a, b = (x[:, 0:8:2], x[:, 1:8:2]) if inter else (x[:, :4], x[:, 4:8])
        z = (a + 1j * b) * np.exp(1j * ang)
        c, d = (y[:, 0:8:2], y[:, 1:8:2]) if inter else (y[:, :4], y[:, 4:8])
        np.testing.assert_allclose(c + 1j * d, z, atol=1e-14)


@pytest.mark.parametrize("ahead", [0, 1, 64])
def test_stage_ahead_is_checked(ahead):
    a = dict(layer=0, loop=0, batch=2, n=0, q=0x1000, qs=768, k=0x2000, ks=384, v=0x3000, vs=384, rope=0x4000, pos=100,
             rot=128, inter=0, ahead=ahead, starts=None, sl=0x5000, bt=0x6000, wk=0x7000, wv=0x8000, qo=0x9000, ev=0xA000,
             slots=0xB000)
    call = lambda **over: B.library().loopvq_append_ahead(ctypes.byref(_cfg().c_struct()), *{**a, **over}.values(), None)
    assert call() == B.LOOPVQ_OK                 # (no tokens: no work)
    assert call(ahead=-1) == call(ahead=65) == E
    assert call(layer=2) == call(rot=-4) == E


@pytest.mark.parametrize("P,R", [(8, 64), (0, 5), (3, 1)])
def test_window_oracle_stages_ahead(P, R):
    # every token once, in order, `ahead` rows before it leaves the window
    for ahead in {1, (R + 1) // 2, R}:
        win = np.full((1, P + R, 1), -1.0)
        out, N = [], 0
        for n in (1, 2, 70, 3, 200, 1, 64):
            toks = np.arange(N, N + n, dtype=float).reshape(n, 1, 1)
            N += n
            for i, (pos, val) in sorted(O.append_sequence_ref(win, toks, N, P, R, ahead).items()):
                assert val[0, 0] == pos == N - n + i - R + ahead
                out.append(pos)
            assert sorted(int(x) for x in win[0, :, 0] if x >= 0) == list(range(min(N, P))) + list(range(max(P, N - R), N))
            assert out == list(range(P, max(P, N - R + ahead)))


def test_more_heads_than_a_grid_holds_are_refused():
    # 2^29 query heads of 8 units: the product must not wrap to a small grid that
    # leaves the queries out
    assert _raw(_cfg(n_q_heads=2 ** 29, n_kv_heads=2 ** 10), qs=0) == U
