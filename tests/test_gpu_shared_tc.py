"""GPU parity of loopvq_decode_attn_shared's tensor-core form: at least four
query rows per group on average and 64 (sequence, query head) pairs, bf16
outputs. The bound is check_shared's; large cases check a sample of the pairs.
"""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import sub_bit_vq_b200 as L
from oracle import loopvq_oracle as O
from sub_bit_vq_b200 import binding as B
from synthetic import Shape

from _cases import sample_pairs
from _guard import workspace, status_word
from _shared_cases import SharedCase, check_shared

pytestmark = pytest.mark.gpu


def shape(h=16, q=None, **kw):
    base = dict(name="tc", n_layers=1, n_kv_heads=h, n_q_heads=q or h, head_dim=128, n_loops=4, loop_group=2,
                chan_group=4, batch=1, context=0)
    base.update(kw)
    return Shape(**base)


H16 = shape()
CASES = {f"prefix_{p}": (H16, [(4, p)], [5, 1, 0, 33]) for p in
         (1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 511, 640)}
CASES.update({
    "own_lengths": (H16, [(9, 300)], [0, 1, 31, 32, 33, 255, 256, 257, 600]),
    "prefix_zero": (H16, [(2, 0), (6, 64)], [100, 3, 7, 0, 1, 2, 90, 64]),
    "ends_inside_a_page": (H16, [(5, 777), (3, 100)], [200, 55, 3, 28, 29, 0, 92, 28]),
    "sixteen_rows": (shape(4), [(16, 260)], [i * 7 % 60 for i in range(16)]),
    "seventeen_rows": (shape(4), [(17, 260)], [i * 7 % 60 for i in range(17)]),
    "thirty_three_rows": (shape(2), [(33, 900)], [i * 5 % 40 for i in range(33)]),
    "sixty_four_rows": (shape(1), [(64, 300)], [i * 5 % 40 for i in range(64)]),
    "sixty_five_rows": (shape(1), [(65, 700), (1, 400)], [i * 5 % 40 for i in range(66)]),
    "two_hundred_rows": (shape(1), [(200, 150)], [i % 4 for i in range(200)]),
    "shorter_than_the_prefix": (H16, [(5, 600)], [10, -100, -599, -600, 3]),
    "first_is_shorter": (H16, [(4, 300)], [-290, 10, 0, 5]),
    "windows_only": (H16, [(6, 300)], [10, 5.0, 1.0, 72.0, None, 0]),
    "behind_the_groups": (H16, [(6, 200)], [30, 4, 2, 1, 0, 9, 150, 90]),
    "gqa3": (shape(8, 24), [(7, 400), (3, 90)], [i * 11 % 70 for i in range(10)]),
    "gqa3_wide": (shape(2, 6), [(30, 300)], [i * 3 % 20 for i in range(30)]),
    "one_sequence_many_heads": (shape(8, 64), [(1, 500)], [40]),
    "d64": (shape(16, head_dim=64), [(5, 600), (3, 33)], [40, 0, 77, 3, 150, 9, 31, 5]),
    "d96_c8": (shape(16, head_dim=96, chan_group=8, page_tokens=96), [(5, 600), (3, 47)], [40, 0, 77, 3, 150, 9, 31, 2]),
    "d96_c8_wide": (shape(2, head_dim=96, chan_group=8, page_tokens=96), [(40, 500)], [i % 50 for i in range(40)]),
    "d96_c4": (shape(16, page_tokens=96, head_dim=96), [(5, 250)], [40, 0, 77, 1, 2]),
    "d128_c8": (shape(16, chan_group=8), [(5, 250)], [40, 0, 77, 1, 2]),
    "page32": (shape(page_tokens=32), [(4, 250)], [40, 0, 77, 5]),
    "page256": (shape(page_tokens=256), [(4, 700)], [40, 0, 300, 5]),
    "long": (H16, [(5, 9000)], [500, 20, 700, 3, 1]),
    "no_window": (shape(prefix=0, recent=0), [(4, 300)], [40, 0, 1, 130]),
    "many_groups": (shape(4, head_dim=64), [(3 + i % 4, 10 + 37 * i) for i in range(14)],
                    [(i * 13) % 90 for i in range(sum(3 + i % 4 for i in range(14)))]),
    "forty_groups_of_heads": (shape(8, head_dim=64), [(4, 20 + 9 * i) for i in range(40)], [(i * 7) % 30 for i in range(160)]),
    "three_hundred_groups": (shape(1, head_dim=64), [(5 if i % 50 else 0, 5 + i % 60) for i in range(300)],
                             [(i * 7) % 9 for i in range(5 * 294)]),
})


@pytest.mark.parametrize("name", list(CASES))
def test_tensor_core_form_matches_the_oracle(name):
    s, groups, own = CASES[name]
    c = SharedCase(s, groups, own, seed=len(name))
    assert c.B * s.n_q_heads >= 64 and c.B * s.n_q_heads / s.n_kv_heads >= 4 * len(groups)
    out, lse = c.run_gpu()
    pairs = None if c.B * s.n_q_heads <= 130 else sample_pairs(c.B, s.n_q_heads, 90, 1, whole=(0, c.B - 1))
    check_shared(c, out, lse, pairs)


@pytest.mark.parametrize("q_scale", [30.0, 1e-3, 0.0])
def test_large_and_small_scores(q_scale):
    c = SharedCase(H16, [(4, 700)], [40, 2, 100, 0], q_scale=q_scale, seed=5)
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("sm_scale,q_scale", [(1e-38, 1.0), (1e-20, 1e-30), (2.0 ** -20, 1e-30), (2.0 ** 20, 1e-7),
                                              (1e25, 1e-26)])
def test_scales_far_from_one(sm_scale, q_scale):
    # one sequence's queries are zero: all of its tokens weigh the same
    c = SharedCase(H16, [(4, 300)], [40, 2, 100, 0], q_scale=q_scale, seed=15)
    c.sm_scale = sm_scale
    c.q[2] = 0
    check_shared(c, *c.run_gpu())


def test_own_tokens_of_many_pairs():
    # chunks of 512 tokens: 32 sequences of 16 heads, ends on either side of them
    own = [0, 1, 255, 256, 257, 511, 512, 513, 700, 1023, 1024, 1025] + [i * 29 % 600 for i in range(20)]
    c = SharedCase(H16, [(20, 300), (10, 90)], own, seed=21)
    check_shared(c, *c.run_gpu(), pairs=sample_pairs(c.B, 16, 60, 5, whole=(7,)))


def test_own_tokens_of_more_than_sixty_four_chunks():
    c = SharedCase(H16, [(4, 300)], [17000, 16640, 100, 0], seed=22)
    check_shared(c, *c.run_gpu(), pairs=sample_pairs(c.B, 16, 24, 6))


@pytest.mark.parametrize("k_scale,v_scale", [(1e-6, 1e5), (3e4, 1e-7)])
def test_codebooks_far_from_one(k_scale, v_scale):
    c = SharedCase(H16, [(4, 300)], [40, 2, 100, 0], q_scale=1e-4 if k_scale > 1 else 1.0, seed=6)
    c.cb[:, :, :, 0] *= k_scale
    c.cb[:, :, :, 1] *= v_scale
    c.win[0] = (c.win[0].float() * k_scale).to(torch.bfloat16)
    c.win[1] = (c.win[1].float() * v_scale).to(torch.bfloat16)
    check_shared(c, *c.run_gpu())


def test_groups_of_channels_of_different_size():
    # one channel group 2^12 times the others, in keys and in values
    c = SharedCase(H16, [(5, 300)], [40, 2, 100, 0, 7], seed=16)
    c.cb[:, :, :, 0, :, 3] *= 4096
    c.cb[:, :, :, 1, :, 9] *= 4096
    c.q[..., 12:16] /= 4096
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("k_scale", [1e-6, 1e-8, 1e-20])
@pytest.mark.parametrize("dead", [[3], [0, 5, 31], list(range(1, 32))])
def test_groups_of_channels_without_any_value(dead, k_scale):
    # key (and value) codewords of some channel groups are all zero, the others small,
    # with queries as large as the small ones ask for: scores of order one
    c = SharedCase(H16, [(4, 300)], [40, 2, 100, 0], q_scale=1.0 / k_scale, seed=26)
    c.cb[:, :, :, 0] *= k_scale
    c.cb[:, :, :, :, :, dead] = 0.0
    c.win[0] = (c.win[0].float() * k_scale).to(torch.bfloat16)
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("k_scale,v_scale", [(1e36, 1.0), (2e38, 1e36), (1e-36, 1e-30)])
def test_codebooks_at_the_ends_of_float32(k_scale, v_scale):
    c = SharedCase(H16, [(4, 300)], [40, 2, 100, 0], q_scale=min(1.0 / k_scale, 1e36), seed=27)
    c.cb.clamp_(-1, 1)
    c.cb[:, :, :, 0] *= k_scale
    c.cb[:, :, :, 1] *= v_scale
    c.win = [(w.float().clamp(-1, 1) * f).to(torch.bfloat16) for w, f in zip(c.win, (k_scale, v_scale))]
    check_shared(c, *c.run_gpu())


def _rows_of(c, code):
    """Gives every token of the shared prefix key code `code[token]` in all groups."""
    for h in range(c.shape.n_kv_heads):
        for b in range(c.B):
            n = min(len(code), c.n_vq[b])
            O.pack_sequence(c.pool[0, h, c.gamma], code[:n, None].repeat(c.shape.J, 1), c.bt[b], c.shape.page_tokens, 0)


@pytest.mark.parametrize("rise", [1.0, -1.0])
@pytest.mark.parametrize("rows,h", [(4, 16), (20, 4), (40, 2)])
def test_rising_and_falling_scores(rise, rows, h):
    # scores that outgrow the reference tile after tile, and ones that fall away
    # below fp16's range of the first tile's
    c = SharedCase(shape(h), [(rows, 2000)], [20, 3, 64, 0] + [5] * (rows - 4), seed=8)
    c.cb[:, :, :, 0] = torch.linspace(-1, 1, 256)[:, None] * 3.0 * rise
    c.q = c.q.abs()
    _rows_of(c, (np.arange(2000) * 255 // 1999).astype(np.uint8))
    check_shared(c, *c.run_gpu(), pairs=sample_pairs(c.B, h, 24, 3))


def test_one_row_far_above_the_others():
    # rows of one group whose scores differ by orders of magnitude: each keeps its
    # own reference
    c = SharedCase(H16, [(6, 900)], [20, 3, 64, 0, 1, 2], seed=18)
    c.q[0] *= 20
    c.q[1] *= 1e-3
    c.q[2] = 0
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("size", [1e9, 1e12, 3e38])
@pytest.mark.parametrize("rows,h,kw", [(6, 16, {}), (20, 4, {}), (40, 2, {}), (6, 16, dict(head_dim=96, chan_group=8, page_tokens=96))])
def test_a_row_does_not_depend_on_its_neighbours_magnitude(rows, h, kw, size):
    # neighbours in one group: an empty sequence whose query was never written, a
    # sequence of windows only and one with tokens, all of a huge finite size
    c = SharedCase(shape(h, **kw), [(rows, 300)], [20, None, 64, 5.0] + [1, 2] * (rows // 2 - 2), seed=17)
    clean, lse = c.run_gpu()
    check_shared(c, clean, lse, pairs=sample_pairs(c.B, h, 20, 2, whole=(0, 1)))
    g = torch.Generator().manual_seed(3)
    for b in (1, 3, 4):
        c.q[b] = (size * (0.5 + 0.5 * torch.rand(c.q[b].shape, generator=g))).to(torch.bfloat16)
    out, lse2 = c.run_gpu()
    keep = [b for b in range(c.B) if b not in (3, 4)]
    np.testing.assert_array_equal(out[keep], clean[keep])
    np.testing.assert_array_equal(lse2[keep], lse[keep])


def test_infinite_and_nan_queries_spoil_their_own_rows_only():
    c = SharedCase(H16, [(6, 300)], [20, 3, 64, 0, 1, 2], seed=19)
    clean, lse = c.run_gpu()
    c.q[1, 3, 5] = float("nan")
    c.q[2, 4, 6] = float("inf")
    out, _ = c.run_gpu()
    assert np.all(np.isnan(out[1, 3]))
    same = np.ones(out.shape[:2], bool)
    same[1, 3] = same[2, 4] = False
    # (the tile's common power-of-two scale leaves out what is not finite)
    check_shared(c, out, lse, pairs=[(b, h) for b in range(6) for h in range(16) if same[b, h]])
    assert not np.all(np.isfinite(out[2, 4]))


def test_nan_in_unused_window_slots():
    c = SharedCase(H16, [(5, 300)], [20, 3.0, 64, 0, None], seed=20)
    c.win[0][1, :, 3:] = float("nan")
    c.win[1][1, :, 3:] = float("inf")
    c.win[0][4] = float("nan")
    check_shared(c, *c.run_gpu())


def test_bad_pages_are_skipped_and_flagged():
    c = SharedCase(H16, [(4, 300)], [100, 40, 0, 7], seed=3, copy_pages=False)
    flag = B.LOOPVQ_DECODE_STATUS_BAD_PAGE
    d = c.device()
    d["block_table"][:, 1] = c.n_pages                     # shared tokens 64 .. 127
    d["block_table"][0, 6] = -3                            # sequence 0's own tokens 384 .. 399
    out, lse = c.run_gpu(status=flag, dev_inputs=d)
    # the oracle without those tokens: sequence 0 alone (its table is the group's)
    for h in range(16):
        q = c.q[0, h].double().numpy()
        parts = [(c.win[0][0, h].double().numpy(), c.win[1][0, h].double().numpy())]
        idx = [O.unpack_sequence(c.pool[0, h, c.gamma], 400, 32, c.bt[0], 64, kv) for kv in range(2)]
        keep = np.r_[0:64, 128:384]
        parts.append(tuple(O.dequant_ref(idx[kv][keep], c.cb[0, h, c.gamma, kv].double().numpy(), c.tau) for kv in range(2)))
        ref, lref = O.attn_ref(q, np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]), c.sm_scale)
        assert np.max(np.abs(out[0, h] - ref)) <= 2e-2
        assert abs(lse[0, h] - lref) <= 2e-2
    d["block_table"].fill_(-1)
    out, lse = c.run_gpu(status=flag, dev_inputs=d)
    c.n_vq = [0] * 4
    check_shared(c, out, lse)


def test_values_past_the_bounds_are_clipped_and_flagged():
    flag = B.LOOPVQ_DECODE_STATUS_BAD_GROUP
    c = SharedCase(H16, [(4, 500)], [130, 4, 60, 1], seed=22)
    out, lse = c.run_gpu(status=flag, bounds=(4, 500, 60))
    c.n_vq[0] = 560
    check_shared(c, out, lse)
    c = SharedCase(H16, [(5, 500)], [60, 4, 60, 0, 60], seed=22)
    out, lse = c.run_gpu(status=flag, bounds=(4, 500, 60))
    c.n_vq[4] = 60                                         # shares nothing
    check_shared(c, out, lse)
    d = c.device()
    for starts in ([-3, 9], [5, 2], [7, 100]):
        d["group_starts"].copy_(torch.tensor(starts, dtype=torch.int32))
        out, lse = c.run_gpu(status=flag, dev_inputs=d)
        assert np.all(np.isfinite(out))
    d["group_starts"].copy_(torch.tensor([0, 5], dtype=torch.int32))
    d["shared_lens"].fill_(-4)
    out, lse = c.run_gpu(status=flag, dev_inputs=d, bounds=(5, 500, 60))
    c.n_vq = [60] * 5
    c.S = [0] * 5
    check_shared(c, out, lse)


def test_other_stream_replay_and_repeat():
    c = SharedCase(H16, [(5, 700)], [40, 0, 77, 3, 150], seed=21)
    most = c.max_own + 100
    out, lse = c.run_gpu(bounds=(5, 700, most))
    again, lse2 = c.run_gpu(bounds=(5, 700, most))
    np.testing.assert_array_equal(out, again)              # no order of atomics in the result
    np.testing.assert_array_equal(lse, lse2)
    d = c.device()
    cfg = c.config()
    o = torch.empty(c.B, 16, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(L.loopvq_decode_shared_workspace_bytes(cfg, c.B, 1, 5, 700, most), dtype=torch.uint8, device="cuda")
    call = lambda **kw: L.loopvq_decode_attn_shared(cfg, 0, c.t, **d, out=o, workspace=ws, max_group=5,
                                                    max_shared_len=700, max_own_len=most, sm_scale=c.sm_scale, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    np.testing.assert_array_equal(o.float().cpu().numpy(), out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()                                             # two calls in a row share the workspace
    for _ in range(3):
        o.fill_(float("nan"))
        ws[256:].fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(o.float().cpu().numpy(), out)
    d["seq_lens"].sub_(40)
    d["shared_lens"].sub_(100)
    g.replay()
    torch.cuda.synchronize()
    c.n_vq = [n - 40 for n in c.n_vq]
    c.seq_lens = [n - 40 for n in c.seq_lens]
    lse = np.array([[c.oracle(b, h)[1] for h in range(16)] for b in range(5)])
    check_shared(c, o.float().cpu().numpy(), lse)
    assert int(ws[:4].view(torch.int32)) == 0


def test_one_workspace_serves_calls_of_every_size_and_form():
    cases = [SharedCase(H16, [(40, 500)], [i * 17 % 600 for i in range(40)], seed=61),
             SharedCase(H16, [(4, 300)], [700, 0, 1, 2], seed=62), SharedCase(H16, [(2, 300)], [70, 0], seed=63),
             SharedCase(H16, [(9, 64), (3, 200)], [3] * 12, seed=64)]
    ws = torch.zeros(max(c.workspace_bytes() for c in cases), dtype=torch.uint8, device="cuda")
    want = [(c.run_gpu()[0], c.run_gpu(out_dtype=torch.float32)[0]) for c in cases]
    for i in (0, 1, 2, 3, 1, 0):
        c, d = cases[i], cases[i].device()
        for dtype, w in zip((torch.bfloat16, torch.float32), want[i]):
            o = torch.full((c.B, 16, 128), float("nan"), dtype=dtype, device="cuda")
            L.loopvq_decode_attn_shared(c.config(), 0, c.t, **d, out=o, workspace=ws, max_group=c.max_group,
                                        max_shared_len=c.max_shared, max_own_len=c.max_own, sm_scale=c.sm_scale)
            np.testing.assert_array_equal(o.float().cpu().numpy(), w)
    assert int(ws[:4].view(torch.int32)) == 0


def test_two_calls_at_once_with_workspaces_of_their_own():
    cases = [SharedCase(H16, [(5, 1500)], [40, 0, 77, 3, 150], seed=31), SharedCase(H16, [(6, 900)], [4, 0, 7, 3, 15, 90], seed=32)]
    want = [c.run_gpu()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ins = [c.device() for c in cases]
    outs = [torch.empty(c.B, 16, 128, dtype=torch.bfloat16, device="cuda") for c in cases]
    wss = [torch.zeros(c.workspace_bytes(), dtype=torch.uint8, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, d, o, w in zip(cases, streams, ins, outs, wss):
            L.loopvq_decode_attn_shared(c.config(), 0, c.t, **d, out=o, workspace=w, max_group=c.max_group,
                                        max_shared_len=c.max_shared, max_own_len=c.max_own, sm_scale=c.sm_scale, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        np.testing.assert_array_equal(o.float().cpu().numpy(), w)


@pytest.mark.parametrize("length", [-1, -2 ** 31])
def test_negative_lengths_are_empty_sequences(length):
    c = SharedCase(H16, [(5, 300)], [60, 4, 60, 0, 60], seed=24)
    d = c.device()
    for b in (0, 2):                                       # the first one's table still names the prefix
        d["seq_lens"][b] = length
        c.seq_lens[b] = c.n_vq[b] = 0
    check_shared(c, *c.run_gpu(dev_inputs=d))


def test_starts_at_the_ends_of_int32():
    # the first two sequences are the group that the bound leaves; nothing lies outside
    flag = B.LOOPVQ_DECODE_STATUS_BAD_GROUP
    c = SharedCase(H16, [(5, 500)], [60, 4, 60, 0, 60], seed=23)
    d = c.device()
    for starts in ([-2 ** 31, 5], [-2 ** 31, 2 ** 31 - 1], [0, 2 ** 31 - 1]):
        d["group_starts"].copy_(torch.tensor(starts, dtype=torch.int32))
        check_shared(c, *c.run_gpu(status=flag, dev_inputs=d, bounds=(2, 500, 560)))


@pytest.mark.parametrize("starts", [[0, -2 ** 31], [5, -2 ** 31], [2 ** 31 - 1, -2], [-2 ** 31, -1], [2 ** 31 - 1, 2 ** 31 - 1],
                                    [4, 2]])
def test_starts_that_leave_no_group(starts):
    # no sequence is in a group: each reads all of its tokens as its own
    c = SharedCase(H16, [(5, 500)], [60, 4, 60, 0, 60], seed=23)
    d = c.device()
    d["group_starts"].copy_(torch.tensor(starts, dtype=torch.int32))
    check_shared(c, *c.run_gpu(status=B.LOOPVQ_DECODE_STATUS_BAD_GROUP, dev_inputs=d, bounds=(5, 500, 560)))


def test_waits_that_run_out_are_reported_and_the_context_stays_usable():
    # the short-wait build gives no wait a try: the call ends with the flag set and
    # poisoned outputs, nothing in flight
    path = os.path.join(os.path.dirname(B.__file__), "libloopvq_shortwait.so")
    if not os.path.exists(path):
        pytest.fail(f"{path} not built")
    lib = B.load_library(path)
    c = SharedCase(H16, [(5, 700)], [40, 0, 77, 3, 150], seed=41)
    d = c.device()
    o = torch.empty(c.B, 16, 128, dtype=torch.bfloat16, device="cuda")
    ws = workspace(c.workspace_bytes())
    p = lambda k: d[k].data_ptr()
    st = lib.loopvq_decode_attn_shared(c.config().c_ref(), 0, c.t, c.B, 1, 5, 700, 150, p("q"), p("pool"), p("codebooks"),
                                       p("block_table"), p("seq_lens"), p("group_starts"), p("shared_lens"), p("win_k"),
                                       p("win_v"), c.sm_scale, 0, o.data_ptr(), None, ws.t.data_ptr(), c.workspace_bytes(), None)
    assert st == B.LOOPVQ_OK
    torch.cuda.synchronize()
    assert status_word(ws) == B.LOOPVQ_DECODE_STATUS_TIMEOUT
    assert bool(torch.isnan(o).all())
    check_shared(c, *c.run_gpu())


def test_a_decode_step_append_then_shared_attention():
    # the two calls as a step makes them: append one token per sequence, then attend;
    # against the oracle's windows and attention
    c = SharedCase(H16, [(5, 300)], [40, 0, 77, 3, 150], seed=51, loop_step=1)
    cfg = c.config()
    d = c.device()
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(5, 16, 128, generator=g).to(torch.bfloat16) for _ in range(3))
    ang = np.arange(1000)[:, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128)
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()
    q_out = torch.empty(5, 16, 128, dtype=torch.bfloat16, device="cuda")
    ev = torch.zeros(1, 2, 2, 2, 5, 16, 128, dtype=torch.bfloat16, device="cuda")
    # the sequences' lengths already count the new token; its window slot is about to
    # be replaced
    L.loopvq_append(cfg, 0, 1, q.cuda(), k.cuda(), v.cuda(), rope.cuda(), d["seq_lens"], d["win_k"], d["win_v"], q_out, ev)
    d["q"] = q_out
    out, lse = c.run_gpu(dev_inputs=d)
    c.q = q_out.cpu()
    c.win = [d["win_k"].cpu(), d["win_v"].cpu()]
    for b in range(5):
        slot = 8 + (c.seq_lens[b] - 1 - 8) % 64
        assert torch.equal(c.win[1][b, :, slot], v[b])
        want = O.rotate_ref(k[b].double().numpy(), rope[c.seq_lens[b] - 1, :64].double().numpy(),
                            rope[c.seq_lens[b] - 1, 64:].double().numpy(), False)
        got = c.win[0][b, :, slot].double().numpy()
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.max(np.abs(want)))
    check_shared(c, out, lse)


def test_a_page_table_of_more_than_two_to_the_31_tokens():
    # 2^23 entries a row for pages of 256: lengths are bounded by the table in 64 bits
    c = SharedCase(shape(page_tokens=256), [(4, 300)], [40, 2, 100, 0], seed=33)
    c.max_pages = 2 ** 23
    c.bt = np.concatenate([c.bt, np.zeros((4, c.max_pages - c.bt.shape[1]), np.int32)], 1)
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("bounds", [(4, 2 ** 30, 100), (4, 300, 2 ** 30), (4, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_bounds_as_loose_as_a_huge_page_table(bounds):
    # counts that the tensor-core form does not hold take the decode kernels
    c = SharedCase(shape(page_tokens=256), [(4, 300)], [40, 2, 100, 0], seed=33)
    c.max_pages = 2 ** 23
    c.bt = np.concatenate([c.bt, np.zeros((4, c.max_pages - c.bt.shape[1]), np.int32)], 1)
    check_shared(c, *c.run_gpu(bounds=bounds))


def _rounded_codebooks(c):
    """The case's codebooks as the tables hold them: per (head, K or V, channel group)
    scaled by the power of two that brings the largest entry into [2^13, 2^14), rounded
    to fp16, scaled back."""
    cb = c.cb.double().numpy()                             # [1][H][G][2][g][J][E][c]
    top = np.abs(cb).max(axis=(-1, -2), keepdims=True)
    ex = 13 - np.floor(np.log2(top))
    return torch.from_numpy((cb * 2.0 ** ex).astype(np.float16).astype(np.float64) * 2.0 ** -ex)


def check_rounding(case, out, lse, pairs):
    """bf16 outputs against the oracle over the rounded codebooks.

    With the codewords' rounding in the oracle what is left is small. A score is off by
    the additions alone: 128 of products of fp16 values (exact), each of which may drop
    a whole step (2^-23) of the sum, and a few scalings: d = S (128 + 12) 2^-23. A weight
    is off by a factor within e^(+-2d) of the softmax and by its own rounding to fp16
    (2^-11) against an unrounded sum; weights below fp16's normal range and the fast
    exponential are within 2^-15 together (see check_shared); the output's own
    rounding is 2^-8."""
    for b, h in pairs:
        ref, lref, A, S = case.oracle(b, h)
        dx = S * 140 * 2.0 ** -23
        e = A * (math.expm1(2 * dx) + 2.0 ** -11 + 2.0 ** -15)
        err = np.abs(out[b, h].astype(np.float64) - ref)
        assert np.all(err <= e + 2.0 ** -8 * (np.abs(ref) + e)), (b, h, float(np.max(err)))
        assert abs(float(lse[b, h]) - lref) <= dx + 2.0 ** -19 + 2.0 ** -23 * abs(lref), (b, h, float(lse[b, h]), lref)


@pytest.mark.parametrize("q_scale", [1.0, 30.0])
@pytest.mark.parametrize("kw,rows,own", [
    (dict(), 9, 300), (dict(h=8, q=24), 7, 70), (dict(head_dim=64), 8, 150),
    (dict(head_dim=96, chan_group=8, page_tokens=96), 8, 150), (dict(head_dim=96, page_tokens=96), 6, 90),
    (dict(chan_group=8), 6, 90), (dict(h=4), 30, 60), (dict(h=2), 70, 60)])
def test_outputs_are_what_the_documented_rounding_gives(kw, rows, own, q_scale):
    c = SharedCase(shape(**{"h": 16, **kw}), [(rows, 700)], [i * 37 % own for i in range(rows)], q_scale=q_scale, seed=40)
    out, lse = c.run_gpu()
    c.cb = _rounded_codebooks(c)
    check_rounding(c, out, lse, sample_pairs(c.B, c.shape.n_q_heads, 60, 4))


def _same_as_decode(c, out):
    """Whether bf16 outputs are loopvq_decode_attn's to the bit: the form of the decode
    kernels (the tensor-core form rounds otherwise somewhere)."""
    d, cfg, n = c.device(), c.config(), max(c.seq_lens)
    ref = torch.empty(c.B, c.shape.n_q_heads, c.shape.head_dim, dtype=torch.bfloat16, device="cuda")
    ws = workspace(L.loopvq_decode_workspace_bytes(cfg, c.B, n))
    L.loopvq_decode_attn(cfg, 0, c.t, d["q"], d["pool"], d["codebooks"], d["block_table"], d["seq_lens"], d["win_k"],
                         d["win_v"], ref, ws.t, n, sm_scale=c.sm_scale)
    return bool(np.array_equal(ref.float().cpu().numpy(), out))


DEEP = shape(40, head_dim=96, chan_group=8, page_tokens=96)
FORMS = {   # far from the tie on both sides
    "own_dominates": (H16, [(8, 512)], [8000, 100, 7000, 6000, 8000, 5000, 7900, 4000], True),
    "one_pair_in_a_batch_of_others": (H16, [(2, 4032)], [50, 9] + [4000, 3900, 4032, 3000], True),
    "forty_heads_of_a_group_of_four": (DEEP, [(4, 16032)], [60, 0, 50, 3], True),
    "nothing_shared": (H16, [(40, 0)], [i * 3 % 90 for i in range(40)], False),
    "nothing_shared_and_no_own": (H16, [(6, 0)], [0] * 6, False),
    "nothing_shared_in_two_groups": (H16, [(9, 0), (5, 0)], [i * 31 % 300 for i in range(15)], False),
    "long_prefix": (H16, [(8, 9024)], [500, 20, 600, 3, 1, 0, 44, 255], False),
    "long_prefix_and_many_chunks": (H16, [(16, 60032)], [17000, 16640, 16500, 100, 0, 1] + [i * 37 % 500 for i in range(10)],
                                    False),
    "long_prefix_of_forty_heads": (DEEP, [(8, 6048)], [60, 0, 50, 3, 300, 299, 1, 2], False),
}


@pytest.mark.parametrize("name", list(FORMS))
def test_the_form_follows_shared_and_own_tokens(name):
    s, groups, own, decode = FORMS[name]
    # (whole pages are shared, so no page has to be copied)
    c = SharedCase(s, groups, own, seed=len(name), copy_pages=False)
    assert all(n % s.page_tokens == 0 for _, n in groups)
    out, lse = c.run_gpu()
    check_shared(c, out, lse, pairs=sample_pairs(c.B, s.n_q_heads, 20, 3))
    assert _same_as_decode(c, out) == decode
