"""GPU parity of loopvq_decode_attn_shared: every sequence of every group
against the float64 oracle (see check_shared for the bound), and against
loopvq_decode_attn on the same page tables."""

import numpy as np
import pytest
import torch

import sub_bit_vq_b200 as L
from sub_bit_vq_b200 import binding as B
from synthetic import Shape

from _guard import Guarded, status_word, workspace
from _shared_cases import SharedCase, check_shared

pytestmark = pytest.mark.gpu


def shape(**kw):
    base = dict(name="sh", n_layers=1, n_kv_heads=2, n_q_heads=2, head_dim=128, n_loops=4, loop_group=2,
                chan_group=4, batch=1, context=0)
    base.update(kw)
    return Shape(**base)


MHA = shape()
GQA = shape(n_q_heads=6)
D64 = shape(head_dim=64)
D96 = shape(head_dim=96, chan_group=8, page_tokens=96)
D96C4 = shape(head_dim=96, page_tokens=96)
D256 = shape(head_dim=256, chan_group=8)
PAGE32 = shape(page_tokens=32)
PAGE256 = shape(page_tokens=256)

CASES = {
    "one_group": (MHA, [(4, 300)], [40, 0, 1, 130]),
    "one_sequence": (MHA, [(1, 500)], [70]),
    "prefix_of_one": (MHA, [(3, 1)], [0, 1, 33]),
    "prefix_31": (MHA, [(3, 31)], [5, 1, 33]),
    "prefix_32": (MHA, [(3, 32)], [5, 32, 64]),
    "prefix_127_128_129": (MHA, [(2, 127), (2, 128), (2, 129)], [5, 1, 0, 0, 64, 63]),
    "prefix_zero": (MHA, [(2, 0), (2, 64)], [100, 3, 7, 0]),
    "ends_inside_a_page": (MHA, [(3, 777), (2, 100)], [200, 55, 3, 28, 29]),
    "seventeen": (MHA, [(17, 260)], [i * 7 % 60 for i in range(17)]),
    "thirty_three": (MHA, [(33, 200)], [i * 5 % 40 for i in range(33)]),
    "sixty_five": (MHA, [(65, 200), (1, 400)], [i * 5 % 40 for i in range(66)]),
    "one_thirty": (MHA, [(130, 150)], [i % 4 for i in range(130)]),
    "shorter_than_the_prefix": (MHA, [(5, 600)], [10, -100, -599, -600, 3]),
    "first_is_shorter": (MHA, [(3, 300)], [-290, 10, 0]),
    "windows_only": (MHA, [(6, 300)], [10, 5.0, 1.0, 72.0, None, 0]),
    "no_groups": (MHA, [], [100, 0, None, 500, 3.0]),
    "behind_the_groups": (MHA, [(2, 200)], [30, 4, 150, 90]),
    "gqa3": (GQA, [(7, 400), (3, 90)], [i * 11 % 70 for i in range(10)]),
    "gqa3_wide": (GQA, [(30, 300)], [i * 3 % 20 for i in range(30)]),
    "d64": (D64, [(5, 600), (2, 33)], [40, 0, 77, 3, 150, 9, 31]),
    "d96_c8": (D96, [(5, 600), (2, 47)], [40, 0, 77, 3, 150, 9, 31]),
    "d96_c4": (D96C4, [(3, 250)], [40, 0, 77]),
    "d256": (D256, [(3, 250)], [40, 0, 77]),
    "page32": (PAGE32, [(3, 250)], [40, 0, 77]),
    "page256": (PAGE256, [(3, 700)], [40, 0, 300]),
    "long": (MHA, [(3, 9000)], [500, 20, 700]),
    "many_groups": (D64, [(1 + i % 3, 10 + 37 * i) for i in range(14)], [(i * 13) % 90 for i in range(27)]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_shared_matches_the_oracle(name):
    s, groups, own = CASES[name]
    c = SharedCase(s, groups, own, seed=len(name))
    out, lse = c.run_gpu()
    check_shared(c, out, lse)


def test_sequences_before_the_first_group():
    c = SharedCase(MHA, [(2, 200)], [150, 30, 4], first=1)
    out, lse = c.run_gpu()
    check_shared(c, out, lse)


@pytest.mark.parametrize("loop_step", [0, 3])
def test_loop_steps(loop_step):
    c = SharedCase(MHA, [(3, 400)], [40, 2, 100], loop_step=loop_step, seed=4)
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("q_scale", [30.0, 1e-3, 0.0])
def test_large_and_small_scores(q_scale):
    c = SharedCase(MHA, [(3, 700)], [40, 2, 100], q_scale=q_scale, seed=5)
    check_shared(c, *c.run_gpu())


@pytest.mark.parametrize("k_scale,v_scale", [(1e-6, 1e5), (3e4, 1e-7)])
def test_codebooks_far_from_one(k_scale, v_scale):
    # keys and values outside fp16's range: the kernel scales them by powers of two
    c = SharedCase(MHA, [(3, 300)], [40, 2, 100], q_scale=1e-4 if k_scale > 1 else 1.0, seed=6)
    c.cb[:, :, :, 0] *= k_scale
    c.cb[:, :, :, 1] *= v_scale
    c.win[0] = (c.win[0].float() * k_scale).to(torch.bfloat16)
    c.win[1] = (c.win[1].float() * v_scale).to(torch.bfloat16)
    check_shared(c, *c.run_gpu())


def test_rising_scores():
    # each tile's keys outgrow the last one's, so the running reference has to rise
    c = SharedCase(MHA, [(4, 2000)], [20, 3, 64, 0], seed=8)
    code = torch.linspace(-1, 1, 256)
    c.cb[:, :, :, 0] = code[:, None] * 3.0
    c.q = c.q.abs()
    order = (np.arange(2000) * 255 // 1999).astype(np.uint8)[:, None].repeat(32, 1)
    from oracle import loopvq_oracle as O
    for h in range(2):
        for b in range(4):
            O.pack_sequence(c.pool[0, h, c.gamma], order, c.bt[b], 64, 0)
    check_shared(c, *c.run_gpu())


def test_equal_scores_give_the_mean():
    c = SharedCase(MHA, [(2, 640)], [0, 64], q_scale=0.0, seed=9)
    out, lse = c.run_gpu()
    check_shared(c, out, lse)
    np.testing.assert_allclose(lse[0], np.log(640 + 72), rtol=1e-6)


def test_float32_output_keeps_float32_precision():
    c = SharedCase(MHA, [(4, 300)], [40, 0, 1, 130], seed=2)
    out, lse = c.run_gpu(torch.float32)
    for b in range(c.B):
        for h in range(2):
            ref, lref, _, _ = c.oracle(b, h)
            assert np.max(np.abs(out[b, h] - ref)) <= 1e-4 * np.max(np.abs(ref))
            assert abs(lse[b, h] - lref) <= 1e-4


def test_agrees_with_decode_on_the_same_tables():
    c = SharedCase(GQA, [(9, 800), (2, 300)], [i * 17 % 90 for i in range(11)], seed=12)
    out, lse = c.run_gpu()
    d = c.device()
    cfg = c.config()
    ref = torch.empty(c.B, 6, 128, dtype=torch.float32, device="cuda")
    n = max(c.seq_lens)
    ws = workspace(L.loopvq_decode_workspace_bytes(cfg, c.B, n))
    L.loopvq_decode_attn(cfg, 0, c.t, d["q"], d["pool"], d["codebooks"], d["block_table"], d["seq_lens"],
                         d["win_k"], d["win_v"], ref, ws.t, n, sm_scale=c.sm_scale)
    assert np.max(np.abs(out - ref.cpu().numpy())) <= 2e-2


def test_bad_pages_are_skipped_and_flagged():
    # a shared page and an own page outside the pool: both are left out
    c = SharedCase(MHA, [(3, 300)], [100, 40, 0], seed=3, copy_pages=False)
    d = c.device()
    d["block_table"][:, 1] = c.n_pages                     # shared tokens 64 .. 127
    d["block_table"][0, 6] = -3                            # sequence 0's own tokens 384 .. 399
    out, _ = c.run_gpu(status=B.LOOPVQ_DECODE_STATUS_BAD_PAGE, dev_inputs=d)
    assert np.all(np.isfinite(out))
    # the same call with those tokens' scores pushed out of reach: keys of the
    # skipped pages cannot matter
    d2 = c.device()
    d2["block_table"][:, 1] = c.n_pages + 7
    d2["block_table"][0, 6] = c.n_pages
    out2, _ = c.run_gpu(status=B.LOOPVQ_DECODE_STATUS_BAD_PAGE, dev_inputs=d2)
    np.testing.assert_array_equal(out, out2)


def test_a_sequence_without_any_valid_page_uses_its_window():
    c = SharedCase(MHA, [(2, 128)], [0, 0], seed=3)
    d = c.device()
    d["block_table"].fill_(-1)
    out, lse = c.run_gpu(status=B.LOOPVQ_DECODE_STATUS_BAD_PAGE, dev_inputs=d)
    c.n_vq = [0, 0]
    check_shared(c, out, lse)


def test_other_stream_replay_and_repeat():
    c = SharedCase(MHA, [(5, 700)], [40, 0, 77, 3, 150], seed=21)
    out, lse = c.run_gpu(bounds=(c.max_group, c.max_shared, c.max_own + 100))
    d = c.device()
    cfg = c.config()
    o = torch.empty(c.B, 2, 128, dtype=torch.bfloat16, device="cuda")
    # (bounds that hold for the lengths of the first and of the last call)
    most = c.max_own + 100
    ws = torch.zeros(L.loopvq_decode_shared_workspace_bytes(cfg, c.B, 1, c.max_group, c.max_shared, most),
                     dtype=torch.uint8, device="cuda")
    call = lambda **kw: L.loopvq_decode_attn_shared(cfg, 0, c.t, **d, out=o, workspace=ws, max_group=c.max_group,
                                                    max_shared_len=c.max_shared, max_own_len=most,
                                                    sm_scale=c.sm_scale, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    np.testing.assert_array_equal(o.float().cpu().numpy(), out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        o.fill_(float("nan"))
        ws[256:].fill_(0xff)                               # nothing is kept in the workspace between calls
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(o.float().cpu().numpy(), out)
    # the graph reads the group and sequence lengths on the device
    d["seq_lens"].sub_(40)
    d["shared_lens"].sub_(100)
    g.replay()
    torch.cuda.synchronize()
    c2 = SharedCase(MHA, [(5, 700)], [40, 0, 77, 3, 150], seed=21)
    c2.n_vq = [n - 40 for n in c.n_vq]
    c2.seq_lens = [n - 40 for n in c.seq_lens]
    c2.groups, c2.S = [(5, 600)], [600] * 5
    lse2 = np.array([[c2.oracle(b, h)[1] for h in range(2)] for b in range(5)])
    check_shared(c2, o.float().cpu().numpy(), lse2)
    assert int(ws[:4].view(torch.int32)) == 0
