"""Host-side tests of loopvq_decode_attn_shared: refusals before any launch,
workspace sizes, the binding's checks."""

import ctypes
import dataclasses
import os
import random
import re
import subprocess

import pytest
import torch

import sub_bit_vq_b200 as L
from sub_bit_vq_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = B.LOOPVQ_ERR_INVALID_ARG


def _cfg(**kw):
    base = dict(n_layers=2, n_kv_heads=3, n_q_heads=6, head_dim=128, n_loops=8, loop_group=4,
                chan_group=4, n_pages=10, max_batch=4, max_pages_per_seq=5)
    base.update(kw)
    return L.LoopVQConfig(**base)


def _raw(cfg=None, **over):
    cfg = cfg or _cfg()
    a = dict(layer=0, loop=0, batch=4, ng=2, mg=3, ms=200, mo=100, q=0x1000, pool=0x2000, cb=0x3000, bt=0x4000,
             sl=0x5000, gs=0x5100, sh=0x5200, wk=0x6000, wv=0x7000, scale=0.1, odt=0, out=0x8000, lse=None,
             ws=0x9000, nbytes=1 << 40)
    a.update(over)
    return B.library().loopvq_decode_attn_shared(cfg.c_ref(), *a.values(), None)


@pytest.mark.parametrize("over", [
    dict(layer=2), dict(loop=8), dict(batch=0), dict(batch=5), dict(ng=-1), dict(ng=5), dict(mg=0), dict(mg=5),
    dict(mg=-1), dict(ms=-1), dict(ms=5 * 64 + 1), dict(mo=-1), dict(mo=5 * 64 + 1), dict(q=None), dict(pool=None),
    dict(cb=None), dict(bt=None), dict(sl=None), dict(gs=None), dict(sh=None), dict(wk=None), dict(wv=None),
    dict(scale=0.0), dict(scale=float("nan")), dict(odt=2), dict(out=None), dict(ws=None), dict(q=0x1008),
    dict(pool=0x2004), dict(cb=0x3004), dict(bt=0x4002), dict(sl=0x5002), dict(gs=0x5101), dict(sh=0x5202),
    dict(wk=0x6008), dict(wv=0x7002), dict(out=0x8004), dict(lse=0xA002), dict(ws=0x9008),
])
def test_rejects_before_launch(over):
    assert _raw(**over) == E


def test_workspace_is_checked_and_grows():
    cfg = _cfg()
    need = L.loopvq_decode_shared_workspace_bytes(cfg, 4, 2, 3, 200, 100)
    assert need > 256
    assert _raw(nbytes=need - 1) == B.LOOPVQ_ERR_WORKSPACE
    assert L.loopvq_decode_shared_workspace_bytes(cfg, 0, 0, 0, 0, 0) == 0
    assert L.loopvq_decode_shared_workspace_bytes(cfg, 4, 2, 3, 5 * 64 + 1, 0) == 0
    assert L.loopvq_decode_shared_workspace_bytes(cfg, 2, 1, 2, 200, 100) <= need
    assert L.loopvq_decode_shared_workspace_bytes(cfg, 2, 0, 0, 0, 100) > 0


def test_a_workspace_of_the_largest_call_serves_smaller_ones():
    cfg = _cfg(n_kv_heads=8, n_q_heads=16, n_pages=2000, max_batch=80, max_pages_per_seq=1500)
    size = lambda *a: L.loopvq_decode_shared_workspace_bytes(cfg, *a)
    r = random.Random(3)
    for _ in range(300):
        b, ms, mo = r.randint(1, 80), r.randint(0, 60000), r.choice([0, 255, 513, 16385, r.randint(1, 90000)])
        ng = r.randint(0, b)
        mg = r.randint(1, b)
        b2 = r.randint(1, b)
        less = (b2, r.randint(0, min(ng, b2)), r.randint(1, min(mg, b2)), r.randint(0, ms), r.randint(0, mo))
        assert 0 < size(*less) <= size(b, ng, mg, ms, mo), (less, (b, ng, mg, ms, mo))


def test_binding_checks_shapes_types_and_device():
    cfg = _cfg()
    bf, i32 = torch.bfloat16, torch.int32

    def call(**over):
        a = dict(q=torch.zeros(4, 6, 128, dtype=bf), pool=torch.zeros(16, dtype=torch.uint8),
                 codebooks=torch.zeros(16), block_table=torch.zeros(4, 5, dtype=i32),
                 seq_lens=torch.zeros(4, dtype=i32), group_starts=torch.zeros(3, dtype=i32),
                 shared_lens=torch.zeros(2, dtype=i32), win_k=torch.zeros(4, 3, 72, 128, dtype=bf),
                 win_v=torch.zeros(4, 3, 72, 128, dtype=bf), out=torch.zeros(4, 6, 128, dtype=bf),
                 workspace=torch.zeros(64, dtype=torch.uint8), max_group=3, max_shared_len=200, max_own_len=100)
        a.update(over)
        L.loopvq_decode_attn_shared(cfg, 0, 0, **a)

    with pytest.raises(ValueError, match="CUDA device"):
        call()
    for over in (dict(out=torch.zeros(4, 6, 128, dtype=torch.float16)), dict(pool=torch.zeros(16)),
                 dict(codebooks=torch.zeros(16, dtype=bf))):
        with pytest.raises(TypeError):
            call(**over)
    for over in (dict(q=torch.zeros(4, 6, 64, dtype=bf)), dict(q=torch.zeros(4, 6, 128)),
                 dict(block_table=torch.zeros(4, 4, dtype=i32)), dict(seq_lens=torch.zeros(3, dtype=i32)),
                 dict(group_starts=torch.zeros(2, dtype=i32)), dict(shared_lens=torch.zeros(2, dtype=torch.int64)),
                 dict(win_k=torch.zeros(4, 3, 64, 128, dtype=bf)), dict(win_v=torch.zeros(3, 3, 72, 128, dtype=bf)),
                 dict(out=torch.zeros(4, 6, 256, dtype=bf)[:, :, ::2]), dict(lse=torch.zeros(4, 5))):
        with pytest.raises(ValueError):
            call(**over)


def test_binding_checks_pool_codebooks_and_workspace(monkeypatch):
    # sizes and density, before the call (the library, which would launch, is replaced)
    cfg = _cfg()
    lay = L.loopvq_cache_layout(cfg)
    bf, i32 = torch.bfloat16, torch.int32
    pool, cb = torch.zeros(lay["pool_bytes"], dtype=torch.uint8), torch.zeros(lay["codebook_bytes"] // 4)
    called = []

    class Lib:
        @staticmethod
        def loopvq_decode_attn_shared(*a):
            called.append(a)
            return 0

    monkeypatch.setattr(B, "_on_current_device", lambda *a: None)
    monkeypatch.setattr(B, "_lib", Lib)

    def call(**over):
        a = dict(q=torch.zeros(4, 6, 128, dtype=bf), pool=pool, codebooks=cb, block_table=torch.zeros(4, 5, dtype=i32),
                 seq_lens=torch.zeros(4, dtype=i32), group_starts=torch.zeros(3, dtype=i32),
                 shared_lens=torch.zeros(2, dtype=i32), win_k=torch.zeros(4, 3, 72, 128, dtype=bf),
                 win_v=torch.zeros(4, 3, 72, 128, dtype=bf), out=torch.zeros(4, 6, 128, dtype=bf),
                 workspace=torch.zeros(64, dtype=torch.uint8), max_group=3, max_shared_len=200, max_own_len=100, stream=0)
        a.update(over)
        L.loopvq_decode_attn_shared(dataclasses.replace(cfg), 0, 0, **a)

    monkeypatch.setattr(B, "loopvq_cache_layout", lambda c: lay)
    call()
    assert len(called) == 1
    for over in (dict(pool=pool[:-1]), dict(codebooks=cb[1:]), dict(pool=torch.zeros(2 * pool.numel(), dtype=torch.uint8)[::2]),
                 dict(codebooks=cb.view(2, -1).t()), dict(workspace=torch.zeros(128, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError, match="dense"):
            call(**over)
    assert len(called) == 1
    call(pool=torch.zeros(1 + pool.numel(), dtype=torch.uint8))
    assert len(called) == 2


def test_status_bit_matches_the_header():
    text = open(os.path.join(ROOT, "include", "loopvq.h")).read()
    m = re.search(r"LOOPVQ_DECODE_STATUS_BAD_GROUP\s*=\s*(\d+)", text)
    assert int(m.group(1)) == B.LOOPVQ_DECODE_STATUS_BAD_GROUP == L.LOOPVQ_DECODE_STATUS_BAD_GROUP


def test_a_group_is_a_part_of_the_batch_whatever_its_starts(tmp_path):
    # the kernels' own arithmetic, compiled for the host: ends at and around the limits
    # of int32 must not wrap into a group outside [0, batch)
    src = tmp_path / "span.cpp"
    src.write_text('#include "group_span.h"\n'
                   'extern "C" void span(int s, int e, int b, int m, int* o) {\n'
                   '  const loopvq::GroupSpan g = loopvq::group_span(s, e, b, m);\n  o[0] = g.lo; o[1] = g.n;\n}\n')
    so = tmp_path / "span.so"
    subprocess.run(["g++", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", os.path.join(ROOT, "sub_bit_vq_b200", "csrc"),
                    str(src), "-o", str(so)], check=True)
    span = ctypes.CDLL(str(so)).span
    ends = [-2 ** 31, -2 ** 31 + 1, -2 ** 30, -3, -1, 0, 1, 2, 4, 5, 6, 7, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1]
    out = (ctypes.c_int * 2)()
    for batch in (1, 5, 2 ** 30):
        for most in (1, 2, 5, batch):
            for s in ends:
                for e in ends:
                    span(s, e, batch, most, out)
                    lo, n = out
                    want = range(max(s, 0), max(max(s, 0), min(e, batch)))[:most]
                    assert 0 <= lo and 0 <= n <= most and lo + n <= batch, (s, e, batch, most, lo, n)
                    assert range(lo, lo + n) == want, (s, e, batch, most, lo, n)   # (empty ranges are equal)


def test_the_longest_lengths_are_counted_in_pages_without_wrapping():
    # 2^31 - 1 tokens and pages of 256: rounding up to pages must not wrap and pass
    # for a short sequence
    cfg = _cfg(page_tokens=256, prefix_tokens=0, recent_tokens=0)
    st = B.library().loopvq_decode_attn(cfg.c_ref(), 0, 0, 4, 2 ** 31 - 1, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, None, None,
                                        0.1, 0, 0x8000, None, 0x9000, 1 << 40, None)
    assert st == E
