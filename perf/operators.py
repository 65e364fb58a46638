"""Cases of the cache-append and shared-prefix decode operators.

Each case is one call pattern of a serving program over the vector-quantised
cache of a looped transformer, with a plain form in elementary torch operations
(``own = False``) and the framework's calls (``own = True``).

append   one decode or verification step of (layer, loop step) that is then
         rolled back (the draft tokens were rejected), so that a pass leaves
         the windows as it found them; or a whole prompt appended at once.
shared   decode attention of a batch whose sequences share quantised prefixes.
"""

import math
import random

import torch

own = False

E, P, R = 256, 8, 64                      # centroids, bf16 prefix and recent tokens
LOOPS = 4                                 # loop steps per loop group, all cases
MODELS = {                                # heads, channels and pages of one layer
    "tiny": dict(hq=1, hkv=1, d=64, c=4, page=64),
    "ouro14": dict(hq=16, hkv=16, d=128, c=4, page=64),
    "gqa2": dict(hq=16, hkv=8, d=128, c=4, page=64),
    "deep025": dict(hq=40, hkv=40, d=96, c=8, page=96),
}


def listed():
    return [
        # one decode step of 8 sequences at 32K context: the call made for every layer and loop step
        dict(name="append_step_b8", op="append", mode="step", model="ouro14", batch=8, spec=1, context=32768,
             rot=128, interleaved=False, shape=1),
        # the largest decode batch of the benchmark's sweep
        dict(name="append_step_b256", op="append", mode="step", model="ouro14", batch=256, spec=1, context=16384,
             rot=128, interleaved=False, shape=2),
        # verification of up to 5 draft tokens per sequence, ragged, d = 96 with half of it rotated in neighbouring pairs
        dict(name="append_draft_deep", op="append", mode="step", model="deep025", batch=32, spec=5, context=16384,
             rot=48, interleaved=True, shape=3),
        # five ragged prompts packed into one call, grouped query heads
        dict(name="append_prompts_gqa", op="append", mode="prompt", model="gqa2", batch=5, spec=0, context=4001,
             rot=128, interleaved=False, shape=4),
        # one prompt of 32768 tokens
        dict(name="append_prompt_32k", op="append", mode="prompt", model="ouro14", batch=1, spec=0, context=32768,
             rot=128, interleaved=False, shape=5),
        # two samples of a short prompt on the smallest shape
        dict(name="shared_tiny_b2", op="shared", model="tiny", groups=1, batch=2, prefix=440, own=40, shape=6),
        # 8 samples of one 32K document, early in their answers
        dict(name="shared_b8_32k", op="shared", model="ouro14", groups=1, batch=8, prefix=32696, own=200, shape=7),
        # 16 users behind an 8K system prompt
        dict(name="shared_b16_8k", op="shared", model="ouro14", groups=1, batch=16, prefix=8120, own=1000, shape=8),
        # seven ragged prompts with ragged numbers of samples, grouped query heads, prefixes that end inside a page
        dict(name="shared_ragged_gqa", op="shared", model="gqa2", groups=7, batch=61, prefix=9001, own=333, shape=9),
        # the 0.25 bit shape: 32 samples of one 16K prompt, 40 heads of 96 channels
        dict(name="shared_deep_b32", op="shared", model="deep025", groups=1, batch=32, prefix=16312, own=300, shape=10),
        # the sweep's largest batch: 256 samples of one 16K prompt
        dict(name="shared_b256_16k", op="shared", model="ouro14", groups=1, batch=256, prefix=16312, own=500, shape=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    shape = rng.randrange(100, 1 << 30)
    model = rng.choice(["ouro14", "gqa2", "deep025", "ouro14", "tiny"])
    d = MODELS[model]["d"]
    kind = rng.choice(["step", "prompt", "shared", "shared"])
    if kind == "step":
        return dict(op="append", mode="step", model=model, batch=_log(rng, 1, 256), spec=rng.choice([1, 1, 2, 5, 8]),
                    context=_log(rng, 300, 32768), rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.3, shape=shape)
    if kind == "prompt":
        batch = rng.randint(1, 8)
        most = 32768 if model != "deep025" else 12000
        return dict(op="append", mode="prompt", model=model, batch=batch, spec=0, context=_log(rng, 65, most) // batch + 1,
                    rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.3, shape=shape)
    groups = rng.choice([1, 1, 2, 3, 6])
    batch = max(groups, _log(rng, 2, 128))
    return dict(op="shared", model=model, groups=groups, batch=batch, prefix=_log(rng, 64, 16384 // (1 + groups // 3)),
                own=_log(rng, 1, 600), shape=shape)


# ---- sizes of a case (from the case alone) -----------------------------------------


def _append_lens(case):
    """Rows appended to each sequence and its length counting them."""
    r = random.Random(case["shape"])
    n, total = [], []
    for _ in range(case["batch"]):
        if case["mode"] == "step":
            n.append(case["spec"] if case["spec"] == 1 else r.randint(1, case["spec"]))
            total.append(r.randint(max(280, case["context"] // 2), max(290, case["context"])))
        else:
            n.append(r.randint(max(1, case["context"] // 3), case["context"]) if case["batch"] > 1 else case["context"])
            total.append(n[-1])
    return n, total


def _shared_lens(case):
    """Group sizes, shared quantised tokens of each group, own quantised tokens of each sequence."""
    r = random.Random(case["shape"])
    g, b = case["groups"], case["batch"]
    cuts = sorted(r.sample(range(1, b), g - 1)) if g > 1 else []
    sizes = [y - x for x, y in zip([0] + cuts, cuts + [b])]
    shared = [case["prefix"] if i == 0 else r.randint(max(1, case["prefix"] // 4), case["prefix"]) for i in range(g)]
    owned = [r.randint(case["own"] // 2, case["own"]) for _ in range(b)]
    return sizes, shared, owned


def work(case):
    m = MODELS[case["model"]]
    hq, hkv, d = m["hq"], m["hkv"], m["d"]
    if case["op"] == "append":
        n, total = _append_lens(case)
        rows = sum(n)
        new_q = rows * hq * d * 2 * 2                                   # q in, q_out out
        new_kv = rows * hkv * d * 2 * 2                                 # k and v in
        if case["mode"] == "step":                                      # append, then the rollback of the same rows
            moved = rows * hkv * d * 2 * 2 * 3                          # window rows out and in, evicted rows out
            nbytes = new_q + new_kv + moved + rows * (4 * case["rot"] + 8) + new_kv + moved
        else:
            kept = sum(min(x, P + R) for x in n)
            gone = sum(max(0, x - P - R) for x in n)
            nbytes = new_q + new_kv + (kept + gone) * hkv * d * 2 * 2 + rows * (4 * case["rot"] + 8)
        return {"bytes": nbytes, "flops": 3 * rows * (hq + hkv) * case["rot"]}
    sizes, shared, owned = _shared_lens(case)
    J = d // m["c"]
    b = case["batch"]
    idx = 2 * J * hkv * (sum(shared) + sum(owned))
    nbytes = idx + 2 * b * hkv * (P + R) * d * 2 + 2 * E * d * 4 * hkv + 2 * b * hq * d * 2
    tokens = sum(s * x for s, x in zip(sizes, shared)) + sum(owned) + b * (P + R)
    return {"bytes": nbytes, "flops": 4 * d * hq * tokens}


# ---- inputs -----------------------------------------------------------------------


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    m = MODELS[case["model"]]
    hq, hkv, d, c, page = m["hq"], m["hkv"], m["d"], m["c"], m["page"]
    J = d // c

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    st = dict(case=case, hq=hq, hkv=hkv, d=d, c=c, J=J, page=page, LB=32 // J * J,
              GR=16 if J % 16 == 0 else 8 if J % 8 == 0 else 4, dev=dev, keep={})
    if case["op"] == "append":
        n, total = _append_lens(case)
        rows, b = sum(n), case["batch"]
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        pages = -(-max(max(total) - P - R, 1) // page)
        st.update(rows=rows, batch=b, rot=case["rot"], n_pages=b * pages, pages=pages, seq_lens=ints(total),
                  token_starts=None if case["spec"] == 1 and case["mode"] == "step" else ints(starts),
                  starts=ints(starts, torch.int64))
        qkv = normal(rows, (hq + 2 * hkv) * d)                          # the fused projection's output
        st["q"] = qkv[:, :hq * d].view(rows, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
        st["v"] = qkv[:, (hq + hkv) * d:].view(rows, hkv, d)
        inv = 10000.0 ** (-torch.arange(0, st["rot"], 2, dtype=torch.float64, device=dev) / st["rot"])
        ang = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * inv
        st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()       # [positions][cos.., sin..]
        st["win_k"], st["win_v"] = normal(b, hkv, P + R, d), normal(b, hkv, P + R, d)
        st["block_table"] = torch.randperm(b * pages, generator=g, device=dev).to(torch.int32).view(b, pages)
        st["q_out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev)
        st["evicted"] = torch.zeros(1, 1, 2, LOOPS, rows, hkv, d, dtype=torch.bfloat16, device=dev)
        st["slots"] = torch.zeros(rows, dtype=torch.int64, device=dev)
        if case["mode"] == "step":
            st["back"] = torch.zeros_like(st["evicted"])
            st["seq_lens_back"] = st["seq_lens"] - R
        return st
    sizes, shared, owned = _shared_lens(case)
    b, ng = case["batch"], case["groups"]
    starts = [0]
    for x in sizes:
        starts.append(starts[-1] + x)
    # page tables: the pages of a shared prefix are the same for its group; a
    # page that the prefix ends in is a copy of each sequence's own
    tables, next_page, copies = [], 0, []
    for i in range(ng):
        full = shared[i] // page
        common = list(range(next_page, next_page + full))
        next_page += full
        first = None
        for k in range(starts[i], starts[i + 1]):
            extra = -(-(shared[i] + owned[k]) // page) - full
            mine = list(range(next_page, next_page + extra))
            next_page += extra
            if shared[i] % page and mine:
                if first is None:
                    first = mine[0]
                else:
                    copies.append((first, mine[0], shared[i] % page))
            tables.append(common + mine)
    cols = max(1, max(len(t) for t in tables))
    n_pages = max(1, next_page)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    st["pool"] = torch.randint(0, 256, (1, hkv, 1, n_pages, 2, page * J), generator=g, device=dev, dtype=torch.uint8)
    if copies:
        src, dst, n_tok = (torch.tensor(x, device=dev) for x in zip(*copies))
        off = _row_offsets(st, torch.arange(page, device=dev))          # [page][J]
        keep = torch.arange(page, device=dev)[None, :] < n_tok[:, None]             # shared slots of the page
        at = torch.nonzero(keep)
        a, z = perm[src].long()[at[:, 0]], perm[dst].long()[at[:, 0]]
        o = off[at[:, 1]]
        for kv in range(2):
            st["pool"][0, :, 0, z[:, None], kv, o] = st["pool"][0, :, 0, a[:, None], kv, o]
    flat = ints([t + [0] * (cols - len(t)) for t in tables], torch.int64)
    st["block_table"] = perm[flat].contiguous()
    st["codebooks"] = normal(1, hkv, 1, 2, LOOPS, J, E, c, dtype=torch.float32)
    scale = torch.rand(1, hkv, 1, 2, 1, 1, 1, 1, generator=g, device=dev) * 1.5 + 0.5   # per head and K/V
    st["codebooks"] *= scale
    st["q"] = normal(b, hq, d)
    st["win_k"] = (normal(b, hkv, P + R, d, dtype=torch.float32) * scale[0, :, 0, 0].reshape(1, hkv, 1, 1)).to(torch.bfloat16)
    st["win_v"] = (normal(b, hkv, P + R, d, dtype=torch.float32) * scale[0, :, 0, 1].reshape(1, hkv, 1, 1)).to(torch.bfloat16)
    group_of = [i for i in range(ng) for _ in range(sizes[i])]
    st.update(batch=b, n_pages=n_pages, pages=cols, loop=LOOPS - 1, sm_scale=d ** -0.5, max_group=max(sizes),
              max_shared=max(shared), max_own=max(owned), group_starts=ints(starts), shared_lens=ints(shared),
              seq_lens=ints([P + R + shared[group_of[i]] + owned[i] for i in range(b)]))
    st["out"] = torch.zeros(b, hq, d, dtype=torch.bfloat16, device=dev)
    return st


def _row_offsets(st, slot):
    """Byte offset in a plane of every channel group's index of the slots: [..][J]."""
    j = torch.arange(st["J"], device=slot.device)
    rot = slot % st["LB"]
    pos = (j - rot[..., None]) % st["J"]
    gr = st["GR"]
    return (slot // st["LB"] * st["LB"] * st["J"] + rot * gr)[..., None] + pos // gr * (st["LB"] * gr) + pos % gr


# ---- one pass ---------------------------------------------------------------------


def run(st):
    if st["case"]["op"] == "append":
        return _append_own(st) if own else _append_plain(st)
    return _shared_own(st) if own else _shared_plain(st)


def _config(st, lib):
    """The framework's handle of the cache, made once and kept."""
    if "cfg" not in st["keep"]:
        st["keep"]["cfg"] = lib.LoopVQConfig(
            n_layers=1, n_kv_heads=st["hkv"], n_q_heads=st["hq"], head_dim=st["d"], n_loops=LOOPS, loop_group=LOOPS,
            chan_group=st["c"], n_pages=st["n_pages"], max_batch=st["batch"], max_pages_per_seq=st["pages"],
            prefix_tokens=P, recent_tokens=R, page_tokens=st["page"])
    return st["keep"]["cfg"]


def _append_own(st):
    import sub_bit_vq_b200 as lib
    cfg = _config(st, lib)
    t = 1
    lib.loopvq_append(cfg, 0, t, st["q"], st["k"], st["v"], st["rope"], st["seq_lens"], st["win_k"], st["win_v"],
                      st["q_out"], st["evicted"], token_starts=st["token_starts"],
                      interleaved=st["case"]["interleaved"], block_table=st["block_table"], slot_mapping=st["slots"])
    ev = st["evicted"][0, 0, :, t]
    if "back" not in st:
        return [st["q_out"], st["win_k"], st["win_v"], ev, st["slots"]]
    lib.loopvq_append(cfg, 0, t, None, ev[0], ev[1], None, st["seq_lens_back"], st["win_k"], st["win_v"], None,
                      st["back"], token_starts=st["token_starts"])
    return [st["q_out"], st["win_k"], st["win_v"], ev, st["slots"], st["back"][0, 0, :, t]]


def _shared_own(st):
    import sub_bit_vq_b200 as lib
    cfg = _config(st, lib)
    if "ws" not in st["keep"]:
        n = lib.loopvq_decode_shared_workspace_bytes(cfg, st["batch"], st["case"]["groups"], st["max_group"],
                                                     st["max_shared"], st["max_own"])
        st["keep"]["ws"] = torch.zeros(n, dtype=torch.uint8, device=st["dev"])
    lib.loopvq_decode_attn_shared(cfg, 0, st["loop"], st["q"], st["pool"], st["codebooks"], st["block_table"],
                                  st["seq_lens"], st["group_starts"], st["shared_lens"], st["win_k"], st["win_v"],
                                  st["out"], st["keep"]["ws"], st["max_group"], st["max_shared"], st["max_own"],
                                  sm_scale=st["sm_scale"])
    return st["out"]


def _rotate(x, cos, sin, rot, interleaved):
    """x [rows][heads][d] in float32, cos and sin [rows][1][rot/2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _put(st, k, v, seq_lens, evicted, slots):
    """Writes rows into the windows, stages the tokens they push out. Works on every row at once."""
    rows, dev = st["rows"], st["dev"]
    r = torch.arange(rows, device=dev)
    b = torch.searchsorted(st["starts"], r, right=True) - 1
    n_new = st["starts"][1:] - st["starts"][:-1]
    total = seq_lens.long()[b]
    p = total - n_new[b] + r - st["starts"][b]                          # positions
    out = p - R                                                         # the token that row r pushes out
    ring = P + (p - P) % R
    old = out < total - n_new[b]
    gone = out >= P
    src = (r - R).clamp(min=0)
    for x, win, ev in ((k, st["win_k"], evicted[0, 0, 0, 1]), (v, st["win_v"], evicted[0, 0, 1, 1])):
        token = torch.where(old[:, None, None], win[b, :, ring], x[src])
        ev.copy_(torch.where(gone[:, None, None], token, ev))
    keep = (p < P) | (p >= total - R)
    at = torch.nonzero(keep)[:, 0]
    slot = torch.where(p < P, p, ring)[at]
    st["win_k"][b[at], :, slot] = k[at]
    st["win_v"][b[at], :, slot] = v[at]
    if slots is not None:
        q = (out - P).clamp(min=0)
        pg = st["block_table"].long()[b, (q // st["page"]).clamp(max=st["pages"] - 1)]
        slots.copy_(torch.where(gone, pg * st["page"] + q % st["page"], -1))
    return p


def _append_plain(st):
    rows, dev, rot = st["rows"], st["dev"], st["rot"]
    r = torch.arange(rows, device=dev)
    b = torch.searchsorted(st["starts"], r, right=True) - 1
    p = st["seq_lens"].long()[b] - (st["starts"][b + 1] - r)
    cos, sin = st["rope"][p, None, :rot // 2], st["rope"][p, None, rot // 2:]
    inter = st["case"]["interleaved"]
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, rot, inter))
    k = _rotate(st["k"].float(), cos, sin, rot, inter).to(torch.bfloat16)
    _put(st, k, st["v"], st["seq_lens"], st["evicted"], st["slots"])
    ev = st["evicted"][0, 0, :, 1]
    if "back" not in st:
        return [st["q_out"], st["win_k"], st["win_v"], ev, st["slots"]]
    _put(st, ev[0], ev[1], st["seq_lens_back"], st["back"], None)
    return [st["q_out"], st["win_k"], st["win_v"], ev, st["slots"], st["back"][0, 0, :, 1]]


def _tokens(st, pages, tok):
    """Keys and values [2][Hkv][n][tokens][d] of tokens `tok` [n][tokens] under page-table rows `pages` [n][..]."""
    page, J = st["page"], st["J"]
    phys = torch.gather(pages.long(), 1, (tok // page).clamp(max=pages.shape[1] - 1))
    flat = phys[..., None] * (2 * page * J) + _row_offsets(st, tok % page)
    pool = st["pool"].view(st["hkv"], -1)
    cb = st["codebooks"][0, :, 0, :, st["loop"]]                        # [Hkv][2][J][E][c]
    h = torch.arange(st["hkv"], device=st["dev"]).view(-1, 1, 1, 1)
    j = torch.arange(J, device=st["dev"])
    k = cb[:, 0][h, j, pool[:, flat].long()].flatten(-2)
    v = cb[:, 1][h, j, pool[:, flat + page * J].long()].flatten(-2)
    return k, v


def _shared_plain(st):
    b, hq, hkv, d, dev = st["batch"], st["hq"], st["hkv"], st["d"], st["dev"]
    ratio, S, N = hq // hkv, st["max_shared"], max(1, st["max_own"])
    starts, lens = st["group_starts"].long(), st["shared_lens"].long()
    seq = torch.arange(b, device=dev)
    grp = torch.searchsorted(starts, seq, right=True) - 1
    i = seq - starts[grp]
    ng, m = lens.shape[0], st["max_group"]
    n_vq = (st["seq_lens"].long() - P - R).clamp(min=0)
    q = st["q"].float() * (st["sm_scale"] * math.log2(math.e))
    # shared tokens, once for every group: rows are the group's sequences and query heads
    qg = torch.zeros(ng, m, hkv, ratio, d, device=dev)
    qg[grp, i] = q.view(b, hkv, ratio, d)
    qg = qg.permute(2, 0, 1, 3, 4).reshape(hkv, ng, m * ratio, d)
    tok = torch.arange(S, device=dev).expand(ng, S)
    ks, vs = _tokens(st, st["block_table"][starts[:-1]], tok)           # [Hkv][ng][S][d]
    xs = (qg @ ks.transpose(-1, -2)).view(hkv, ng, m, ratio, S)
    del ks
    lim = torch.zeros(ng, m, dtype=torch.int64, device=dev)
    lim[grp, i] = torch.minimum(lens[grp], n_vq)
    xs.masked_fill_(tok[None, :, None, None] >= lim[None, :, :, None, None], -math.inf)
    # own tokens and window of every sequence
    qs = q.view(b, hkv, ratio, d).transpose(0, 1)                       # [Hkv][b][ratio][d]
    own_tok = lens[grp][:, None] + torch.arange(N, device=dev)
    ko, vo = _tokens(st, st["block_table"], own_tok)
    xo = qs @ ko.transpose(-1, -2)
    del ko
    xo.masked_fill_(own_tok[None, :, None] >= n_vq[None, :, None, None], -math.inf)
    wk, wv = st["win_k"].transpose(0, 1).float(), st["win_v"].transpose(0, 1).float()
    xw = qs @ wk.transpose(-1, -2)
    xw.masked_fill_(torch.arange(P + R, device=dev) >= st["seq_lens"].long()[None, :, None, None], -math.inf)
    # one softmax over all three
    top = torch.maximum(torch.maximum(xs.amax(-1)[:, grp, i], xo.amax(-1)), xw.amax(-1))     # [Hkv][b][ratio]
    top_g = torch.zeros(hkv, ng, m, ratio, device=dev)
    top_g[:, grp, i] = top
    xs.sub_(top_g[..., None]).exp2_()
    po, pw = torch.exp2(xo - top[..., None]), torch.exp2(xw - top[..., None])
    total = xs.sum(-1)[:, grp, i] + po.sum(-1) + pw.sum(-1)
    o = (xs.view(hkv, ng, m * ratio, S) @ vs).view(hkv, ng, m, ratio, d)[:, grp, i]
    o = (o + po @ vo + pw @ wv) / total[..., None]
    st["out"].copy_(o.transpose(0, 1).reshape(b, hq, d))
    return st["out"]


# ---- the operators' definition in 64 bits -------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return _append_exact(st) if case["op"] == "append" else _shared_exact(st)


def _append_exact(st):
    rot, inter, d = st["rot"], st["case"]["interleaved"], st["d"]
    n, total = _append_lens(st["case"])
    step = st["case"]["mode"] == "step"
    f8 = torch.float64
    pair = torch.arange(rot // 2, device=st["dev"])
    first, second = (2 * pair, 2 * pair + 1) if inter else (pair, pair + rot // 2)

    def turned(x, lo, hi, p0):
        y = x[lo:hi].to(f8)
        z = y.clone()
        cs = st["rope"][p0:p0 + hi - lo].to(f8)[:, None]
        z[..., first] = y[..., first] * cs[..., :rot // 2] - y[..., second] * cs[..., rot // 2:]
        z[..., second] = y[..., second] * cs[..., :rot // 2] + y[..., first] * cs[..., rot // 2:]
        return z

    q_out = st["q_out"].to(f8)
    win = [st["win_k"].to(f8), st["win_v"].to(f8)]
    ev = torch.zeros(2, st["rows"], st["hkv"], d, dtype=f8, device=st["dev"])
    back = torch.zeros_like(ev)
    slots = [-1] * st["rows"]
    table = st["block_table"].tolist()
    r0 = 0
    for b in range(st["batch"]):
        r1, p0 = r0 + n[b], total[b] - n[b]
        q_out[r0:r1] = turned(st["q"], r0, r1, p0)
        new = [turned(st["k"], r0, r1, p0), st["v"][r0:r1].to(f8)]
        for a in range(2):
            if step:                                 # every row replaces its ring slot, and is taken back
                at = [P + (p0 + x - P) % R for x in range(n[b])]
                ev[a, r0:r1] = win[a][b][:, at].transpose(0, 1)
                back[a, r0:r1] = new[a]
            else:                                    # a fresh prompt: first P, last R, and the tokens between
                last = max(P, total[b] - R)
                win[a][b][:, :min(P, n[b])] = new[a][:P].transpose(0, 1)
                at = [P + (x - P) % R for x in range(last, n[b])]
                win[a][b][:, at] = new[a][last:].transpose(0, 1)
                if n[b] > P + R:
                    ev[a, r0 + P + R:r1] = new[a][P:n[b] - R]
        for x in range(n[b]):
            v = p0 + x - R - P
            if v >= 0:
                slots[r0 + x] = table[b][v // st["page"]] * st["page"] + v % st["page"]
        r0 = r1
    out = [q_out, win[0], win[1], ev, torch.tensor(slots, dtype=torch.int64, device=st["dev"])]
    return out + [back] if step else out


def _shared_exact(st):
    sizes, shared, owned = _shared_lens(st["case"])
    f8, dev, page, J, c = torch.float64, st["dev"], st["page"], st["J"], st["c"]
    hq, hkv, d = st["hq"], st["hkv"], st["d"]
    pool = st["pool"][0, :, 0]                                          # [Hkv][pages][2][page*J]
    cb = st["codebooks"][0, :, 0, :, st["loop"]].to(f8)                 # [Hkv][2][J][E][c]

    def tokens(row, lo, hi, kv):
        got = torch.empty(hkv, hi - lo, J, c, dtype=f8, device=dev)
        v = torch.arange(lo, hi, device=dev)
        phys, slot = row.long()[v // page], v % page
        turn = slot % st["LB"]
        for j in range(J):                                              # group j's byte of every token
            pos = torch.remainder(j - turn, J)
            byte = slot // st["LB"] * (st["LB"] * J) + pos // st["GR"] * (st["LB"] * st["GR"]) + turn * st["GR"] + pos % st["GR"]
            code = pool[:, phys, kv, byte].long()
            got[:, :, j] = torch.gather(cb[:, kv, j], 1, code[..., None].expand(-1, -1, c))
        return got.reshape(hkv, hi - lo, d)

    out = torch.empty(st["batch"], hq, d, dtype=f8, device=dev)
    b = 0
    for g, size in enumerate(sizes):
        ks, vs = (tokens(st["block_table"][b], 0, shared[g], kv) for kv in range(2))
        for _ in range(size):
            row = st["block_table"][b]
            parts = [(ks, vs), (st["win_k"][b].to(f8), st["win_v"][b].to(f8))]
            if owned[b]:
                parts.append(tuple(tokens(row, shared[g], shared[g] + owned[b], kv) for kv in range(2)))
            q = st["q"][b].to(f8).view(hkv, hq // hkv, d)
            z = torch.cat([q @ k.transpose(1, 2) for k, _ in parts], -1) * st["sm_scale"]
            p = torch.softmax(z, -1)
            at, o = 0, 0
            for k, v in parts:
                o = o + p[..., at:at + k.shape[1]] @ v
                at += k.shape[1]
            out[b] = o.reshape(hq, d)
            b += 1
    return out
