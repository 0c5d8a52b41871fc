"""Jagged attention with a sliding window and attention sinks, and the paged key/value cache it
serves from: the measured cases, the plain forms, and the framework's calls.

Four calls make the set: the prompt's forward pass over jagged sequences ("forward"), a training
step ("train": forward and backward), the appending of new keys and values to a paged cache with
the position rotation applied on the way ("append"), and one decoding step's attention over that
cache ("attend").  Grouped heads throughout: `heads` query heads share `kv_heads` key/value heads.

Definitions.  Query i of a sequence with Lq queries and Lk keys stands at position
p = i + Lk - Lq; it sees key j where j <= p and (j > p - window or j < sinks).
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEVICE = "cuda:0"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short user histories of the smallest workload: latency
        dict(name="forward_tiny", op="forward", batch=4, dist="uniform", lo=1, hi=64, past_hi=0, heads=2, kv_heads=2,
             dim=64, window=16, sinks=2, lens_seed=1),
        # ragged histories of the mid-sized workload (U[1, 2048], d = 64), shared key/value heads
        dict(name="forward_ragged", op="forward", batch=128, dist="uniform", lo=1, hi=2048, past_hi=0, heads=4,
             kv_heads=2, dim=64, window=255, sinks=4, lens_seed=2),
        # long-tailed histories (log-normal, up to 16384 tokens), as in the long-tail workload
        dict(name="forward_longtail", op="forward", batch=64, dist="lognormal", lo=16, hi=16384, past_hi=0, heads=8,
             kv_heads=8, dim=128, window=1024, sinks=4, lens_seed=3),
        # new events of each user after a longer known history: fewer queries than keys
        dict(name="forward_continued", op="forward", batch=48, dist="uniform", lo=1, hi=777, past_hi=6000, heads=8,
             kv_heads=2, dim=128, window=600, sinks=33, lens_seed=4),
        # one training step on ragged histories, d = 64
        dict(name="train_ragged", op="train", batch=64, dist="uniform", lo=1, hi=2048, past_hi=0, heads=4, kv_heads=2,
             dim=64, window=256, sinks=4, lens_seed=5),
        # one training step on long-tailed histories, d = 128
        dict(name="train_longtail", op="train", batch=64, dist="lognormal", lo=16, hi=16384, past_hi=0, heads=8,
             kv_heads=4, dim=128, window=512, sinks=16, lens_seed=6),
        # one new token of each of 64 users into the cache: latency
        dict(name="append_token", op="append", batch=64, dist="uniform", lo=1, hi=1, past_hi=4000, heads=8, kv_heads=8,
             dim=128, page=16, lens_seed=7),
        # whole prompts into the cache, queries rotated as well
        dict(name="append_prompt", op="append", batch=64, dist="uniform", lo=1, hi=2048, past_hi=100, heads=16,
             kv_heads=4, dim=128, page=64, lens_seed=8),
        # a decoding step of four short sequences: latency
        dict(name="attend_tiny", op="attend", batch=4, dist="uniform", lo=1, hi=64, heads=2, kv_heads=2, dim=64,
             page=16, window=1 << 30, sinks=0, lens_seed=9),
        # a decoding step of a wide batch over everything cached
        dict(name="attend_wide", op="attend", batch=128, dist="uniform", lo=1, hi=16384, heads=16, kv_heads=4, dim=128,
             page=64, window=1 << 30, sinks=0, lens_seed=10),
        # two very long sequences: the key axis has to be split
        dict(name="attend_long", op="attend", batch=2, dist="uniform", lo=100000, hi=131072, heads=8, kv_heads=8,
             dim=128, page=32, window=1 << 30, sinks=0, lens_seed=11),
        # a decoding step with a window and sinks over long caches
        dict(name="attend_window", op="attend", batch=192, dist="uniform", lo=1, hi=20000, heads=8, kv_heads=2, dim=64,
             page=16, window=2048, sinks=4, lens_seed=12),
    ]


def draw(rng):
    """One more case: sizes log-uniform over the ranges that the listed cases span."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["forward", "train", "append", "attend"])
    most = [work(c) for c in listed() if c["op"] == op]
    most_bytes, most_flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 1, 2, 3, 4, 8])
        c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([64, 128]), batch=log_int(1, 192),
                 dist="uniform", lo=1, lens_seed=rng.randrange(1 << 30))
        if op in ("forward", "train"):
            c.update(hi=log_int(1, 8192), past_hi=rng.choice([0, 0, log_int(1, 6000)]), window=log_int(1, 2048),
                     sinks=rng.choice([0, 1, 4, log_int(1, 128)]))
            if rng.random() < 0.3:
                c.update(dist="lognormal", lo=16, hi=16384)
            if op == "train":  # a row that sees one key alone has no gradient but its rounding
                c.update(hi=max(c["hi"], 8), window=max(c["window"], 4))
        elif op == "append":
            c.update(hi=rng.choice([1, log_int(1, 2048)]), past_hi=log_int(1, 4000), page=rng.choice([16, 32, 64, 128]))
        else:
            c.update(hi=log_int(1, 131072), page=rng.choice([16, 32, 64, 128]), window=1 << 30, sinks=0)
            if rng.random() < 0.5:
                c.update(window=log_int(1, 8192), sinks=rng.choice([0, 1, 4, log_int(1, 128)]))
        lens = _lens(c)
        w = work(c)
        # the plain form works on 256-query blocks with whole windows of keys: bound its scores too
        blocks = sum((n + 255) // 256 for n in lens[0])
        if op in ("forward", "train") and blocks * c["heads"] * 256 * (min(c["window"], max(lens[1])) + 256) > 3e9:
            continue
        if op == "attend" and c["batch"] * min(max(lens[0]), c["window"] + c["sinks"]) * kv_heads * c["dim"] > 1.1e9:
            continue
        if op == "append" and sum(lens[1]) * kv_heads * c["dim"] > 2e8:
            continue
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and sum(lens[0]) > 0:
            return c


def _lens(case):
    """(new tokens, all tokens) of each sequence, from the case alone."""
    r = random.Random(case["lens_seed"])
    n = []
    for _ in range(case["batch"]):
        if case["dist"] == "lognormal":
            x = int(round(math.exp(math.log(512.0) + 1.2 * r.gauss(0.0, 1.0))))
            n.append(min(max(x, case["lo"]), case["hi"]))
        else:
            n.append(r.randint(case["lo"], case["hi"]))
    past = case.get("past_hi", 0)
    return n, [x + (r.randint(0, past) if past else 0) for x in n]


def _seen_by(p, window, sinks):
    """How many keys a query at position p sees."""
    w = min(p + 1, window)
    return w + min(sinks, p + 1 - w)


def _pairs(case):
    """Visible (query, key) pairs of one head, and the keys that some query sees."""
    pairs = keys = 0
    W, S = case["window"], case["sinks"]
    for lq, lk in zip(*_lens(case)):
        if lk <= W:  # plain causal
            pairs += lq * (lk - lq) + lq * (lq + 1) // 2
        else:
            pairs += sum(_seen_by(p, W, S) for p in range(lk - lq, lk)) if lq < 4096 else \
                _seen_sum(lk - lq, lk, W, S)
        first = max(0, lk - lq - W + 1)
        keys += (lk - first) + min(S, first)
    return pairs, keys


def _seen_sum(p0, p1, window, sinks):
    """sum of _seen_by over positions p0 .. p1 - 1, without the loop."""
    def tri(n, cap):  # sum over p < n of min(p + 1, cap)
        m = min(n, cap)
        return m * (m + 1) // 2 + (n - m) * cap
    cap = window + sinks
    return tri(p1, cap) - tri(p0, cap)


def work(case):
    """What a pass cannot do without: each input that counts read once, each output written once."""
    H, G, d = case["heads"], case["kv_heads"], case["dim"]
    new, all_ = _lens(case)
    if case["op"] in ("forward", "train"):
        pairs, keys = _pairs(case)
        tq, tk = sum(new), sum(all_)
        q, kv, lse = tq * H * d * 2, keys * G * d * 2, tq * H * 4
        if case["op"] == "forward":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * H * pairs}
        # out and lse, then q, k, v, dout again into dq, dk, dv; five products in the backward pass
        return {"bytes": 4 * q + 2 * kv + lse + 2 * tk * G * d * 2, "flops": 14 * d * H * pairs}
    if case["op"] == "append":
        n = sum(new)
        return {"bytes": n * d * 2 * (2 * H + 4 * G) + 12 * case["batch"], "flops": 3 * n * d * (H + G)}
    W, S = case["window"], case["sinks"]
    keys = sum(_seen_by(x - 1, W, S) for x in new)
    return {"bytes": keys * G * d * 4 + case["batch"] * H * (4 * d + 4), "flops": 4 * d * H * keys}


# ------------------------------------------------------------------ inputs

def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int64, device=DEVICE)


def _cache_layout(case, gen, tokens):
    """A page table over shuffled pages with room for `tokens[b]` tokens of each sequence."""
    page = case["page"]
    need = [(n + page - 1) // page for n in tokens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((case["batch"], max(need)), -1, dtype=torch.int32, device=DEVICE)
    b = torch.repeat_interleave(torch.arange(case["batch"], device=DEVICE), torch.tensor(need, device=DEVICE))
    first = _offsets(need)[:-1]
    i = torch.arange(sum(need), device=DEVICE)
    table[b, i - first[b]] = perm[:sum(need)]
    return pages, table


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    H, G, d = case["heads"], case["kv_heads"], case["dim"]
    new, all_ = _lens(case)

    def normal(*shape):
        x = torch.empty(shape, dtype=BF16, device=DEVICE)
        return x.normal_(generator=gen)

    s = dict(op=case["op"], scale=1.0 / math.sqrt(d))
    if case["op"] in ("forward", "train"):
        s.update(q=normal(sum(new), H, d), k=normal(sum(all_), G, d), v=normal(sum(all_), G, d),
                 q_offsets=_offsets(new), kv_offsets=_offsets(all_), window=case["window"], sinks=case["sinks"],
                 blocks=sum((n + 255) // 256 for n in new), longest=max(all_))
        if case["op"] == "train":
            s["dout"] = normal(sum(new), H, d)
        if own:
            from jagged_attention_recsys_jfa_gb300 import new_window_workspace
            args = (case["batch"], H, G, d, sum(new), sum(all_), case["sinks"])
            s["workspace"] = new_window_workspace(*args, False, DEVICE)
            if case["op"] == "train":
                s["workspace_bwd"] = new_window_workspace(*args, True, DEVICE)
        return s
    # theta_i = 10000^(-2i/d), as the angle in radians that a step of one position turns pair i
    freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=F64) / d)
    if case["op"] == "append":
        pages, table = _cache_layout(case, gen, all_)
        s.update(k=normal(sum(new), G, d), v=normal(sum(new), G, d), q=normal(sum(new), H, d), offsets=_offsets(new),
                 lengths=torch.tensor([a - n for a, n in zip(all_, new)], dtype=torch.int32, device=DEVICE),
                 frequencies=freq, frequencies_gpu=freq.to(DEVICE), page_table=table,
                 k_cache=normal(pages, G, case["page"], d), v_cache=normal(pages, G, case["page"], d))
    else:
        pages, table = _cache_layout(case, gen, new)
        s.update(q=normal(case["batch"], H, d), k_cache=normal(pages, G, case["page"], d),
                 v_cache=normal(pages, G, case["page"], d), page_table=table,
                 lengths=torch.tensor(new, dtype=torch.int32, device=DEVICE), window=case["window"],
                 sinks=case["sinks"], longest=max(new))
    if own:
        from jagged_attention_recsys_jfa_gb300 import new_cache_workspace
        s["workspace"] = new_cache_workspace(case["batch"], H, G, d, DEVICE)
    return s


# ------------------------------------------------------------------ the passes

def run(s):
    if own:
        return _run_own(s)
    if s["op"] in ("forward", "train"):
        return _plain_window(s)
    return _plain_append(s) if s["op"] == "append" else _plain_attend(s)


def _run_own(s):
    import jagged_attention_recsys_jfa_gb300 as jfa

    if s["op"] in ("forward", "train"):
        seqs, mask = (s["q_offsets"], s["kv_offsets"]), (s["window"], s["sinks"], s["scale"])
        out, lse, _ = jfa.jfa_window_forward(s["q"], s["k"], s["v"], *seqs, *mask, workspace=s["workspace"])
        if s["op"] == "forward":
            return {"out": out, "lse": lse}
        dq, dk, dv, _ = jfa.jfa_window_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, *seqs, *mask,
                                                workspace=s["workspace_bwd"])
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    if s["op"] == "append":
        q, _, lengths, _ = jfa.jfa_cache_append(s["k"], s["v"], s["offsets"], s["k_cache"], s["v_cache"],
                                                s["page_table"], s["lengths"], q=s["q"], frequencies=s["frequencies"],
                                                workspace=s["workspace"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": lengths}
    out, lse, _ = jfa.jfa_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"],
                                          s["window"], s["sinks"], s["scale"], workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _softmax_parts(x, mask):
    """exp(x - lse) over the last axis where `mask`, and lse; rows without a visible key get 0 and -inf."""
    x.masked_fill_(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    return p, (m + total.log()).squeeze(-1)


def _plain_window(s):
    """Blocks of 256 queries, each against the sinks and the keys that its windows span."""
    q, k, v, W, S, scale = s["q"], s["k"], s["v"], min(s["window"], s["longest"]), s["sinks"], s["scale"]
    c, N = 256, s["blocks"]
    (Tq, H, d), G = q.shape, k.shape[1]
    qo, ko = s["q_offsets"], s["kv_offsets"]
    lq, lk = qo.diff(), ko.diff()
    nb = (lq + c - 1) // c
    b = torch.repeat_interleave(torch.arange(lq.numel(), device=q.device), nb, output_size=N)
    start = (torch.arange(N, device=q.device) - (nb.cumsum(0) - nb)[b]) * c
    i = start[:, None] + torch.arange(c, device=q.device)
    q_ok = i < lq[b, None]
    pos = i + (lk - lq)[b, None]
    at = start + (lk - lq)[b] - W + 1
    j = torch.cat([torch.arange(S, device=q.device).expand(N, S),
                   at[:, None] + torch.arange(W + c - 1, device=q.device)], 1)
    j_ok = (j >= 0) & (j < lk[b, None])
    j_ok[:, S:] &= j[:, S:] >= S
    near = j[:, None, :] > pos[:, :, None] - W
    near[:, :, :S] = True
    mask = (q_ok[:, :, None] & j_ok[:, None, :] & near & (j[:, None, :] <= pos[:, :, None]))[:, None, None]
    qi = (qo[b, None] + i).clamp(0, max(Tq - 1, 0))
    kj = (ko[b, None] + j).clamp(0, max(k.shape[0] - 1, 0))
    qg = q[qi].view(N, c, G, H // G, d).float()
    kg, vg = k[kj].float(), v[kj].float()
    p, lse_g = _softmax_parts(torch.einsum("nqghd,nkgd->nghqk", qg, kg).mul_(scale), mask)
    og = torch.einsum("nghqk,nkgd->nqghd", p, vg)
    rows = qi[q_ok]
    out = torch.empty((Tq, H, d), dtype=F32, device=q.device)
    out[rows] = og.reshape(N, c, H, d)[q_ok]
    if s["op"] == "forward":
        lse = torch.empty((Tq, H), dtype=F32, device=q.device)
        lse[rows] = lse_g.permute(0, 3, 1, 2).reshape(N, c, H)[q_ok]
        return {"out": out.to(BF16), "lse": lse.t().contiguous()}
    do = s["dout"][qi].view(N, c, G, H // G, d).float()
    do.mul_(q_ok[:, :, None, None, None])
    dvg = torch.einsum("nghqk,nqghd->nkgd", p, do)
    delta = (do * og).sum(-1).permute(0, 2, 3, 1)[..., None]
    ds = torch.einsum("nqghd,nkgd->nghqk", do, vg).sub_(delta).mul_(p).mul_(scale)
    dqg = torch.einsum("nghqk,nkgd->nqghd", ds, kg).reshape(N, c, H, d)
    dkg = torch.einsum("nghqk,nqghd->nkgd", ds, qg)
    dq = torch.empty((Tq, H, d), dtype=F32, device=q.device)
    dq[rows] = dqg[q_ok]
    dk = torch.zeros(k.shape, dtype=F32, device=q.device).index_add_(0, kj.reshape(-1), dkg.reshape(-1, G, d))
    dv = torch.zeros(k.shape, dtype=F32, device=q.device).index_add_(0, kj.reshape(-1), dvg.reshape(-1, G, d))
    return {"out": out.to(BF16), "dq": dq.to(BF16), "dk": dk.to(BF16), "dv": dv.to(BF16)}


def _rotate(x, angle):
    """Pair (x_i, x_{i + d/2}) of every head turned by the token's angle i; angles in 64 bits."""
    a, b = x.float().chunk(2, -1)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(BF16)


def _plain_append(s):
    off, page, T = s["offsets"], s["k_cache"].shape[2], s["k"].shape[0]
    n = off.diff()
    b = torch.repeat_interleave(torch.arange(n.numel(), device=off.device), n, output_size=T)
    pos = s["lengths"][b].long() + torch.arange(T, device=off.device) - off[b]
    angle = pos.to(F64)[:, None] * s["frequencies_gpu"]
    slot = s["page_table"][b, pos // page].long(), pos % page
    s["k_cache"][slot[0], :, slot[1]] = _rotate(s["k"], angle)
    s["v_cache"][slot[0], :, slot[1]] = s["v"]
    return {"q": _rotate(s["q"], angle), "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "lengths": (s["lengths"] + n).to(torch.int32)}


def _plain_attend(s):
    q, L, S, page = s["q"], s["lengths"].long()[:, None], s["sinks"], s["k_cache"].shape[2]
    (B, H, d), G = q.shape, s["k_cache"].shape[1]
    W = min(s["window"], s["longest"])
    ar = torch.arange(W, device=q.device)
    first = (L - W).clamp(min=0)
    near = first + ar
    j = torch.cat([torch.arange(S, device=q.device).expand(B, S), near], 1)
    ok = j < L
    ok[:, :S] &= j[:, :S] < first  # a sink inside the window is counted there
    j = j.clamp(max=s["page_table"].shape[1] * page - 1)
    pages = torch.gather(s["page_table"], 1, j // page).long().clamp(min=0)
    k, v = s["k_cache"][pages, :, j % page].float(), s["v_cache"][pages, :, j % page].float()
    x = torch.einsum("bghd,bkgd->bghk", q.view(B, G, H // G, d).float(), k).mul_(s["scale"])
    p, lse = _softmax_parts(x, ok[:, None, None])
    out = torch.einsum("bghk,bkgd->bghd", p, v).reshape(B, H, d)
    return {"out": out.to(BF16), "lse": lse.reshape(B, H).t().contiguous()}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, all_ = _lens(case)
    H, G, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        k_cache, v_cache = s["k_cache"].to(F64), s["v_cache"].to(F64)
        q_out, row = torch.zeros(s["q"].shape, dtype=F64, device=DEVICE), 0
        half = d // 2
        theta = torch.tensor([10000.0 ** (-2.0 * i / d) for i in range(half)], dtype=F64, device=DEVICE)
        for b, (n, total) in enumerate(zip(new, all_)):
            p = torch.arange(total - n, total, device=DEVICE)
            z = torch.exp(1j * (p.to(F64)[:, None] * theta))[:, None]  # one turn per token and pair
            def turn(x):
                w = torch.complex(x[..., :half].to(F64), x[..., half:].to(F64)) * z
                return torch.cat([w.real, w.imag], -1)
            where = s["page_table"][b].long()[p // case["page"]]
            k_cache[where, :, p % case["page"]] = turn(s["k"][row:row + n])
            v_cache[where, :, p % case["page"]] = s["v"][row:row + n].to(F64)
            q_out[row:row + n] = turn(s["q"][row:row + n])
            row += n
        return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache, "lengths": None}
    if case["op"] == "attend":
        out = torch.zeros(s["q"].shape, dtype=F64, device=DEVICE)
        lse = torch.full((H, case["batch"]), -math.inf, dtype=F64, device=DEVICE)
        for b, n in enumerate(new):
            seen = [x for x in range(min(case["sinks"], n))]
            rest = max(0, n - case["window"])
            seen = torch.tensor([x for x in seen if x < rest] + list(range(rest, n)), device=DEVICE)
            where = s["page_table"][b].long()[seen // case["page"]]
            for h in range(H):
                g = h // (H // G)
                x = s["k_cache"][where, g, seen % case["page"]].to(F64) @ s["q"][b, h].to(F64) * s["scale"]
                lse[h, b] = torch.logsumexp(x, 0)
                out[b, h] = torch.exp(x - lse[h, b]) @ s["v_cache"][where, g, seen % case["page"]].to(F64)
        return {"out": out, "lse": lse}
    q, k, v = s["q"], s["k"], s["v"]
    train = case["op"] == "train"
    out = torch.zeros(q.shape, dtype=F64, device=DEVICE)
    lse = torch.full((H, q.shape[0]), -math.inf, dtype=F64, device=DEVICE)
    if train:
        dq, dk, dv = (torch.zeros(x.shape, dtype=F64, device=DEVICE) for x in (q, k, v))
    q0 = k0 = 0
    for n, total in zip(new, all_):
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            p = torch.arange(r0, r1, device=DEVICE)[:, None] + (total - n)
            low = max(0, r0 + total - n - case["window"] + 1)
            cols = torch.cat([torch.arange(min(case["sinks"], low), device=DEVICE),
                              torch.arange(low, r1 + total - n, device=DEVICE)])
            see = (cols <= p) & ((cols > p - case["window"]) | (cols < case["sinks"]))
            rows, at = slice(q0 + r0, q0 + r1), k0 + cols
            # all heads of the block at once: [H, rows, keys]
            Q = q[rows].to(F64).transpose(0, 1)
            K = k[at].to(F64).transpose(0, 1).repeat_interleave(H // G, 0)
            V = v[at].to(F64).transpose(0, 1).repeat_interleave(H // G, 0)
            x = (Q @ K.transpose(1, 2) * s["scale"]).masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, -1)
            P = torch.exp(x - z[..., None])
            O = P @ V
            out[rows], lse[:, rows] = O.transpose(0, 1), z
            if train:
                D = s["dout"][rows].to(F64).transpose(0, 1)
                dS = P * (D @ V.transpose(1, 2) - (D * O).sum(-1, keepdim=True)) * s["scale"]
                dq[rows] = (dS @ K).transpose(0, 1)
                for into, grad in ((dk, dS.transpose(1, 2) @ Q), (dv, P.transpose(1, 2) @ D)):
                    into[at] += grad.view(G, H // G, -1, d).sum(1).transpose(0, 1)
        q0, k0 = q0 + n, k0 + total
    if train:
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    return {"out": out, "lse": lse}
