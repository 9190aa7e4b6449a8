"""What is measured of the operators that serve and train the window layers of
a hybrid stack next to plain attention: attention with a sliding window and a
few first tokens that stay visible (sinks; whole sequences with gradients, and
over the paged cache), the append that norms, rotates and stores new tokens'
keys and values in one pass, and attention of a batch whose sequences share a
long prefix in the cache.

Each case is one pass through one operator.  ``own`` false: elementary torch
operations in 32 bits (rotary angles in 64); ``own`` true: the package's
entry points.  Shapes follow this repository's layer workload (16 heads,
d = 128, 8 x 4096 training tokens, 32K long sequences, decode batches, the
pages' 2K window) and their ragged, small and float32 relatives.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
F8_MAX = 448.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "f8": 1}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a training step (forward and backward) of the hybrid's 2K-window layer, four sink tokens
        dict(name="sink_train_2k", op="sink", nseq=8, tokens=32768, ragged=False, Hq=16, Hk=4, d=128, window=2048,
             sinks=4, dt="bf16", bwd=True),
        # the same on one long sequence, where every row but the first sees the sinks from afar: the largest
        dict(name="sink_train_32k", op="sink", nseq=1, tokens=32768, ragged=False, Hq=16, Hk=4, d=128, window=2048,
             sinks=4, dt="bf16", bwd=True),
        # packed sequences of different lengths, d = 64, more sinks than a tile has rows
        dict(name="sink_packed_d64", op="sink", nseq=11, tokens=9973, ragged=True, Hq=12, Hk=4, d=64, window=500,
             sinks=33, dt="bf16", bwd=True),
        # float32, ungrouped heads, short ragged sequences
        dict(name="sink_packed_f32", op="sink", nseq=5, tokens=1543, ragged=True, Hq=4, Hk=4, d=64, window=100, sinks=7,
             dt="f32", bwd=True),
        # decode of a ragged batch over a quantised cache whose middle pages are freed
        dict(name="sink_decode_f8", op="paged", nseq=64, q=1, ctx=16384, Hq=16, Hk=4, d=128, page=64, window=2048,
             sinks=4, dt="bf16", cache="f8"),
        # one sequence's decode step: latency
        dict(name="sink_decode_one", op="paged", nseq=1, q=1, ctx=9000, Hq=16, Hk=4, d=128, page=16, window=1024,
             sinks=20, dt="bf16", cache="bf16"),
        # a serving batch's new tokens at far positions: latency
        dict(name="append_decode", op="append", B=32, T=1, Hq=16, Hk=4, d=128, rot=128, inter=False, page=16, dt="bf16",
             cache="bf16", far=1 << 20),
        # a prompt's tokens into a quantised cache
        dict(name="append_prompt_f8", op="append", B=1, T=32768, Hq=16, Hk=4, d=128, rot=128, inter=False, page=64,
             dt="bf16", cache="f8", far=0),
        # float32, half of the head rotated in the interleaved layout, odd lengths and head counts
        dict(name="append_partial_f32", op="append", B=3, T=1001, Hq=6, Hk=3, d=64, rot=32, inter=True, page=32,
             dt="f32", cache="f32", far=1 << 15),
        # decode of a batch behind one long common prompt
        dict(name="prefix_decode", op="prefix", groups=1, nseq=64, q=1, chunk=0, prefix=32768, ctx=1500, Hq=16, Hk=4,
             d=128, page=64, dt="bf16", cache="bf16"),
        # three common prompts, a new request's chunk among single tokens, quantised cache
        dict(name="prefix_groups_f8", op="prefix", groups=3, nseq=41, q=1, chunk=200, prefix=9000, ctx=700, Hq=16, Hk=4,
             d=128, page=64, dt="bf16", cache="f8"),
        # a few sequences behind a short prompt: latency
        dict(name="prefix_few", op="prefix", groups=1, nseq=5, q=1, chunk=0, prefix=1000, ctx=90, Hq=12, Hk=4, d=64,
             page=16, dt="bf16", cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sink", "sink", "paged", "append", "prefix", "prefix"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
    if Hq > 16:
        Hq = Hk = 1 + rng.randint(0, 7)
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "sink":
        nseq = rng.randint(1, 20)
        tokens = max(nseq, _log(rng, 64, 12000 if dt == "bf16" else 4000))
        return dict(op=op, nseq=nseq, tokens=tokens, ragged=True, Hq=Hq, Hk=Hk, d=d, window=_log(rng, 1, 2048),
                    sinks=_log(rng, 1, 200), dt=dt, bwd=rng.random() < 0.7)
    if op == "paged":
        return dict(op=op, nseq=_log(rng, 1, 200), q=rng.choice([1, 1, 1, 2, 5, 40]), ctx=_log(rng, 100, 16000), Hq=Hq,
                    Hk=Hk, d=d, page=rng.choice([16, 32, 64, 128]), window=_log(rng, 30, 2048), sinks=_log(rng, 1, 200),
                    dt=dt, cache=rng.choice(["f8", dt]))
    if op == "append":
        return dict(op=op, B=rng.randint(1, 9), T=_log(rng, 1, 4000), Hq=Hq, Hk=Hk, d=d, rot=rng.choice([16, d // 2, d]),
                    inter=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]), dt=dt, cache=rng.choice(["f8", dt]),
                    far=rng.choice([0, 1 << 16, 1 << 22]))
    groups = rng.choice([1, 1, 2, 4])
    return dict(op=op, groups=groups, nseq=groups * _log(rng, 1, 40), q=rng.choice([1, 1, 1, 3]),
                chunk=rng.choice([0, 0, 150]), prefix=_log(rng, 50, 16000), ctx=_log(rng, 150, 2000), Hq=Hq, Hk=Hk, d=d,
                page=rng.choice([16, 32, 64, 128]), dt=dt, cache=rng.choice(["f8", dt]))


def _lens(case):
    """Sequence lengths of a whole-sequence case: equal, or ragged from one token up."""
    n, tot = case["nseq"], case["tokens"]
    if not case["ragged"]:
        return [tot // n] * n
    r = random.Random(n * 1000003 + tot)
    w = [math.exp(r.uniform(0.0, 4.0)) for _ in range(n)]
    lens = [1 + int((tot - n) * x / sum(w)) for x in w]
    lens[-1] += tot - sum(lens)
    return lens


def _paged_lens(case):
    """Keys of every sequence of a paged case, its new tokens among them."""
    r = random.Random(case["nseq"] * 7919 + case["ctx"])
    return [max(case["q"], case["ctx"] if case["nseq"] == 1 else r.randint(case["ctx"] // 4, case["ctx"]))
            for _ in range(case["nseq"])]


def _prefix_lens(case):
    """(new tokens, own keys with the new ones) of every sequence, the prefix
    keys of every group, and the first sequence of each group."""
    r = random.Random(case["nseq"] * 104729 + case["prefix"])
    lq = [case["q"]] * case["nseq"]
    if case["chunk"]:
        lq[case["nseq"] // 2] = case["chunk"]
    lk = [max(a, r.randint(1, case["ctx"])) for a in lq]
    pre = [r.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["groups"])]
    pre[0] = case["prefix"]
    cuts = sorted(r.sample(range(1, case["nseq"]), case["groups"] - 1)) if case["groups"] > 1 else []
    return lq, lk, pre, [0] + cuts + [case["nseq"]]


def _visible(lq, lk, window, sinks):
    """Visible (query, key) pairs of queries at positions lk-lq .. lk-1."""
    pos = np.arange(lk - lq, lk, dtype=np.int64)
    near = np.minimum(pos + 1, window) if window else pos + 1
    return int((near + np.minimum(sinks, pos + 1 - near)).sum())


def work(case):
    s = SIZE[case["dt"]]
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "sink":
        tot = case["tokens"]
        pairs = sum(_visible(n, n, case["window"], case["sinks"]) for n in _lens(case))
        fwd_b = tot * d * (2 * Hq + 2 * Hk) * s + tot * Hq * 4
        bwd_b = tot * d * (4 * Hq + 4 * Hk) * s + tot * Hq * 4   # q, o, dout, dq; k, v, dk, dv
        return {"bytes": fwd_b + (bwd_b if case["bwd"] else 0), "flops": pairs * Hq * d * (14 if case["bwd"] else 4)}
    row = d * SIZE[case["cache"]] + (1 if case["cache"] == "f8" else 0)
    if case["op"] == "paged":
        lk, a, w, sk = _paged_lens(case), case["q"], case["window"], case["sinks"]
        keys = sum(min(b, a - 1 + w + sk) for b in lk)
        flops = sum(_visible(a, b, w, sk) for b in lk) * Hq * d * 4
        return {"bytes": 2 * keys * Hk * row + 2 * a * len(lk) * Hq * d * s, "flops": flops}
    if case["op"] == "append":
        n = case["B"] * case["T"]
        # read q, k, v; write q and the rows (quantised rows are read back as the values they stand for)
        back = 2 * n * Hk * (row + 2 * d) if case["cache"] == "f8" else 0
        return {"bytes": n * d * s * (2 * Hq + 2 * Hk) + 2 * n * Hk * row + back, "flops": n * d * (8 * Hq + 12 * Hk)}
    lq, lk, pre, cuts = _prefix_lens(case)
    flops = sum(_visible(a, b, 0, 0) for a, b in zip(lq, lk))
    flops += sum(p * sum(lq[a:b]) for p, a, b in zip(pre, cuts, cuts[1:]))
    return {"bytes": 2 * (sum(pre) + sum(lk)) * Hk * row + 2 * sum(lq) * Hq * d * s, "flops": flops * Hq * d * 4}


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dt, mul=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * mul).to(dt)


def _cache(x, g, case, npages):
    """A cache of npages pages of keys and values, filled."""
    for n in ("k", "v"):
        c = torch.randn((npages, case["Hk"], case["page"], case["d"]), generator=g, device="cuda")
        x[n + "_scale"] = None
        if case["cache"] == "f8":
            x[n + "_cache"], x[n + "_scale"] = _quantise(c)
        else:
            x[n + "_cache"] = c.to(DT[case["dt"]])


def _table(need, perm):
    """Block table [N, max pages] of sequences of `need` pages each, from the
    page numbers perm; -1 behind a sequence's last page."""
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    g = _gen(seed)
    dt = DT[case["dt"]]
    x = {"case": case}
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "sink":
        lens = _lens(case)
        B, T = (1, case["tokens"]) if case["ragged"] else (case["nseq"], lens[0])
        x["q"], x["k"] = _randn(g, (B, T, Hq, d), dt), _randn(g, (B, T, Hk, d), dt)
        # the first tokens' keys stand out, as those of trained sinks do
        x["k"][:, :case["sinks"]] *= 1.5
        x["v"] = _randn(g, (B, T, Hk, d), dt)
        x["lens"] = lens
        x["cu"] = _ints([0] + list(np.cumsum(lens))) if case["ragged"] else None
        if case["bwd"]:
            x["dout"] = _randn(g, (B, T, Hq, d), dt)
    elif case["op"] == "paged":
        lk, page = _paged_lens(case), case["page"]
        need = [-(-n // page) for n in lk]
        npages = sum(need) + 3
        table = _table(need, torch.randperm(npages, generator=g, device="cuda").to(torch.int32).cpu())
        for i, n in enumerate(lk):
            # pages behind the sinks and before the first query's window are freed
            first = max(0, n - case["q"] + 1 - case["window"])
            table[i, -(-case["sinks"] // page):first // page] = -1
        x["table"], x["seq_lens"], x["lk"] = table.cuda(), _ints(lk), lk
        x["q"] = _randn(g, (case["nseq"], case["q"], Hq, d), dt)
        _cache(x, g, case, npages)
    elif case["op"] == "append":
        B, T, page = case["B"], case["T"], case["page"]
        # q, k and v as one projection leaves them, head by head of every token
        x["qkv"] = _randn(g, (B, T, Hq + 2 * Hk, d), dt, torch.exp(0.5 * torch.randn((B, T, 1, 1), generator=g, device="cuda")))
        x["wq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        x["wk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        x["freqs"] = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        x["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        npages = -(-B * T // page) + 2
        x["slots"] = torch.randperm(npages * page, generator=g, device="cuda")[:B * T].to(torch.int64)
        for n in ("k", "v"):
            x[n + "_cache"] = torch.zeros((npages, Hk, page, d), device="cuda").to(
                torch.float8_e4m3fn if case["cache"] == "f8" else dt)
            x[n + "_scale"] = None
            if case["cache"] == "f8":
                x[n + "_scale"] = torch.full((npages, Hk, page), 127, dtype=torch.uint8, device="cuda")
    else:
        lq, lk, pre, cuts = _prefix_lens(case)
        page = case["page"]
        need, need_pre = [-(-n // page) for n in lk], [-(-n // page) for n in pre]
        npages = sum(need) + sum(need_pre) + 3
        perm = torch.randperm(npages, generator=g, device="cuda").to(torch.int32).cpu()
        x["prefix_table"] = _table(need_pre, perm).cuda()
        x["table"] = _table(need, perm[sum(need_pre):]).cuda()
        x["prefix_lens"], x["seq_lens"] = _ints(pre), _ints(lk)
        x["groups"] = _ints(cuts) if case["groups"] > 1 else None
        x["lq"], x["lk"], x["pre"], x["cuts"] = lq, lk, pre, cuts
        x["cu"] = _ints([0] + list(np.cumsum(lq))) if case["chunk"] else None
        x["q"] = _randn(g, (1, sum(lq), Hq, d) if case["chunk"] else (case["nseq"], case["q"], Hq, d), dt)
        _cache(x, g, case, npages)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    # the buffers a serving or training loop keeps for its outputs
    if case["op"] == "append":
        B, T, Hq = case["B"], case["T"], case["Hq"]
        x["out"] = torch.empty((B, T, Hq, case["d"]), dtype=DT[case["dt"]], device="cuda")
    else:
        x["out"] = torch.empty_like(x["q"])
        x["lse"] = torch.empty(x["q"].shape[:3], dtype=torch.float32, device="cuda")
    if own and case["op"] != "append":
        import gated_delta_rule_07_amd as g
        need = 0
        if case["op"] == "sink" and case["bwd"]:
            B, T, Hq, d = x["q"].shape
            need = g.attn_bwd_workspace_bytes(B, T, Hq, case["Hk"], d, DT[case["dt"]], sinks=case["sinks"],
                                              num_seqs=case["nseq"] if case["ragged"] else 0)
        elif case["op"] == "paged":
            need = g.attn_paged_workspace_bytes(x["q"], x["k_cache"], x["table"], None, case["window"], case["sinks"])
        elif case["op"] == "prefix":
            need = g.attn_paged_prefix_workspace_bytes(x["q"], x["k_cache"], x["prefix_table"], x["table"], x["cu"])
        x["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return x


# ------------------------------------------------------------- plain forms --
def _quantise(c):
    """Rows of c (float32, last axis) as e4m3 codes and the exponent byte e +
    127 of their scale 2^e, e the smallest with amax <= 448 * 2^e."""
    m, k = torch.frexp(c.abs().amax(-1))
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(m == 0, torch.zeros_like(e), e.clamp(min=-126))
    codes = (c * torch.exp2(-e.double()).float()[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _stand_for(codes, e):
    """The values e4m3 codes and their exponent bytes stand for (or a plain cache's own)."""
    if e is None:
        return codes.float()
    return codes.float() * torch.exp2(e.double() - 127).float()[..., None]


def _attn_seq(q, k, v, window, sinks, scale):
    """Attention of one sequence, heads first, 32 bits: q [H, L, d], k, v
    [H, L, d] -> p [H, L, L], o [H, L, d], lse [H, L]."""
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    n = torch.arange(k.shape[1], device=k.device)
    i, j = n[:, None], n[None, :]
    s.masked_fill_((j > i) | ((j <= i - window) & (j >= sinks)), float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(m))
    l = p.sum(-1, keepdim=True)
    p /= l
    return p, torch.matmul(p, v), (m + torch.log(l))[..., 0]


def _head_blocks(Hq, G, elems):
    """Query heads in blocks of whole-group parts whose scores fit."""
    step = max(1, min(Hq, int(2 ** 31 // max(elems, 1))))
    while step > 1 and (step > G and step % G or step <= G and G % step):
        step -= 1
    return [slice(h, min(h + step, Hq)) for h in range(0, Hq, step)]


def _sink_plain(x):
    case = x["case"]
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    G, scale, dt, shape = Hq // Hk, d ** -0.5, x["q"].dtype, x["q"].shape
    q, k, v = (x[n].reshape(-1, x[n].shape[2], d) for n in ("q", "k", "v"))
    o, lse = x["out"].reshape(-1, Hq, d), x["lse"].reshape(-1, Hq)
    if case["bwd"]:
        do = x["dout"].reshape(-1, Hq, d)
        dq = torch.empty_like(q)
        dk, dv = (torch.zeros(k.shape, dtype=torch.float32, device="cuda") for _ in range(2))
    t0 = 0
    for n in x["lens"]:
        t = slice(t0, t0 + n)
        for hs in _head_blocks(Hq, G, n * n):
            hk = torch.arange(hs.start, hs.stop, device="cuda") // G
            qf, kf, vf = (y.float().transpose(0, 1).contiguous() for y in (q[t, hs], k[t][:, hk], v[t][:, hk]))
            p, of, ls = _attn_seq(qf, kf, vf, case["window"], case["sinks"], scale)
            o[t, hs], lse[t, hs] = of.transpose(0, 1).to(dt), ls.t()
            if case["bwd"]:
                dof = do[t, hs].float().transpose(0, 1).contiguous()
                dp = torch.matmul(dof, vf.transpose(1, 2))
                dv[t].index_add_(1, hk, torch.matmul(p.transpose(1, 2), dof).transpose(0, 1))
                ds = dp.sub_((dof * of).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[t, hs] = torch.matmul(ds, kf).transpose(0, 1).to(dt)
                dk[t].index_add_(1, hk, torch.matmul(ds.transpose(1, 2), qf).transpose(0, 1))
        t0 += n
    res = (x["out"], x["lse"])
    if case["bwd"]:
        res += (dq.reshape(shape), dk.to(dt).reshape(x["k"].shape), dv.to(dt).reshape(x["k"].shape))
    return res


def _gather(x, n, table, j):
    """Keys (n = "k") or values at the places j [N, m] of the table's [N, pages] sequences: [N, m, Hk, d] in 32 bits."""
    page = x["case"]["page"]
    pg, off = torch.gather(table.long(), 1, j // page), j % page
    c, e = x[n + "_cache"], x[n + "_scale"]
    if e is None:
        return c[pg, :, off].float()
    return _stand_for(c.view(torch.uint8)[pg, :, off].view(torch.float8_e4m3fn), e[pg, :, off])


def _softmax_sum(s, v):
    """Weights of the scores s [N, Hk, rows, m] (-inf where masked) on v [N, m, Hk, d]: o [N, Hk, rows, d], lse."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p / l, v.transpose(1, 2).contiguous()), (m + torch.log(l))[..., 0]


def _paged_plain(x):
    """All sequences at once: their sinks and the keys from the first query's window on, padded to the same number."""
    case = x["case"]
    Hq, Hk, d, T, W, S = case["Hq"], case["Hk"], case["d"], case["q"], case["window"], case["sinks"]
    N, G = case["nseq"], Hq // Hk
    lk = x["seq_lens"].long()[:, None]
    first = (lk - T + 1 - W).clamp(min=S)
    j = torch.cat((torch.arange(S, device="cuda").expand(N, S), first + torch.arange(W + T - 1, device="cuda")), 1)
    there = j < lk
    j = torch.where(there, j, 0)
    k, v = _gather(x, "k", x["table"], j), _gather(x, "v", x["table"], j)
    # rows: (token, head of the group) of every kv head
    q = x["q"].float().reshape(N, T, Hk, G, d).transpose(1, 2).reshape(N, Hk, T * G, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * d ** -0.5
    pos = (lk - T + torch.arange(T, device="cuda")).repeat_interleave(G, 1)[:, None, :, None]
    j, there = j[:, None, None, :], there[:, None, None, :]
    s = s.masked_fill(~(there & (j <= pos) & ((j > pos - W) | (j < S))), float("-inf"))
    o = _softmax_sum(s, v)[0].reshape(N, Hk, T, G, d).transpose(1, 2).reshape(N, T, Hq, d)
    x["out"].copy_(o)
    return (x["out"],)


def _rotate(x, cos, sin, inter):
    """The first 2 * cos.shape[-1] channels of x [B, T, H, d] rotated."""
    h = cos.shape[-1]
    cos, sin = cos[:, :, None], sin[:, :, None]
    r, rest = x[..., :2 * h], x[..., 2 * h:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :h], r[..., h:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _split(x):
    """q, k and v, views of the projection's output."""
    Hq, Hk = x["case"]["Hq"], x["case"]["Hk"]
    return x["qkv"][:, :, :Hq], x["qkv"][:, :, Hq:Hq + Hk], x["qkv"][:, :, Hq + Hk:]


def _append_plain(x):
    case = x["case"]
    page, Hk, d = case["page"], case["Hk"], case["d"]
    ang = x["positions"].double()[..., None] * x["freqs"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def turned(y, w):
        f = y.float()
        return _rotate(f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w, cos, sin, case["inter"])

    q, k, v = _split(x)
    x["out"].copy_(turned(q, x["wq"]))
    pg, off = x["slots"] // page, x["slots"] % page
    k, v = turned(k, x["wk"]).reshape(-1, Hk, d), v.float().reshape(-1, Hk, d)
    if case["cache"] != "f8":
        x["k_cache"][pg, :, off] = k.to(x["k_cache"].dtype)
        x["v_cache"][pg, :, off] = v.to(x["v_cache"].dtype)
        return x["out"], x["k_cache"], x["v_cache"]
    back = []
    for n, y in (("k", k), ("v", v)):
        codes, byte = _quantise(y)
        c, e = x[n + "_cache"].view(torch.uint8), x[n + "_scale"]
        c[pg, :, off] = codes.view(torch.uint8)
        e[pg, :, off] = byte
        back.append(_stand_for(c[pg, :, off].view(torch.float8_e4m3fn), e[pg, :, off]).to(torch.bfloat16))
    return x["out"], back[0], back[1]


def _prefix_plain(x):
    """A group at a time: its prefix once for all rows, its sequences' own keys padded to the longest."""
    case = x["case"]
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    G, scale = Hq // Hk, d ** -0.5
    q, o, lse = x["q"].reshape(-1, Hq, d), x["out"].reshape(-1, Hq, d), x["lse"].reshape(-1, Hq)
    t0 = 0
    for m, p in enumerate(x["pre"]):
        a, b = x["cuts"][m], x["cuts"][m + 1]
        N, T, L = b - a, max(x["lq"][a:b]), max(x["lk"][a:b])
        lq, lk = _ints(x["lq"][a:b]).long()[:, None], x["seq_lens"][a:b].long()[:, None]
        R = sum(x["lq"][a:b])
        rows = slice(t0, t0 + R)
        j = torch.arange(p, device="cuda")[None]
        kp, vp = _gather(x, "k", x["prefix_table"][m:m + 1], j), _gather(x, "v", x["prefix_table"][m:m + 1], j)
        qf = q[rows].float().reshape(R, Hk, G, d).transpose(0, 1).reshape(1, Hk, R * G, d)
        op, lp = _softmax_sum(torch.matmul(qf, kp.permute(0, 2, 3, 1).contiguous()) * scale, vp)
        op, lp = op.reshape(Hk, R, G, d).transpose(0, 1), lp.reshape(Hk, R, G).transpose(0, 1)
        # the sequences' rows, padded to T tokens each (a padded row stands for the sequence's last token)
        tok = torch.arange(T, device="cuda")[None]
        real = tok < lq
        at = t0 + (torch.cumsum(lq, 0) - lq) + torch.minimum(tok, lq - 1)
        qf = q[at].float().reshape(N, T, Hk, G, d).transpose(1, 2).reshape(N, Hk, T * G, d)
        j = torch.arange(L, device="cuda").expand(N, L)
        there = torch.where(j < lk, j, 0)
        k, v = _gather(x, "k", x["table"][a:b], there), _gather(x, "v", x["table"][a:b], there)
        s = torch.matmul(qf, k.permute(0, 2, 3, 1).contiguous()) * scale
        pos = (lk - lq + torch.minimum(tok, lq - 1)).repeat_interleave(G, 1)[:, None, :, None]
        oo, lo = _softmax_sum(s.masked_fill(j[:, None, None, :] > pos, float("-inf")), v)
        oo = oo.reshape(N, Hk, T, G, d).transpose(1, 2)[real]
        lo = lo.reshape(N, Hk, T, G).transpose(1, 2)[real]
        top = torch.maximum(lp, lo)
        wp, wo = torch.exp(lp - top), torch.exp(lo - top)
        o[rows] = ((op * wp[..., None] + oo * wo[..., None]) / (wp + wo)[..., None]).reshape(R, Hq, d).to(q.dtype)
        lse[rows] = (top + torch.log(wp + wo)).reshape(R, Hq)
        t0 += R
    return x["out"], x["lse"]


# --------------------------------------------------------------- one pass --
def run(x):
    case = x["case"]
    if not own:
        return {"sink": _sink_plain, "paged": _paged_plain, "append": _append_plain, "prefix": _prefix_plain}[case["op"]](x)
    import gated_delta_rule_07_amd as g
    if case["op"] == "sink":
        kw = dict(cu_seqlens=x["cu"], window=case["window"], sinks=case["sinks"])
        res = g.attn_fwd(x["q"], x["k"], x["v"], out=x["out"], lse=x["lse"], **kw)
        if case["bwd"]:
            gr = g.attn_bwd(x["q"], x["k"], x["v"], res[0], res[1], x["dout"], workspace=x["ws"], **kw)
            res = res + (gr["dq"], gr["dk"], gr["dv"])
        return res
    if case["op"] == "paged":
        o, _ = g.attn_paged(x["q"], x["k_cache"], x["v_cache"], x["table"], x["seq_lens"], k_scale=x["k_scale"],
                            v_scale=x["v_scale"], window=case["window"], sinks=case["sinks"], out=x["out"],
                            workspace=x["ws"])
        return (o,)
    if case["op"] == "append":
        q, k, v = _split(x)
        o = g.kv_cache_append(q, k, v, x["slots"], x["k_cache"], x["v_cache"], x["freqs"], wq=x["wq"], wk=x["wk"],
                              positions=x["positions"], interleaved=case["inter"], eps=EPS, k_scale=x["k_scale"],
                              v_scale=x["v_scale"], out=x["out"])
        if case["cache"] != "f8":
            return o, x["k_cache"], x["v_cache"]
        k, v = g.kv_cache_read(x["slots"], x["k_cache"], x["v_cache"], k_scale=x["k_scale"], v_scale=x["v_scale"],
                               dtype=torch.bfloat16)
        return o, k, v
    return g.attn_paged_prefix(x["q"], x["k_cache"], x["v_cache"], x["prefix_table"], x["prefix_lens"], x["table"],
                               x["seq_lens"], cu_groups=x["groups"], cu_seqlens=x["cu"], k_scale=x["k_scale"],
                               v_scale=x["v_scale"], out=x["out"], lse=x["lse"], workspace=x["ws"])


# ---------------------------------------------------------------- 64 bits --
def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "append":
        return _exact_append(x)
    Hq, d = case["Hq"], case["d"]
    if case["op"] == "sink":
        q, k, v = (x[n].reshape(-1, x[n].shape[2], d).double() for n in ("q", "k", "v"))
        do = x["dout"].reshape(q.shape).double() if case["bwd"] else None
        parts, t0 = [], 0
        for n in x["lens"]:
            t = slice(t0, t0 + n)
            parts.append(_exact_attn(q[t], k[t], v[t], case["window"], case["sinks"], None if do is None else do[t]))
            t0 += n
        shapes = [x["q"].shape, x["q"].shape[:3], x["q"].shape, x["k"].shape, x["k"].shape]
        return tuple(torch.cat(c).reshape(s) for c, s in zip(zip(*parts), shapes))
    q = x["q"].reshape(-1, Hq, d).double()
    if case["op"] == "paged":
        T = case["q"]
        outs = [_exact_attn(q[i * T:i * T + T], _exact_rows(x, "k", x["table"][i], n), _exact_rows(x, "v", x["table"][i], n),
                            case["window"], case["sinks"])[0] for i, n in enumerate(x["lk"])]
        return (torch.cat(outs).reshape(x["q"].shape),)
    outs, t0 = [], 0
    for m, p in enumerate(x["pre"]):
        kp, vp = (_exact_rows(x, n, x["prefix_table"][m], p) for n in ("k", "v"))
        for i in range(x["cuts"][m], x["cuts"][m + 1]):
            k, v = (torch.cat((c, _exact_rows(x, n, x["table"][i], x["lk"][i]))) for n, c in (("k", kp), ("v", vp)))
            outs.append(_exact_attn(q[t0:t0 + x["lq"][i]], k, v, 0, 0))
            t0 += x["lq"][i]
    return tuple(torch.cat(c).reshape(s) for c, s in zip(zip(*outs), (x["q"].shape, x["q"].shape[:3])))


def _exact_rows(x, n, table, lk):
    """The values of a sequence's first lk rows of the cache, [lk, Hk, d]
    (rows of freed pages are zeros: nothing may see them)."""
    at = torch.arange(lk, device="cuda")
    pg, off = table.long()[at // x["case"]["page"]], at % x["case"]["page"]
    held = pg >= 0
    pg = torch.where(held, pg, 0)
    if x[n + "_scale"] is None:
        c = x[n + "_cache"][pg, :, off].double()
    else:
        c = x[n + "_cache"].view(torch.uint8)[pg, :, off].view(torch.float8_e4m3fn).double()
        c = c * torch.exp2(x[n + "_scale"][pg, :, off].double() - 127.0)[..., None]
    return torch.where(held[:, None, None], c, 0.0)


def _exact_attn(q, k, v, window, sinks, do=None):
    """The definition for one sequence, one query head and a block of rows at
    a time: scores by explicit visibility, weights exp(s) / sum exp(s) and the
    gradients of sum(o * do)."""
    (lq, Hq, d), (lk, Hk, _) = q.shape, k.shape
    G = Hq // Hk
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    key = torch.arange(lk, device=q.device)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        for r0 in range(0, lq, 8192):
            rows = slice(r0, min(r0 + 8192, lq))
            pos = torch.arange(lk - lq, lk, device=q.device)[rows]
            vis = key[None, :] <= pos[:, None]
            if window:
                vis = vis & ((key[None, :] > pos[:, None] - window) | (key[None, :] < sinks))
            s = (q[rows, h] @ kh.t()) / math.sqrt(d)
            z = torch.logsumexp(torch.where(vis, s, float("-inf")), 1)
            a = torch.where(vis, torch.exp(s - z[:, None]), 0.0)
            o[rows, h], lse[rows, h] = a @ vh, z
            if do is not None:
                gr = do[rows, h]
                da = gr @ vh.t()
                ds = a * (da - (a * da).sum(1, keepdim=True)) / math.sqrt(d)
                dv[:, h // G] += a.t() @ gr
                dk[:, h // G] += ds.t() @ q[rows, h]
                dq[rows, h] = ds @ kh
    return (o, lse) if do is None else (o, lse, dq, dk, dv)


def _exact_append(x):
    """By definition.  The scale of a quantised row is the smallest power of
    two that brings its largest value to at most 448; a value becomes its
    nearest e4m3 number (ties to even): 3 bits of fraction, exponents from -6
    up, steps of 2^-9 below."""
    case = x["case"]
    rot, d, Hk, page = case["rot"], case["d"], case["Hk"], case["page"]
    ang = x["positions"].double()[..., None] * x["freqs"]
    # the rotation of each position as complex numbers on the pairs
    turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]
    if case["inter"]:
        ia, ib = torch.arange(0, rot, 2, device="cuda"), torch.arange(1, rot, 2, device="cuda")
    else:
        ia, ib = torch.arange(0, rot // 2, device="cuda"), torch.arange(rot // 2, rot, device="cuda")

    def spin(y, w):
        y = y.double()
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    def kept(f):
        amax = f.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(amax > 0, amax, F8_MAX) / F8_MAX))
        y = f * torch.exp2(-e)
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -40))), min=-6.0) - 3.0)
        return torch.round(y / step) * step * torch.exp2(e)

    q, k, v = _split(x)
    rows = [spin(k, x["wk"]).reshape(-1, Hk, d), v.double().reshape(-1, Hk, d)]
    if case["cache"] == "f8":
        return spin(q, x["wq"]), kept(rows[0]), kept(rows[1])
    held = []
    for n, y in zip(("k", "v"), rows):
        c = torch.zeros(x[n + "_cache"].shape, dtype=torch.float64, device="cuda")
        c[x["slots"] // page, :, x["slots"] % page] = y
        held.append(c)
    return spin(q, x["wq"]), held[0], held[1]
