"""Measured cases of the paged key-value cache: appending to it, attention of one
new token over it, and eviction from it by accumulated attention weight.

A case is a dict of plain values.  Sequence lengths come from the case alone
("lo", "hi", "lens_seed"); every tensor's values, and the order of the pages,
come from the seed.  With `own` false, run() computes each operator in plain
torch operations; with `own` true it calls this repository's kernels.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a chat's first tokens, one user: latency of one call
        dict(name="attn_single_short", op="attn", N=1, H=16, H_kv=16, d=128, page=16, lo=100, hi=100,
             lens_seed=1, io="bf16", layout="NHD", window=0, weights=False),
        # a serving batch of mixed lengths, one value head per key head
        dict(name="attn_batch_ragged", op="attn", N=64, H=16, H_kv=16, d=128, page=16, lo=1, hi=8192,
             lens_seed=2, io="bf16", layout="NHD", window=0, weights=False),
        # one user with a very long document, 8 query heads to a key head
        dict(name="attn_long_grouped", op="attn", N=1, H=16, H_kv=2, d=128, page=64, lo=131071, hi=131071,
             lens_seed=3, io="bf16", layout="HND", window=0, weights=False),
        # the hybrid's sliding-window blocks in a large batch (2K window)
        dict(name="attn_window_2k", op="attn", N=128, H=16, H_kv=4, d=128, page=32, lo=1, hi=16384,
             lens_seed=4, io="bf16", layout="NHD", window=2048, weights=False),
        # float32 caches with the small head size, odd page size
        dict(name="attn_f32_d64", op="attn", N=16, H=16, H_kv=4, d=64, page=24, lo=1, hi=4097,
             lens_seed=5, io="f32", layout="NHD", window=0, weights=False),
        # attention that also adds up what each cached token received
        dict(name="attn_weights", op="attn", N=32, H=16, H_kv=4, d=128, page=16, lo=1, hi=8192,
             lens_seed=6, io="bf16", layout="NHD", window=0, weights=True),
        # one decode step's keys and values, 256 sequences x 16 heads
        dict(name="append_step", op="append", N=256, H_kv=16, d=128, page=16, lo=0, hi=127, lens_seed=7,
             new_lo=1, new_hi=1, packed=False, io="bf16", layout="NHD", weights=True),
        # prompts packed back to back (16384 tokens or so) into the pages
        dict(name="append_prompts", op="append", N=16, H_kv=16, d=128, page=16, lo=0, hi=0, lens_seed=8,
             new_lo=1, new_hi=2048, packed=True, io="bf16", layout="NHD", weights=True),
        # a small cache brought back to its budget
        dict(name="evict_small", op="evict", N=4, H_kv=4, d=64, page=16, lo=200, hi=600, lens_seed=9,
             budget=256, sink=4, recent=32, io="bf16", layout="NHD"),
        # a batch brought back from up to 8K tokens to 2K, 16 heads
        dict(name="evict_batch", op="evict", N=16, H_kv=16, d=128, page=16, lo=2048, hi=8192, lens_seed=10,
             budget=2048, sink=4, recent=256, io="bf16", layout="NHD"),
        # one very long sequence halved
        dict(name="evict_long", op="evict", N=1, H_kv=2, d=128, page=64, lo=131072, hi=131072, lens_seed=11,
             budget=65536, sink=16, recent=1024, io="bf16", layout="HND"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "evict", "evict"])
    H_kv = rng.choice([1, 2, 3, 4, 8, 16])
    d = rng.choice([32, 64, 128, 128])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    io = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, H_kv=H_kv, d=d, page=page, io=io, layout=rng.choice(["NHD", "HND"]),
             lens_seed=rng.randrange(1 << 30))
    most = 1 << 28  # elements of K that a drawn case holds at most
    if op == "attn":
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c["H"], most = H_kv * G, most // max(1, G // 4)
        c["N"] = _log(rng, 1, 256)
        c["hi"] = _log(rng, 1, max(1, min(131072, most // (c["N"] * H_kv * d))))
        c["lo"] = rng.choice([0, 1, c["hi"] // 2, c["hi"]])
        c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
        c["weights"] = rng.choice([False, False, True])
        if c["lo"] == 0 and c["hi"] <= 2:
            c["lo"] = c["hi"]
    elif op == "append":
        c["packed"] = rng.choice([False, True])
        c["N"] = _log(rng, 1, 256 if not c["packed"] else 48)
        c["new_lo"], c["new_hi"] = (0, _log(rng, 1, 2048)) if c["packed"] else (1, 1)
        c["lo"], c["hi"] = 0, _log(rng, 1, 256)
        c["weights"] = rng.choice([False, True])
    else:
        c["budget"] = _log(rng, 8, 16384)
        c["hi"] = int(c["budget"] * rng.choice([1.01, 1.25, 2.0, 4.0])) + 1
        c["lo"] = rng.choice([1, c["budget"], c["hi"]])
        c["N"] = _log(rng, 1, max(1, min(64, (most >> 2) // (c["hi"] * H_kv * d))))
        c["sink"] = min(4, c["budget"] // 4)
        c["recent"] = c["budget"] // rng.choice([2, 8, 16])
    return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])]


def _news(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["N"])]


def work(case):
    e = 4 if case["io"] == "f32" else 2
    N, H_kv, d, lens = case["N"], case["H_kv"], case["d"], _lens(case)
    if case["op"] == "attn":
        seen = sum(min(x, case["window"]) if case["window"] else x for x in lens)
        H = case["H"]
        pages = sum(-(-(min(x, case["window"]) if case["window"] else x) // case["page"]) for x in lens)
        b = seen * H_kv * 2 * d * e + 2 * N * H * d * e + 4 * N * H + 4 * pages + 4 * N
        if case["weights"]:
            b += seen * H_kv * 8
        return {"bytes": b, "flops": 4 * d * H * seen}
    if case["op"] == "append":
        T = sum(_news(case))
        return {"bytes": T * H_kv * (4 * d * e + (4 if case["weights"] else 0)) + 4 * T + 12 * N, "flops": 0}
    kept = sum(min(x, case["budget"]) for x in lens)
    over = sum(x for x in lens if x > case["budget"])
    b = kept * H_kv * (4 * d * e + 8) + over * H_kv * 4 + N * H_kv * case["budget"] * 4 + 8 * N
    return {"bytes": b, "flops": 0}


# ------------------------------------------------------------------ inputs

def _pool(g, pages, case, blank=False):
    """One cache pool, seen as [pages, slot, head, channel] whatever its layout in memory."""
    P, H_kv, d, dt = case["page"], case["H_kv"], case["d"], DTYPES[case["io"]]
    shape = (pages, H_kv, P, d) if case["layout"] == "HND" else (pages, P, H_kv, d)
    if blank:
        t = torch.zeros(shape, dtype=dt, device="cuda")
    else:
        t = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    return t.transpose(1, 2) if case["layout"] == "HND" else t


def _table(g, lens, case):
    """Pages in random order, -1 behind each sequence's last page; and their number."""
    need = [max(0, -(-x // case["page"])) for x in lens]
    pages, width = max(1, sum(need)), max(1, max(need))
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).cpu()
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for n, k in enumerate(need):
        t[n, :k] = perm[at:at + k]
        at += k
    return t.cuda(), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, H_kv, d, N = DTYPES[case["io"]], case["H_kv"], case["d"], case["N"]
    lens = _lens(case)
    s = {"case": case}
    if case["op"] == "append":
        news = _news(case)
        s["table"], pages = _table(g, [a + b for a, b in zip(lens, news)], case)
        T = sum(news)
        s["k_new"] = torch.randn(T, H_kv, d, dtype=dt, device="cuda", generator=g)
        s["v_new"] = torch.randn(T, H_kv, d, dtype=dt, device="cuda", generator=g)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda") \
            if case["packed"] else None
        s["lens_out"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    else:
        s["table"], pages = _table(g, lens, case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k"], s["v"] = _pool(g, pages, case), _pool(g, pages, case)
    s["w"] = None
    if case["op"] == "evict" or case["weights"]:
        # sums of attention weights: a few tokens hold most, new ones have none yet
        s["w"] = torch.exp(2 * torch.randn(pages, H_kv, case["page"], device="cuda", generator=g) - 4)
        s["w"] *= torch.rand(pages, H_kv, case["page"], device="cuda", generator=g) > 0.02
    if case["op"] == "attn":
        s["q"] = torch.randn(N, case["H"], d, dtype=dt, device="cuda", generator=g)
        s["scale"] = d ** -0.5
    if case["op"] == "evict":
        kept = [min(x, case["budget"]) for x in lens]
        s["table2"], pages2 = _table(g, kept, case)
        s["k2"], s["v2"] = _pool(g, pages2, case, True), _pool(g, pages2, case, True)
        s["w2"] = torch.zeros(pages2, H_kv, case["page"], device="cuda")
        s["lens2"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    if own:  # the handle that a program makes once for its cache
        import gated_delta_rule_128_b200 as gdn
        s["kv"] = gdn.PagedKV(s["k"], s["v"], s["table"], s["lens"], s["w"])
        if case["op"] == "evict":
            s["kv2"] = gdn.PagedKV(s["k2"], s["v2"], s["table2"], s["lens2"], s["w2"])
    return s


# -------------------------------------------------------------- plain forms

def _gather(pool, table, at):
    """Rows of `pool` ([page, slot, ...]) at positions at [N, L] of each sequence; positions
    without a page read page 0 (the caller masks them)."""
    P = pool.shape[1]
    page = table.long().gather(1, (at // P).clamp(0, table.shape[1] - 1)).clamp_min(0)
    return pool[page, at % P]


def _plain_attn(s):
    c, q, lens, table = s["case"], s["q"], s["lens"].long(), s["table"]
    N, H, d = q.shape
    H_kv, P = c["H_kv"], c["page"]
    L = table.shape[1] * P
    first = (lens - c["window"]).clamp_min(0) if c["window"] else torch.zeros_like(lens)
    span = min(L, c["window"]) if c["window"] else L
    at = first[:, None] + torch.arange(span, device=q.device)[None]          # [N, span]
    seen = at < lens[:, None]
    k = _gather(s["k"], table, at).float()                                   # [N, span, H_kv, d]
    v = _gather(s["v"], table, at).float()
    qg = q.float().view(N, H_kv, H // H_kv, d)
    sc = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]                # [N, H_kv, G, span]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    e = torch.exp(sc - m)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(N, H, d).to(q.dtype)
    out = {"o": o, "lse": (m + torch.log(total)).reshape(N, H)}
    if c["weights"]:
        slot = at % P
        page = table.long().gather(1, (at // P).clamp(0, table.shape[1] - 1))
        n, j = torch.nonzero(seen, as_tuple=True)
        s["w"][page[n, j], :, slot[n, j]] += p.sum(2)[n, :, j]
        out["w"] = s["w"]
    return out


def _plain_append(s):
    c, lens, table, P = s["case"], s["lens"].long(), s["table"], s["case"]["page"]
    T = s["k_new"].shape[0]
    i = torch.arange(T, device=lens.device)
    if s["cu"] is None:
        n, at, count = i, lens, 1
    else:
        n = torch.searchsorted(s["cu"][1:].long(), i, right=True)
        at, count = lens[n] + i - s["cu"].long()[n], (s["cu"][1:] - s["cu"][:-1]).long()
    page, slot = table.long()[n, at // P], at % P
    s["k"][page, slot] = s["k_new"]
    s["v"][page, slot] = s["v_new"]
    if c["weights"]:
        s["w"][page, :, slot] = 0
    s["lens_out"].copy_(lens + count)
    out = {"k": s["k"], "v": s["v"], "lens": s["lens_out"]}
    if c["weights"]:
        out["w"] = s["w"]
    return out


def _plain_evict(s):
    c, lens, table, P = s["case"], s["lens"].long(), s["table"], s["case"]["page"]
    N, H_kv, budget = c["N"], c["H_kv"], c["budget"]
    L = table.shape[1] * P
    at = torch.arange(L, device=lens.device)[None].expand(N, L)
    w = _gather(s["w"].transpose(1, 2), table, at).permute(0, 2, 1)          # [N, H_kv, L]
    inside = (at < lens[:, None])[:, None]
    fixed = ((at < c["sink"]) | (at >= lens[:, None] - c["recent"]))[:, None]
    rank = torch.where(fixed, torch.full_like(w, math.inf), w)
    rank = torch.where(inside, rank, torch.full_like(w, -math.inf))
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.sort(kept, dim=-1).values                                   # [N, H_kv, <= budget]
    if kept.shape[-1] < budget:
        kept = torch.cat([kept, kept.new_zeros(N, H_kv, budget - kept.shape[-1])], -1)
    to = torch.arange(budget, device=lens.device)
    short = (lens <= budget)[:, None, None]
    kept = torch.where(short, to.expand_as(kept), kept)
    valid = to[None] < lens[:, None]                                         # [N, budget]
    n, j = torch.nonzero(valid, as_tuple=True)
    page2, slot2 = s["table2"].long()[n, j // P], j % P
    src = kept[n, :, j]                                                      # [rows, H_kv]
    page, slot = table.long()[n[:, None], src // P], src % P
    h = torch.arange(H_kv, device=lens.device)[None]
    s["k2"][page2, slot2] = s["k"][page, slot, h]
    s["v2"][page2, slot2] = s["v"][page, slot, h]
    s["w2"][page2, :, slot2] = s["w"][page, h, slot]
    s["lens2"].copy_(lens.clamp_max(budget))
    kept = torch.where(valid[:, None], kept, torch.full_like(kept, -1)).to(torch.int32)
    return {"k": s["k2"], "v": s["v2"], "w": s["w2"], "lens": s["lens2"], "kept": kept}


def run(s):
    c = s["case"]
    if own:
        import gated_delta_rule_128_b200 as gdn
        if c["op"] == "attn":
            o, lse = gdn.attn_decode_step(s["q"], s["kv"], scale=s["scale"], window=c["window"],
                                          add_weights=c["weights"], want_lse=True)
            return {"o": o, "lse": lse, "w": s["w"]} if c["weights"] else {"o": o, "lse": lse}
        if c["op"] == "append":
            gdn.kv_append(s["kv"], s["k_new"], s["v_new"], cu_seqlens=s["cu"], lens_out=s["lens_out"])
            out = {"k": s["k"], "v": s["v"], "lens": s["lens_out"]}
            return {**out, "w": s["w"]} if c["weights"] else out
        kept = gdn.kv_evict(s["kv"], c["budget"], sink=c["sink"], recent=c["recent"], dst=s["kv2"],
                            want_kept=True)
        return {"k": s["k2"], "v": s["v2"], "w": s["w2"], "lens": s["lens2"], "kept": kept}
    return {"attn": _plain_attn, "append": _plain_append, "evict": _plain_evict}[c["op"]](s)


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What run() returns on a fresh state, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    P, lens, table = case["page"], _lens(case), s["table"].cpu().numpy()

    def rows(n, idx):
        return (torch.from_numpy(table[n, idx // P].astype(np.int64)).cuda(),
                torch.from_numpy(idx % P).cuda())

    if case["op"] == "attn":
        N, H, d = s["q"].shape
        G = H // case["H_kv"]
        o = torch.zeros(N, H, d, dtype=torch.float64, device="cuda")
        lse = torch.full((N, H), -math.inf, dtype=torch.float64, device="cuda")
        w = s["w"].double() if case["weights"] else None
        for n, x in enumerate(lens):
            lo = max(0, x - case["window"]) if case["window"] else 0
            if x == 0:
                continue
            page, slot = rows(n, np.arange(lo, x))
            for h in range(case["H_kv"]):
                k, v = s["k"][page, slot, h].double(), s["v"][page, slot, h].double()
                z = s["q"][n, h * G:(h + 1) * G].double() @ k.T * s["scale"]
                lse[n, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                o[n, h * G:(h + 1) * G] = p @ v
                if w is not None:
                    w[page, h, slot] += p.sum(0)
        return {"o": o, "lse": lse, "w": w} if w is not None else {"o": o, "lse": lse}
    if case["op"] == "append":
        k, v, w = s["k"].double(), s["v"].double(), s["w"].double() if case["weights"] else None
        at = 0
        for n, (x, y) in enumerate(zip(lens, _news(case))):
            page, slot = rows(n, np.arange(x, x + y))
            k[page, slot], v[page, slot] = s["k_new"][at:at + y].double(), s["v_new"][at:at + y].double()
            if w is not None:
                w[page, :, slot] = 0
            at += y
        return {"k": k, "v": v, "lens": None, "w": w} if w is not None else {"k": k, "v": v, "lens": None}
    k2, v2, w2 = s["k2"].double(), s["v2"].double(), s["w2"].double()
    table2, wh, budget = s["table2"].cpu().numpy(), s["w"].cpu().numpy(), case["budget"]
    for n, x in enumerate(lens):
        new = np.arange(min(x, budget))
        p2 = torch.from_numpy(table2[n, new // P].astype(np.int64)).cuda()
        s2 = torch.from_numpy(new % P).cuda()
        for h in range(case["H_kv"]):
            old = np.arange(x)
            if x > budget:
                first, last = case["sink"], x - case["recent"]
                mid = np.arange(first, last)
                weight = wh[table[n, mid // P], h, mid % P]
                best = mid[np.lexsort((mid, -weight))[:budget - case["sink"] - case["recent"]]]
                old = np.concatenate([np.arange(first), np.sort(best), np.arange(last, x)])
            page, slot = rows(n, old)
            k2[p2, s2, h], v2[p2, s2, h] = s["k"][page, slot, h].double(), s["v"][page, slot, h].double()
            w2[p2, h, s2] = s["w"][page, h, slot].double()
    return {"k": k2, "v": v2, "w": w2, "lens": None, "kept": None}
