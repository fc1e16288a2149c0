"""Helpers of the paged-cache tests: a cache on the GPU, the same in fp64, and
the error bounds of one-token attention."""

import numpy as np
import torch

import gated_delta_rule_128_b200 as gdn

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def cache(lens, page, H_kv, d, io, seed, *, layout="NHD", spare=2, room=0, fill=None, device="cuda"):
    """(PagedKV, the fp64 dict of oracle.paged).  Pages are shuffled; `room` more tokens a
    sequence have pages; slots that hold no token are `fill` (NaN where it says so)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(x + room) // page) for x in lens]
    width, pages = max(1, max(need)), sum(need) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    at = 0
    for n, y in enumerate(need):
        table[n, :y] = perm[at:at + y]
        at += y
    k = torch.randn(pages, page, H_kv, d, generator=g).to(DT[io])
    v = torch.randn(pages, page, H_kv, d, generator=g).to(DT[io])
    w = torch.rand(pages, H_kv, page, generator=g)
    if fill is not None:
        used = torch.zeros(pages, page, dtype=torch.bool)
        for n, x in enumerate(lens):
            for j in range(x):
                used[table[n, j // page], j % page] = True
        k[~used], v[~used] = fill, fill
        w.transpose(1, 2)[~used] = fill
    kv = on_gpu(k, v, w, table, lens, layout, device)
    return kv, dict(k=k.double().numpy(), v=v.double().numpy(), w=w.double().numpy(), table=table.numpy().copy(),
                    lens=np.array(lens))


def on_gpu(k, v, w, table, lens, layout, device="cuda"):
    def place(t):
        if layout == "HND":      # heads before slots
            return t.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        if layout == "padded":   # rows and pages further apart than they need be
            P, S, H, d = t.shape
            big = torch.full((P, S + 1, H + 2, d + 8), float("nan"), dtype=t.dtype, device=device)
            big[:, :S, :H, :d] = t.to(device)
            return big[:, :S, :H, :d]
        return t.to(device)
    if layout == "interleaved":  # one pool [pages, 2, slots, heads, d]
        both = torch.stack([k, v], 1).to(device)
        kd, vd = both[:, 0], both[:, 1]
    else:
        kd, vd = place(k), place(v)
    return gdn.PagedKV(kd, vd, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device),
                       w.to(device))


def host(kv):
    """The cache's present contents as the fp64 dict."""
    return dict(k=kv.k.double().cpu().numpy(), v=kv.v.double().cpu().numpy(), w=kv.weights.double().cpu().numpy(),
                table=kv.block_table.cpu().numpy(), lens=kv.seq_lens.cpu().numpy().astype(np.int64))


def bounds(io, o, lse, a, smax, length, d):
    """Elementwise bounds on |o - ref| and |lse - ref|, and the relative one on a softmax weight.

    Scores: a dot of d float32 products and sums, in any order, is off by at most d 2^-24 of
    sum |q_i k_i| times 1 + small (doubled for the tensor cores' truncating sums), and the
    multiplications by scale and log2 e by 2^-23 of |s|: ds below, smax being the largest sum.
    A softmax weight before normalisation, e^(s - m): m is one of the computed scores, so the
    exponent is off by 2 ds, and e^x itself by 2^-21 (exp2 and the subtraction's rounding are
    relative to the exponent, again within ds).  Sums over the tokens: `length` 2^-24, twice
    (numerator and denominator), and the rescalings and joins 64 2^-24.  bf16 takes
    each weight in two parts, the second rounded (2^-8 of the at most 2^-8 that the first
    leaves), and rounds the result (2^-8 |o|)."""
    ds = (2 * d * 2.0 ** -24 + 2.0 ** -22) * smax
    p = 4 * ds + 2 * 2.0 ** -21 + (2 * length + 64) * 2.0 ** -24
    half = 2.0 ** -8 if io == "bf16" else 2.0 ** -24
    b = (p[..., None] + (2.0 ** -16 if io == "bf16" else 0.0)) * a * (1 + 2.0 ** -7) + half * np.abs(o) * (1 + 2.0 ** -7)
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return b + 1e-30, 2 * ds + 2.0 ** -21 + (length + 64) * 2.0 ** -24 + 2.0 ** -23 * (1 + fin), p
