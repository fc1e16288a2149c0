"""The paged-cache kernels against the fp64 oracle on the GPU."""

import numpy as np
import pytest
import torch

import gated_delta_rule_128_b200 as gdn
from gated_delta_rule_128_b200 import workloads
from _paged import DT, bounds, cache, host, on_gpu
from oracle import paged

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.lib()


@pytest.fixture(autouse=True)
def _status():
    gdn.gdn2_get_device_status()
    yield
    torch.cuda.synchronize()


def query(N, H, d, io, seed, mul=1.0):
    q = (torch.randn(N, H, d, generator=torch.Generator().manual_seed(seed)) * mul).to(DT[io])
    return q.cuda(), q.double().numpy()


def same(a, b):
    """Equal, NaN equal to NaN."""
    return np.array_equal(a, b, equal_nan=True)


def check(kv, c, q, q64, io, scale, window=0, add=False, status=0):
    o, lse = gdn.attn_decode_step(q, kv, scale=scale, window=window, add_weights=add, want_lse=True)
    assert gdn.gdn2_get_device_status() == status
    w0 = c["w"].copy()
    r, rl, a, smax = paged.attention(c, q64, scale, window, add)
    longest = max([paged.length(c, n) for n in range(len(c["lens"]))] + [1])
    bo, bl, bp = bounds(io, r, rl, a, smax, longest, q64.shape[2])
    err = np.abs(o.double().cpu().numpy() - r)
    assert (err <= bo).all(), float((err / bo).max())
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert (np.abs(got[fin] - rl[fin]) <= bl[fin]).all()
    if add:
        w = kv.weights.double().cpu().numpy()
        fin = np.isfinite(c["w"])
        added = c["w"] - w0
        G = q64.shape[1] // c["k"].shape[2]
        lim = bp.max() * added + (G + 2) * 2.0 ** -24 * np.abs(c["w"]) + 1e-30
        assert (np.abs(w - c["w"])[fin] <= lim[fin]).all()
        assert np.array_equal(np.isnan(w), np.isnan(c["w"]))
    return o, lse


LENS = [0, 1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H_kv,G", [(1, 1), (3, 2), (2, 7), (2, 8), (1, 9), (1, 16), (2, 17), (1, 40), (33, 3)])
def test_attention_heads_and_sizes(io, d, H_kv, G):
    kv, c = cache(LENS, 16, H_kv, d, io, d + G, fill=NAN)
    q, q64 = query(len(LENS), H_kv * G, d, io, 5)
    check(kv, c, q, q64, io, d ** -0.5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 5, 8, 24, 64, 100, 512])
@pytest.mark.parametrize("layout", ["NHD", "HND", "padded", "interleaved"])
def test_attention_pages_and_layouts(io, page, layout):
    lens = [130, 0, 7, 100, 101]
    kv, c = cache(lens, page, 2, 64, io, page, layout=layout, fill=NAN)
    q, q64 = query(len(lens), 6, 64, io, 6)
    check(kv, c, q, q64, io, 0.125, add=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 199, 200, 100000])
@pytest.mark.parametrize("add", [False, True])
def test_attention_window(io, window, add):
    """Tokens before the window (NaN here) are not looked at."""
    kv, c = cache(LENS, 24, 2, 64, io, window)
    for n, x in enumerate(LENS):
        for j in range(max(0, x - window)):
            p, s = paged.place(c, n, j)
            kv.k[p, s], kv.v[p, s], c["k"][p, s], c["v"][p, s] = NAN, NAN, NAN, NAN
    q, q64 = query(len(LENS), 8, 64, io, 7)
    check(kv, c, q, q64, io, 0.125, window, add)


@pytest.mark.parametrize("io,N,H_kv,G,d,lens", [
    ("bf16", 1, 1, 4, 128, (9001,)), ("bf16", 1, 2, 8, 64, (20011,)), ("f32", 1, 1, 3, 128, (7003,)),
    ("bf16", 3, 2, 1, 32, (12000, 1, 333)), ("f32", 4, 2, 16, 32, (0, 5000, 0, 2)),
    ("bf16", 2, 1, 33, 128, (4097, 6000)), ("bf16", 2, 1, 256, 32, (600, 70)), ("f32", 1, 2, 100, 64, (900,)),
])
@pytest.mark.parametrize("add", [False, True])
def test_attention_long_caches_are_split_and_joined(io, N, H_kv, G, d, lens, add):
    kv, c = cache(list(lens), 16, H_kv, d, io, N + G, fill=NAN)
    q, q64 = query(N, H_kv * G, d, io, 8)
    check(kv, c, q, q64, io, d ** -0.5, 0, add)


@pytest.mark.parametrize("width", [1, 100])
@pytest.mark.parametrize("add", [False, True])
def test_attention_of_empty_sequences_only(width, add):
    kv, c = cache([0] * 5, 16, 2, 64, "bf16", 24, fill=NAN)
    kv = gdn.PagedKV(kv.k, kv.v, torch.full((5, width), -1, dtype=torch.int32, device="cuda"), kv.seq_lens, kv.weights)
    q, _ = query(5, 4, 64, "bf16", 25)
    o, lse = gdn.attn_decode_step(q, kv, add_weights=add, want_lse=True, o=torch.full_like(q, NAN))
    assert (o == 0).all() and torch.isneginf(lse).all() and torch.isnan(kv.weights).all()
    assert gdn.gdn2_get_device_status() == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_many_sequences(io):
    """More sequences than blocks and than one pass of a block's threads over the lengths."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 1500)]
    kv, c = cache(lens, 8, 1, 32, io, 21, fill=NAN)
    q, q64 = query(len(lens), 2, 32, io, 9)
    check(kv, c, q, q64, io, 0.2, 0, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_large_scores(io):
    """Scores of several hundred either way: the softmax is nearly one-hot, e^s alone would
    overflow, and a maximum late in the cache rescales what came before."""
    kv, c = cache([700, 3, 1], 16, 2, 64, io, 11, fill=NAN)
    q, q64 = query(3, 8, 64, io, 10, 8.0)
    check(kv, c, q, q64, io, 2.0, 0, True)
    check(kv, c, q, q64, io, -2.0)
    check(kv, c, q, q64, io, 0.0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_infinite_scores(io):
    """Keys of -inf leave their tokens out, all of them an empty sequence."""
    kv, c = cache([70, 40], 16, 1, 32, io, 12)
    q = torch.ones(2, 2, 32).to(DT[io])
    for n, which in ((0, range(0, 70, 3)), (1, range(40))):
        for j in which:
            p, s = paged.place(c, n, j)
            kv.k[p, s, 0, 0], c["k"][p, s, 0, 0] = float("-inf"), float("-inf")
    r, rl, a, _ = paged.attention(c, q.double().numpy(), 0.1)
    o, lse = gdn.attn_decode_step(q.cuda(), kv, scale=0.1, add_weights=True, want_lse=True)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    got = o.double().cpu().numpy()
    # rounding o, and 1e-4 of sum p |v| for scores of at most sum |q k| / 10 < 20
    assert (np.abs(got - r) <= (2.0 ** -8 if io == "bf16" else 0) * np.abs(r) * 1.01 + 1e-4 * a + 1e-30).all()
    assert torch.isfinite(kv.weights).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_nan_stays_in_its_sequence(io):
    kv, c = cache([50, 50, 50], 16, 2, 32, io, 13)
    p, s = paged.place(c, 1, 20)
    kv.k[p, s, 1, 3] = NAN
    q, _ = query(3, 4, 32, io, 11)
    o, lse = gdn.attn_decode_step(q, kv, want_lse=True)
    assert torch.isnan(o[1, 2:]).all() and torch.isnan(lse[1, 2:]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all() and torch.isfinite(o[1, :2]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
def test_attention_bad_pages_and_lengths(io, add):
    """A page outside the pool is left out, a length outside the table is an empty sequence;
    both are reported, and the other sequences are right."""
    lens = [100, 60, 33, 5]
    kv, c = cache(lens, 16, 2, 64, io, 14, fill=NAN)
    for t in (c["table"], kv.block_table):
        t[0, 2], t[0, 6], t[1, 0] = -1, c["k"].shape[0], 2 ** 31 - 1
    for t in (c["lens"], kv.seq_lens):
        t[2], t[3] = -4, 16 * c["table"].shape[1] + 1
    q, q64 = query(4, 4, 64, io, 12)
    check(kv, c, q, q64, io, 0.125, 0, add, status=1)


def test_attention_repeats_bit_for_bit_and_leaves_the_cache():
    kv, c = cache([3000, 1, 700], 16, 2, 128, "bf16", 15)
    q, _ = query(3, 16, 128, "bf16", 13)
    k0, v0 = kv.k.clone(), kv.v.clone()
    a = gdn.attn_decode_step(q, kv, want_lse=True)
    b = gdn.attn_decode_step(q, kv, want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(k0, kv.k) and torch.equal(v0, kv.v)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_shared_pages_collect_every_sequences_weight(io):
    kv, c = cache([48, 48, 20], 16, 2, 32, io, 16)
    for t in (kv.block_table, c["table"]):
        t[1, :2] = t[0, :2]
    q, q64 = query(3, 4, 32, io, 14)
    check(kv, c, q, q64, io, 0.2, 0, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(32, 1), (64, 5), (128, 20)])
def test_a_long_prompt_shared_by_many_sequences(io, d, G):
    """Together the sequences hold many times the tokens of the pool."""
    N, lens = 30, 300
    kv, c = cache([lens], 16, 2, d, io, 17, spare=0, fill=NAN)
    table = np.repeat(c["table"], N, 0)
    kv = gdn.PagedKV(kv.k, kv.v, torch.tensor(table, dtype=torch.int32).cuda(),
                     torch.full((N,), lens, dtype=torch.int32, device="cuda"), kv.weights)
    c["table"], c["lens"] = table, np.full(N, lens)
    q, q64 = query(N, 2 * G, d, io, 18)
    check(kv, c, q, q64, io, d ** -0.5, 0, True)


def test_a_wide_table_needs_no_more_workspace_than_the_pool():
    kv, _ = cache([100, 30], 16, 2, 64, "bf16", 19)
    wide = torch.zeros(2, 1 << 16, dtype=torch.int32, device="cuda")
    wide[:, :kv.block_table.shape[1]] = kv.block_table
    big = gdn.PagedKV(kv.k, kv.v, wide, kv.seq_lens, kv.weights.clone())
    assert gdn.gdn2_attn_decode_workspace_bytes(big, 8, True) < 32 << 20
    q, _ = query(2, 8, 64, "bf16", 20)
    a, b = (gdn.attn_decode_step(q, x, add_weights=True, want_lse=True) for x in (kv, big))
    # the narrow table takes each head in one block, the wide one in parts
    assert torch.allclose(a[0].float(), b[0].float(), rtol=2 ** -7, atol=2 ** -8)
    assert torch.allclose(a[1], b[1], rtol=0, atol=1e-5)
    assert torch.allclose(kv.weights, big.weights, rtol=1e-5, atol=1e-6)


def test_attention_takes_the_callers_buffers():
    kv, _ = cache([2000, 3], 16, 2, 64, "bf16", 22)
    q, _ = query(2, 8, 64, "bf16", 23)
    n = kv.workspace_bytes("gdn2_attn_decode_workspace_bytes", 8, False)
    ws, o = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.full_like(q, NAN)
    a = gdn.attn_decode_step(q, kv)[0]
    b, lse = gdn.attn_decode_step(q, kv, o=o, ws=ws)
    assert b is o and lse is None and torch.equal(a, b)
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.attn_decode_step(q, kv, ws=ws[:n - 256])
    assert e.value.status == 3
    with pytest.raises(ValueError):
        gdn.attn_decode_step(q, kv, o=torch.empty(2, 8, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        gdn.attn_decode_step(q, kv, ws=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn.attn_decode_step(q.cpu(), kv)
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.attn_decode_step(q, gdn.PagedKV(kv.k, kv.v, kv.block_table, kv.seq_lens), add_weights=True)
    assert e.value.status == 1


# ----------------------------------------------------------------------- append

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,H_kv,page,layout", [(32, 1, 1, "NHD"), (64, 3, 24, "HND"), (128, 16, 16, "padded"),
                                                (128, 2, 7, "interleaved")])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_one_token(io, d, H_kv, page, layout, in_place):
    lens = [0, 1, page - 1, page, 3 * page, 40]
    kv, c = cache(lens, page, H_kv, d, io, 30 + d, layout=layout, room=1)
    k, v = (torch.randn(6, H_kv, d, generator=torch.Generator().manual_seed(x)).to(DT[io]) for x in (1, 2))
    out = None if in_place else torch.full((6,), -3, dtype=torch.int32, device="cuda")
    gdn.kv_append(kv, k.cuda(), v.cuda(), lens_out=out)
    assert gdn.gdn2_get_device_status() == 0
    assert list((kv.seq_lens if in_place else out).cpu()) == [x + 1 for x in lens]
    if not in_place:
        assert list(kv.seq_lens.cpu()) == lens
    paged.append(c, k.double().numpy(), v.double().numpy())
    h = host(kv)
    assert all(same(h[x], c[x]) for x in ("k", "v", "w"))   # every other slot as it was


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("news", [[3, 0, 41, 1, 0, 100], [0, 0, 0, 0, 0, 0], [1, 1, 1, 1, 1, 1], [0, 0, 0, 0, 0, 1900]])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_packed(io, news, in_place):
    lens = [5, 0, 17, 16, 3, 1]
    kv, c = cache(lens, 16, 2, 64, io, 31, room=max(news))
    T = sum(news)
    k, v = (torch.randn(T, 2, 64, generator=torch.Generator().manual_seed(x)).to(DT[io]) for x in (3, 4))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32)
    out = None if in_place else torch.zeros(6, dtype=torch.int32, device="cuda")
    gdn.kv_append(kv, k.cuda(), v.cuda(), cu_seqlens=cu.cuda(), lens_out=out)
    assert gdn.gdn2_get_device_status() == 0
    assert list((kv.seq_lens if in_place else out).cpu()) == [x + y for x, y in zip(lens, news)]
    paged.append(c, k.double().numpy(), v.double().numpy(), cu.tolist())
    h = host(kv)
    assert all(same(h[x], c[x]) for x in ("k", "v", "w"))


def test_append_what_does_not_fit_or_has_no_page():
    lens = [16, 31, 32, -1, 2 ** 31 - 1]
    kv, c = cache([16, 31, 32, 0, 0], 16, 2, 32, "f32", 32)
    kv.block_table[0, 1] = 10 ** 6
    kv.block_table[1, 1] = -2
    c["table"][0, 1], c["table"][1, 1] = 10 ** 6, -2
    kv.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c["lens"][:] = lens
    k = torch.ones(5, 2, 32)
    paged.append(c, k.double().numpy(), k.double().numpy())
    gdn.kv_append(kv, k.cuda(), k.cuda())
    assert gdn.gdn2_get_device_status() == 1
    h = host(kv)
    assert all(same(h[x], c[x]) for x in ("k", "v", "w", "lens"))
    # a table that does not rise appends nothing
    cu = torch.tensor([0, 3, 2, 4, 4, 5], dtype=torch.int32, device="cuda")
    gdn.kv_append(kv, k.cuda(), k.cuda(), cu_seqlens=cu)
    assert gdn.gdn2_get_device_status() == 1
    h = host(kv)
    assert all(same(h[x], c[x]) for x in ("k", "v", "w", "lens"))


# ------------------------------------------------------------------------ evict

def weighted(kv, c, kind, seed):
    w = torch.rand(kv.weights.shape, generator=torch.Generator().manual_seed(seed))
    if kind == "ties":
        w = torch.floor(w * 4)
    elif kind == "equal":
        w = torch.ones_like(w)
    elif kind == "special":
        pick = torch.tensor([NAN, float("inf"), float("-inf"), 0.0, -0.0, 1e-40, -1e-40, 3e38, -3e38, 1.0, -1.0])
        w = pick[(w * len(pick)).long().clamp_max(len(pick) - 1)]
    elif kind == "close":   # neighbours in float32
        w = (torch.ones_like(w).view(torch.int32) + (w * 7).int()).view(torch.float32)
    kv.weights.copy_(w)
    c["w"][:] = w.double().numpy()


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special", "close"])
@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (40, 0, 0), (40, 4, 8), (40, 40, 0), (40, 0, 40), (40, 10, 30),
                                                (64, 1, 0), (300, 0, 1)])
def test_evict(kind, into, budget, sink, recent):
    lens = [0, 1, 39, 40, 41, 64, 65, 300, 301]
    io, d = ("bf16", 64) if budget != 64 else ("f32", 128)
    kv, c = cache(lens, 16, 2, d, io, 40, fill=NAN)
    weighted(kv, c, kind, 1)
    dst = c2 = None
    if into:   # another page size and layout
        dst, c2 = cache([min(x, budget) for x in lens], 5, 2, d, io, 41, layout="HND")
        dst.seq_lens.fill_(-9)
        before = host(kv)
    ref = paged.evict(c, budget, sink, recent, c2)
    kept = gdn.kv_evict(kv, budget, sink=sink, recent=recent, dst=dst, want_kept=True)
    assert gdn.gdn2_get_device_status() == 0
    assert np.array_equal(kept.cpu().numpy(), ref)
    h = host(dst if into else kv)
    want = c2 if into else c
    assert all(same(h[x], want[x]) for x in ("k", "v", "w", "lens"))   # other slots as they were
    if into:
        h = host(kv)
        assert all(same(h[x], before[x]) for x in ("k", "v", "w", "lens"))


@pytest.mark.parametrize("io,d,H_kv,page,layout", [("bf16", 32, 1, 1, "NHD"), ("bf16", 128, 3, 24, "padded"),
                                                   ("f32", 32, 4, 64, "interleaved"), ("f32", 128, 1, 7, "HND")])
@pytest.mark.parametrize("into", [False, True])
def test_evict_larger(io, d, H_kv, page, layout, into):
    lens = [2500, 5, 4096, 3999]
    kv, c = cache(lens, page, H_kv, d, io, 42, layout=layout)
    weighted(kv, c, "ties", 2)
    dst, c2 = cache([min(x, 1999) for x in lens], page, H_kv, d, io, 43, layout=layout) if into else (None, None)
    ref = paged.evict(c, 1999, 3, 100, c2)
    kept = gdn.kv_evict(kv, 1999, sink=3, recent=100, dst=dst, want_kept=True)
    assert np.array_equal(kept.cpu().numpy(), ref)
    h, want = host(dst if into else kv), c2 if into else c
    assert all(same(h[x], want[x]) for x in ("k", "v", "w", "lens"))
    assert gdn.kv_evict(kv, 10 ** 4, dst=None) is None     # within the budget: nothing changes
    assert list(kv.seq_lens.cpu()) == (lens if into else list(c["lens"]))


@pytest.mark.parametrize("length,budget", [(60000, 30000), (120001, 119999)])
def test_evict_very_long(length, budget):
    kv, c = cache([length], 64, 1, 32, "bf16", 44)
    weighted(kv, c, "random", 3)
    w = np.array([c["w"][paged.place(c, 0, j)[0], 0, paged.place(c, 0, j)[1]] for j in range(length)])
    k0 = c["k"].copy()
    kept = gdn.kv_evict(kv, budget, sink=2, recent=64, want_kept=True)[0, 0].cpu().numpy()
    mid = np.arange(2, length - 64)
    best = mid[np.lexsort((mid, -w[mid]))[:budget - 66]]
    assert np.array_equal(kept, np.concatenate([[0, 1], np.sort(best), np.arange(length - 64, length)]))
    h = host(kv)
    P = 64
    new = np.arange(budget)
    assert np.array_equal(h["k"][c["table"][0, new // P], new % P, 0], k0[c["table"][0, kept // P], kept % P, 0])


@pytest.mark.parametrize("lens,budget,H_kv,page", [([20000, 19000, 1], 18990, 3, 16), ([9000] * 5, 4500, 4, 64),
                                                   ([30000], 29999, 1, 7), ([3000] * 40, 100, 8, 32)])
def test_evict_in_place_agrees_with_another_cache(lens, budget, H_kv, page):
    """Many blocks shift rows at once, down to one row a token: what they read must not have
    been written over."""
    for seed in range(3):
        kv, _ = cache_on_gpu(lens, page, H_kv, 128, 70 + seed)
        dst, _ = cache_on_gpu([min(x, budget) for x in lens], page, H_kv, 128, 80 + seed)
        a = gdn.kv_evict(kv, budget, sink=2, recent=3, dst=dst, want_kept=True)
        b = gdn.kv_evict(kv, budget, sink=2, recent=3, want_kept=True)
        assert gdn.gdn2_get_device_status() == 0
        assert torch.equal(a, b) and torch.equal(kv.seq_lens, dst.seq_lens)
        for n, x in enumerate(lens):
            j = torch.arange(min(x, budget), device="cuda")
            p, p2 = kv.block_table[n, j // page].long(), dst.block_table[n, j // page].long()
            assert torch.equal(kv.k[p, j % page], dst.k[p2, j % page])
            assert torch.equal(kv.v[p, j % page], dst.v[p2, j % page])
            assert torch.equal(kv.weights[p, :, j % page], dst.weights[p2, :, j % page])


def cache_on_gpu(lens, page, H_kv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // page) for x in lens]
    perm = torch.randperm(sum(need), device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for n, y in enumerate(need):
        table[n, :y] = perm[at:at + y]
        at += y
    k, v = (torch.randn(sum(need), page, H_kv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(sum(need), H_kv, page, device="cuda", generator=g)
    return gdn.PagedKV(k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), w), None


def test_evict_into_other_pages_of_the_same_pool():
    """Two sequences that share their prompt's pages, evicted into pages of their own."""
    kv, c = cache([64, 64, 0], 16, 2, 32, "f32", 49, room=32)
    for t in (kv.block_table, c["table"]):
        t[1, :4] = t[0, :4]
    free = sorted(set(range(c["k"].shape[0])) - set(c["table"][:2, :4].ravel().tolist()))
    dst_table = torch.tensor([free[:2], free[2:4], free[4:6]], dtype=torch.int32, device="cuda")
    dst = gdn.PagedKV(kv.k, kv.v, dst_table, torch.zeros(3, dtype=torch.int32, device="cuda"), kv.weights)
    c2 = dict(c, table=dst_table.cpu().numpy(), lens=np.zeros(3, dtype=np.int64))
    weighted(kv, c, "random", 5)
    ref = paged.evict(c, 20, 2, 3, c2)
    kept = gdn.kv_evict(kv, 20, sink=2, recent=3, dst=dst, want_kept=True)
    assert np.array_equal(kept.cpu().numpy(), ref)
    h = host(dst)
    assert all(same(h[x], c2[x]) for x in ("k", "v", "w", "lens"))


def test_evict_with_a_budget_beyond_the_table():
    kv, c = cache([50, 20], 16, 1, 32, "f32", 53)
    dst, c2 = cache([50, 20], 16, 1, 32, "f32", 54)
    before = host(kv)
    assert torch.equal(gdn.kv_evict(kv, 70, want_kept=True)[1, 0, :22].cpu(), torch.tensor(list(range(20)) + [-1, -1], dtype=torch.int32))
    h = host(kv)
    assert all(same(h[x], before[x]) for x in ("k", "v", "w", "lens"))
    paged.evict(c, 10 ** 5, 7, 9, c2)
    gdn.kv_evict(kv, 10 ** 5, sink=7, recent=9, dst=dst)
    h = host(dst)
    assert all(same(h[x], c2[x]) for x in ("k", "v", "w", "lens"))


def test_evict_keys_that_one_block_cannot_hold():
    """Many sequences, so one block each, and two of them longer than its shared memory has keys."""
    lens = [50000] + [3] * 150 + [45000, 0]
    kv, _ = cache_on_gpu(lens, 64, 1, 32, 90)
    kv.weights.copy_(torch.floor(kv.weights * 50))
    budget = 20000
    w = kv.weights.cpu().numpy()
    table = kv.block_table.cpu().numpy()
    kept = gdn.kv_evict(kv, budget, sink=1, recent=5, want_kept=True).cpu().numpy()
    assert gdn.gdn2_get_device_status() == 0
    for n, x in enumerate(lens):
        j = np.arange(x)
        ref = np.array(paged.kept(w[table[n, j // 64], 0, j % 64], x, budget, 1, 5))
        assert np.array_equal(kept[n, 0, :len(ref)], ref) and (kept[n, 0, len(ref):] == -1).all()
    assert kv.seq_lens.tolist() == [min(x, budget) for x in lens]


@pytest.mark.parametrize("into", [False, True])
def test_evict_bad_pages_and_lengths(into):
    lens = [100, 60, 33, 5]
    kv, c = cache(lens, 16, 2, 64, "f32", 45)
    for t in (c["table"], kv.block_table):
        t[0, 2], t[1, 0] = -1, 10 ** 7
    for t in (c["lens"], kv.seq_lens):
        t[2], t[3] = -4, 16 * c["table"].shape[1] + 1
    dst, c2 = cache([30, 30, 30, 30], 16, 2, 64, "f32", 46) if into else (None, None)
    if into:
        for t in (c2["table"], dst.block_table):
            t[0, 1] = 10 ** 6
    ref = paged.evict(c, 30, 2, 5, c2)
    kept = gdn.kv_evict(kv, 30, sink=2, recent=5, dst=dst, want_kept=True)
    assert gdn.gdn2_get_device_status() == 1
    assert np.array_equal(kept.cpu().numpy(), ref)
    h, want = host(dst if into else kv), c2 if into else c
    assert all(same(h[x], want[x]) for x in ("k", "v", "w", "lens"))


def test_evict_into_a_cache_that_is_too_small():
    kv, c = cache([50, 20], 16, 1, 32, "f32", 47)
    dst, c2 = cache([16, 16], 16, 1, 32, "f32", 48)
    paged.evict(c, 30, 0, 0, c2)
    gdn.kv_evict(kv, 30, dst=dst)
    assert gdn.gdn2_get_device_status() == 1
    h = host(dst)
    assert all(same(h[x], c2[x]) for x in ("k", "v", "w", "lens"))


# ------------------------------------------------- together, streams and graphs

def decode_inputs(N, H, H_kv, d, seed, step):
    g = torch.Generator().manual_seed(seed * 1000 + step)
    return tuple(torch.randn(N, h, d, generator=g).to(torch.bfloat16) for h in (H, H_kv, H_kv))


@pytest.mark.parametrize("mode", ["plain", "stream", "graph"])
def test_a_decode_loop_of_both_mixers(mode):
    """Steps of a hybrid: the recurrent block's step, then the attention block's append and
    attention with weights, and an eviction whenever 8 tokens are over the budget."""
    N, H, H_kv, d, budget = 5, 4, 2, 64, 24
    kv, c = cache([0, 3, 24, 17, 9], 8, H_kv, d, "bf16", 50, room=40, fill=0.0)
    x = {n: t.cuda() for n, t in workloads.decode_step_inputs(N, H, d, d, 51, 0).items()}
    S = torch.zeros(N, H, d, d, device="cuda")
    bufs = [t.cuda() for t in decode_inputs(N, H, H_kv, d, 52, 0)]
    side = torch.cuda.Stream() if mode == "stream" else None
    out = {}

    def step():
        y = gdn.decode_step(x["q"], x["k"], x["v"], x["g"], x["b"], x["w"], S, stream=side)
        gdn.kv_append(kv, bufs[1], bufs[2], stream=side)
        out["o"], out["lse"] = gdn.attn_decode_step(bufs[0], kv, add_weights=True, want_lse=True, stream=side)
        return y

    graph = None
    if mode == "graph":
        saved = kv.seq_lens.clone(), kv.weights.clone(), kv.k.clone(), kv.v.clone()
        step()   # first use of the kernels outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, s in zip((kv.seq_lens, kv.weights, kv.k, kv.v), saved):
            t.copy_(s)
    for i in range(30):
        q, k, v = decode_inputs(N, H, H_kv, d, 52, i)
        torch.cuda.synchronize()
        for b, t in zip(bufs, (q, k, v)):
            b.copy_(t)
        torch.cuda.synchronize()
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        paged.append(c, k.double().numpy(), v.double().numpy())
        r, rl, a, smax = paged.attention(c, q.double().numpy(), d ** -0.5, 0, True)
        bo, bl, _ = bounds("bf16", r, rl, a, smax, 64, d)
        assert (np.abs(out["o"].double().cpu().numpy() - r) <= bo).all(), i
        assert (np.abs(out["lse"].double().cpu().numpy() - rl) <= bl).all(), i
        h = host(kv)
        used = np.array([[p for p in (paged.place(c, n, j) for j in range(int(c["lens"][n])))] for n in [2]][0])
        assert np.allclose(h["w"][used[:, 0], :, used[:, 1]], c["w"][used[:, 0], :, used[:, 1]], rtol=1e-4)
        if max(c["lens"]) >= budget + 8:
            c["w"][:] = h["w"]   # the choice is made from the GPU's own sums
            kept = paged.evict(c, budget, 2, 6)
            mine = gdn.kv_evict(kv, budget, sink=2, recent=6, want_kept=True, stream=side)
            torch.cuda.synchronize()
            assert np.array_equal(mine.cpu().numpy(), kept), i
        h = host(kv)
        assert np.array_equal(h["lens"], c["lens"])
        for n in range(N):
            for j in range(int(c["lens"][n])):
                p, s = paged.place(c, n, j)
                assert np.array_equal(h["k"][p, s], c["k"][p, s]) and np.array_equal(h["v"][p, s], c["v"][p, s])
    assert gdn.gdn2_get_device_status() == 0


def test_a_captured_step_with_eviction_repeats_the_eager_one():
    """Append, attention with weights and an eviction in one graph, against the same calls
    made one by one on a copy: every tensor equal, bit for bit, at every step."""
    a, _ = cache([0, 90, 700, 33], 16, 2, 64, "bf16", 67, room=60, fill=0.0)
    b = gdn.PagedKV(a.k.clone(), a.v.clone(), a.block_table, a.seq_lens.clone(), a.weights.clone())
    bufs = [torch.zeros(4, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)]

    def step(kv):
        gdn.kv_append(kv, bufs[1], bufs[2])
        o, lse = gdn.attn_decode_step(bufs[0], kv, add_weights=True, want_lse=True)
        return o, lse, gdn.kv_evict(kv, 96, sink=1, recent=20, want_kept=True)

    saved = [t.clone() for t in (a.k, a.v, a.seq_lens, a.weights)]
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    for t, x in zip((a.k, a.v, a.seq_lens, a.weights), saved):
        t.copy_(x)
    for i in range(25):
        for t, x in zip(bufs, decode_inputs(4, 8, 2, 64, 68, i)):
            t.copy_(x)
        graph.replay()
        ref = step(b)
        assert all(torch.equal(x, y) for x, y in zip(out, ref)), i
        assert all(torch.equal(x, y) for x, y in ((a.k, b.k), (a.v, b.v), (a.seq_lens, b.seq_lens), (a.weights, b.weights))), i
    assert max(a.seq_lens.tolist()) == 96 and gdn.gdn2_get_device_status() == 0


def test_evictions_on_two_streams_at_once():
    lens = [6000, 5000]
    caches = [cache_on_gpu(lens, 16, 4, 128, 95 + i)[0] for i in range(2)]
    dst = [cache_on_gpu([3000, 3000], 16, 4, 128, 97 + i)[0] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [gdn.kv_evict(c, 3000, recent=10, dst=x, want_kept=True) for c, x in zip(caches, dst)]
    torch.cuda.synchronize()
    got = [gdn.kv_evict(c, 3000, recent=10, want_kept=True, stream=s) for c, s in zip(caches, streams)]
    torch.cuda.synchronize()
    j = torch.arange(3000, device="cuda")
    for c, x, a, b in zip(caches, dst, want, got):
        assert torch.equal(a, b)
        for n in range(2):
            p, p2 = c.block_table[n, j // 16].long(), x.block_table[n, j // 16].long()
            assert torch.equal(c.k[p, j % 16], x.k[p2, j % 16]) and torch.equal(c.v[p, j % 16], x.v[p2, j % 16])


def test_launches_are_counted_and_timed():
    kv, _ = cache([3000, 40], 16, 2, 64, "bf16", 65, room=1)
    q, _ = query(2, 4, 64, "bf16", 66)
    kn = torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)
    before = gdn.gdn2_kernel_launches()
    gdn.gdn2_set_kernel_timer(True)
    try:
        gdn.kv_append(kv, kn, kn)
        gdn.attn_decode_step(q, kv, add_weights=True)
        gdn.kv_evict(kv, 1000)
        times = gdn.gdn2_kernel_times()
    finally:
        gdn.gdn2_set_kernel_timer(False)
    assert gdn.gdn2_kernel_launches() - before == 5
    assert set(times) == {"kv_append", "attn_split", "attn_finish", "evict_select", "evict_move"}
    assert all(n == 1 and ms > 0 for n, ms in times.values())


def test_two_streams_at_once():
    """Two caches on two streams, each call with a workspace of its own."""
    a, ca = cache([4000, 1], 16, 2, 128, "bf16", 60)
    b, cb = cache([3000, 2000], 16, 2, 128, "bf16", 61)
    qa, qa64 = query(2, 8, 128, "bf16", 62)
    qb, qb64 = query(2, 8, 128, "bf16", 63)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(20):
        res.append((gdn.attn_decode_step(qa, a, stream=sa)[0], gdn.attn_decode_step(qb, b, stream=sb)[0]))
    torch.cuda.synchronize()
    one = gdn.attn_decode_step(qa, a)[0], gdn.attn_decode_step(qb, b)[0]
    assert all(torch.equal(x, one[0]) and torch.equal(y, one[1]) for x, y in res)
    check(a, ca, qa, qa64, "bf16", 128 ** -0.5)
    check(b, cb, qb, qb64, "bf16", 128 ** -0.5)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes (and, float32, 2^30 elements): the last pages are read
    and written where they are."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB free")
    pages = (1 << 32) // (16 * 4 * 128 * 2) * 2 + 3    # 8 GB each of k and v
    k = torch.zeros(pages, 16, 4, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[pages - 1, 0, pages // 2 + 1, pages - 2]], dtype=torch.int32, device="cuda")
    w = torch.zeros(pages, 4, 16, device="cuda")
    kv = gdn.PagedKV(k, v, table, torch.zeros(1, dtype=torch.int32, device="cuda"), w)
    g = torch.Generator().manual_seed(5)
    kn, vn = (torch.randn(60, 4, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    gdn.kv_append(kv, kn.cuda(), vn.cuda(), cu_seqlens=torch.tensor([0, 60], dtype=torch.int32, device="cuda"))
    small = on_gpu(torch.zeros(4, 16, 4, 128, dtype=torch.bfloat16), torch.zeros(4, 16, 4, 128, dtype=torch.bfloat16),
                   torch.zeros(4, 4, 16), torch.tensor([[0, 1, 2, 3]], dtype=torch.int32), [0], "NHD")
    gdn.kv_append(small, kn.cuda(), vn.cuda(), cu_seqlens=torch.tensor([0, 60], dtype=torch.int32, device="cuda"))
    q, _ = query(1, 8, 128, "bf16", 64)
    for x in (kv, small):
        x_o = gdn.attn_decode_step(q, x, add_weights=True)[0]
        if x is kv:
            first = x_o
    assert torch.equal(first, x_o) and float(first.float().abs().max()) > 0
    assert torch.equal(gdn.kv_evict(kv, 33, sink=1, recent=4, want_kept=True),
                       gdn.kv_evict(small, 33, sink=1, recent=4, want_kept=True))
    assert torch.equal(gdn.attn_decode_step(q, kv)[0], gdn.attn_decode_step(q, small)[0])


# ------------------------------------------------- values that are not numbers

def agree(o, r, bo):
    """Equal where the reference is infinite or not a number, within bounds elsewhere."""
    got, fin = o.double().cpu().numpy(), np.isfinite(r)
    assert np.array_equal(got[~fin], r[~fin], equal_nan=True)
    assert (np.abs(got[fin] - r[fin]) <= bo[fin]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(32, 1), (64, 5), (128, 8), (128, 9), (128, 16), (64, 20)])
@pytest.mark.parametrize("last", [70, 2500])
def test_attention_infinite_values(io, d, G, last):
    """A value of +-inf makes its channel +-inf, whatever its token's weight (1 in a sequence of
    one token), both signs or NaN make it NaN; the other channels are not touched.  In one
    launch, and (2500 tokens) in parts that are joined."""
    lens = [1, 40, last]
    kv, c = cache(lens, 16, 2, d, io, 71, fill=NAN)
    inf, big = float("inf"), float(torch.finfo(DT[io]).max)
    for n, j, ch, x in ((0, 0, 3, inf), (0, 0, 4, -inf), (0, 0, 5, NAN), (0, 0, 6, big), (0, 0, 7, -big),
                        (1, 7, 0, inf), (1, 8, 0, inf), (1, 39, 1, -inf), (1, 0, 2, inf), (1, 31, 2, -inf), (1, 5, 9, NAN),
                        (2, 0, 1, inf), (2, last - 1, 2, -inf), (2, last // 2, 8, inf), (2, 3, 9, inf), (2, last - 3, 9, -inf)):
        p, s = paged.place(c, n, j)
        kv.v[p, s, 1, ch], c["v"][p, s, 1, ch] = x, x
    q, q64 = query(3, 2 * G, d, io, 72)
    with np.errstate(invalid="ignore"):
        r, rl, a, smax = paged.attention(c, q64, d ** -0.5)
    bo, bl, _ = bounds(io, r, rl, a, smax, last, d)
    o, lse = gdn.attn_decode_step(q, kv, want_lse=True)
    agree(o, r, bo)
    assert (np.abs(lse.double().cpu().numpy() - rl) <= bl).all()
    assert gdn.gdn2_get_device_status() == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(32, 2), (128, 8), (64, 16)])
@pytest.mark.parametrize("length", [70, 2500])
def test_attention_scores_of_plus_infinity(io, d, G, length):
    """Where a score is +inf, log sum e^s is, e^(s - lse) is 0 for every other token and NaN for
    that one, and so is o.  Heads that give the same keys -inf leave them out, and what a score
    that is no number makes of its heads stays NaN."""
    kv, c = cache([length, 5, 40], 16, 2, d, io, 73, fill=NAN)
    q, q64 = query(3, 2 * G, d, io, 74)
    q[:, :, 0], q64[:, :, 0] = 1, 1                      # even heads: +inf
    q[:, 1::2, 0], q64[:, 1::2, 0] = -1, -1              # odd heads: -inf
    top = [(0, 3), (0, length // 2), (0, length - 1), (1, 4)]
    for n, j in top:
        p, s = paged.place(c, n, j)
        kv.k[p, s, 1, 0], c["k"][p, s, 1, 0] = float("inf"), float("inf")
    p, s = paged.place(c, 2, 20)
    kv.k[p, s, 0, 0], c["k"][p, s, 0, 0] = NAN, NAN
    w0 = c["w"].copy()
    finite = dict(c, k=np.where(np.isfinite(c["k"]), c["k"], 0.0), w=w0.copy())
    smax = paged.attention(finite, q64, d ** -0.5)[3]
    with np.errstate(invalid="ignore"):
        r, rl, a, _ = paged.attention(c, q64, d ** -0.5, 0, True)
    hot = np.zeros(rl.shape, dtype=bool)
    hot[:2, G::2] = True
    assert np.isnan(rl[hot]).all()                       # the oracle's inf - inf
    rl[hot] = np.inf
    bo, bl, bp = bounds(io, r, rl, a, smax, length, d)
    o, lse = gdn.attn_decode_step(q, kv, add_weights=True, want_lse=True)
    assert gdn.gdn2_get_device_status() == 0
    agree(o, r, bo)
    agree(lse, rl, bl)
    # weights of the second key-value head: the odd heads' alone, NaN on the +inf tokens
    got = kv.weights.double().cpu().numpy()
    odd = dict(finite, k=c["k"], w=w0.copy())
    q_odd = q64.copy()
    q_odd[:, G::2] = q_odd[:, G + 1::2]                  # each odd head twice
    paged.attention(odd, q_odd, d ** -0.5, 0, True)
    for n, x in ((0, length), (1, 5)):
        for j in range(x):
            p, s = paged.place(c, n, j)
            if (n, j) in top:
                assert np.isnan(got[p, 1, s])
            else:
                add = (odd["w"][p, 1, s] - w0[p, 1, s]) / 2
                lim = bp[n].max() * add + (G + 2) * 2.0 ** -24 * (w0[p, 1, s] + add) + 1e-30
                assert abs(got[p, 1, s] - w0[p, 1, s] - add) <= lim


def test_eviction_in_place_gives_up_a_wait_and_says_so():
    """Nobody reads the first chunk of rows, so whoever would write over it gives up: the status
    says so, no row has moved (a write before its read would show), and the context is usable."""
    lens, budget = [3000, 40, 2000], 1200
    kv, _ = cache_on_gpu(lens, 16, 2, 64, 110)
    before = [t.clone() for t in (kv.k, kv.v, kv.weights, kv.seq_lens)]
    ws = torch.empty(kv.workspace_bytes("gdn2_kv_evict_workspace_bytes", budget), dtype=torch.uint8, device="cuda")
    gdn.gdn2_selftest_evict_timeout(kv, budget, ws, ws.nbytes)
    assert gdn.gdn2_get_device_status() == 5          # GDN2_ERR_TIMEOUT
    for t, x in zip((kv.k, kv.v, kv.weights), before):
        assert torch.equal(t, x)
    assert kv.seq_lens.tolist() == [1200, 40, 1200]
    kv.seq_lens.copy_(before[3])
    dst, _ = cache_on_gpu([min(x, budget) for x in lens], 16, 2, 64, 111)
    a = gdn.kv_evict(kv, budget, dst=dst, want_kept=True)
    b = gdn.kv_evict(kv, budget, want_kept=True, ws=ws)
    assert gdn.gdn2_get_device_status() == 0 and torch.equal(a, b)
    for n, x in enumerate(lens):
        j = torch.arange(min(x, budget), device="cuda")
        p, p2 = kv.block_table[n, j // 16].long(), dst.block_table[n, j // 16].long()
        assert torch.equal(kv.k[p, j % 16], dst.k[p2, j % 16]) and torch.equal(kv.v[p, j % 16], dst.v[p2, j % 16])


@pytest.mark.parametrize("into", [False, True])
def test_the_c_calls_under_their_own_names(into):
    """gdn2_kv_append, gdn2_attn_decode_step and gdn2_kv_evict with the caller's buffers, on a
    stream of the caller's: what kv_append, attn_decode_step and kv_evict leave, bit for bit."""
    budget = 64
    cu = torch.tensor([0, 900, 900, 930], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(930, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    q, _ = query(3, 8, 64, "bf16", 118)
    a, _ = cache([5, 0, 17], 16, 2, 64, "bf16", 119, room=900, fill=0.0)
    b = gdn.PagedKV(a.k.clone(), a.v.clone(), a.block_table, a.seq_lens.clone(), a.weights.clone())
    dst = [cache_on_gpu([budget] * 3, 16, 2, 64, 120)[0] for _ in range(2)] if into else [None, None]
    gdn.kv_append(a, k, v, cu_seqlens=cu)
    o, lse = gdn.attn_decode_step(q, a, scale=0.1, window=700, add_weights=True, want_lse=True)
    kept = gdn.kv_evict(a, budget, sink=2, recent=7, dst=dst[0], want_kept=True)
    side = torch.cuda.Stream()
    o2, lse2, kept2 = torch.full_like(o, NAN), torch.full_like(lse, NAN), torch.full_like(kept, -5)
    n1, n2 = gdn.gdn2_attn_decode_workspace_bytes(b, 8, True), gdn.gdn2_kv_evict_workspace_bytes(b, budget)
    ws1, ws2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (n1, n2))
    torch.cuda.synchronize()
    gdn.gdn2_kv_append(b, k, v, cu, 930, b.seq_lens, stream=side)
    gdn.gdn2_attn_decode_step(b, q, o2, lse2, 8, 0.1, 700, True, ws1, n1, stream=side)
    gdn.gdn2_kv_evict(b, dst[1], budget, 2, 7, kept2, ws2, n2, stream=side)
    assert gdn.gdn2_get_device_status(side) == 0
    for x, y in ((o, o2), (lse, lse2), (kept, kept2)):
        assert torch.equal(x, y)
    for x, y in ((a, b), dst) if into else ((a, b),):
        assert all(torch.equal(s, t) for s, t in ((x.k, y.k), (x.v, y.v), (x.weights, y.weights), (x.seq_lens, y.seq_lens)))
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.gdn2_attn_decode_step(b, q, o2, lse2, 8, 0.1, 700, True, ws1, n1 - 256)
    assert e.value.status == 3
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.gdn2_kv_append(b, k, v, None, 930, b.seq_lens)
    assert e.value.status == 1
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.gdn2_kv_evict(b, None, 0, 0, 0, None, ws2, n2)
    assert e.value.status == 1
