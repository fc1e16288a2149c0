"""One-token attention where a call is split and its parts are joined: what short tables, which
go to blocks whole, do not reach.  Each test asserts that its call was split."""

import numpy as np
import pytest
import torch

import gated_delta_rule_128_b200 as gdn
from _paged import bounds, cache
from oracle import paged
from test_paged_gpu import NAN, _lib, _status, cache_on_gpu, check, query  # noqa: F401  (the fixtures apply here too)

pytestmark = pytest.mark.gpu


def widened(kv, c, reach=4096):
    """The same cache under a table that could hold `reach` tokens a sequence."""
    more = -(-reach // kv.k.shape[1]) - kv.block_table.shape[1]
    if more <= 0:
        return kv
    table = torch.nn.functional.pad(kv.block_table, (0, more), value=-7).contiguous()
    c["table"] = np.pad(c["table"], ((0, 0), (0, more)), constant_values=-7)
    return gdn.PagedKV(kv.k, kv.v, table, kv.seq_lens, kv.weights)


def check_split(kv, c, q, q64, io, scale, window=0, add=False, status=0):
    """check(), and the call took two launches (a whole one without weights takes one; one with
    weights is laid out by the same rule whatever the window)."""
    before = gdn.gdn2_kernel_launches()
    gdn.attn_decode_step(q, kv, scale=scale, window=0 if add else window)
    assert gdn.gdn2_kernel_launches() - before == 2
    gdn.gdn2_get_device_status()
    return check(kv, c, q, q64, io, scale, window, add, status)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [31, 32, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("add", [False, True])
def test_runs_of_many_sequences(io, N, add):
    """Up to 32 sequences a warp looks for its run alone, beyond that a block, and beyond 128 in
    several passes.  A few long sequences among empty and short ones, the first and last empty."""
    rng = np.random.default_rng(N)
    lens = [int(x) for x in rng.choice([0, 0, 1, 17, 63, 64, 65, 90], N)]
    for n, x in ((1, 2100), (N // 2, 3001), (N - 2, 2049), (N - 3, 700)):
        lens[n] = x
    lens[0] = lens[-1] = 0
    kv, c = cache(lens, 16, 2, 32, io, N, fill=NAN)
    q, q64 = query(N, 2 * 20, 32, io, 100)             # two blocks of query heads
    check_split(kv, c, q, q64, io, 32 ** -0.5, 0, add)


@pytest.mark.parametrize("io,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("H_kv,G", [(1, 1), (3, 2), (2, 7), (1, 16), (2, 17)])
def test_heads_and_short_sequences(io, d, H_kv, G):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]
    kv, c = cache(lens, 16, H_kv, d, io, d + G, fill=NAN)
    q, q64 = query(len(lens), H_kv * G, d, io, 101)
    check_split(widened(kv, c), c, q, q64, io, d ** -0.5, 0, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window,add", [(x, True) for x in (1, 63, 64, 65, 199, 700, 2048, 2049)] +
                         [(x, False) for x in (513, 700, 2048, 2049)])
def test_windows(io, window, add):
    """Tokens before the window (NaN here) are not looked at.  (Without weights a window of up
    to 512 tokens is not split.)"""
    lens = [0, 1, 62, 64, 66, 200, 699, 701, 2500, 3100]
    kv, c = cache(lens, 24, 2, 64, io, window)
    for n, x in enumerate(lens):
        for j in range(max(0, x - window)):
            p, s = paged.place(c, n, j)
            c["k"][p, s], c["v"][p, s] = NAN, NAN
    kv.k.copy_(torch.from_numpy(c["k"]).to(kv.k))
    kv.v.copy_(torch.from_numpy(c["v"]).to(kv.v))
    q, q64 = query(len(lens), 8, 64, io, 102)
    check_split(kv, c, q, q64, io, 0.125, window, add)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 5, 24, 64, 512])
@pytest.mark.parametrize("layout", ["NHD", "HND", "padded", "interleaved"])
def test_pages_and_layouts(io, page, layout):
    lens = [130, 0, 7, 100, 101, 1500]
    kv, c = cache(lens, page, 2, 64, io, page, layout=layout, fill=NAN)
    q, q64 = query(len(lens), 6, 64, io, 103)
    check_split(widened(kv, c), c, q, q64, io, 0.125, 0, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
def test_bad_pages_and_lengths(io, add):
    """Pages outside the pool inside long and short sequences, and lengths outside the table."""
    lens = [2400, 60, 33, 5, 900]
    kv, c = cache(lens, 16, 2, 64, io, 104, fill=NAN)
    kv = widened(kv, c)
    for t in (c["table"], kv.block_table):
        t[0, 2], t[0, 77], t[0, 149], t[1, 0], t[4, 0] = -1, c["k"].shape[0], -5, 2 ** 31 - 1, -1
    for t in (c["lens"], kv.seq_lens):
        t[2], t[3] = -4, 16 * c["table"].shape[1] + 1
    q, q64 = query(5, 4, 64, io, 105)
    check_split(kv, c, q, q64, io, 0.125, 0, add, status=1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_keys_of_minus_infinity_and_nan(io):
    """-inf leaves a token out: some of a sequence's, a whole part's, all of one; NaN stays in
    its sequence and key-value head."""
    kv, c = cache([2500, 2600, 40, 2200], 16, 2, 32, io, 106)
    which = [(0, j) for j in range(0, 2500, 3)] + [(0, j) for j in range(64, 640)] + [(1, j) for j in range(2600)]
    for n, j in which:
        p, s = paged.place(c, n, j)
        c["k"][p, s, :, 0] = -np.inf
    p, s = paged.place(c, 3, 1111)
    c["k"][p, s, 1, 3] = NAN
    kv.k.copy_(torch.from_numpy(c["k"]).to(kv.k))
    q, q64 = query(4, 4, 32, io, 107)
    q[:, :, 0], q64[:, :, 0] = 1, 1
    o, lse = gdn.attn_decode_step(q, kv, scale=0.1, add_weights=True, want_lse=True)
    assert gdn.gdn2_get_device_status() == 0
    r, rl, a, _ = paged.attention(c, q64, 0.1)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert torch.isnan(o[3, 2:]).all() and torch.isnan(lse[3, 2:]).all()
    got = o.double().cpu().numpy()
    # rounding o, and 1e-4 of sum p |v|: scores of at most sum |q k| / 10 < 20 in float32, as
    # where a call is not split, and 2 * 2500 * 2^-24 = 3e-4 at the very most for the sums
    for at in (np.s_[0], np.s_[2], np.s_[3, :2]):
        lim = (2.0 ** -8 if io == "bf16" else 0) * np.abs(r[at]) * 1.01 + 4e-4 * a[at] + 1e-30
        assert (np.abs(got[at] - r[at]) <= lim).all()
        assert (np.abs(lse.double().cpu().numpy()[at] - rl[at]) <= 1e-3).all()
    w = kv.weights.cpu().numpy()
    for n, x, heads in ((0, 2500, (0, 1)), (1, 2600, (0, 1)), (2, 40, (0, 1)), (3, 2200, (0,))):
        for j in range(x):
            p, s = paged.place(c, n, j)
            assert all(np.isfinite(w[p, h, s]) for h in heads)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(32, 1), (64, 5), (128, 20)])
@pytest.mark.parametrize("prompt,N", [(2100, 12), (600, 40)])
def test_shared_prompts_hold_more_than_the_pool(io, d, G, prompt, N):
    """The scores that a call keeps for the weights are bounded by the pool, so most sequences'
    scores are computed once more.  Each sequence has some tokens of its own behind the prompt."""
    own, page = 40, 16
    first = prompt // page
    kv, c = cache([prompt] + [own] * N, page, 2, d, io, 108, spare=0, fill=NAN)
    more = kv.block_table[1:, :-(-own // page)]
    shared = kv.block_table[:1, :first].expand(N, first)
    lens = [first * page + own - n % 7 for n in range(N)]
    table = torch.cat([shared, more], 1).contiguous()
    kv = gdn.PagedKV(kv.k, kv.v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), kv.weights)
    c["table"], c["lens"] = table.cpu().numpy(), np.array(lens)
    HB = -(-G // 16)
    units = N * 2 * HB * (-(-table.shape[1] * page // 64) + 2)      # all that there can be
    kept = gdn.gdn2_attn_decode_workspace_bytes(kv, 2 * G, True) - gdn.gdn2_attn_decode_workspace_bytes(kv, 2 * G, False)
    assert kept < units * -(-G // HB) * 64 * 4 / 2
    q, q64 = query(N, 2 * G, d, io, 109)
    for window in (0, 1000):
        check_split(kv, c, q, q64, io, d ** -0.5, window if window > 512 else 0)
        w0 = c["w"].copy()
        r, rl, a, smax = paged.attention(c, q64, d ** -0.5, window, True)
        bp = bounds(io, r, rl, a, smax, max(lens), d)[2].max()
        gdn.attn_decode_step(q, kv, window=window, add_weights=True)
        got, fin = kv.weights.double().cpu().numpy(), np.isfinite(c["w"])
        # each head's weight is off by bp of itself; the sum over G heads rounds G times, and each
        # of up to N sequences adds its sum to a shared token with one rounding more, every one by
        # 2^-24 of what is there, which only grows; w0 is the GPU's own for the second window
        lim = bp * (c["w"] - w0) + (N + G + 2) * 2.0 ** -24 * np.abs(c["w"]) + 1e-30
        assert (np.abs(got - c["w"])[fin] <= lim[fin]).all()
        assert np.array_equal(np.isnan(got), ~fin)
        c["w"][:] = got


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[100, 3], [3000, 3, 0, 700]])
def test_the_output_may_take_the_queries_place(io, lens):
    kv, _ = cache(lens, 16, 2, 64, io, 112)
    q, _ = query(len(lens), 2 * 20, 64, io, 113)
    want, lse = gdn.attn_decode_step(q, kv, want_lse=True)
    o, lse2 = gdn.attn_decode_step(q, kv, o=q, want_lse=True)
    assert o is q and torch.equal(o, want) and torch.equal(lse, lse2)
    with pytest.raises(gdn.Gdn2Error) as e:
        gdn.attn_decode_step(q, kv, o=q, add_weights=True)
    assert e.value.status == 1


# ------------------------------------------------------------- the longest tables

PAGE = 1 << 20


def one_page_many_times(io, seed):
    """A sequence of 2^30 tokens, the most that a table may reach: one page of 2^20 tokens 1024
    times over."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(1, PAGE, 1, 32, device="cuda", generator=g).to({"bf16": torch.bfloat16, "f32": torch.float32}[io])
            for _ in range(2))
    v += 1
    return gdn.PagedKV(k, v, torch.zeros(1, 1024, dtype=torch.int32, device="cuda"),
                       torch.full((1,), 1 << 30, dtype=torch.int32, device="cuda"),
                       torch.zeros(1, 1, PAGE, device="cuda")), g


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, (1 << 30) - 5])
def test_attention_over_two_to_the_thirty_tokens(io, window):
    """Every page's tokens again and again: o is that of one page, lse log 1024 more, each weight
    1024 times the page's."""
    kv, g = one_page_many_times(io, 114)
    q = torch.randn(1, 2, 32, device="cuda", generator=g).to(kv.k.dtype)
    o, lse = gdn.attn_decode_step(q, kv, window=window, add_weights=True, want_lse=True)
    assert gdn.gdn2_get_device_status() == 0
    z = q[0].double() @ kv.k[0, :, 0].double().T * 32 ** -0.5
    p, v = torch.softmax(z, -1), kv.v[0, :, 0].double()
    ref, spread = p @ v, p @ v.abs()
    # A lane adds 2^30 / (148 * 4 blocks * 4 warps) tokens in steps of 16 or 8, two sums a step, so
    # fewer than 2^18 additions in a row, each off by at most 2^-23 (the tensor cores' truncate)
    # of sums that grow evenly (half of the last on average): 2^-6 of sum p |v| for o's numerator
    # and of l alike.  A block's tokens left out or read twice would change lse by 1/600.
    assert ((o[0].double() - ref).abs() <= 2.0 ** -5 * spread + 2.0 ** -8 * ref.abs()).all()
    assert ((lse[0].double() - torch.logsumexp(z, -1) - np.log(1024)).abs() <= 2.0 ** -6).all()
    # 1024 additions to each weight, each rounding by 2^-24 of what is there, after lse's error
    want = p.sum(0)
    assert ((kv.weights[0, 0].double() - want).abs() <= (2.0 ** -5 + 1024 * 2.0 ** -24) * want).all()


def test_eviction_from_two_to_the_thirty_tokens():
    """The heaviest tokens are the page's heaviest one, 1024 times; equal weights go by index."""
    kv, g = one_page_many_times("bf16", 115)
    kv.weights.copy_(torch.randperm(PAGE, device="cuda", generator=g).float())
    best = int(kv.weights.argmax())
    k, v = (torch.zeros(11, 100, 1, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dst = gdn.PagedKV(k, v, torch.arange(11, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.zeros(11, 1, 100, device="cuda"))
    kept = gdn.kv_evict(kv, 1003, sink=1, recent=2, dst=dst, want_kept=True)
    assert gdn.gdn2_get_device_status() == 0
    want = [0] + [best + i * PAGE for i in range(1000)] + [(1 << 30) - 2, (1 << 30) - 1]
    assert best not in (0, PAGE - 1, PAGE - 2) and kept[0, 0].tolist() == want
    assert dst.seq_lens.tolist() == [1003] and kv.seq_lens.tolist() == [1 << 30]
    j = torch.arange(1003, device="cuda")
    src = kept[0, 0].long() % PAGE
    assert torch.equal(dst.k[j // 100, j % 100, 0], kv.k[0, src, 0]) and torch.equal(dst.v[j // 100, j % 100, 0], kv.v[0, src, 0])


@pytest.mark.parametrize("into", [False, True])
def test_eviction_of_keys_that_a_cluster_cannot_hold(into):
    """A sequence of a million tokens: 16 blocks share it, and each has more keys than its shared
    memory takes."""
    x, budget, P = 1000003, 300000, 64
    kv, _ = cache_on_gpu([x], P, 1, 32, 116)
    kv.weights.copy_(torch.floor(kv.weights * 5000))
    dst = cache_on_gpu([budget], P, 1, 32, 117)[0] if into else None
    k0, w0, table = kv.k.clone(), kv.weights.clone(), kv.block_table[0].long()
    kept = gdn.kv_evict(kv, budget, sink=3, recent=100, dst=dst, want_kept=True)[0, 0].long()
    assert gdn.gdn2_get_device_status() == 0
    j = torch.arange(x, device="cuda")
    w = w0[table[j // P], 0, j % P][3:x - 100]
    best = torch.sort(w, descending=True, stable=True).indices[:budget - 103] + 3
    assert torch.equal(kept, torch.cat([j[:3], best.sort().values, j[x - 100:]]))
    to = dst if into else kv
    i = torch.arange(budget, device="cuda")
    assert torch.equal(to.k[to.block_table[0].long()[i // P], i % P], k0[table[kept // P], kept % P])
    assert to.seq_lens.tolist() == [budget]
