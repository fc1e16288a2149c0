"""The paged-cache calls without a GPU: the oracle against hand-made values, the
host checks of the C entry points, and what the binding refuses."""

import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_128_b200 as gdn
from gated_delta_rule_128_b200 import build
from oracle import paged

FAKE = 1 << 20   # an aligned, never-dereferenced address: host checks fail first
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return gdn.lib()


def desc(**kw):
    a = dict(k=FAKE, v=FAKE, weight=FAKE, block_table=FAKE, seq_lens=FAKE, stride_page=16 * 4 * 64,
             stride_slot=4 * 64, stride_head=64, num_pages=10, page_size=16, max_pages=5, N=2, H_kv=4, d=64, io=1)
    a.update(kw)
    return gdn._PagedKVStruct(*a.values())


def attn(L, kv=None, q=FAKE, o=FAKE, lse=FAKE, H=8, scale=0.125, window=0, add=0, ws=FAKE, ws_bytes=BIG):
    return L.gdn2_attn_decode_step(ctypes.byref(kv or desc()), q, o, lse, H, scale, window, add, ws, ws_bytes, None)


def evict(L, kv=None, dst=None, budget=8, sink=1, recent=2, kept=None, ws=FAKE, ws_bytes=BIG):
    return L.gdn2_kv_evict(ctypes.byref(kv or desc()), ctypes.byref(dst) if dst else None, budget, sink, recent, kept,
                           ws, ws_bytes, None)


def append(L, kv=None, k=FAKE, v=FAKE, cu=FAKE, T=7, lens=FAKE):
    return L.gdn2_kv_append(ctypes.byref(kv or desc()), k, v, cu, T, lens, None)


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1), (dict(v=FAKE + 2), 1),
    (dict(block_table=None), 1), (dict(seq_lens=None), 1), (dict(seq_lens=FAKE + 2), 1),
    (dict(block_table=FAKE + 1), 1), (dict(weight=FAKE + 2), 1),
    (dict(io=2), 1), (dict(N=0), 1), (dict(H_kv=0), 1), (dict(num_pages=0), 1), (dict(page_size=-1), 1),
    (dict(max_pages=0), 1), (dict(d=48), 2), (dict(d=256), 2),
    (dict(max_pages=1 << 20, page_size=1 << 11, stride_page=1 << 20), 2),
    (dict(max_pages=(1 << 26) + 1), 2),
    (dict(N=1 << 25, H_kv=4), 2),
    (dict(stride_head=60), 1),          # rows overlap
    (dict(stride_head=65), 1),          # not 16 bytes
    (dict(stride_slot=2 * 64), 1),      # slots overlap the heads
    (dict(stride_page=15 * 256), 1),    # pages overlap
    (dict(stride_slot=-256), 1), (dict(stride_page=0), 1),
    (dict(stride_page=1 << 41), 1),
    (dict(stride_page=64, stride_slot=64 * 10 * 4), 1),   # pages inside the heads
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_checks_the_cache(L, kw, status):
    kv = desc(**kw)
    assert attn(L, kv) == status
    assert append(L, kv) == status
    assert evict(L, kv) == status
    assert evict(L, dst=desc(seq_lens=FAKE + 64, **{k: v for k, v in kw.items() if k != "seq_lens"})) == status \
        if not ("seq_lens" in kw or "N" in kw or "H_kv" in kw or "d" in kw) else True
    assert L.gdn2_attn_decode_workspace_bytes(ctypes.byref(kv), 8, 0) == 0
    assert L.gdn2_kv_evict_workspace_bytes(ctypes.byref(kv), 8) == 0


def test_null_cache(L):
    assert L.gdn2_attn_decode_step(None, FAKE, FAKE, None, 8, 1.0, 0, 0, FAKE, BIG, None) == 1
    assert L.gdn2_kv_append(None, FAKE, FAKE, None, 2, FAKE, None) == 1
    assert L.gdn2_kv_evict(None, None, 8, 0, 0, None, FAKE, BIG, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(q=FAKE + 4), 1), (dict(o=FAKE + 8), 1), (dict(lse=FAKE + 2), 1),
    (dict(H=0), 1), (dict(H=6), 1), (dict(H=-4), 1), (dict(window=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(scale=-3e38), 1),
    (dict(H=4 * 257), 2), (dict(kv=desc(N=1 << 20, max_pages=1 << 16)), 2),
    (dict(kv=desc(weight=None), add=1), 1),
    (dict(ws=None), 3), (dict(ws_bytes=0), 3), (dict(ws=FAKE + 8), 3),
    (dict(H=1 << 26), 2),
])
def test_attention_refuses(L, kw, status):
    assert attn(L, **kw) == status


def test_attention_refuses_an_output_over_its_queries(L):
    """The weights of tokens whose scores were not kept need q after o has been written."""
    size = 2 * 8 * 64 * 2
    for o, add, status in ((FAKE, 1, 1), (FAKE, 0, 3), (FAKE + 128, 0, 1), (FAKE - 128, 0, 1), (FAKE + size - 16, 1, 1),
                           (FAKE + 16 - size, 0, 1), (FAKE + size, 1, 3), (FAKE - size, 1, 3)):
        assert attn(L, o=o, add=add, ws_bytes=0) == status, (o - FAKE, add)


@pytest.mark.parametrize("N,H_kv,G,page_size,max_pages", [
    (1 << 20, 1, 1, 64, 1021), ((1 << 20) - 1, 1, 1, 64, 1022),      # N * H_kv * (units + 2)
    (1 << 20, 1, 1, 32, 2042), (1, 1, 1, 1 << 15, 1 << 15),
    (1 << 16, 2, 32, 64, 4093), (1 << 16, 2, 33, 64, 2728), (64, 1, 256, 64, (1 << 20) - 3),
    ((1 << 18) - 1, 1, 128, 16, 1), (3, 4, 256, 16, 100),             # N * H
])
def test_attention_takes_what_the_header_promises(L, N, H_kv, G, page_size, max_pages):
    """Sizes at the stated limits are taken (as far as the workspace check), one step beyond is
    refused, by the call and by the workspace query alike."""
    def status(n, table):
        kv = desc(N=n, H_kv=H_kv, page_size=page_size, max_pages=table, stride_head=64, stride_slot=64 * H_kv,
                  stride_page=64 * H_kv * page_size)
        size = L.gdn2_attn_decode_workspace_bytes(ctypes.byref(kv), H_kv * G, 0)
        rc = attn(L, kv, H=H_kv * G, ws_bytes=0)
        assert (size == 0) == (rc == 2) and rc in (2, 3)
        return rc

    def fits(n, table):
        units = -(-table * page_size // 64) + 2
        return G <= 256 and n * H_kv * G < 1 << 25 and n * H_kv * -(-G // 16) * units < 1 << 30

    for n in (1, N, N + 1, N + 2, 2 * N):
        for table in (1, max_pages, max_pages + 1, max_pages + 4):
            if n * H_kv < 1 << 25 and table * page_size <= 1 << 30:
                assert status(n, table) == (3 if fits(n, table) else 2)
    assert fits(N, max_pages)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 4), 1), (dict(v=FAKE + 4), 1), (dict(lens=None), 1),
    (dict(lens=FAKE + 2), 1), (dict(cu=FAKE + 2), 1), (dict(T=-1), 1), (dict(cu=None, T=3), 1), (dict(cu=None, T=0), 1),
])
def test_append_refuses(L, kw, status):
    assert append(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(budget=0), 1), (dict(sink=-1), 1), (dict(recent=-1), 1), (dict(sink=5, recent=4), 1),
    (dict(sink=1 << 30, recent=1 << 30, budget=100), 1), (dict(kept=FAKE + 2), 1),
    (dict(kv=desc(weight=None)), 1), (dict(dst=desc(weight=None, seq_lens=FAKE + 64)), 1),
    (dict(dst=desc()), 1),                              # the same lengths as the source
    (dict(dst=desc(seq_lens=FAKE + 64, N=3)), 1), (dict(dst=desc(seq_lens=FAKE + 64, io=0)), 1),
    (dict(dst=desc(seq_lens=FAKE + 64, H_kv=2)), 1), (dict(dst=desc(seq_lens=FAKE + 64, d=32)), 1),
    (dict(ws=None), 3), (dict(ws_bytes=16), 3), (dict(ws=FAKE + 8), 3),
    (dict(kv=desc(N=1 << 20, max_pages=1 << 20), budget=1 << 24), 2),
])
def test_evict_refuses(L, kw, status):
    assert evict(L, **kw) == status


@pytest.mark.parametrize("dst", [None, desc(seq_lens=FAKE + 64)])
def test_evict_refuses_a_kept_list_that_the_kernels_cannot_count(L, dst):
    """A list of kept tokens has `budget` entries.  Counted in steps of up to 16384 threads, a
    32-bit index would pass 2^31 and come back below the list.  Without a list any budget goes."""
    for budget in (2 ** 30 + 1, 2 ** 31 - 16384, 2 ** 31 - 1):
        assert evict(L, dst=dst, budget=budget, kept=FAKE, ws_bytes=0) == 2
        assert evict(L, dst=dst, budget=budget, ws_bytes=0) == 3      # as far as the workspace check
    assert evict(L, dst=dst, budget=2 ** 30, kept=FAKE, ws_bytes=0) == 3


def test_binding_refuses_a_kept_list_before_it_allocates_one():
    with pytest.raises(ValueError, match="want_kept"):
        gdn.kv_evict(cpu_cache(), 2 ** 30 + 1, want_kept=True)


@pytest.mark.parametrize("kw,status", [
    (dict(kv=desc(d=48)), 2), (dict(kv=desc(weight=None)), 1), (dict(budget=0), 1), (dict(ws=None), 3),
    (dict(ws_bytes=16), 3), (dict(kv=desc(N=1 << 20, max_pages=1 << 20), budget=1 << 24), 2),
])
def test_the_evictions_selftest_refuses(L, kw, status):
    a = dict(kv=desc(), budget=8, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    assert L.gdn2_selftest_evict_timeout(ctypes.byref(a["kv"]), a["budget"], a["ws"], a["ws_bytes"], 1000, None) == status


def test_strides_along_single_axes_are_not_read(L):
    """An axis of extent 1 may carry any stride (frameworks leave anything there); the call
    then gets as far as its own arguments."""
    kv = desc(H_kv=1, stride_head=3, stride_slot=64, stride_page=1024)
    assert attn(L, kv, H=4, ws_bytes=0) == 3
    kv = desc(num_pages=1, stride_page=-5)
    assert attn(L, kv, ws_bytes=0) == 3


def test_workspace_sizes(L):
    kv = ctypes.byref(desc())
    plain, more = (L.gdn2_attn_decode_workspace_bytes(kv, 8, x) for x in (0, 1))
    assert 256 <= plain <= more
    assert L.gdn2_attn_decode_workspace_bytes(kv, 6, 0) == 0
    a, b = (L.gdn2_kv_evict_workspace_bytes(kv, x) for x in (8, 8000))
    assert 256 <= a < b and L.gdn2_kv_evict_workspace_bytes(kv, 0) == 0


def cpu_cache(**kw):
    a = dict(k=torch.zeros(6, 16, 2, 32), v=torch.zeros(6, 16, 2, 32), block_table=torch.zeros(3, 2, dtype=torch.int32),
             seq_lens=torch.zeros(3, dtype=torch.int32), weights=torch.zeros(6, 2, 16))
    a.update(kw)
    return gdn.PagedKV(*a.values())


@pytest.mark.parametrize("kw,error", [
    (dict(k=torch.zeros(6, 16, 2, 32, dtype=torch.float16), v=torch.zeros(6, 16, 2, 32, dtype=torch.float16)), TypeError),
    (dict(v=torch.zeros(6, 16, 2, 64)), ValueError), (dict(v=torch.zeros(6, 16, 2, 32, dtype=torch.bfloat16)), TypeError),
    (dict(v=torch.zeros(6, 2, 16, 32).transpose(1, 2)), ValueError),
    (dict(k=torch.zeros(6, 16, 2, 64)[..., ::2], v=torch.zeros(6, 16, 2, 64)[..., ::2]), ValueError),
    (dict(k=torch.zeros(6, 16, 64)), ValueError),
    (dict(block_table=torch.zeros(3, 2)), TypeError), (dict(block_table=torch.zeros(6, dtype=torch.int32)), ValueError),
    (dict(block_table=torch.zeros(3, 4, dtype=torch.int32)[:, ::2]), ValueError),
    (dict(seq_lens=torch.zeros(4, dtype=torch.int32)), ValueError), (dict(seq_lens=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(weights=torch.zeros(6, 16, 2)), ValueError), (dict(weights=torch.zeros(6, 2, 16, dtype=torch.float64)), TypeError),
])
def test_binding_refuses_a_cache(kw, error):
    with pytest.raises(error):
        cpu_cache(**kw)


def test_binding_refuses_arguments(L):
    kv = cpu_cache()
    with pytest.raises(ValueError):
        gdn.attn_decode_step(torch.zeros(3, 4, 64), kv)
    with pytest.raises(ValueError):
        gdn.attn_decode_step(torch.zeros(2, 4, 32), kv)
    with pytest.raises(TypeError):
        gdn.attn_decode_step(torch.zeros(3, 4, 32, dtype=torch.bfloat16), kv)
    with pytest.raises(ValueError):   # a slice of a wider projection: not contiguous
        gdn.attn_decode_step(torch.zeros(3, 12, 32)[:, :4], kv)
    with pytest.raises(ValueError):
        gdn.kv_append(kv, torch.zeros(3, 2, 32), torch.zeros(3, 1, 32))
    with pytest.raises(TypeError):
        gdn.kv_append(kv, torch.zeros(3, 2, 32), torch.zeros(3, 2, 32), cu_seqlens=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.attn_decode_step(torch.zeros(3, 4, 32), kv)
    for kw in (dict(budget=0), dict(budget=2 ** 31), dict(budget=8, recent=2 ** 32), dict(budget=8, sink=-2 ** 33)):
        with pytest.raises(ValueError):
            gdn.kv_evict(kv, **kw)
    with pytest.raises(ValueError, match="window"):
        gdn.attn_decode_step(torch.zeros(3, 4, 32), kv, window=2 ** 32 + 4)
    with pytest.raises(ValueError):
        gdn.kv_append(kv, torch.zeros(3, 2, 32), torch.zeros(3, 2, 32), lens_out=torch.zeros(2, dtype=torch.int32))


# ------------------------------------------------------------------ the oracle

def small(lens, seed=0, P=4, H=2, d=3, pages=12):
    rng = np.random.default_rng(seed)
    return dict(k=rng.normal(size=(pages, P, H, d)), v=rng.normal(size=(pages, P, H, d)),
                w=rng.random((pages, H, P)), table=rng.permutation(pages)[:len(lens) * 3].reshape(len(lens), 3),
                lens=np.array(lens))


def test_oracle_attention_is_the_softmax_of_gathered_rows():
    c = small([7, 0, 12])
    q = np.random.default_rng(1).normal(size=(3, 4, 3))
    o, lse, a, _ = paged.attention(c, q, 0.7, window=5)
    rows = [(int(c["table"][0, j // 4]), j % 4) for j in range(2, 7)]
    k = np.array([c["k"][p, s, 1] for p, s in rows])
    v = np.array([c["v"][p, s, 1] for p, s in rows])
    e = np.exp(0.7 * k @ q[0, 2])
    assert np.allclose(o[0, 2], e @ v / e.sum(), rtol=1e-13)
    assert np.isclose(lse[0, 2], np.log(e.sum()), rtol=1e-13)
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()


def test_oracle_weights_sum_to_the_heads():
    c = small([7, 0, 12])
    before = c["w"].sum()
    paged.attention(c, np.random.default_rng(2).normal(size=(3, 4, 3)), 1.0, add_weights=True)
    assert np.isclose(c["w"].sum() - before, 2 * 4)


def test_oracle_evict_by_hand():
    w = np.array([9.0, 1.0, 5.0, 5.0, np.nan, 0.0, -0.0, 2.0])
    assert paged.kept(w, 8, 4, 1, 1) == [0, 2, 3, 7]
    assert paged.kept(w, 8, 3, 0, 0) == [0, 2, 3]
    assert paged.kept(w, 8, 2, 0, 0) == [0, 2]
    assert paged.kept(w, 8, 6, 0, 0) == [0, 1, 2, 3, 5, 7]
    assert paged.kept(w, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]
    assert paged.kept(w, 8, 2, 1, 1) == [0, 7]
    c = small([10, 3])
    k0 = c["k"].copy()
    idx = paged.evict(c, 6, 1, 2)
    assert list(c["lens"]) == [6, 3] and list(idx[1, 0]) == [0, 1, 2, -1, -1, -1]
    for i, j in enumerate(idx[0, 1]):
        assert (c["k"][c["table"][0, i // 4], i % 4, 1] == k0[c["table"][0, j // 4], j % 4, 1]).all()


def test_oracle_append_leaves_a_full_sequence():
    c = small([12, 11, 5])
    k = np.ones((4, 2, 3))
    paged.append(c, k, -k, [0, 1, 2, 4])
    assert list(c["lens"]) == [12, 12, 7]
    assert (c["v"][c["table"][1, 2], 3] == -1).all() and (c["w"][c["table"][2, 1], :, 1] == 0).all()
    paged.append(c, k, k, [0, 2, 1, 4])
    assert list(c["lens"]) == [12, 12, 7]
