"""Per-head key-value caches on the GPU against the fp64 oracle: append, one-token
attention with accumulated weights, eviction, and the three as a decode loop.

Moved data (append, eviction, its weights and positions) has to be equal bit for
bit.  The attention's tolerances are derived per element (`attend_bounds`), from
u = half an ulp of the cache's type and e = 2^-24 of fp32:
  * a score is a d-term fp32 dot product of exact products, scaled twice, so it
    is off by at most dz = (d + 4) e scale sum|q k| + 4 e |z|;
  * exp2 of the difference to a running maximum adds 2 ulp and the rounding of
    its argument: a probability's relative error is at most
    dp = 2 dz + 8 e (1 + |z - lse|), with n more roundings in its sums: n e;
  * a probability is rounded to the type before the product with the values: u
    relative, and in fp16 below 2^-14 half a subnormal step, 2^-25 absolute
    relative to the largest one (whose denominator is at least 1);
  * the output is rounded once: u |out|.
"""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def make_cache(g, B, cap, page, Hkv, d, dtype=torch.bfloat16, layout="token", shared=False, spare=2):
    """(KVCache, page table or None): shuffled pages, or contiguous for page 0."""
    import compressed_sparse_kv_03_b200 as csa
    table = None
    n, ps = B, cap
    if page:
        per = -(-cap // page)
        n, ps = B * per + spare, page
        table = torch.randperm(n, generator=g)[:B * per].to(torch.int32).reshape(B, per).cuda()

    def one():
        if layout == "head":          # [pages, heads, page_size, d]
            return torch.randn(n, Hkv, ps, d, generator=g).to(dtype).cuda().transpose(1, 2)
        return torch.randn(n, ps, Hkv, d, generator=g).to(dtype).cuda()
    if layout == "interleaved":       # keys and values in one allocation, with room between rows
        both = torch.randn(n, 2, ps, Hkv, d + 8, generator=g).to(dtype).cuda()
        k, v = both[:, 0, :, :, :d], both[:, 1, :, :, :d]
    else:
        k = one()
        v = k if shared else one()
    return csa.KVCache(k, v, table), table


def attend_bounds(q, k, v, table, lens, scale, window, sink, prob, lse, out, dtype):
    """(out, lse, probability) tolerances per element, as derived above."""
    u = torch.finfo(dtype).eps / 2
    B, H, d = q.shape
    G = H // k.shape[2]
    t_out, t_lse, t_p = np.zeros_like(out), np.zeros_like(lse), []
    for b in range(B):
        n = int(lens[b])
        kb, vb = np.abs(oracle.kv_rows(k, table, b, n)), np.abs(oracle.kv_rows(v, table, b, n))
        z0 = oracle.kv_rows(k, table, b, n)
        tp = np.zeros((H, n))
        for h in range(H):
            seen = prob[b][h] > 0
            if not n or not seen.any():
                continue
            z = scale * (z0[:, h // G] @ q[b, h])
            dz = (d + 4) * E * abs(scale) * (kb[:, h // G] @ np.abs(q[b, h])) + 4 * E * np.abs(z)
            dp = 2 * dz + 8 * E * (1 + np.abs(z - lse[b, h])) + n * E + 2 * dz[seen].max()
            tp[h] = prob[b][h] * dp
            t_lse[b, h] = dz[seen].max() + (n + 16) * E + 4 * E * abs(lse[b, h])
            sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
            t_out[b, h] = u * np.abs(out[b, h]) + ((prob[b][h] * (u + dp) + sub * seen)[:, None] * vb[:, h // G]).sum(0) \
                + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133)
        t_p.append(tp)
    return t_out, t_lse, t_p


def check_attend(cache, table, q, lens, scale, window=0, sink=None, weigh=False, inplace=False, got=None, **kw):
    import compressed_sparse_kv_03_b200 as csa
    B, H, d = q.shape
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ds = None if sink is None else sink.cuda()
    ws = csa.Workspace("cuda")
    w0 = None
    if weigh:
        w0 = torch.rand(B, cache.n_kv_heads, cache.capacity + 3, generator=torch.Generator().manual_seed(9)).cuda()
        wo = w0.clone() if inplace else torch.full_like(w0, -7.0)
        w_in = wo if inplace else w0
        out, lse = csa.kv_attn_decode(q, cache, dl, scale, window=window, sink=ds, weights=w_in, weights_out=wo,
                                      return_lse=True, ws=ws, **kw)
    else:
        out, lse = csa.kv_attn_decode(q, cache, dl, scale, window=window, sink=ds, return_lse=True, ws=ws, **kw)
    ws.check()
    tb = None if table is None else table.cpu().numpy()
    k, v, qq = f64(cache.k), f64(cache.v), f64(q)
    zs = None if sink is None else f64(sink)
    ro, rl, rp = oracle.kv_attend(qq, k, v, tb, lens, scale, window, zs)
    to, tl, tp = attend_bounds(qq, k, v, tb, lens, scale, window, zs, rp, rl, ro, cache.dtype)
    go, gl = f64(out), f64(lse)
    assert np.all(np.isfinite(go))
    bad = np.abs(go - ro) > to
    assert not bad.any(), f"output: {bad.sum()} of {bad.size}, worst {np.max(np.abs(go - ro) - to):.3g}"
    empty = np.isinf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(np.abs(gl[~empty] - rl[~empty]) <= tl[~empty] + 4 * E * np.abs(rl[~empty]))
    if weigh:
        gw = f64(wo)
        for b in range(B):
            n = int(lens[b])
            want = f64(w0)[b, :, :n] + rp[b].reshape(cache.n_kv_heads, -1, n).sum(1) if n else None
            if n:
                tol = tp[b].reshape(cache.n_kv_heads, -1, n).sum(1) + 4 * E * np.abs(want) + (H // cache.n_kv_heads) * E * want
                assert np.all(np.abs(gw[b, :, :n] - want) <= tol)
            rest = f64(w0)[b, :, n:] if inplace else -7.0
            assert np.all(gw[b, :, n:] == rest)     # behind the sequence: as it was
    return out, lse


# B, H, Hkv, d, lens (or max), page, layout
ATTEND = [
    (1, 1, 1, 8, [1], 1, "token"),
    (1, 4, 4, 64, [17], 16, "token"),
    (2, 8, 1, 128, [0, 300], 64, "token"),
    (3, 16, 2, 128, [129, 1, 640], 16, "token"),
    (3, 20, 4, 96, [700, 15, 16], 0, "token"),
    (2, 20, 20, 72, [65, 64], 5, "token"),
    (2, 34, 2, 128, [513, 250], 64, "token"),            # 17 heads a group: two warps side by side
    (2, 64, 2, 64, [100, 1100], 32, "head"),
    (2, 64, 1, 128, [1000, 777], 64, "token"),           # 64 heads: four
    (1, 128, 1, 128, [900], 16, "token"),                # 128: two head blocks
    (3, 51, 3, 96, [1, 300, 511], 48, "interleaved"),    # 17 heads on the tensor cores, boxes of 16 rows
    (3, 66, 2, 64, [257, 640, 0], 128, "token"),         # 33 heads, boxes of 128
    (2, 64, 1, 8, [700, 129], 0, "token"),
    (2, 40, 1, 72, [100, 255], 0, "head"),               # a CTA per sequence
    (2, 200, 2, 128, [1500, 130], 32, "head"),           # 100 heads: two blocks
    (5, 64, 1, 128, [9000, 1, 128, 127, 129], 256, "token"),
    (2, 64, 1, 128, [600, 200], 9, "token"),             # pages without a 16-row box
    (2, 280, 8, 128, [30000, 5000], 16, "token"),        # 16 tiles of 128 slots a CTA, and 17
    (1, 272, 16, 64, [20000], 64, "head"),
    (2, 64, 32, 128, [5000, 4000], 64, "token"),         # many tiles a CTA on mma.sync as well
    (2, 100, 1, 192, [400, 33], 7, "token"),
    (2, 12, 3, 192, [333, 2], 64, "token"),
    (2, 16, 4, 256, [450, 31], 100, "token"),
    (1, 40, 1, 256, [200], 0, "head"),
    (1, 64, 1, 256, [300], 16, "interleaved"),
    (4, 8, 2, 128, [80, 0, 1, 200], 3, "interleaved"),
    (70, 8, 2, 64, None, 16, "token"),                   # more sequences than a warp; ragged
    (2, 8, 8, 128, [5000, 40], 64, "token"),             # many CTAs per unit
    (300, 4, 2, 64, None, 16, "token"),                  # several sequences a thread where runs are cut
    (200, 20, 1, 64, None, 16, "token"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c[:4]) + f"-p{c[5]}{c[6][0]}")
def test_attention_matches_oracle(case, dtype):
    B, H, Hkv, d, lens, page, layout = case
    g = torch.Generator().manual_seed(11)
    if lens is None:
        lens = torch.randint(0, 400, (B,), generator=g).tolist()
    cache, table = make_cache(g, B, max(lens), page, Hkv, d, dtype, layout)
    q = (2 * torch.randn(B, H, d, generator=g)).to(dtype).cuda()
    check_attend(cache, table, q, lens, 1 / math.sqrt(d))


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("G", [8, 20, 40])
@pytest.mark.parametrize("window", [1, 15, 16, 100, 128, 500, 5000])
def test_attention_window_and_sink(window, G, sink):
    g = torch.Generator().manual_seed(12)
    lens = [0, 1, 16, 99, 250, 1001]
    for page in (16, 7):
        cache, table = make_cache(g, 6, 1001, page, 2, 128)
        q = (2 * torch.randn(6, 2 * G, 128, generator=g)).bfloat16().cuda()
        check_attend(cache, table, q, lens, 0.09, window=window, sink=torch.randn(2 * G, generator=g) * 3 if sink else None)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", [(3, 8, 2, 128, [40, 0, 64], 16), (3, 16, 2, 64, [900, 1, 333], 16),
                                  (2, 34, 2, 128, [1500, 20], 64), (2, 64, 1, 128, [1030, 600], 64),
                                  (2, 128, 1, 64, [300, 1200], 5), (40, 4, 4, 96, None, 0), (3, 96, 1, 128, [200, 1, 3000], 32),
                                  (2, 40, 2, 64, [129, 900], 16), (2, 32, 1, 128, [100, 255], 0)],
                         ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_accumulated_weights(case, inplace):
    B, H, Hkv, d, lens, page = case
    g = torch.Generator().manual_seed(13)
    if lens is None:
        lens = torch.randint(0, 300, (B,), generator=g).tolist()
    cache, table = make_cache(g, B, max(lens), page, Hkv, d)
    q = (2 * torch.randn(B, H, d, generator=g)).bfloat16().cuda()
    sink = torch.randn(H, generator=g) if inplace else None
    check_attend(cache, table, q, lens, 1 / math.sqrt(d), sink=sink, weigh=True, inplace=inplace)


def test_weights_without_an_input_start_at_zero():
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(14)
    cache, _ = make_cache(g, 2, 500, 16, 2, 64)
    q = torch.randn(2, 8, 64, generator=g).bfloat16().cuda()
    lens = torch.tensor([500, 3], dtype=torch.int32, device="cuda")
    wo = torch.full((2, 2, cache.capacity), 5.0, device="cuda")
    csa.kv_attn_decode(q, cache, lens, 0.125, weights_out=wo)
    zero = torch.zeros_like(wo)
    csa.kv_attn_decode(q, cache, lens, 0.125, weights=zero)
    assert torch.equal(wo[0, :, :500], zero[0, :, :500]) and torch.equal(wo[1, :, :3], zero[1, :, :3])
    assert torch.all(wo[1, :, 3:] == 5) and torch.all(zero[1, :, 3:] == 0)
    assert torch.allclose(wo[0, :, :500].sum(-1), torch.full((2,), 4.0, device="cuda"), atol=1e-4)


@pytest.mark.parametrize("G", [1, 16, 32, 40])
def test_masked_slots_are_never_read(G):
    """Infinities and NaN in free slots, in other pages and before the window."""
    g = torch.Generator().manual_seed(15)
    lens = [33, 200, 0]
    cache, table = make_cache(g, 3, 200, 16, 1, 128)
    for b, n in enumerate(lens):
        for s in range(n, cache.capacity):
            page, row = table[b, s // 16], s % 16
            cache.k[page, row] = float("nan")
            cache.v[page, row] = float("inf") if s % 2 else float("nan")
    free = sorted(set(range(cache.k.shape[0])) - set(table.flatten().tolist()))
    cache.k[free] = float("nan")
    q = torch.randn(3, G, 128, generator=g).bfloat16().cuda()
    clean_k, clean_v = torch.nan_to_num(cache.k, 0, 0, 0), torch.nan_to_num(cache.v, 0, 0, 0)
    import compressed_sparse_kv_03_b200 as csa
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = csa.kv_attn_decode(q, cache, dl, 0.1, return_lse=True)
    b = csa.kv_attn_decode(q, csa.KVCache(clean_k, clean_v, table), dl, 0.1, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0]).all()
    # before a window
    cache.k[table[1, :5].long()] = float("nan")
    cache.v[table[1, :5].long()] = float("inf")
    out = csa.kv_attn_decode(q, cache, dl, 0.1, window=100)
    assert torch.isfinite(out[1]).all()


@pytest.mark.parametrize("G", [2, 24, 64])
def test_nan_of_a_seen_slot_reaches_the_output(G):
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(16)
    cache, table = make_cache(g, 2, 300, 16, 2, 64)
    cache.k[table[0, 3], 1, 0, 5] = float("nan")
    q = torch.randn(2, 2 * G, 64, generator=g).bfloat16().cuda()
    out = csa.kv_attn_decode(q, cache, torch.tensor([300, 300], dtype=torch.int32, device="cuda"), 0.1)
    assert torch.isnan(out[0, :G]).all() and torch.isfinite(out[0, G:]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("G", [4, 24, 64])
def test_scores_that_grow_along_the_cache(G):
    """Every block of slots scores far above the ones before it, so the running
    maximum moves again and again (and once, in the last block, downwards)."""
    g = torch.Generator().manual_seed(31)
    n, d = 1500, 128
    cache, table = make_cache(g, 2, n, 64, 1, d)
    q = torch.randn(2, G, d, generator=g).abs().bfloat16().cuda()
    level = (torch.arange(n) // 100).float() * 0.05
    level[-100:] = -0.3
    for b in range(2):
        for s in range(n):
            cache.k[table[b, s // 64], s % 64] += level[s]
    check_attend(cache, table, q, [n, 1023], 1.0, weigh=True)


def test_shared_key_value_memory_and_strided_queries():
    g = torch.Generator().manual_seed(17)
    cache, table = make_cache(g, 3, 700, 64, 1, 128, shared=True)
    qkv = torch.randn(3, 70, 128, generator=g).bfloat16().cuda()
    check_attend(cache, table, qkv[:, 2:66], [700, 64, 5], 0.088)
    check_attend(cache, table, qkv[:, 1:65:4], [700, 64, 5], 0.088, weigh=True)
    cache, table = make_cache(g, 1, 12000, 64, 8, 64, shared=True)      # several tiles a CTA on one copy
    q = torch.randn(1, 8 * 40, 64, generator=g).bfloat16().cuda()
    check_attend(cache, table, q, [12000], 0.125)


def test_equal_scores_and_a_dominant_slot():
    """All keys equal: the mean of the values; one key far above: its value."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(18)
    cache, table = make_cache(g, 1, 333, 16, 1, 64)
    q = torch.ones(1, 3, 64, dtype=torch.bfloat16, device="cuda")
    cache.k.fill_(0.25)
    check_attend(cache, table, q, [333], 1.0)
    cache.k[table[0, 7], 3] = 4.0    # score 256 against 16
    out, lse = check_attend(cache, table, q, [333], 1.0)
    assert torch.equal(out[0, 0], cache.v[table[0, 7], 3, 0])
    assert abs(float(lse[0, 0]) - 256) < 1e-3


@pytest.mark.parametrize("H", [4, 48, 80])
def test_bad_lengths_and_pages_are_recorded(H):
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(19)
    cache, table = make_cache(g, 3, 160, 16, 2, 64)
    q = torch.randn(3, H, 64, generator=g).bfloat16().cuda()
    ws = csa.Workspace("cuda")
    lens = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = csa.kv_attn_decode(q, cache, lens(160, 100, 7), 0.1, ws=ws)
    ws.check()
    out = csa.kv_attn_decode(q, cache, lens(-5, 100, 1000), 0.1, ws=ws)
    with pytest.raises(csa.CsaError, match="sequence length"):
        ws.check()
    assert torch.all(out[0] == 0) and torch.equal(out[1], good[1])
    assert torch.equal(out[2], csa.kv_attn_decode(q, cache, lens(1, 1, 160), 0.1)[2])
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 2] = bad     # slots 32..47 of sequence 1
        out = csa.kv_attn_decode(q, csa.KVCache(cache.k, cache.v, t), lens(160, 100, 7), 0.1, ws=ws)
        with pytest.raises(csa.CsaError, match="page id"):
            ws.check()
        rows = [s for s in range(100) if not 32 <= s < 48]
        k = torch.stack([cache.k[table[1, s // 16], s % 16] for s in rows])[None].contiguous()
        v = torch.stack([cache.v[table[1, s // 16], s % 16] for s in rows])[None].contiguous()
        want = csa.kv_attn_decode(q[1:2], csa.KVCache(k, v), lens(len(rows)), 0.1)
        assert torch.allclose(out[1].float(), want[0].float(), atol=2e-2)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


@pytest.mark.parametrize("G", [8, 40])
def test_runs_are_bit_identical_and_batch_invariant_mode(G):
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(20)
    lens = [3000, 1, 0, 511, 512, 513, 1400]
    cache, table = make_cache(g, 7, 3000, 64, 2, 128)
    q = torch.randn(7, 2 * G, 128, generator=g).bfloat16().cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = csa.kv_attn_decode(q, cache, dl, 0.09, return_lse=True)
    b = csa.kv_attn_decode(q, cache, dl, 0.09, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    csa.set_batch_invariant(True)
    try:
        check_attend(cache, table, q, lens, 0.09, weigh=True)
        check_attend(cache, table, q, lens, 0.09, window=700)
        w = torch.zeros(7, 2, 3008, device="cuda")
        full = csa.kv_attn_decode(q, cache, dl, 0.09, return_lse=True, weights_out=w)
        for i in range(7):
            one = csa.KVCache(cache.k, cache.v, table[i:i + 1].contiguous())
            w1 = torch.zeros(1, 2, 3008, device="cuda")
            o, l = csa.kv_attn_decode(q[i:i + 1], one, dl[i:i + 1], 0.09, return_lse=True, weights_out=w1)
            assert torch.equal(o[0], full[0][i]) and torch.equal(l[0], full[1][i]) and torch.equal(w1[0], w[i])
    finally:
        csa.set_batch_invariant(False)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements, read at its far end."""
    import compressed_sparse_kv_03_b200 as csa
    pages, page, Hkv, d = 17000, 128, 8, 128          # 2.2e9 elements, 4.5 GB each for keys and values
    k = torch.empty(pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = [pages - 1, 3, pages - 7]
    g = torch.Generator().manual_seed(21)
    for p in used:
        k[p] = torch.randn(page, Hkv, d, generator=g).bfloat16().cuda()
        v[p] = torch.randn(page, Hkv, d, generator=g).bfloat16().cuda()
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, d, generator=g).bfloat16().cuda()
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    out = csa.kv_attn_decode(q, csa.KVCache(k, v, table), n, 0.09)
    near = csa.KVCache(k[used].contiguous(), v[used].contiguous(), torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, csa.kv_attn_decode(q, near, n, 0.09))
    # append and evict there
    new = torch.randn(1, 2 * Hkv, d, generator=g).bfloat16().cuda()
    cache = csa.KVCache(k, v, table)
    assert csa.kv_append(new[:, :Hkv], new[:, Hkv:], cache, n).tolist() == [301]
    assert torch.equal(k[pages - 7, 300 - 256], new[0, :Hkv]) and torch.equal(v[pages - 7, 300 - 256], new[0, Hkv:])
    w = torch.zeros(1, Hkv, 384, device="cuda")
    w[:, :, 1:] = 1
    sp = torch.arange(384, dtype=torch.int32, device="cuda").expand(1, Hkv, 384).contiguous()
    csa.kv_evict(cache, n, w, sp, torch.tensor([300], dtype=torch.int32, device="cuda"), 300, 1)
    assert n.tolist() == [300] and torch.equal(k[pages - 1, 0], new[0, :Hkv])


# ---- append -------------------------------------------------------------------
@pytest.mark.parametrize("page,layout", [(16, "token"), (5, "interleaved"), (0, "token"), (64, "head"), (1, "token")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_matches_oracle(page, layout, dtype):
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(22)
    B, Hkv, d, cap = 5, 3, 72, 120
    for new, track, inplace in (([1] * B, True, True), ([3, 0, 40, 1, 17], True, False), ([0] * B, False, True),
                                ([9, 100, 2, 0, 30], False, True)):
        cache, table = make_cache(g, B, cap, page, Hkv, d, dtype, layout)
        lens = [0, 7, 60, 33, 90]
        one = new == [1] * B
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(start[-1])
        kv = torch.randn(T, 2 * Hkv + 1, d, generator=g).to(dtype).cuda()
        kn, vn = kv[:, :Hkv], kv[:, Hkv + 1:]
        dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        w = torch.rand(B, Hkv, cap, generator=g).cuda() if track else None
        sp = torch.randint(0, 99, (B, Hkv, cap), generator=g, dtype=torch.int32).cuda() if track else None
        pos = [100, 7, 61, 1000, 90]
        want = oracle.kv_append(f64(cache.k), f64(cache.v), None if table is None else table.cpu().numpy(), lens, f64(kn),
                                f64(vn), None if one else start, None if w is None else f64(w),
                                None if sp is None else sp.cpu().numpy(), pos)
        ws = csa.Workspace("cuda")
        out = csa.kv_append(kn, vn, cache, dl, token_start=None if one else torch.from_numpy(start).cuda(),
                            pos=torch.tensor(pos, dtype=torch.int32, device="cuda") if track else None, weights=w, slot_pos=sp,
                            lens_out=None if inplace else torch.empty_like(dl), ws=ws)
        dropped = any(a + b > (cap if track or not page else -(-cap // page) * page) for a, b in zip(lens, new))
        if dropped:
            with pytest.raises(csa.CsaError, match="no room"):
                ws.check()
        ws.check()
        assert np.array_equal(f64(cache.k), want[0]) and np.array_equal(f64(cache.v), want[1])
        assert out.cpu().tolist() == want[2].tolist() and (inplace or dl.tolist() == lens)
        if track:
            assert np.array_equal(f64(w), want[3]) and np.array_equal(sp.cpu().numpy(), want[4])


def test_append_records_bad_lengths_and_pages():
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(23)
    cache, table = make_cache(g, 3, 48, 16, 2, 64)
    before = cache.k.clone()
    kv = torch.randn(3, 4, 64, generator=g).bfloat16().cuda()
    ws = csa.Workspace("cuda")
    lens = torch.tensor([-1, 10, 48], dtype=torch.int32, device="cuda")
    out = csa.kv_append(kv[:, :2], kv[:, 2:], cache, lens, ws=ws, lens_out=torch.empty_like(lens))
    with pytest.raises(csa.CsaError):
        ws.check()
    assert out.tolist() == [-1, 11, 48]
    before[table[1, 0], 10] = kv[1, :2]
    assert torch.equal(cache.k, before)
    t = table.clone()
    t[1, 0] = cache.k.shape[0]
    csa.kv_append(kv[:, :2], kv[:, 2:], csa.KVCache(cache.k, cache.v, t),
                  torch.tensor([48, 10, 48], dtype=torch.int32, device="cuda"), ws=ws)
    with pytest.raises(csa.CsaError):
        ws.check()
    assert torch.equal(cache.k, before)


# ---- eviction -------------------------------------------------------------------
def evict_state(g, B, Hkv, n, slots, lens, budget, recent, ties=False, settled=True):
    w = torch.rand(B, Hkv, slots, generator=g) ** 4
    if ties:
        w = (w * 4).floor()
    sp = torch.arange(slots, dtype=torch.int32).expand(B, Hkv, slots).clone()
    if settled:
        for b in range(B):
            for h in range(Hkv):
                m = max(1, min(budget, lens[b]) - recent)
                sp[b, h, :m] = torch.randperm(m, generator=g).to(torch.int32)
    return w.cuda(), sp.cuda(), torch.tensor([max(x - 1, 0) for x in lens], dtype=torch.int32, device="cuda")


EVICT = [  # B, Hkv, d, lens, page, budget, recent, first, ties
    (1, 1, 8, [2], 1, 1, 1, 0, False),
    (2, 2, 64, [33, 32], 16, 32, 4, 0, False),
    (3, 2, 128, [100, 10, 41], 16, 40, 8, 2, True),
    (2, 3, 72, [300, 299], 5, 100, 99, 1, False),
    (2, 2, 128, [2000, 700], 64, 700, 64, 4, True),
    (1, 2, 64, [5000], 0, 1000, 100, 4, True),
    (1, 1, 256, [9000], 64, 2048, 512, 0, False),
    (9, 8, 64, [65, 64, 80, 1, 0, 70, 66, 79, 67], 16, 64, 16, 4, True),
    (1, 2, 64, [5001], 0, 5000, 100, 4, True),           # one slot too many, over a cluster
    (3, 2, 64, [1500, 1501, 1600], 16, 1500, 100, 4, False),
    (40, 8, 8, [700] * 40, 16, 90, 10, 4, True),         # more moves than are listed in shared memory
    (2, 2, 64, [50, 64], 16, 100, 10, 4, False),         # a budget above the cache's room
]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("layout", ["token", "head", "interleaved"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{max(c[3])}to{c[5]}")
def test_evict_matches_oracle(case, layout, inplace):
    import compressed_sparse_kv_03_b200 as csa
    B, Hkv, d, lens, page, budget, recent, first, ties = case
    g = torch.Generator().manual_seed(24)
    cache, table = make_cache(g, B, max(lens), page, Hkv, d, torch.float16 if layout == "head" else torch.bfloat16, layout)
    slots = cache.capacity + 5
    w, sp, pos = evict_state(g, B, Hkv, max(lens), slots, lens, budget, recent, ties)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ml = cache.capacity
    want = oracle.kv_evict(f64(cache.k), f64(cache.v), None if table is None else table.cpu().numpy(), np.array(lens), f64(w),
                           sp.cpu().numpy(), pos.tolist(), budget, recent, first, ml, inplace)
    wo, so, lo = (w, sp, dl) if inplace else (w.clone(), sp.clone(), torch.empty_like(dl))
    ws = csa.Workspace("cuda")
    n, src = csa.kv_evict(cache, dl, w, sp, pos, budget, recent, keep_first=first, max_len=ml, lens_out=lo, weights_out=wo,
                          slot_pos_out=so, return_src=True, ws=ws)
    ws.check()
    assert n.tolist() == want[2].tolist()
    assert np.array_equal(src.cpu().numpy(), want[5])
    assert np.array_equal(f64(wo), want[3]) and np.array_equal(so.cpu().numpy(), want[4])
    assert np.array_equal(f64(cache.k), want[0]) and np.array_equal(f64(cache.v), want[1])


@pytest.mark.parametrize("n", [700, 301])
@pytest.mark.parametrize("kind", ["zero", "nan", "inf", "negative", "held", "tail"])
def test_evict_of_special_weights(kind, n):
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(25)
    B, Hkv, budget = 2, 2, 300
    cache, table = make_cache(g, B, n, 64, Hkv, 64)
    w, sp, pos = evict_state(g, B, Hkv, n, n, [n, n], budget, 10)
    if kind == "zero":
        w.zero_()
        w[:, :, ::3] = -0.0
    elif kind == "nan":
        w[:, :, 5::2] = float("nan")
    elif kind == "inf":
        w[:, :, 3::5] = float("inf")
        w[:, :, 4::5] = -float("inf")
        w[0, 0, 9] = float("nan")
    elif kind == "negative":
        w.sub_(0.5)
    elif kind == "tail":     # the newest tokens lie low, the highest slots weigh least
        sp.copy_(sp.flip(-1))
        w[:, :, budget:] *= 1e-6
    else:
        sp.fill_(n)      # every slot claims to be recent: the lower ones stay
    dl = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    want = oracle.kv_evict(f64(cache.k), f64(cache.v), table.cpu().numpy(), np.array([n, n]), f64(w), sp.cpu().numpy(),
                           pos.tolist(), budget, 10)
    _, src = csa.kv_evict(cache, dl, w, sp, pos, budget, 10, return_src=True)
    assert np.array_equal(src.cpu().numpy(), want[5])
    assert np.array_equal(f64(w), want[3], equal_nan=True) and np.array_equal(f64(cache.k), want[0])


def test_evict_of_more_slots_than_shared_memory_holds():
    """300000 slots in one head: keys beyond the cached ones are read again."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(26)
    n, budget, recent, first = 300000, 1234, 100, 3
    k = torch.randn(1, n, 1, 8, generator=g).bfloat16().cuda()
    cache = csa.KVCache(k, k.clone())
    w = torch.randint(0, 5000, (1, 1, n), generator=g).float().cuda()     # many ties
    sp = torch.arange(n, dtype=torch.int32, device="cuda")[None, None].contiguous()
    rank = w[0, 0].double().clone()
    rank[n - recent:] = 1e9
    rank[:first] = 1e9
    stay = rank.sort(descending=True, stable=True).indices[:budget].sort().values
    low = stay[stay < budget]
    src = torch.arange(budget, device="cuda")
    hole = torch.ones(budget, dtype=torch.bool, device="cuda")
    hole[low] = False
    src[hole] = stay[stay >= budget]
    k0 = k.clone()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for inplace in (False, True):
        k.copy_(k0)
        w1, s1 = (w, sp) if inplace else (torch.empty_like(w), torch.empty_like(sp))
        w0 = w.clone()
        new, got = csa.kv_evict(cache, lens, w, sp, torch.tensor([n - 1], dtype=torch.int32, device="cuda"), budget, recent,
                                keep_first=first, return_src=True, weights_out=w1, slot_pos_out=s1, lens_out=torch.empty_like(lens))
        assert new.tolist() == [budget] and torch.equal(got[0, 0].long(), src)
        assert torch.equal(w1[0, 0, :budget], w0[0, 0, src]) and torch.all(w1[0, 0, budget:] == 0)
        assert torch.equal(s1[0, 0, :budget].long(), src) and torch.all(s1[0, 0, budget:] == 0)
        assert torch.equal(k[0, :budget], k0[0, src]) and torch.equal(k[0, budget:], k0[0, budget:])


def test_evict_with_shared_memory_bad_lengths_and_pages():
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(27)
    cache, table = make_cache(g, 2, 200, 16, 1, 128, shared=True)
    w, sp, pos = evict_state(g, 2, 1, 200, 208, [200, 200], 100, 10)
    k0 = cache.k.clone()
    dl = torch.tensor([200, 200], dtype=torch.int32, device="cuda")
    w0 = w.clone()
    _, src = csa.kv_evict(cache, dl, w, sp, pos, 100, 10, return_src=True)
    for b in range(2):
        for j, s in enumerate(src[b, 0].tolist()):
            assert torch.equal(cache.k[table[b, j // 16], j % 16], k0[table[b, s // 16], s % 16])
            assert w[b, 0, j] == w0[b, 0, s]
    ws = csa.Workspace("cuda")
    out = csa.kv_evict(cache, torch.tensor([-3, 999], dtype=torch.int32, device="cuda"), w, sp, pos, 100, 10, ws=ws)
    with pytest.raises(csa.CsaError, match="sequence length"):
        ws.check()
    assert out.tolist() == [0, 100]
    t = table.clone()
    t[0] = -1
    k1 = cache.k.clone()
    w, sp, pos = evict_state(g, 2, 1, 200, 208, [200, 200], 100, 10)
    out = csa.kv_evict(csa.KVCache(cache.k, cache.v, t), torch.tensor([200, 0], dtype=torch.int32, device="cuda"), w, sp, pos,
                       100, 10, ws=ws)
    with pytest.raises(csa.CsaError, match="page id"):
        ws.check()
    assert torch.equal(cache.k, k1) and out.tolist() == [100, 0]


# ---- together -------------------------------------------------------------------
@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop_with_eviction(graph):
    """Prompts appended, then steps of append, attention with accumulated weights
    and eviction, all in place and (graph) captured once and replayed; the
    oracle does the same with its own cache, taking the weights that the GPU
    accumulated, so that the choices can be compared exactly."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(28)
    B, H, Hkv, d, page, budget, recent, cap = 3, 16, 4, 64, 16, 48, 8, 64
    cache, table = make_cache(g, B, cap, page, Hkv, d)
    tb = table.cpu().numpy()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, cap, device="cuda")
    sp = torch.zeros(B, Hkv, cap, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    prompt = [40, 47, 1]
    start = torch.tensor([0, 40, 87, 88], dtype=torch.int32, device="cuda")
    kv = torch.randn(88, 2 * Hkv, d, generator=g).bfloat16().cuda()
    ok, ov = f64(cache.k), f64(cache.v)
    ok, ov, on, ow, osp = oracle.kv_append(ok, ov, tb, [0, 0, 0], f64(kv[:, :Hkv]), f64(kv[:, Hkv:]), start.cpu().numpy(), f64(w),
                                           sp.cpu().numpy(), [0, 0, 0])
    csa.kv_append(kv[:, :Hkv], kv[:, Hkv:], cache, lens, token_start=start, pos=pos, weights=w, slot_pos=sp)
    pos.copy_(lens)
    q = torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda")
    kn, vn = torch.empty(B, Hkv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hkv, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = csa.Workspace("cuda")
    w_seen = torch.empty_like(w)

    def step():
        csa.kv_append(kn, vn, cache, lens, pos=pos, weights=w, slot_pos=sp, ws=ws)
        csa.kv_attn_decode(q, cache, lens, 0.2, weights=w, out=out, ws=ws)
        w_seen.copy_(w)
        csa.kv_evict(cache, lens, w, sp, pos, budget, recent, keep_first=2, ws=ws)

    replay = step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        keep = [x.clone() for x in (cache.k, cache.v, lens, w, sp)]
        with torch.cuda.stream(side):
            kn.zero_(), vn.zero_(), q.zero_()
            step()                   # sizes the workspace before the capture
        torch.cuda.current_stream().wait_stream(side)
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        for x, y in zip((cache.k, cache.v, lens, w, sp), keep):
            x.copy_(y)
        replay = cg.replay
    for i in range(20):
        q.copy_(torch.randn(B, H, d, generator=g).bfloat16())
        kn.copy_(torch.randn(B, Hkv, d, generator=g).bfloat16())
        vn.copy_(torch.randn(B, Hkv, d, generator=g).bfloat16())
        replay()
        at = [p + i for p in prompt]
        ok, ov, on, ow, osp = oracle.kv_append(ok, ov, tb, on, f64(kn), f64(vn), None, ow, osp, at)
        ro, _, rp = oracle.kv_attend(f64(q), ok, ov, tb, on, 0.2)
        want = oracle.kv_weigh(ow, rp, Hkv)
        got = f64(w_seen)
        assert np.abs(f64(out) - ro).max() < 2e-2
        assert np.abs(got - want).max() < 1e-4      # 20 steps of at most 4 (2 dz + ..): about 1e-5
        ok, ov, on, ow, osp, _ = oracle.kv_evict(ok, ov, tb, on, got, osp, at, budget, recent, 2, cap, inplace=True)
        assert lens.tolist() == list(on)
        assert np.array_equal(f64(w), ow) and np.array_equal(sp.cpu().numpy(), osp)
        assert np.array_equal(f64(cache.k), ok) and np.array_equal(f64(cache.v), ov)
        pos.add_(1)
    ws.check()


def test_two_streams_and_default_workspaces():
    """Calls on two streams at once, without workspaces of their own."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(29)
    jobs = []
    for n in (3000, 2500):
        cache, _ = make_cache(g, 2, n, 16, 2, 128)
        q = torch.randn(2, 16, 128, generator=g).bfloat16().cuda()
        lens = torch.tensor([n, n // 3], dtype=torch.int32, device="cuda")
        w = torch.zeros(2, 2, cache.capacity, device="cuda")
        jobs.append((cache, q, lens, w, csa.kv_attn_decode(q, cache, lens, 0.1, weights_out=w.clone()), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (cache, q, lens, w, _, s) in enumerate(jobs):
            outs[i].append(csa.kv_attn_decode(q, cache, lens, 0.1, weights_out=w, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, jobs[i][4]) for o in outs[i])


def test_a_captured_first_call():
    """Kernels whose first launch is captured, without a workspace of their own."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(32)
    for G, n in ((3, 900), (30, 1300)):
        cache, _ = make_cache(g, 2, n, 16, 2, 88, torch.float16)
        q = torch.randn(2, 2 * G, 88, generator=g).half().cuda()
        lens = torch.tensor([n, n // 3], dtype=torch.int32, device="cuda")
        w = torch.zeros(2, 2, n, device="cuda")     # fewer slots than the pages hold
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            out = csa.kv_attn_decode(q, cache, lens, 0.1, weights=w)
        cg.replay()
        cg.replay()
        w2 = torch.zeros_like(w)
        assert torch.equal(out, csa.kv_attn_decode(q, cache, lens, 0.1, weights=w2))
        assert torch.allclose(w, 2 * w2)


def test_python_argument_checks():
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(30)
    cache, _ = make_cache(g, 2, 64, 16, 2, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    for bad in (q.half(), q.cpu(), q.float()):
        with pytest.raises(TypeError):
            csa.kv_attn_decode(bad, cache, lens, 0.1)
    for bad in (q[:, :, :32], q[0], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            csa.kv_attn_decode(bad, cache, lens, 0.1)
    with pytest.raises(TypeError):
        csa.kv_attn_decode(q, cache, lens.long(), 0.1)
    with pytest.raises(ValueError):
        csa.kv_attn_decode(q, cache, lens[:1], 0.1)
    with pytest.raises(ValueError):
        csa.kv_attn_decode(torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), cache, torch.cat([lens, lens])[:3], 0.1)
    with pytest.raises(csa.CsaError, match="multiple of n_kv_heads"):
        csa.kv_attn_decode(q[:, :3], cache, lens, 0.1)
    with pytest.raises(csa.CsaError, match="window"):
        csa.kv_attn_decode(q, cache, lens, 0.1, window=4, weights_out=torch.zeros(2, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        csa.kv_attn_decode(q, cache, lens, 0.1, sink=torch.zeros(3, device="cuda"))
    w, sp = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")
    with pytest.raises(csa.CsaError, match="budget"):
        csa.kv_evict(cache, lens, w, sp, lens, 4, 5)
    with pytest.raises(TypeError):
        csa.kv_evict(cache, lens, w, w, lens, 4, 2)
    with pytest.raises(csa.CsaError, match="one token per sequence"):
        csa.kv_append(q[:1, :2], q[:1, :2], cache, lens)
    with pytest.raises(csa.CsaError, match="needs pos"):
        csa.kv_append(q[:, :2], q[:, 2:], cache, lens, slot_pos=sp)
    with pytest.raises(csa.CsaError, match="same memory"):
        csa.kv_append(q[:, :2], q[:, 2:], csa.KVCache(cache.k, cache.k, cache.page_table), lens)
    wide = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16, device="cuda").expand(8, 16, 2, 64)
    with pytest.raises(csa.CsaError, match="overlap"):
        csa.kv_append(q[:, :2], q[:, 2:], csa.KVCache(wide, cache.v[:8], cache.page_table), lens)
    # nothing to do
    assert csa.kv_attn_decode(q[:0], cache, lens[:0], 0.1).shape == (0, 4, 64)
    assert csa.kv_append(q[:0, :2], q[:0, 2:], cache, lens[:0]).shape == (0,)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    full = torch.ones(2, 2, 64, device="cuda")
    assert torch.all(csa.kv_attn_decode(q, cache, none, 0.1, max_len=0, weights=full) == 0) and torch.all(full == 1)
    assert csa.kv_evict(cache, none.clone(), full, sp, none, 4, 2, max_len=0).tolist() == [0, 0]
    # broadcast heads can be read
    out = csa.kv_attn_decode(q, csa.KVCache(wide, wide, cache.page_table), lens, 0.1)
    assert torch.all(out == 0)


# ---- promises that hold whatever the batch, the bounds and the free pages --------
@pytest.mark.parametrize("G", [8, 20, 40])
def test_batch_invariant_mode_beside_many_sequences_and_other_bounds(G):
    """A sequence's bits alone, beside 23 others, and under a tighter max_len: the
    order in which slices are joined follows none of these."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(33)
    B, Hkv, d, page, per = 24, 8, 128, 64, 128
    k, v = (torch.randn(160, page, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randint(0, 160, (B, per), generator=g, dtype=torch.int32).cuda()   # reading: pages may be shared
    lens = [3000, 1, 0, 511, 512, 513, 8192] + torch.randint(600, 3000, (B - 7,), generator=g).tolist()
    q = (2 * torch.randn(B, Hkv * G, d, generator=g)).bfloat16().cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(rows, **kw):
        w = torch.zeros(len(rows), Hkv, 8192, device="cuda")
        o, l = csa.kv_attn_decode(q[rows], csa.KVCache(k, v, table[rows]), dl[rows], 0.09, return_lse=True, weights_out=w, **kw)
        plain = csa.kv_attn_decode(q[rows], csa.KVCache(k, v, table[rows]), dl[rows], 0.09, **kw)
        assert torch.equal(o, plain)
        return o, l, w

    csa.set_batch_invariant(True)
    try:
        o, l, w = run(list(range(B)))
        for rows, kw in [([i], {}) for i in range(B)] + [([i], {"max_len": 3000}) for i in (0, 8, 15)] + [
                (list(range(7, B)), {"max_len": 3000}), ([0, 5, 6, 9], {}), ([23, 0, 7], {"max_len": 3001})]:
            o1, l1, w1 = run(rows, **kw)
            for j, i in enumerate(rows):
                assert torch.equal(o1[j], o[i]) and torch.equal(l1[j], l[i]) and torch.equal(w1[j], w[i]), (i, rows, kw)
    finally:
        csa.set_batch_invariant(False)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 7])
@pytest.mark.parametrize("G", [8, 20, 40])
def test_pages_behind_a_window_may_be_gone(G, page):
    """Page ids of slots that no query sees are never looked up: a sliding window's
    cache whose older pages were given back has no page error, and the same bits."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(34)
    lens = [1000, 517, 130, 300, 0, 129]
    cache, table = make_cache(g, 6, 1000, page, 2, 64)
    q = torch.randn(6, 2 * G, 64, generator=g).bfloat16().cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = csa.Workspace("cuda")
    for window in (1, 17, 100, 128, 200):
        want = csa.kv_attn_decode(q, cache, dl, 0.1, window=window, return_lse=True, ws=ws)
        ws.check()
        for gone in (-1, cache.k.shape[0], 2 ** 31 - 1):
            t = table.clone()
            for b, n in enumerate(lens):
                t[b, :max(0, n - window) // page] = gone      # pages wholly before the window
                t[b, -(-n // page):] = gone                   # and behind the sequence
            got = csa.kv_attn_decode(q, csa.KVCache(cache.k, cache.v, t), dl, 0.1, window=window, return_lse=True, ws=ws)
            ws.check()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_used_on_a_second_stream():
    """Memory of a workspace that a call on another stream still uses does not go to
    the first stream's next tensor when the workspace is dropped or grows."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(37)
    cache, _ = make_cache(g, 2, 4000, 16, 2, 64)
    q = torch.randn(2, 16, 64, generator=g).bfloat16().cuda()
    lens = torch.tensor([4000, 99], dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 2, cache.capacity, device="cuda")
    want = csa.kv_attn_decode(q, cache, lens, 0.1)
    for grow in (False, True):
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        ws = csa.Workspace("cuda")
        csa.kv_attn_decode(q, cache, lens, 0.1, ws=ws, stream=a)
        torch.cuda.synchronize()
        at, size = ws.buf.data_ptr(), ws.buf.numel()
        with torch.cuda.stream(b):
            torch.cuda._sleep(400000000)      # some 0.2 s
        out = csa.kv_attn_decode(q, cache, lens, 0.1, ws=ws, stream=b)
        if grow:
            csa.kv_attn_decode(q, cache, lens, 0.1, ws=ws, stream=b, weights=w)
            assert ws.buf.data_ptr() != at
        else:
            del ws
        with torch.cuda.stream(a):
            other = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() != at for t in other)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_sizes_beyond_32_bits_are_refused():
    """An int that does not fit the C argument is refused, not cut to its low bits."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(36)
    cache, _ = make_cache(g, 2, 64, 16, 2, 64)
    lens = torch.tensor([60, 33], dtype=torch.int32, device="cuda")
    w, sp = torch.rand(2, 2, 64, generator=g).cuda(), torch.arange(64, dtype=torch.int32).expand(2, 2, 64).contiguous().cuda()
    k0, w0 = cache.k.clone(), w.clone()
    for kw in (dict(budget=2 ** 32 + 20, recent=4), dict(budget=20, recent=2 ** 32 + 4), dict(budget=20, recent=4, keep_first=2 ** 32),
               dict(budget=20, recent=4, max_len=2 ** 64 + 64), dict(budget=-2 ** 32 + 20, recent=4)):
        with pytest.raises(ValueError, match="out of range"):
            csa.kv_evict(cache, lens, w, sp, lens, **kw)
    q = torch.randn(2, 4, 64, generator=g).bfloat16().cuda()
    for kw in (dict(window=2 ** 32 + 4), dict(max_len=2 ** 64 + 4), dict(window=-2 ** 33)):
        with pytest.raises(ValueError, match="out of range"):
            csa.kv_attn_decode(q, cache, lens, 0.1, **kw)
    assert lens.tolist() == [60, 33] and torch.equal(cache.k, k0) and torch.equal(w, w0)
    # numpy's integers are taken
    a = csa.kv_attn_decode(q, cache, lens, 0.1, window=np.int64(7), max_len=np.int32(64))
    assert torch.equal(a, csa.kv_attn_decode(q, cache, lens, 0.1, window=7))


@pytest.mark.parametrize("G", [8, 12, 40])
@pytest.mark.parametrize("page", [64, 7])
def test_many_small_probabilities_in_fp16(G, page):
    """Four slots 18 nats above 19996 others, whose probabilities (2^-26 of the
    largest) lie below fp16's subnormals and together make the whole output.

    Maxima belong to a run of slots and, up to 16 heads, to a warp that sees 16 of
    every 64, so enough sequences are given that a run holds whole ones, and the
    four slots are 16 apart.  With S = 19996 exp(-18) the output is 16 S / (4 + S).
    On mma.sync the probabilities are scaled by 2^14 and normal numbers, off by u
    relative; on tcgen05 by 2^7 and subnormal, off by at most 2^-25 / 2^7 each.  The
    rest: one rounding of the output, u, and the fp32 exponent, sums and quotient, a
    few dozen roundings and one per summand (E each)."""
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(35)
    n, d, B, Hkv = 20000, 64, 40, 8
    cache, table = make_cache(g, 1, n, page, Hkv, d, torch.float16)
    cache.k.zero_(), cache.v.fill_(16.0)
    for s in (0, 16, 32, 48):
        at = (table[0, s // page].long(), s % page)
        cache.k[at] = torch.tensor([18.0] + [0.0] * (d - 1)).half().cuda()
        cache.v[at] = 0.0
    cache = csa.KVCache(cache.k, cache.v, table.expand(B, -1).contiguous())
    q = torch.zeros(B, Hkv * G, d, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    out, lse = csa.kv_attn_decode(q, cache, torch.full((B,), n, dtype=torch.int32, device="cuda"), 1.0, return_lse=True)
    s = (n - 4) * math.exp(-18.0)
    want, u = 16 * s / (4 + s), 2.0 ** -11
    each = 0.0 if G <= 16 or page == 7 else 2.0 ** -32
    tol = want * (2 * u + (n + 64) * E) + (n - 4) * each * 16 / 4
    assert np.abs(f64(out) - want).max() <= tol, (np.abs(f64(out) - want).max(), want, tol)
    assert np.abs(f64(lse) - (18 + math.log(4 + s))).max() <= (n + 16) * E


def test_two_threads_on_one_stream_with_default_workspaces():
    """Calls of two host threads on the default stream, without workspaces: launches of
    one may come between those of the other."""
    import threading
    import compressed_sparse_kv_03_b200 as csa
    g = torch.Generator().manual_seed(38)
    jobs, errors = [], []
    for n, G in ((5000, 4), (7000, 20)):
        cache, _ = make_cache(g, 3, n, 16, 2, 64)
        q = torch.randn(3, 2 * G, 64, generator=g).bfloat16().cuda()
        lens = torch.tensor([n, n // 3, 5], dtype=torch.int32, device="cuda")
        w, sp, pos = evict_state(g, 3, 2, n, cache.capacity, [n, n // 3, 5], 1000, 100)
        k0, v0 = cache.k.clone(), cache.v.clone()

        def step(cache=cache, q=q, lens=lens, w=w, sp=sp, pos=pos, k0=k0, v0=v0):
            wo, so, lo = torch.zeros_like(w), torch.zeros_like(sp), torch.empty_like(lens)
            cache.k.copy_(k0), cache.v.copy_(v0)
            out = csa.kv_attn_decode(q, cache, lens, 0.1, weights=w, weights_out=wo)
            csa.kv_evict(cache, lens, wo, sp, pos, 1000, 100, lens_out=lo, weights_out=wo, slot_pos_out=so)
            return [out, wo, so, lo, cache.k.clone(), cache.v.clone()]
        jobs.append((step, step()))
    torch.cuda.synchronize()

    def run(step, want):
        try:
            for got in [step() for _ in range(40)]:
                assert all(torch.equal(x, y) for x, y in zip(got, want))
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]
