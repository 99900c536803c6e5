"""Per-head key-value caches without a GPU: the host-side argument checks of
csa_kv_append, csa_kv_attn_decode and csa_kv_evict (nothing is launched), their
workspace sizes, and pins of the fp64 oracle that the GPU tests compare with."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_kv_03_b200 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from compressed_sparse_kv_03_b200 import build
        build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def mem():
    buf = (C.c_uint8 * (1 << 16))()
    base = (C.addressof(buf) + 255) // 256 * 256
    return buf, base


def cache(base, **kw):
    from compressed_sparse_kv_03_b200._lib import KvCacheT
    d, heads, page = kw.pop("head_dim", 64), kw.pop("n_kv_heads", 2), kw.pop("page_size", 4)
    f = dict(k=base, v=base + 16384, n_pages=4, k_page_stride=page * heads * d, k_slot_stride=heads * d, k_head_stride=d,
             v_page_stride=page * heads * d, v_slot_stride=heads * d, v_head_stride=d, page_table=base + 32768, max_pages=2,
             page_size=page, n_kv_heads=heads, head_dim=d, dtype=0)
    f.update(kw)
    return KvCacheT(*[f[n] for n, _ in KvCacheT._fields_])


def rows(base, **kw):
    from compressed_sparse_kv_03_b200._lib import KvRowsT
    f = dict(data=base, token_stride=128, head_stride=64)
    f.update(kw)
    return KvRowsT(f["data"], f["token_stride"], f["head_stride"])


# what every call refuses of a cache: fields, status
BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(dtype=2), 1), (dict(n_pages=0), 1), (dict(page_size=0), 1),
    (dict(n_kv_heads=0), 1), (dict(max_pages=0), 1), (dict(head_dim=12), 1), (dict(head_dim=0), 1), (dict(head_dim=264), 2),
    (dict(k_head_stride=60), 1), (dict(v_page_stride=-8), 1), (dict(max_pages=1 << 30), 2),
]


def bad_caches(base):
    for kw, st in BAD_CACHES:
        yield kw, cache(base, **kw), st
    yield "misaligned", cache(base, k=base + 8), 1


def test_append_refuses_bad_arguments_without_launching(lib, mem):
    _, base = mem
    before = lib.csa_launch_count()
    p = C.c_void_p
    kv, r = cache(base), rows(base)
    # k_new, v_new, kv, token_start, n_tokens, B, lens, lens_out, pos, weights, slot_pos, slots, ws, ws_bytes, stream
    args = [C.byref(r), C.byref(r), C.byref(kv), None, 2, 2, p(base), p(base + 64), None, None, None, 0, p(base), 256, None]

    def st(**kw):
        a = list(args)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return lib.csa_kv_append(*a)

    for what, c, want in bad_caches(base):
        assert st(_2=C.byref(c)) == want, what
        assert b"csa_kv_append" in lib.csa_last_error()
    assert st(_2=None) == 1
    assert st(_2=C.byref(cache(base, k_slot_stride=64))) == 1 and b"overlap" in lib.csa_last_error()
    assert st(_2=C.byref(cache(base, v_page_stride=0))) == 1 and b"overlap" in lib.csa_last_error()
    assert st(_2=C.byref(cache(base, v=base))) == 1 and b"same memory" in lib.csa_last_error()
    assert st(_2=C.byref(cache(base, page_table=None, n_pages=1))) == 1 and b"page per sequence" in lib.csa_last_error()
    assert st(_4=3) == 1 and b"one token per sequence" in lib.csa_last_error()
    assert st(_4=-1) == 1
    assert st(_5=-1) == 1
    assert st(_5=70000, _4=70000) == 2
    assert st(_0=None) == 1 and b"k_new" in lib.csa_last_error()
    assert st(_1=C.byref(rows(base, token_stride=12))) == 1 and b"v_new" in lib.csa_last_error()
    assert st(_0=C.byref(rows(base + 2))) == 1
    assert st(_6=None) == 1 and st(_7=None) == 1
    assert st(_7=p(base + 4)) == 1 and b"apart" in lib.csa_last_error()
    assert st(_10=p(base), _11=8) == 1 and b"needs pos" in lib.csa_last_error()
    assert st(_9=p(base), _11=0) == 1 and b"slots" in lib.csa_last_error()
    assert st(_13=128) == 5
    assert st(_12=p(base + 16)) == 5 and b"aligned" in lib.csa_last_error()
    assert st(_5=0, _4=0) == 0      # nothing to do
    assert lib.csa_launch_count() == before


def test_attention_refuses_bad_arguments_without_launching(lib, mem):
    _, base = mem
    before = lib.csa_launch_count()
    p = C.c_void_p
    kv, r = cache(base), rows(base)
    # q, kv, lens, B, H, max_len, window, sm_scale, sink, out, lse, weights, weights_out, slots, ws, ws_bytes, stream
    out = p(base + 4096)
    args = [C.byref(r), C.byref(kv), p(base), 2, 4, 8, 0, 0.1, None, out, None, None, None, 0, p(base), 1 << 30, None]

    def st(**kw):
        a = list(args)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return lib.csa_kv_attn_decode(*a)

    for what, c, want in bad_caches(base):
        assert st(_1=C.byref(c)) == want, what
        assert b"csa_kv_attn_decode" in lib.csa_last_error()
    assert st(_0=None) == 1
    assert st(_0=C.byref(rows(base, head_stride=4))) == 1
    assert st(_2=None) == 1 and st(_9=None) == 1 and st(_9=p(base + 2)) == 1
    assert st(_9=p(base)) == 1 and b"overlap" in lib.csa_last_error()
    assert st(_3=-1) == 1 and st(_3=65536) == 2
    assert st(_4=0) == 1 and st(_4=3) == 1 and b"multiple" in lib.csa_last_error()
    assert st(_4=258) == 2 and b"128" in lib.csa_last_error()
    assert st(_5=9) == 1 and st(_5=-1) == 1 and b"max_len" in lib.csa_last_error()
    assert st(_6=-1) == 1
    assert st(_7=float("nan")) == 1
    assert st(_11=p(base)) == 1 and b"weights_out" in lib.csa_last_error()
    assert st(_12=p(base), _13=7) == 1 and b"slots" in lib.csa_last_error()
    assert st(_12=p(base), _13=8, _6=4) == 2 and b"window" in lib.csa_last_error()
    assert st(_11=p(base + 64), _12=p(base), _13=8) == 1 and b"apart" in lib.csa_last_error()
    assert st(_15=128) == 5
    assert st(_3=0) == 0
    # a call that needs scores needs more workspace than the plain one
    plain = lib.csa_kv_attn_decode_workspace_size(2, 4, C.byref(kv), 8, 0)
    weigh = lib.csa_kv_attn_decode_workspace_size(2, 4, C.byref(kv), 8, 1)
    assert 256 <= plain < weigh
    assert st(_12=p(base), _13=8, _15=plain) == 5
    assert lib.csa_launch_count() == before


def test_evict_refuses_bad_arguments_without_launching(lib, mem):
    _, base = mem
    before = lib.csa_launch_count()
    p = C.c_void_p
    kv = cache(base)
    # kv, lens, lens_out, weights, weights_out, slot_pos, slot_pos_out, slots, pos, B, budget, recent, keep_first, max_len,
    # src_out, ws, ws_bytes, stream
    args = [C.byref(kv), p(base), p(base + 64), p(base), p(base + 512), p(base), p(base + 512), 8, p(base), 2, 6, 2, 1, 8, None,
            p(base), 1 << 20, None]

    def st(**kw):
        a = list(args)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return lib.csa_kv_evict(*a)

    for what, c, want in bad_caches(base):
        assert st(_0=C.byref(c)) == want, what
        assert b"csa_kv_evict" in lib.csa_last_error()
    assert st(_0=C.byref(cache(base, v_head_stride=0))) == 1 and b"overlap" in lib.csa_last_error()
    assert st(_0=C.byref(cache(base, v=base, v_page_stride=1024, v_slot_stride=256))) == 1
    for i in (1, 2, 3, 4, 5, 6, 8):
        assert st(**{f"_{i}": None}) == 1, i
    assert st(_2=p(base + 4)) == 1 and st(_4=p(base + 64)) == 1 and st(_6=p(base + 64)) == 1
    assert st(_9=-1) == 1 and st(_9=65536) == 2
    assert st(_10=0) == 1 and st(_11=0) == 1 and st(_12=-1) == 1
    assert st(_11=6, _12=1) == 1 and b"budget" in lib.csa_last_error()
    assert st(_11=2147483647, _12=2147483647) == 1
    assert st(_10=(1 << 24) + 1) == 2
    assert st(_13=9) == 1 and st(_13=-1) == 1
    assert st(_16=256) == 5
    assert st(_9=0) == 0
    # per sequence and head min(max_len - budget, budget) moves, two slots each, and their number
    assert lib.csa_kv_evict_workspace_size(2, 8, 100, 90) == 512
    assert lib.csa_kv_evict_workspace_size(2, 8, 100, 132) == 512 + 2 * 8 * 2 * 32 * 4
    assert lib.csa_kv_evict_workspace_size(2, 8, 100, 10000) == 512 + 12800
    assert lib.csa_launch_count() == before


def test_python_entry_points_refuse_host_tensors():
    import compressed_sparse_kv_03_b200 as csa
    k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        csa.KVCache(k, k)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        csa.KVCache(k.float(), k.float())


# ---- oracle pins -------------------------------------------------------------
def test_oracle_attention_is_softmax_attention():
    rng = np.random.default_rng(0)
    B, H, Hkv, d, page, n = 2, 6, 3, 8, 4, 11
    q = rng.standard_normal((B, H, d))
    table = np.array([[5, 0, 3], [1, 4, 2]])
    k, v = rng.standard_normal((6, page, Hkv, d)), rng.standard_normal((6, page, Hkv, d))
    out, lse, prob = oracle.kv_attend(q, k, v, table, [n, 0], 0.3)
    full = lambda x: torch.tensor(x[table[0]].reshape(-1, Hkv, d)[:n]).repeat_interleave(2, 1).transpose(0, 1)  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q[0])[:, None], full(k), full(v), scale=0.3)[:, 0]
    assert np.allclose(out[0], want.numpy(), atol=1e-12)
    assert np.allclose(prob[0].sum(1), 1) and np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
    # a sink takes its share, and alone gives its own logit
    z = rng.standard_normal(H)
    o2, l2, p2 = oracle.kv_attend(q, k, v, table, [n, 0], 0.3, sink=z)
    assert np.allclose(np.exp(l2[0]), np.exp(lse[0]) + np.exp(z)) and np.allclose(l2[1], z)
    assert np.allclose(o2[0], out[0] * np.exp(lse[0] - l2[0])[:, None])
    # the window sees the last slots only
    o3, _, p3 = oracle.kv_attend(q, k, v, table, [n, 0], 0.3, window=3)
    one = k[table[0]].reshape(1, -1, Hkv, d)[:, n - 3:n], v[table[0]].reshape(1, -1, Hkv, d)[:, n - 3:n]
    o4, _, _ = oracle.kv_attend(q[:1], *one, None, [3], 0.3)
    assert np.allclose(o3[0], o4[0]) and np.all(p3[0][:, :n - 3] == 0)
    w = oracle.kv_weigh(np.ones((B, Hkv, 12)), prob, Hkv)
    assert np.allclose(w[0, :, :n].sum(-1), n + 2) and np.all(w[0, :, n:] == 1) and np.all(w[1] == 1)


def test_oracle_eviction_by_hand():
    # one head, budget 4, the newest token held: slots 0..5 with weights 5 1 1 0 4 0
    k = np.arange(6.0).reshape(1, 6, 1, 1)
    w = np.array([[[5.0, 1, 1, 0, 4, 0]]])
    sp = np.arange(6)[None, None]
    k2, v2, n, w2, p2, src = oracle.kv_evict(k, k * 10, None, np.array([6]), w, sp, np.array([5]), 4, 1)
    # stay: 0 (5), 4 (4), 5 (held) and 1 (first of the two ones); 2 and 3 are holes, filled by 4 and 5
    assert src[0, 0].tolist() == [0, 1, 4, 5] and n.tolist() == [4]
    assert k2[0, :4, 0, 0].tolist() == [0, 1, 4, 5] and v2[0, :4, 0, 0].tolist() == [0, 10, 40, 50]
    assert k2[0, 4:, 0, 0].tolist() == [4, 5]       # above the budget: as it was
    assert w2[0, 0].tolist() == [5, 1, 4, 0, 0, 0] and p2[0, 0].tolist() == [0, 1, 4, 5, 0, 0]
    # within the budget nothing moves
    k3, _, n3, w3, _, s3 = oracle.kv_evict(k, k, None, np.array([3]), w, sp, np.array([2]), 4, 1)
    assert n3.tolist() == [3] and np.array_equal(k3, k) and s3[0, 0].tolist() == [0, 1, 2, -1] and w3[0, 0].tolist() == [5, 1, 1, 0, 0, 0]
    # a NaN weight counts above every number, the first token can be kept by position
    w[0, 0, 3], w[0, 0, 0] = np.nan, 0
    s = oracle.kv_evict(k, k, None, np.array([6]), w, sp, np.array([5]), 3, 1)[-1]
    assert sorted(s[0, 0].tolist()) == [3, 4, 5]
    s = oracle.kv_evict(k, k, None, np.array([6]), w, sp, np.array([5]), 3, 1, keep_first=1)[-1]
    assert sorted(s[0, 0].tolist()) == [0, 3, 5]


def test_oracle_append_by_hand():
    k = np.zeros((3, 2, 1, 1))
    table = np.array([[2, 0], [1, 1]])
    new = np.array([1.0, 2, 3, 4]).reshape(4, 1, 1)
    k2, v2, n, w, sp = oracle.kv_append(k, k, table, [1, 0], new, -new, [0, 3, 4], np.ones((2, 1, 4)), np.zeros((2, 1, 4), int), [7, 9])
    assert k2[:, :, 0, 0].tolist() == [[2, 3], [4, 0], [0, 1]] and np.array_equal(v2, -k2) and n.tolist() == [4, 1]
    assert w[:, 0].tolist() == [[1, 0, 0, 0], [0, 1, 1, 1]] and sp[:, 0].tolist() == [[0, 7, 8, 9], [9, 0, 0, 0]]
    # no room: dropped
    assert oracle.kv_append(k, k, table, [3, 0], new, new, [0, 3, 4])[2].tolist() == [4, 1]


def test_the_batch_invariant_switch_is_read_once_per_call():
    """Another thread may change the switch while a call is under way; the workspace
    layout and the kernel's indexes into it have to follow one reading of it.  (A
    call that read it twice could write past its workspace, so this is read from
    the source instead of run.)"""
    from compressed_sparse_kv_03_b200 import build
    with open(os.path.join(build.CSRC, "kv_api.cu")) as f:
        text = f.read()
    assert text.count("batch_invariant()") == 1
    body = text[text.index("AttnLayout attn_layout("):]
    assert "batch_invariant()" in body[:body.index("\n}")]
    assert "a.invariant = l.plan.invariant;" in text
    for name in ("kv_attention.cu", "kv_attention.cuh", "kv_attention_tc.cu"):
        with open(os.path.join(build.CSRC, name)) as f:
            assert "batch_invariant()" not in f.read()


# ---- the Python calls' scratch, streams and devices ------------------------------
@pytest.fixture
def no_capture(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_threads_on_one_stream_have_scratch_of_their_own(no_capture):
    """A call makes several launches over its scratch, and the interpreter runs other
    threads meanwhile: two threads on one stream must not share it.  (Shown on
    host memory: shared scratch would let one thread's join or row moves run on
    another's lists.)"""
    import threading
    from compressed_sparse_kv_03_b200 import api
    host, got, both = torch.device("cpu"), {}, threading.Barrier(2, timeout=30)

    def job(name):
        at, size = api._kv_scratch(None, host, 7, 1000)
        both.wait()      # the other thread has its own by now
        again, _ = api._kv_scratch(None, host, 7, 500)
        more, big = api._kv_scratch(None, host, 7, 100000)
        other, _ = api._kv_scratch(None, host, 8, 500)
        got[name] = (at.value, size, again.value, more.value, big, other.value)
        both.wait()

    threads = [threading.Thread(target=job, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 2
    for at, size, again, more, big, other in got.values():
        assert again == at and size >= 1000 and big >= 100000 and other != more   # `at` is free again by then
    spans = [(got[i][k], got[i][k] + got[i][k + 1]) for i in range(2) for k in (0, 3)]
    assert spans[0][0] != spans[2][0] and (spans[1][1] <= spans[3][0] or spans[3][1] <= spans[1][0])


def test_workspaces_and_streams_of_another_device_are_refused(no_capture):
    """Before anything is allocated or launched: a workspace without memory yet goes
    by the device it was made for."""
    import compressed_sparse_kv_03_b200 as csa
    from compressed_sparse_kv_03_b200 import api
    first = torch.device("cuda", 0)
    for where in ("cuda:1", "cpu", torch.device("cuda", 3)):
        ws = csa.Workspace(where)
        with pytest.raises(ValueError, match="workspace is on"):
            api._kv_scratch(ws, first, 7, 256)
        assert ws.buf is None
    ws = csa.Workspace("cpu")
    ws.get(256)      # and one with memory by that
    with pytest.raises(ValueError, match="workspace is on"):
        api._kv_scratch(ws, first, 7, 256)

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7

    with pytest.raises(ValueError, match="stream is on"):
        api._kv_run(first, Stream(), lambda s: pytest.fail("ran"))


# ---- arrays that one call both reads and writes ----------------------------------
def test_new_lengths_do_not_share_memory_with_what_the_call_still_reads(lib, mem):
    """Blocks write lens_out while others read pos and token_start (host checks: nothing
    is launched, workspaces that are too small stop the calls that pass)."""
    _, base = mem
    before = lib.csa_launch_count()
    p = C.c_void_p
    kv, r = cache(base), rows(base)
    at = {"lens": base, "out": base + 64, "pos": base + 128, "start": base + 192}

    def append(start=None, n=2, pos=at["pos"], lens=at["lens"], out=at["out"], slot_pos=base + 2048):
        return lib.csa_kv_append(C.byref(r), C.byref(r), C.byref(kv), start and p(start), n, 2, p(lens), p(out), p(pos),
                                 p(base + 1024), slot_pos and p(slot_pos), 8, p(base), 128, None)

    ws = 5   # what a call that passes the checks before it gives
    assert append() == ws and append(at["start"], 5) == ws
    assert append(at["start"], 5, out=at["pos"]) == 1 and b"pos" in lib.csa_last_error()
    assert append(at["start"], 5, out=at["pos"] + 4) == 1
    assert append(at["start"], 5, out=at["start"]) == 1 and b"token_start" in lib.csa_last_error()
    assert append(at["start"], 5, out=at["start"] + 8) == 1      # its last entry
    assert append(at["start"], 5, out=at["start"] + 12) == ws
    assert append(out=at["pos"] + 4) == 1                        # another sequence's position
    assert append(out=at["pos"]) == ws                           # one block reads and writes a sequence's
    assert append(at["start"], 5, out=at["pos"], slot_pos=None) == ws   # pos is not read
    # in place the lengths are written when everything has been read
    assert append(at["start"], 5, out=at["lens"], pos=at["lens"]) == ws
    assert append(at["start"], 5, lens=at["start"], out=at["start"]) == 1

    def evict(pos=at["pos"], lens=at["lens"], out=at["out"]):
        return lib.csa_kv_evict(C.byref(kv), p(lens), p(out), p(base + 1024), p(base + 1024), p(base + 2048), p(base + 2048), 8, p(pos),
                                2, 6, 2, 1, 8, None, p(base), 128, None)

    assert evict() == ws
    assert evict(out=at["pos"]) == 1 and b"pos" in lib.csa_last_error()
    assert evict(out=at["pos"] - 4) == 1
    assert evict(out=at["lens"], pos=at["lens"]) == ws
    assert lib.csa_launch_count() == before
