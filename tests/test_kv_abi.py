"""The paged cache's and its attention's argument checks, on the host: nothing here reaches a device."""
import ctypes

import pytest
import torch

import kda_gated_delta_gate_b200 as kda

BOGUS = 0x10000


@pytest.fixture(scope="module")
def L():
    from kda_gated_delta_gate_b200 import build
    build.build()
    return kda.lib()


def _c(**kw):
    f = dict(k=BOGUS, v=BOGUS, page_table=BOGUS, seq_len=BOGUS, ref=BOGUS, scratch=BOGUS, layer_stride=1 << 20, layers=2,
             num_pages=64, page_size=16, kv_heads=2, head_dim=64, max_seqs=4, max_pages=8)
    f.update(kw)
    return ctypes.byref(kda.KdaKvCache(*[f[n] for n, _ in kda.KdaKvCache._fields_]))


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(page_table=None), 1), (dict(seq_len=None), 1), (dict(ref=None), 1),
              (dict(k=BOGUS + 8), 7), (dict(v=BOGUS + 2), 7), (dict(layers=0), 1), (dict(num_pages=0), 1),
              (dict(page_size=8), 4), (dict(page_size=48), 4), (dict(page_size=512), 4), (dict(head_dim=96), 4),
              (dict(kv_heads=0), 1), (dict(max_seqs=0), 1), (dict(max_pages=-1), 1), (dict(num_pages=1 << 27), 4),
              (dict(max_pages=1 << 28), 4), (dict(layer_stride=64 * 2 * 16 * 64 - 8), 1), (dict(layer_stride=(1 << 20) + 4), 7)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(L, kw, code):
    c, d = _c(**kw), ctypes.byref(kda.dims(4, kw.get("head_dim", 64)))
    assert L.kda_kv_reserve(c, BOGUS, BOGUS, 1, None) == code
    assert L.kda_kv_fork(c, BOGUS, BOGUS, 1, None) == code
    assert L.kda_kv_truncate(c, BOGUS, BOGUS, 1, None) == code
    assert L.kda_kv_compact(c, None, None) == code
    assert L.kda_kv_append(c, 0, BOGUS, BOGUS, 128, BOGUS, BOGUS, 1, 1, None) == code
    assert L.kda_attn_decode(c, 0, BOGUS, None, 1, 1, 0, 0, BOGUS, None, BOGUS, 1 << 30, d, None) == code
    assert L.kda_attn_prefill(c, 0, BOGUS, BOGUS, None, 1, 1, 1, 0, 0, BOGUS, None, BOGUS, 1 << 30, d, None) == code
    assert L.kda_attn_decode_scratch_bytes(1, 1, d, c) == 0 == L.kda_attn_prefill_scratch_bytes(1, 1, 1, d, c)


def test_bookkeeping_arguments(L):
    assert L.kda_kv_scratch_bytes(0, 4) == 0 and L.kda_kv_scratch_bytes(4, 0) == 0
    assert L.kda_kv_scratch_bytes(64, 4) >= 4 * (4 * 64 + 4 * 4)
    for f, two in ((L.kda_kv_reserve, 1), (L.kda_kv_fork, 0), (L.kda_kv_truncate, 1)):
        assert f(_c(), BOGUS, None, 1, None) == 1
        assert f(_c(), BOGUS, BOGUS, -1, None) == 1
        assert f(_c(), BOGUS, BOGUS, 5, None) == 1  # more than max_seqs
        assert f(_c(), BOGUS, BOGUS, 0, None) == 0
        assert f(None, BOGUS, BOGUS, 1, None) == 1
    assert L.kda_kv_fork(_c(), None, BOGUS, 1, None) == 1
    assert L.kda_kv_reserve(_c(scratch=None), BOGUS, BOGUS, 1, None) == 1
    assert L.kda_kv_compact(_c(scratch=BOGUS + 4), None, None) == 7


def test_append_arguments(L):
    f = L.kda_kv_append
    assert f(_c(), 2, BOGUS, BOGUS, 128, BOGUS, None, 1, 1, None) == 1      # layer
    assert f(_c(), -1, BOGUS, BOGUS, 128, BOGUS, None, 1, 1, None) == 1
    assert f(_c(), 0, None, BOGUS, 128, BOGUS, None, 1, 1, None) == 1
    assert f(_c(), 0, BOGUS, BOGUS, 128, None, None, 1, 1, None) == 1
    assert f(_c(), 0, BOGUS, BOGUS, 120, BOGUS, None, 1, 1, None) == 1      # rows would overlap
    assert f(_c(), 0, BOGUS, BOGUS, 132, BOGUS, None, 1, 1, None) == 7
    assert f(_c(), 0, BOGUS + 8, BOGUS, 128, BOGUS, None, 1, 1, None) == 7
    assert f(_c(), 0, BOGUS, BOGUS, 128, BOGUS, None, -1, 1, None) == 1
    assert f(_c(), 0, BOGUS, BOGUS, 128, BOGUS, None, 0, 1, None) == 0
    assert f(_c(), 0, BOGUS, BOGUS, 128, BOGUS, None, 1, 0, None) == 0


def test_attention_arguments(L):
    d = kda.dims(4, 64)
    dp = ctypes.byref(d)

    def dec(c=None, layer=0, q=BOGUS, N=1, K=1, w=0, s=0, out=BOGUS, scr=BOGUS, nb=1 << 30, dims=dp):
        return L.kda_attn_decode(c or _c(), layer, q, None, N, K, w, s, out, None, scr, nb, dims, None)

    def pre(c=None, layer=0, q=BOGUS, cu=BOGUS, B=1, rows=1, total=1, w=0, s=0, out=BOGUS, scr=BOGUS, nb=1 << 30,
            dims=dp):
        return L.kda_attn_prefill(c or _c(), layer, q, cu, None, B, rows, total, w, s, out, None, scr, nb, dims, None)

    for f in (dec, pre):
        assert f(layer=2) == 1 and f(layer=-1) == 1 and f(q=None) == 1 and f(out=None) == 1
        assert f(w=-1) == 1 and f(s=-1) == 1 and f(q=BOGUS + 8) == 7 and f(out=BOGUS + 4) == 7
        assert f(dims=None) == 1
        assert f(dims=ctypes.byref(kda.dims(5, 64))) == 1    # heads not a multiple of kv_heads
        assert f(dims=ctypes.byref(kda.dims(4, 128))) == 1   # not the cache's head_dim
        assert f(dims=ctypes.byref(kda.dims(4, 32))) == 4
    assert dec(N=-1) == 1 and dec(K=-1) == 1 and dec(N=0) == 0 and dec(K=0) == 0
    assert dec(K=33) == 4 and dec(dims=ctypes.byref(kda.dims(130, 64))) == 4  # more than 64 rows per kv head
    need = L.kda_attn_decode_scratch_bytes(1, 1, dp, _c())
    assert need > 0 and L.kda_attn_decode_scratch_bytes(0, 1, dp, _c()) == 0
    assert dec(scr=None) == 1 and dec(scr=BOGUS + 8) == 7 and dec(nb=need - 16) == 3
    assert pre(cu=None) == 1 and pre(B=-1) == 1 and pre(rows=-1) == 1 and pre(total=-1) == 1
    need = L.kda_attn_prefill_scratch_bytes(1, 1, 1, dp, _c())
    assert need > 0 and L.kda_attn_prefill_scratch_bytes(0, 1, 1, dp, _c()) == 0
    assert L.kda_attn_prefill_scratch_bytes(1, 50000, 50000, dp, _c()) == 0  # the rows fill the SMs
    assert pre(scr=None) == 1 and pre(scr=BOGUS + 8) == 7 and pre(nb=need - 16) == 3
    assert pre(B=0) == 0 and pre(total=0) == 0 and pre(rows=0) == 1 and pre(B=70000) == 4


def test_cache_object_checks_its_tensors(L):
    def make(**kw):
        t = dict(k=torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16), v=torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16),
                 page_table=torch.zeros(3, 5, dtype=torch.int32), seq_len=torch.zeros(3, dtype=torch.int32),
                 ref=torch.zeros(4, dtype=torch.int32))
        t.update(kw)
        return kda.KVCache(**t)

    c = make().struct
    assert (c.layers, c.num_pages, c.kv_heads, c.page_size, c.head_dim, c.max_seqs, c.max_pages) == (2, 4, 2, 16, 64, 3, 5)
    assert c.layer_stride == 4 * 2 * 16 * 64
    wide = torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)[:, :4]  # layers further apart than a pool is long
    assert make(k=wide, v=wide).struct.layer_stride == 6 * 2 * 16 * 64
    for kw in (dict(k=torch.zeros(2, 4, 2, 16, 64)), dict(v=torch.zeros(2, 4, 2, 16, 32, dtype=torch.bfloat16)),
               dict(ref=torch.zeros(5, dtype=torch.int32)), dict(seq_len=torch.zeros(3, dtype=torch.int64)),
               dict(page_table=torch.zeros(5, 3, dtype=torch.int32).T), dict(k=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)),
               dict(v=torch.zeros(2, 4, 16, 2, 64, dtype=torch.bfloat16).transpose(2, 3))):
        with pytest.raises(ValueError):
            make(**kw)


def test_binding_checks_types_and_sizes():
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
    d = kda.dims(4, 64)
    c = kda.KVCache(bf(1, 4, 2, 16, 64), bf(1, 4, 2, 16, 64), torch.zeros(3, 5, dtype=torch.int32),
                    torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    stride = lambda k, v: kda._rows_stride(c, k, v, 4)
    wide = bf(4, 384)
    assert stride(wide[:, 128:256], wide[:, 256:]) == 384
    assert stride(bf(5, 2, 64), bf(5, 2, 64)) == 128
    assert stride(bf(4, 6, 64)[:, 2:4], bf(4, 6, 64)[:, 4:]) == 384
    assert kda._rows_stride(c, wide[:1, :128], bf(1, 128), 1) == 128
    for k in (bf(4, 128).float(), bf(3, 128), bf(4, 64), bf(128, 4).T, bf(4, 64, 2).transpose(1, 2), bf(4, 256)[:, ::2],
              bf(4, 2, 128)[:, :, :64], bf(5, 128)):
        with pytest.raises(ValueError):
            stride(k, bf(4, 128))
    with pytest.raises(ValueError):
        stride(bf(4, 128), wide[:, :128])  # two row strides
    kda._attn_rows(c, 3, d, bf(3, 4, 64), bf(3, 4, 64), None)
    for q, o, l in ((bf(3, 4, 32), bf(3, 4, 64), None), (bf(3, 4, 64).float(), bf(3, 4, 64), None),
                    (bf(3, 4, 128)[:, :, ::2], bf(3, 4, 64), None), (bf(3, 4, 64), bf(2, 4, 64), None),
                    (bf(3, 4, 64), bf(3, 4, 64), torch.zeros(3, 3)), (bf(3, 4, 64), bf(3, 4, 64), bf(3, 4))):
        with pytest.raises(ValueError):
            kda._attn_rows(c, 3, d, q, o, l)
    assert kda._ints(c, None, torch.zeros(2, dtype=torch.int32))[0] is None
    for t in (torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            kda._ints(c, t)


def test_calls_refuse_short_or_foreign_tensors(monkeypatch):
    """Arrays with fewer entries than the call reads, and tensors on another device than the cache's."""
    bf = lambda *shape, dev="cpu": torch.zeros(*shape, dtype=torch.bfloat16, device=dev)
    ints = lambda n, dev="cpu": torch.zeros(n, dtype=torch.int32, device=dev)
    d = kda.dims(4, 64)
    c = kda.KVCache(bf(1, 4, 2, 16, 64), bf(1, 4, 2, 16, 64), ints(15).view(3, 5), ints(3), ints(4))
    calls = []
    monkeypatch.setattr(kda, "_on", lambda cache, stream: (cache._ref, 0))
    monkeypatch.setattr(kda, "_call", lambda name, *args: calls.append(name))
    q, scr = bf(4, 4, 64), torch.zeros(64, dtype=torch.uint8)
    kda.kda_kv_reserve(c, ints(2), ints(2), 2)
    kda.kda_kv_fork(c, ints(2), ints(2), 2)
    kda.kda_kv_truncate(c, None, ints(2), 2)
    kda.kda_kv_compact(c, ints(1))
    kda.kda_kv_append(c, 0, bf(4, 128), bf(4, 128), ints(3), ints(2), 2, 4)
    kda.kda_attn_decode(c, 0, q, ints(4), 4, 1, q.clone(), d, scratch=scr)
    kda.kda_attn_prefill(c, 0, q, ints(3), ints(2), 2, 4, 4, q.clone(), d, scratch=scr)
    assert len(calls) == 7
    m = "meta"  # stands for another device
    for bad in (lambda: kda.kda_kv_reserve(c, ints(1), ints(2), 2), lambda: kda.kda_kv_reserve(c, None, ints(1), 2),
                lambda: kda.kda_kv_reserve(c, None, ints(2, m), 2),
                lambda: kda.kda_kv_fork(c, ints(2), ints(1), 2), lambda: kda.kda_kv_fork(c, ints(2, m), ints(2), 2),
                lambda: kda.kda_kv_truncate(c, ints(2), ints(1), 2), lambda: kda.kda_kv_compact(c, ints(0)),
                lambda: kda.kda_kv_append(c, 0, bf(4, 128), bf(4, 128), ints(2), ints(2), 2, 4),
                lambda: kda.kda_kv_append(c, 0, bf(4, 128), bf(4, 128), ints(3), ints(1), 2, 4),
                lambda: kda.kda_kv_append(c, 0, bf(4, 128, dev=m), bf(4, 128, dev=m), ints(3), ints(2), 2, 4),
                lambda: kda.kda_attn_decode(c, 0, q, ints(3), 4, 1, q.clone(), d, scratch=scr),
                lambda: kda.kda_attn_decode(c, 0, bf(4, 4, 64, dev=m), None, 4, 1, q.clone(), d, scratch=scr),
                lambda: kda.kda_attn_decode(c, 0, q, None, 4, 1, q.clone(), d, scratch=scr.to(m)),
                lambda: kda.kda_attn_prefill(c, 0, q, ints(2), None, 2, 4, 4, q.clone(), d, scratch=scr),
                lambda: kda.kda_attn_prefill(c, 0, q, ints(3), ints(1), 2, 4, 4, q.clone(), d, scratch=scr),
                lambda: kda.kda_attn_prefill(c, 0, q, ints(3), None, 2, 4, 4, q.clone(), d, scratch=scr[::2])):
        with pytest.raises(ValueError):
            bad()
    assert len(calls) == 7


@pytest.mark.parametrize("B,rows,total,heads,kv_heads,dim", [(256, 1, 1, 64, 1, 128), (1024, 2, 2, 64, 1, 128), (4096, 3, 3, 16, 1, 128),
                                                             (65535, 40, 40, 1, 1, 64), (300, 9, 700, 48, 8, 64), (65535, 7, 900, 32, 2, 128)])
def test_scratch_does_not_grow_with_sequences_without_rows(L, B, rows, total, heads, kv_heads, dim):
    """Parts are kept for at most twice the tiles that can hold rows, and these with their splits fill the SMs once:
    148 CTAs of 256 rows at head_dim 128, 296 of 128 rows at 64, (dim + 4) FP32 values a row."""
    c = _c(num_pages=1 << 14, page_size=64, kv_heads=kv_heads, head_dim=dim, max_seqs=65536, max_pages=2048, layer_stride=1 << 40)
    need = L.kda_attn_prefill_scratch_bytes(B, rows, total, ctypes.byref(kda.dims(heads, dim)), c)
    assert need <= 2 * 148 * 256 * (dim + 4) * 4
    busy = min(B, total)  # the same rows without the empty sequences
    assert need <= L.kda_attn_prefill_scratch_bytes(busy, rows, total, ctypes.byref(kda.dims(heads, dim)), c)


def test_calls_of_two_threads_that_share_scratch_do_not_mix(L, monkeypatch):
    """A call that takes the stream's cached scratch launches several kernels on it: another thread's call on the stream comes
    before or after all of them. With scratch of their own, calls of two threads may run side by side."""
    import threading
    import time
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)
    scr, d = torch.zeros(64, dtype=torch.uint8), kda.dims(4, 64)
    c = kda.KVCache(bf(1, 4, 2, 16, 64), bf(1, 4, 2, 16, 64), torch.zeros(3, 5, dtype=torch.int32), ints(0, 0, 0), ints(0, 0, 0, 0))
    inside, most = [0], [0]

    def slow_call(name, *args):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        time.sleep(0.02)
        inside[0] -= 1

    monkeypatch.setattr(kda, "_on", lambda cache, stream: (cache._ref, 5))
    monkeypatch.setattr(kda, "_call", slow_call)
    monkeypatch.setattr(kda, "_attn_scratch", lambda *a: scr)
    monkeypatch.setattr(kda, "scratch_buffer", lambda *a: scr)
    q, x = bf(4, 4, 64), torch.zeros(64, 4, 64)
    calls = [lambda **k: kda.kda_attn_decode(c, 0, q, None, 4, 1, q, d, **k),
             lambda **k: kda.kda_attn_prefill(c, 0, q, ints(0, 1, 4), None, 2, 4, 4, q, d, **k),
             lambda **k: kda.kda_chunk_prefill(x, x, x, x, x, x, x, 1, 64, d, stream=5, **k),
             lambda **k: kda.kda_chunk_prefill_fused(x, x, x, x, x, x, x, 1, 64, d, stream=5, **k),
             lambda **k: kda.kda_chunk_prefill_graw(x, x, x, x, x, x, x, x, x, 1, 64, d, stream=5, **k),
             lambda **k: kda.kda_chunk_prefill_varlen(x, x, x, x, x, x, 1, 1, 64, x, x, d, stream=5, **k),
             lambda **k: kda.kda_chunk_verify(x, x, x, x, x, x, 1, 64, x, x, x, d, stream=5, **k)]

    def together(**k):
        inside[0] = most[0] = 0
        ts = [threading.Thread(target=f, kwargs=k) for f in calls for _ in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        return most[0]

    assert together() == 1
    assert together(scratch=scr) > 1


def test_capture_id_arguments(L):
    assert L.kda_stream_capture_id(None, None) == 1
    n = ctypes.c_ulonglong(7)
    assert L.kda_stream_capture_id(None, ctypes.byref(n)) == 0 and n.value == 0


def test_scratch_of_a_graph_is_kept_where_the_allocator_has_no_pool_for_it(monkeypatch):
    made, pooled, capture = [], [True], [1]
    monkeypatch.setattr(kda, "_empty_on", lambda n, dev, st: made.append(torch.zeros(n, dtype=torch.uint8)) or made[-1])
    monkeypatch.setattr(kda, "_of_a_pool", lambda t: pooled[0])
    monkeypatch.setattr(kda, "_capture_id", lambda st: capture[0])
    monkeypatch.setattr(kda, "_GRAPHS", {})
    monkeypatch.setattr(kda, "_KEPT", [])
    assert kda._graph_scratch(64, 0, 5) is made[0] and kda._graph_scratch(64, 0, 5) is made[1] and not kda._KEPT
    pooled[0], capture[0] = False, 2
    a = kda._graph_scratch(64, 0, 5)
    assert kda._graph_scratch(32, 0, 5) is a and kda._graph_scratch(64, 0, 6) is not a  # another stream of the capture
    b = kda._graph_scratch(96, 0, 5)
    assert b is not a and kda._graph_scratch(96, 0, 5) is b and any(x is a for x in kda._KEPT) and any(x is b for x in kda._KEPT)
    capture[0] = 3
    assert kda._graph_scratch(64, 0, 5) is not b and len(kda._KEPT) == 4
