"""kda_attn_decode against the FP64 oracle: lengths from none to long ones, odd head groups, windows
and sinks, pages of every size, hidden rows that hold NaN, refusals, and calls side by side."""
import numpy as np
import pytest
import torch

import kda_gated_delta_gate_b200 as kda
import oracle
from tests.attn_harness import Case, check, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status(cuda_ok):
    kda.device_status(clear=True)
    yield
    assert kda.device_status(clear=True) == 0


def run(c, K, **kw):
    out = torch.full((len(c.order) * K, c.heads, c.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(c.order) * K, c.heads), float("nan"), device="cuda")
    kda.kda_attn_decode(c.cache, c.layer, c.qd, kw.pop("slots", i32(c.order)), len(c.order), K, out, c.d, window=c.window,
                        sinks=c.sinks, lse=lse, **kw)
    return out, lse


# lengths, K, heads, kv_heads, dim, page, window, sinks
CASES = [
    ([0, 1, 15, 16, 17, 63, 64, 65, 200], 1, 4, 2, 64, 16, 0, 0),
    ([0, 1, 2, 127, 128, 129], 1, 6, 6, 128, 32, 0, 0),
    ([1000], 1, 8, 1, 128, 64, 0, 0),
    ([700, 3, 0, 321], 1, 10, 2, 128, 128, 0, 0),
    ([515, 64], 1, 32, 2, 64, 256, 0, 0),
    ([0, 1, 2, 3, 100, 777], 3, 4, 2, 128, 16, 0, 0),   # fewer tokens than rows among them
    ([300, 5, 64], 4, 10, 2, 128, 64, 0, 0),             # 20 rows per kv head
    ([300, 5, 64, 129], 4, 32, 2, 128, 16, 0, 0),        # 64
    ([300, 5, 64, 129], 8, 16, 2, 64, 32, 0, 0),
    ([257, 31], 2, 48, 3, 64, 16, 0, 0),
    ([0, 1, 40, 300, 641], 1, 4, 2, 64, 16, 1, 0),
    ([0, 1, 40, 300, 641], 1, 4, 2, 128, 16, 7, 1),
    ([10, 64, 300, 641], 1, 4, 2, 64, 32, 64, 4),
    ([10, 64, 300, 641], 3, 6, 2, 128, 16, 100, 5),
    ([10, 190, 300, 641], 2, 4, 1, 64, 64, 33, 70),
    ([10, 190, 300, 1641], 1, 4, 1, 128, 128, 130, 200),
    ([500, 600], 1, 4, 1, 128, 256, 5000, 3),            # a window longer than the cache
]


@pytest.mark.parametrize("lens,K,heads,kv_heads,dim,page,window,sinks", CASES)
def test_matches_the_oracle(lens, K, heads, kv_heads, dim, page, window, sinks):
    c = Case(lens, [K] * len(lens), heads, kv_heads, dim, page, window, sinks, seed=len(lens) + dim)
    check(*run(c, K), c.expected())


def test_one_long_sequence_beside_short_ones():
    c = Case([3, 40000, 0, 777, 64], [1] * 5, 4, 2, 128, 16, seed=2)
    out, lse = run(c, 1)
    check(out, lse, c.expected())
    for _ in range(3):  # the parts are added in one order
        again = run(c, 1)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_many_sequences_more_than_threads():
    lens = [(i * 29) % 150 for i in range(300)]
    c = Case(lens, [1] * 300, 4, 2, 64, 16, seed=9)
    check(*run(c, 1), c.expected())


def test_layers_slots_and_optional_arguments():
    c = Case([70, 130, 33], [2] * 3, 4, 2, 64, 16, layers=3, layer=1, order=[2, 0, 2, 1], seed=4)
    out, lse = run(c, 2)
    check(out, lse, c.expected())
    c = Case([70, 130, 33], [2] * 3, 4, 2, 64, 16, layers=2, layer=1, seed=4)
    out, lse = run(c, 2, slots=None)
    check(out, lse, c.expected())
    out2 = torch.empty_like(out)
    kda.kda_attn_decode(c.cache, 1, c.qd, None, 3, 2, out2, c.d)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("evicted", [-1, -2 ** 31, 10 ** 9])
def test_pages_that_left_the_window_are_not_looked_at(evicted):
    c = Case([900, 640, 300], [1] * 3, 4, 2, 128, 16, 64, 20, evicted=evicted, seed=6)
    check(*run(c, 1), c.expected())


def test_bad_slots_lengths_and_pages_leave_their_rows():
    c = Case([700, 130, 64, 90, 200], [1] * 5, 4, 2, 64, 16, seed=11)
    o = c.expected()
    c.cache.seq_len[3] = -5
    c.cache.page_table[0, 20] = 10 ** 8
    c.cache.seq_len[4] = 10 ** 9
    slots = i32([0, 1, 2, 3, 4])
    out, lse = run(c, 1, slots=slots)
    assert kda.device_status(clear=True) == 1
    assert torch.isnan(out[[0, 3, 4]]).all() and torch.isnan(lse[[0, 3, 4]]).all()
    check(out[1:3], lse[1:3], tuple(x[1:3] for x in o))
    out, lse = run(c, 1, slots=i32([1, -1, 2, 5, 2 ** 31 - 1]))
    assert kda.device_status(clear=True) == 1
    assert torch.isnan(out[[1, 3, 4]]).all()
    out, lse = run(c, 1, slots=i32([-1] * 5))
    assert kda.device_status(clear=True) == 1 and torch.isnan(out).all()


def test_far_pages():
    """Rows past the 2^32nd element of a pool."""
    pages = 2 ** 32 // (8 * 64 * 128) + 40
    cache = kda.KVCache.empty(pages, 64, 8, 128, 2, 30)
    gen = torch.Generator(device="cuda").manual_seed(1)
    far = torch.arange(pages - 30, pages, device="cuda")
    for t in (cache.k, cache.v):
        t[0, far] = torch.randn((30, 8, 64, 128), generator=gen, device="cuda").bfloat16()
    cache.page_table[1] = far.int()
    cache.seq_len[1] = 1900
    near = kda.KVCache(cache.k[:, far].contiguous(), cache.v[:, far].contiguous(),
                       torch.arange(30, dtype=torch.int32, device="cuda")[None], i32([1900]), i32([1] * 30))
    q = torch.randn((1, 16, 128), generator=gen, device="cuda").bfloat16()
    d, a, b = kda.dims(16, 128, scale=0.09), torch.empty_like(q), torch.empty_like(q)
    kda.kda_attn_decode(cache, 0, q, i32([1]), 1, 1, a, d)
    kda.kda_attn_decode(near, 0, q, None, 1, 1, b, d)
    assert torch.equal(a, b) and a.float().abs().sum() > 0


def test_streams_graphs_and_guard_bands():
    """Two streams at once, two graphs replayed at once, and outputs inside canaries."""
    cs = [Case([900, 31, 2000], [1] * 3, 8, 2, 128, 16, seed=s) for s in (1, 2)]
    want = [c.expected() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                outs[i] = run(c, 1)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        check(*o, w)
    graphs, held = [], []
    for c in cs:
        out, lse = torch.zeros_like(c.qd), torch.zeros((3, 8), device="cuda")
        slots = i32(c.order)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_attn_decode(c.cache, 0, c.qd, slots, 3, 1, out, c.d, lse=lse)
        graphs.append(g)
        held.append((out, lse, slots))
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (out, lse, _), w in zip(held, want):
        check(out, lse, w)
    c, M = cs[0], 4096
    n = kda.kda_attn_decode_scratch_bytes(3, 1, c.d, c.cache)
    raw = [torch.full((2 * M + b,), 0xA5, dtype=torch.uint8, device="cuda") for b in (c.qd.numel() * 2, 3 * 8 * 4, n)]
    out = raw[0][M:-M].view(torch.bfloat16).view(c.qd.shape)
    lse = raw[1][M:-M].view(torch.float32).view(3, 8)
    kda.kda_attn_decode(c.cache, 0, c.qd, None, 3, 1, out, c.d, lse=lse, scratch=raw[2][M:-M])
    check(out, lse, want[0])
    for r in raw:
        assert (r[:M] == 0xA5).all() and (r[-M:] == 0xA5).all()


def test_extreme_scores():
    """Scores far apart and large: nothing overflows on the way, and one weight takes all."""
    c = Case([400, 77], [1, 1], 4, 2, 64, 16, spread=2000.0, seed=8)
    out, lse = run(c, 1)
    o, l, _ = c.expected()
    assert torch.isfinite(out).all()
    assert np.allclose(lse.double().cpu().numpy(), l, rtol=2.0 ** -17, atol=0)


def test_calls_on_another_device_are_refused(monkeypatch):
    c = Case([20], [1], 4, 2, 64, 16)
    run(c, 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: c.cache.k.device.index + 1)
    one = i32([1])
    for call in (lambda: kda.kda_attn_decode(c.cache, 0, c.qd, None, 1, 1, torch.empty_like(c.qd), c.d, stream=0),
                 lambda: kda.kda_attn_prefill(c.cache, 0, c.qd, i32([0, 1]), None, 1, 1, 1, torch.empty_like(c.qd), c.d, stream=0),
                 lambda: kda.kda_kv_reserve(c.cache, None, one, 1, stream=0),
                 lambda: kda.kda_kv_fork(c.cache, one, one, 1, stream=0),
                 lambda: kda.kda_kv_truncate(c.cache, None, one, 1, stream=0),
                 lambda: kda.kda_kv_compact(c.cache, stream=0),
                 lambda: kda.kda_kv_append(c.cache, 0, c.qd[:, :2], c.qd[:, 2:], i32([0, 1]), None, 1, 1, stream=0)):
        with pytest.raises(ValueError):
            call()


def test_scratch_belongs_to_the_stream_of_the_call():
    """Scratch for an explicit stream is not memory that the current stream has just given back with work still queued on it."""
    side = torch.cuda.Stream()
    n = 48 << 20
    freed = torch.empty(n, dtype=torch.uint8, device="cuda")
    at = freed.data_ptr()
    del freed
    buf = kda.scratch_buffer(n, "cuda", side.cuda_stream)
    assert buf.data_ptr() != at and buf.numel() >= n
    again = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == at  # the freed block was there to be had
    assert kda.scratch_buffer(n, "cuda", side.cuda_stream) is buf
    kda._SCRATCH.pop((torch.cuda.current_device(), side.cuda_stream))


def test_an_explicit_stream_and_its_capture():
    """Calls on another stream than the current one, eager and captured on a branch of a graph beside one on the trunk."""
    cs = [Case([900, 31, 2000], [1] * 3, 8, 2, 128, 16, seed=s) for s in (11, 12)]
    want = [c.expected() for c in cs]
    side = torch.cuda.Stream()
    outs = [(torch.empty_like(c.qd), torch.empty((3, 8), device="cuda")) for c in cs]
    slots = [i32(c.order) for c in cs]
    torch.cuda.synchronize()

    def call(i, stream=None):
        kda.kda_attn_decode(cs[i].cache, 0, cs[i].qd, slots[i], 3, 1, outs[i][0], cs[i].d, lse=outs[i][1], stream=stream)

    call(0)
    call(1, side)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        check(*o, w)
        o[0].zero_(), o[1].zero_()
    g, fork, join = torch.cuda.CUDAGraph(), torch.cuda.Event(), torch.cuda.Event()
    with torch.cuda.graph(g):
        trunk = torch.cuda.current_stream()
        fork.record(trunk)
        side.wait_event(fork)
        call(1, side)
        call(0)
        join.record(side)
        trunk.wait_event(join)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        check(*o, w)


def test_scratch_of_the_default_stream_asked_for_on_another():
    """stream=0 (the handle of the default stream) while another stream is current: the scratch is the default stream's memory."""
    n, key = 48 << 20, (torch.cuda.current_device(), 0)
    kda._SCRATCH.pop(key, None)
    with torch.cuda.stream(torch.cuda.Stream()):
        at = kda.scratch_buffer(n, "cuda", 0).data_ptr()
    kda._SCRATCH.pop(key)
    assert torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr() == at  # given back to where it came from


def test_two_threads_on_one_stream():
    """Decode, draft rows and packed rows from two host threads whose current stream is the same one."""
    import threading
    cs = [Case([1900, 31, 2500], [2] * 3, 8, 2, 128, 16, seed=s) for s in (21, 22)]
    more = [Case([3000, 40], [90, 40], 4, 1, 64, 16, seed=s) for s in (23, 24)]
    want, want_more = [run(c, 2) for c in cs], []

    def packed(c):
        out, lse = torch.empty_like(c.qd), torch.empty(c.qd.shape[:2], device="cuda")
        kda.kda_attn_prefill(c.cache, 0, c.qd, cu, None, 2, 90, c.total, out, c.d, lse=lse)
        return out, lse

    cu = i32(more[0].cu)
    want_more = [packed(c) for c in more]
    stream, got = torch.cuda.current_stream(), [[], []]

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(40):
                got[i].append((run(cs[i], 2), packed(more[i])))

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        check(*want[i], cs[i].expected())
        check(*want_more[i], more[i].expected())
        assert len(got[i]) == 40
        for a, b in got[i]:
            assert torch.equal(a[0], want[i][0]) and torch.equal(a[1], want[i][1])
            assert torch.equal(b[0], want_more[i][0]) and torch.equal(b[1], want_more[i][1])


def test_a_stream_captured_through_the_cuda_api(monkeypatch):
    """Captured by cudaStreamBeginCapture, no allocator pool stands behind the graph: its scratch stays its own."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.12")
    ok = lambda rc: rc == 0 or pytest.fail(f"cuda error {rc}")
    c = Case([900, 31, 2000], [1] * 3, 8, 2, 128, 16, seed=31)
    want, slots = c.expected(), i32(c.order)
    out, lse = torch.zeros_like(c.qd), torch.zeros((3, 8), device="cuda")
    made, empty_on = [], kda._empty_on

    def noted(*a):
        buf = empty_on(*a)
        made.append((buf.data_ptr(), buf.numel()))
        return buf

    monkeypatch.setattr(kda, "_empty_on", noted)
    side = torch.cuda.Stream()
    call = lambda: kda.kda_attn_decode(c.cache, 0, c.qd, slots, 3, 1, out, c.d, lse=lse, stream=side)
    call()
    torch.cuda.synchronize()
    made.clear()
    st, graph, ex = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
    ok(rt.cudaStreamBeginCapture(st, 1))  # thread-local mode
    call()
    call()
    ok(rt.cudaStreamEndCapture(st, ctypes.byref(graph)))
    assert len(made) == 1  # both calls are on one stream
    ok(rt.cudaGraphInstantiate(ctypes.byref(ex), graph, ctypes.c_ulonglong(0)))
    at, n = made[0]
    with torch.cuda.stream(side):
        later = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for t in later:
        assert t.data_ptr() + n <= at or at + n <= t.data_ptr()
    out.zero_(), lse.zero_()
    torch.cuda.synchronize()
    ok(rt.cudaGraphLaunch(ex, st))
    torch.cuda.synchronize()
    check(out, lse, want)
    for t in later:
        assert (t == 255).all()
    ok(rt.cudaGraphExecDestroy(ex))
    ok(rt.cudaGraphDestroy(graph))
    # torch's own capture: the graph's pool has the memory, nothing is kept
    before, g = len(kda._KEPT), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_attn_decode(c.cache, 0, c.qd, slots, 3, 1, out, c.d, lse=lse)
    out.zero_()
    g.replay()
    check(out, lse, want)
    assert len(kda._KEPT) == before


def test_more_sequences_than_a_grid_dimension_has():
    """70000 sequences, a few of them long, one of them refused."""
    n, page = 70000, 16
    lens = [1 + i % 3 for i in range(n)]
    for i, x in ((17, 160), (40000, 90), (69999, 33)):
        lens[i] = x
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    pages, heads = n + 20, 2
    cache = kda.KVCache.empty(pages, page, 1, 64, n, 10)
    cache.k.copy_(rand(*cache.k.shape))
    cache.v.copy_(rand(*cache.v.shape))
    kda.kda_kv_reserve(cache, None, i32(lens), n)
    q = rand(n, heads, 64)
    d, out, lse = kda.dims(heads, 64, scale=0.125), torch.full_like(q, float("nan")), torch.empty((n, heads), device="cuda")
    cache.seq_len[123] = -1
    kda.kda_attn_decode(cache, 0, q, None, n, 1, out, d, lse=lse)
    assert kda.device_status(clear=True) == 1 and torch.isnan(out[123]).all()
    out[123] = 0
    assert torch.isfinite(out).all()
    table = cache.page_table.cpu()
    for i in (0, 1, 17, 122, 124, 33333, 40000, 69998, 69999):
        rows = [cache.k[0, table[i, j], 0].cpu().double() for j in range(-(-lens[i] // page))]
        vals = [cache.v[0, table[i, j], 0].cpu().double() for j in range(-(-lens[i] // page))]
        k, v = torch.cat(rows)[:lens[i]].numpy(), torch.cat(vals)[:lens[i]].numpy()
        o, l, sp = zip(*[oracle.attention(q[i, h:h + 1].double().cpu().numpy(), k, v, [lens[i] - 1], 0.125) for h in range(heads)])
        check(out[i:i + 1], lse[i:i + 1], (np.stack(o, 1), np.stack(l, 1), np.stack(sp, 1)))


def test_capture_numbers():
    """A stream's capture is told apart from the next, and asking about another stream leaves it as it is."""
    seen, x = set(), torch.zeros(4, device="cuda")
    assert kda._capture_id(torch.cuda.current_stream().cuda_stream) == 0
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            seen.add(kda._capture_id(torch.cuda.current_stream().cuda_stream))
            assert kda._capture_id(0) == 0  # the default stream
            x.add_(1)
        g.replay()
    assert len(seen) == 2 and 0 not in seen
    torch.cuda.synchronize()
    assert (x == 2).all()


def test_graphs_do_not_share_the_core_calls_scratch(monkeypatch):
    """Graphs of the chunked prefill captured one after the other on torch's capture stream, and what that stream's calls take
    afterwards: three buffers."""
    d, at = kda.dims(2, 64), []
    q, k, v = (torch.randn((64, 2, 64), device="cuda") for _ in range(3))
    gate, beta, core = -torch.rand((64, 2, 64), device="cuda"), torch.rand((64, 2), device="cuda"), torch.empty((64, 2, 64), device="cuda")
    state = torch.zeros((2, 64, 64), device="cuda")
    ptrs, call, side = kda.ptr_array([state]), kda._call, torch.cuda.Stream()
    f = lambda: kda.kda_chunk_prefill(q, k, v, gate, beta, ptrs, core, 1, 64, d)
    f()
    want, end = core.clone(), state.clone()

    def noted(name, *args):
        if name == "kda_chunk_prefill":
            at.append(args[9])
        return call(name, *args)

    monkeypatch.setattr(kda, "_call", noted)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=side):
            f()
    with torch.cuda.stream(side):
        f()
    torch.cuda.synchronize()
    assert len(set(at)) == 3
    for g in graphs:
        core.zero_(), state.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(core, want) and torch.equal(state, end)
