"""kda_attn_prefill against the FP64 oracle: packed prompts, chunks behind cached tokens, odd head
groups, windows and sinks, hidden rows that hold NaN, refusals, and a run of the cache's calls."""
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


def run(c, lse=True, more_rows=0, **kw):
    out = torch.full(c.qd.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    l = torch.full(c.qd.shape[:2], float("nan"), device="cuda") if lse else None
    kda.kda_attn_prefill(c.cache, c.layer, c.qd, kw.pop("cu", i32(c.cu)), kw.pop("slots", i32(c.order)), len(c.order),
                         kw.pop("max_rows", max(c.rows) + more_rows), c.total, out, c.d, window=c.window, sinks=c.sinks,
                         lse=l, **kw)
    return out, l


# lengths, query rows, heads, kv_heads, dim, page, window, sinks
CASES = [
    ([1], [1], 2, 1, 64, 16, 0, 0),
    ([63, 64, 65], [63, 64, 65], 4, 2, 64, 16, 0, 0),
    ([127, 128, 129, 0, 5], [127, 128, 129, 0, 5], 4, 4, 128, 32, 0, 0),
    ([300, 700], [300, 1], 8, 2, 128, 64, 0, 0),
    ([300, 700, 257], [17, 200, 257], 10, 2, 128, 16, 0, 0),
    ([500], [333], 6, 2, 64, 128, 0, 0),
    ([400, 130], [130, 130], 14, 2, 128, 256, 0, 0),
    ([300], [129], 16, 1, 64, 16, 0, 0),
    ([260], [40], 33, 1, 128, 16, 0, 0),
    ([3, 2, 0, 10], [5, 2, 1, 12], 4, 2, 64, 16, 0, 0),           # more query rows than tokens
    ([300, 40], [300, 40], 4, 2, 64, 16, 1, 0),
    ([500, 40], [400, 40], 4, 2, 128, 16, 50, 4),
    ([900, 640], [100, 640], 8, 2, 128, 32, 128, 1),
    ([900, 640], [100, 300], 4, 1, 64, 64, 130, 200),
    ([1500, 20], [70, 20], 4, 2, 128, 16, 257, 129),
    ([600], [600], 4, 2, 128, 64, 5000, 7),
    ([700, 900], [700, 900], 16, 8, 64, 32, 0, 0),                # enough rows for one CTA per walk
    ([700, 400], [700, 400], 24, 8, 128, 64, 200, 3),
    ([9000, 40], [300, 2], 8, 2, 128, 64, 0, 0),                  # a chunk behind many cached tokens: shared walks
    ([5000], [130], 2, 1, 64, 16, 2000, 10),
    ([300, 7, 0, 900, 64], [3, 0, 2, 1, 4], 8, 2, 128, 16, 0, 0),  # few rows per sequence
    ([300, 7, 0, 900, 64], [3, 0, 5, 16, 4], 8, 2, 64, 32, 40, 2),
    ([200, 1000], [64, 1], 4, 4, 128, 16, 0, 0),
]


@pytest.mark.parametrize("lens,rows,heads,kv_heads,dim,page,window,sinks", CASES)
def test_matches_the_oracle(lens, rows, heads, kv_heads, dim, page, window, sinks):
    c = Case(lens, rows, heads, kv_heads, dim, page, window, sinks, seed=len(lens) + dim + heads)
    check(*run(c), c.expected())


def test_long_prompt():
    """Many tiles: the rows of a few heads against the oracle, the same bits again, and the last row as a decode."""
    c = Case([2500], [2500], 4, 2, 128, 64, seed=3)
    out, lse = run(c)
    check(out, lse, c.expected())
    again = run(c, more_rows=900)  # a looser bound on the rows changes nothing
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    one, l1 = torch.empty((1, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 4), device="cuda")
    kda.kda_attn_decode(c.cache, 0, c.qd[-1:].contiguous(), None, 1, 1, one, c.d, lse=l1)
    o, l, sp = c.expected()
    check(one, l1, (o[-1:], l[-1:], sp[-1:]))


def test_many_sequences():
    """More sequences than one round of a warp looks at, in both forms."""
    rows = [(i * 5) % 4 for i in range(1100)]
    rows[700] = 40
    c = Case([r + (i * 3) % 50 for i, r in enumerate(rows)], rows, 2, 1, 64, 16, seed=5)
    check(*run(c), c.expected())
    out, lse = run(c, max_rows=40)
    c.cache.seq_len[1000] = -1
    again = run(c, max_rows=40)
    assert kda.device_status(clear=True) == 1
    hit = slice(c.cu[1000], c.cu[1001])
    assert torch.isnan(again[0][hit]).all() and torch.equal(torch.nan_to_num(again[0], 9.0)[:hit.start], out[:hit.start])
    few = Case([r + 20 for r in rows[:600]], rows[:600], 2, 1, 64, 16, seed=6)
    check(*run(few), few.expected())


def test_layers_slots_and_optional_arguments():
    c = Case([70, 130, 33], [20, 130, 3], 4, 2, 64, 16, layers=3, layer=1, order=[2, 0, 2, 1], seed=4)
    c.total = c.cu[-1]
    check(*run(c), c.expected())
    c = Case([70, 130, 33], [20, 130, 3], 4, 2, 64, 16, layers=2, layer=1, seed=4)
    out, lse = run(c, slots=None)
    check(out, lse, c.expected())
    assert torch.equal(out, run(c, lse=False)[0])


@pytest.mark.parametrize("evicted", [-1, -2 ** 31, 10 ** 9])
def test_pages_that_left_the_window_are_not_looked_at(evicted):
    c = Case([900, 640, 300], [30, 64, 1], 4, 2, 128, 16, 64, 20, evicted=evicted, seed=6)
    check(*run(c), c.expected())


def test_bad_sequences_and_rows_behind_the_last_are_left():
    c = Case([300, 130, 64, 90, 200], [60, 130, 30, 90, 20], 4, 2, 64, 16, seed=11)
    o = c.expected()
    c.cache.seq_len[2] = -5
    c.cache.page_table[0, 3] = 10 ** 8
    c.cache.seq_len[4] = 10 ** 9
    out, lse = run(c)
    assert kda.device_status(clear=True) == 1
    hit = lambda i: slice(c.cu[i], c.cu[i + 1])
    for i in (0, 2, 4):
        assert torch.isnan(out[hit(i)]).all() and torch.isnan(lse[hit(i)]).all()
    for i in (1, 3):
        check(out[hit(i)], lse[hit(i)], tuple(x[hit(i)] for x in o))
    out, lse = run(c, slots=i32([-1, 1, 5, 3, 2 ** 31 - 1]))
    assert kda.device_status(clear=True) == 1
    for i in (0, 2, 4):
        assert torch.isnan(out[hit(i)]).all()
    check(out[hit(3)], lse[hit(3)], tuple(x[hit(3)] for x in o))
    # a sequence of more rows than max_rows, bounds that are none, and fewer rows than the call has
    out, lse = run(c, slots=i32([1] * 5), max_rows=60)
    assert kda.device_status(clear=True) == 1 and torch.isnan(out[hit(1)]).all() and not torch.isnan(out[hit(0)]).any()
    for cu in ([0, 60, 40, 40, 40, 50], [-7, 10, 10, 10, 10, 10], [0, 0, 0, 0, 0, 10 ** 6], [2 ** 31 - 1, -2 ** 31, 0, 0, 0, 0]):
        run(c, cu=i32(cu), slots=i32([1] * 5))
        assert kda.device_status(clear=True) == 1
    out, lse = run(c, cu=i32([0, 0, 130, 130, 130, 130]), slots=i32([3, 1, 1, 1, 3]))
    assert torch.isnan(out[130:]).all() and torch.isnan(lse[130:]).all() and not torch.isnan(out[:130]).any()


def test_bad_sequences_of_few_rows():
    c = Case([300, 130, 64, 90, 200], [3, 2, 4, 1, 2], 4, 2, 64, 16, seed=12)
    o = c.expected()
    hit = lambda i: slice(c.cu[i], c.cu[i + 1])
    c.cache.seq_len[2] = 10 ** 9
    c.cache.page_table[0, 3] = -3
    out, lse = run(c)
    assert kda.device_status(clear=True) == 1
    for i in range(5):
        if i in (0, 2):
            assert torch.isnan(out[hit(i)]).all() and torch.isnan(lse[hit(i)]).all()
        else:
            check(out[hit(i)], lse[hit(i)], tuple(x[hit(i)] for x in o))
    for cu in ([0, 6, 4, 4, 4, 5], [-7, 1, 1, 1, 1, 1], [0, 0, 0, 0, 0, 10 ** 6], [2 ** 31 - 1, -2 ** 31, 0, 0, 0, 0]):
        run(c, cu=i32(cu), slots=i32([1] * 5))
        assert kda.device_status(clear=True) == 1
    out, lse = run(c, cu=i32([0, 0, 2, 2, 2, 3]), slots=i32([3, 1, 1, 1, 3]))
    assert torch.isnan(out[3:]).all() and not torch.isnan(out[:3]).any()


def test_a_bad_page_in_one_part_of_a_shared_walk_leaves_the_tile():
    c = Case([6000, 500], [100, 100], 4, 2, 64, 16, seed=13)
    o = c.expected()
    c.cache.page_table[0, 200] = 10 ** 8
    out, lse = run(c)
    assert kda.device_status(clear=True) == 1
    assert torch.isnan(out[:100]).all() and torch.isnan(lse[:100]).all()
    check(out[100:], lse[100:], tuple(x[100:] for x in o))


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("rows", [[300, 40], [7, 3]])
def test_negative_and_zero_scales(scale, rows):
    c = Case([300, 40], rows, 8, 2, 64, 16, seed=14)
    c.scale = scale
    c.d = kda.dims(8, 64, scale=scale)
    check(*run(c), c.expected())


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
    q = torch.randn((200, 16, 128), generator=gen, device="cuda").bfloat16()
    d, a, b = kda.dims(16, 128, scale=0.09), torch.empty_like(q), torch.empty_like(q)
    kda.kda_attn_prefill(cache, 0, q, i32([0, 200]), i32([1]), 1, 200, 200, a, d)
    kda.kda_attn_prefill(near, 0, q, i32([0, 200]), None, 1, 200, 200, b, d)
    assert torch.equal(a, b) and a.float().abs().sum() > 0


def test_streams_graph_and_guard_bands():
    cs = [Case([400, 31, 500], [400, 31, 100], 8, 2, 128, 16, seed=s) for s in (1, 2)]
    want = [c.expected() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                outs[i] = run(c)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        check(*o, w)
    c, M = cs[0], 4096
    raw = [torch.full((2 * M + b,), 0xA5, dtype=torch.uint8, device="cuda") for b in (c.qd.numel() * 2, c.total * 8 * 4)]
    out = raw[0][M:-M].view(torch.bfloat16).view(c.qd.shape)
    lse = raw[1][M:-M].view(torch.float32).view(c.total, 8)
    cu, g = i32(c.cu), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_attn_prefill(c.cache, 0, c.qd, cu, None, 3, 400, c.total, out, c.d, lse=lse)
    for _ in range(3):
        g.replay()
    check(out, lse, want[0])
    for r in raw:
        assert (r[:M] == 0xA5).all() and (r[-M:] == 0xA5).all()


def test_extreme_scores():
    c = Case([400, 77], [200, 77], 4, 2, 64, 16, spread=2000.0, seed=8)
    out, lse = run(c)
    _, l, _ = c.expected()
    assert torch.isfinite(out).all()
    assert np.allclose(lse.double().cpu().numpy(), l, rtol=2.0 ** -17, atol=0)


def test_serving_run():
    """The calls together, as a serving loop makes them: prompts in two chunks, a decode step, samples forked
    from one prompt, draft rows of which some are rejected, a sequence that leaves, compaction, and
    decoding on. Every step's attention in both layers against the oracle on rows kept on the host."""
    H, Hk, D, L, page = 8, 2, 64, 2, 16
    cache = kda.KVCache.empty(60, page, Hk, D, 6, 20, L)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    d, rng = kda.dims(H, D, scale=D ** -0.5), torch.Generator().manual_seed(5)
    host = {}  # slot -> per layer [tokens, 2, Hk, D] as appended

    def step(slots, rows, prefill=True, window=0, sinks=0):
        kda.kda_kv_reserve(cache, i32(slots), i32(rows), len(slots))
        cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
        for layer in range(L):
            qkv = torch.randn((cu[-1], H + 2 * Hk, D), generator=rng).bfloat16()
            dev = qkv.cuda()
            kda.kda_kv_append(cache, layer, dev[:, H:H + Hk], dev[:, H + Hk:], i32(cu), i32(slots), len(slots), cu[-1])
            q, out = dev[:, :H].contiguous(), torch.empty((cu[-1], H, D), dtype=torch.bfloat16, device="cuda")
            lse = torch.empty((cu[-1], H), device="cuda")
            if prefill:
                kda.kda_attn_prefill(cache, layer, q, i32(cu), i32(slots), len(slots), max(rows), cu[-1], out, d,
                                     window=window, sinks=sinks, lse=lse)
            else:
                kda.kda_attn_decode(cache, layer, q, i32(slots), len(slots), rows[0], out, d, window=window, sinks=sinks,
                                    lse=lse)
            for i, s in enumerate(slots):
                new = torch.stack([qkv[cu[i]:cu[i + 1], H:H + Hk], qkv[cu[i]:cu[i + 1], H + Hk:]], 1)
                old = host.setdefault(s, {}).get(layer)
                host[s][layer] = new if old is None else torch.cat([old, new])
                kv, n = host[s][layer].double().numpy(), len(host[s][layer])
                o, l, sp = (np.zeros((rows[i], H, D)), np.zeros((rows[i], H)), np.zeros((rows[i], H, D)))
                for h in range(H):
                    o[:, h], l[:, h], sp[:, h] = oracle.attention(
                        qkv[cu[i]:cu[i + 1], h].double().numpy(), kv[:, 0, h // 4], kv[:, 1, h // 4], np.arange(n - rows[i], n),
                        d.scale, window, sinks)
                check(out[cu[i]:cu[i + 1]], lse[cu[i]:cu[i + 1]], (o, l, sp))

    step([0, 1, 2], [70, 33, 5])
    step([0, 2], [50, 100])                 # second chunks
    step([0, 1, 2], [1, 1, 1], prefill=False)
    kda.kda_kv_fork(cache, i32([0, 0, 1]), i32([3, 4, 5]), 3)
    for p, c in ((0, 3), (0, 4), (1, 5)):
        host[c] = dict(host[p])
    step([0, 3, 4, 5], [4, 4, 4, 4], prefill=False)   # draft rows
    keep = {0: 123, 3: 122, 4: 121, 5: 38}             # 1 to 4 of them accepted
    kda.kda_kv_truncate(cache, i32(keep), i32(keep.values()), 4)
    for s, n in keep.items():
        host[s] = {layer: x[:n] for layer, x in host[s].items()}
    step([0, 3, 4, 5], [1, 1, 1, 1], prefill=False)
    kda.kda_kv_truncate(cache, i32([0, 2]), i32([0, 0]), 2)  # two sequences end
    host.pop(0), host.pop(2)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_kv_compact(cache, live)
    assert int(live) == int((cache.ref > 0).sum()) and int(cache.page_table.max()) < int(live)
    step([3, 4, 5, 1, 0], [1, 1, 1, 1, 1], prefill=False)
    step([5, 2, 3], [30, 61, 2], window=40, sinks=3)
    step([5, 2, 3], [1, 1, 1], prefill=False, window=40, sinks=3)
    assert cache.seq_len.tolist() == [len(host[s][0]) for s in range(6)]


@pytest.mark.parametrize("B,busy,heads,kv_heads,dim", [(2000, {3: (2100, 3), 1998: (700, 2)}, 32, 2, 128),
                                                       (300, {0: (900, 140), 150: (40, 1), 299: (1300, 60)}, 4, 1, 64),
                                                       (70, {64: (600, 1)}, 33, 1, 64),
                                                       (6000, {4000: (300, 1)}, 33, 1, 128)])
def test_few_sequences_with_rows_among_many_without(B, busy, heads, kv_heads, dim):
    """A fixed list of slots, most of them without rows: fewer row tiles than sequences, walks shared by several CTAs."""
    lens, rows = [i % 3 for i in range(B)], [0] * B
    for s, (n, r) in busy.items():
        lens[s], rows[s] = n, r
    c = Case(lens, rows, heads, kv_heads, dim, 16, seed=B)
    out, lse = run(c)
    check(out, lse, c.expected())
    c.cache.seq_len[B - 2 if B - 2 not in busy else B - 3] = -1  # one without rows that is refused all the same
    again = run(c)
    assert kda.device_status(clear=True) == 1
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("lens,rows,heads,kv_heads,dim,window", [([2500], [2500], 8, 2, 128, 0), ([2500], [2500], 8, 2, 64, 0),
                                                                 ([900, 640], [300, 640], 8, 4, 64, 200), ([6000], [140], 4, 1, 128, 0),
                                                                 ([5000], [300], 2, 1, 64, 0), ([900, 31, 2000], [4, 4, 4], 8, 2, 128, 0),
                                                                 ([900, 31, 2000], [1, 1, 1], 8, 2, 64, 0), ([700, 90], [16, 16], 8, 2, 128, 0)])
def test_equal_values_come_out_as_they_are(lens, rows, heads, kv_heads, dim, window):
    """V rows that are all c: the weights, whatever they are rounded to, are divided by their own sum, and o is c. Weights and
    products are summed in FP32, each sum within 6000 2^-24 < 2^-11 of the terms, so o is within 2^-10 of c before its own
    rounding, and what is nearer than 2^-9 to a BF16 value rounds to it."""
    c = Case(lens, rows, heads, kv_heads, dim, 16, window, seed=dim + heads, spread=4.0)
    value = torch.randn((kv_heads, dim), generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    c.cache.v.copy_(value[:, None].expand(kv_heads, 16, dim).expand_as(c.cache.v))
    out, lse = run(c)
    want = value.repeat_interleave(heads // kv_heads, 0).expand_as(out)
    assert torch.equal(out, want), f"{int((out != want).sum())} of {out.numel()} values differ"
    if len(set(rows)) == 1:
        n = rows[0]
        if heads // kv_heads * n <= 64:
            o = torch.empty_like(out)
            kda.kda_attn_decode(c.cache, 0, c.qd, None, len(lens), n, o, c.d, window=window)
            assert torch.equal(o, want)


def test_both_head_sizes_and_the_short_form_at_once():
    """Packed calls at head_dim 64 and 128 (256 and 512 TMEM columns per CTA) and decodes, on three streams."""
    cs = [Case([700, 31, 900], [500, 31, 200], 8, 2, dim, 32, seed=dim) for dim in (64, 128)]
    one = Case([900, 31, 2000], [1] * 3, 8, 2, 128, 16, seed=41)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, o1, l1 = [None, None], torch.empty_like(one.qd), torch.empty((3, 8), device="cuda")
    slots = i32(one.order)
    torch.cuda.synchronize()
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                outs[i] = run(c)
        kda.kda_attn_decode(one.cache, 0, one.qd, slots, 3, 1, o1, one.d, lse=l1, stream=streams[2])
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        check(*o, c.expected())
    check(o1, l1, one.expected())


def test_more_heads_per_kv_head_than_a_tile_has_rows():
    c = Case([150, 3, 40], [3, 1, 0], 600, 2, 64, 16, seed=42)
    check(*run(c), c.expected())


def test_rows_before_the_first_sequence_are_left():
    c = Case([300, 40], [100, 40], 4, 2, 64, 16, seed=43)
    o, total = c.expected(), c.total
    c.qd = torch.cat([c.qd[:7], c.qd])
    c.total += 7
    out, lse = run(c, cu=i32([x + 7 for x in c.cu]))
    assert torch.isnan(out[:7]).all() and torch.isnan(lse[:7]).all() and len(out) == total + 7
    check(out[7:], lse[7:], o)
