"""The paged key-value cache's bookkeeping and row writing against tests/kv_model.py: every array
and every page bit for bit, over random sequences of calls and the cases that a call refuses."""
import numpy as np
import pytest
import torch

import kda_gated_delta_gate_b200 as kda
import oracle
from tests.attn_harness import check
from tests.kv_model import KvModel

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status(cuda_ok):
    kda.device_status(clear=True)
    yield
    assert kda.device_status(clear=True) == 0


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Pair:
    """A cache on the GPU and its model, kept in step."""

    def __init__(self, pages=40, page=16, heads=2, dim=64, seqs=8, max_pages=12, layers=2, seed=0):
        self.cache = kda.KVCache.empty(pages, page, heads, dim, seqs, max_pages, layers)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        self.rng = np.random.default_rng(seed)
        c = self.cache
        self.model = KvModel(_bits(c.k), _bits(c.v), c.page_table.cpu().numpy(), c.seq_len.cpu().numpy(),
                             c.ref.cpu().numpy())

    def call(self, name, *args):
        c, n = self.cache, len(args[0]) if args else 0
        if name == "compact":
            live = torch.full((1,), -7, dtype=torch.int32, device="cuda")
            kda.kda_kv_compact(c, live)
            assert int(live) == self.model.compact()
        else:
            getattr(kda, "kda_kv_" + name)(c, *[_i32(a) for a in args], n)
            getattr(self.model, name)(*args)
        self.check()

    def append(self, layer, slots, rows, ids=True):
        c, total = self.cache, sum(rows)
        w = c.k.shape[2] * c.k.shape[4]
        wide = torch.from_numpy(self.rng.standard_normal((total + 3, 3 * w), dtype=np.float32)).cuda().bfloat16()
        k_new, v_new = wide[:, w:2 * w], wide[:, 2 * w:]
        cu = np.concatenate([[0], np.cumsum(rows)])
        kda.kda_kv_append(c, layer, k_new, v_new, _i32(cu), _i32(slots) if ids else None, len(rows), total + 3)
        shape = (-1, c.k.shape[2], c.k.shape[4])
        self.model.append(layer, _bits(k_new).reshape(shape), _bits(v_new).reshape(shape), cu, slots)
        self.check()

    def check(self):
        c, m = self.cache, self.model
        assert kda.device_status(clear=True) == m.status
        m.status = 0
        assert np.array_equal(c.seq_len.cpu().numpy(), m.seq_len)
        assert np.array_equal(c.ref.cpu().numpy(), m.ref)
        assert np.array_equal(c.page_table.cpu().numpy(), m.table)
        assert np.array_equal(_bits(c.k), m.k) and np.array_equal(_bits(c.v), m.v)


@pytest.mark.parametrize("page,dim,heads,layers", [(16, 64, 2, 2), (32, 128, 1, 1), (64, 128, 3, 1), (128, 64, 1, 2),
                                                     (256, 64, 1, 1)])
def test_random_calls_match_the_model(page, dim, heads, layers):
    p = Pair(pages=30, page=page, heads=heads, dim=dim, seqs=7, max_pages=9, layers=layers, seed=page)
    rng = p.rng
    for _ in range(40):
        m = p.model
        op = rng.choice(["reserve", "reserve", "fork", "truncate", "compact", "append"])
        n = int(rng.integers(1, 6))
        slots = [int(x) for x in rng.choice(np.arange(-1, 8), n)]  # out of range and repeated ones among them
        if op == "reserve":
            p.call(op, slots, [int(x) for x in rng.choice([0, 1, 5, page - 1, page, 2 * page + 3, 5 * page], n)])
        elif op == "fork":
            p.call(op, [int(x) for x in rng.integers(0, 7, n)], slots)
        elif op == "truncate":
            lens = [int(rng.integers(-1 if rng.random() < .05 else 0, m.seq_len[s] + 1)) if 0 <= s < 7 else 0 for s in slots]
            p.call(op, slots, [0 if rng.random() < .3 else x for x in lens])
        elif op == "compact":
            p.call(op)
        else:
            slots = [int(x) for x in rng.permutation(7)[:n]]
            p.append(int(rng.integers(layers)), slots, [int(rng.integers(0, min(4, m.seq_len[s]) + 1)) for s in slots])


def test_reserve_without_slot_list_and_out_of_pages():
    p = Pair(pages=10, page=16, seqs=4, max_pages=8)
    kda.kda_kv_reserve(p.cache, None, _i32([16, 17, 64, 5]), 4)  # 1 + 2 + 4 + 1 pages
    p.model.reserve([0, 1, 2, 3], [16, 17, 64, 5])
    p.check()
    p.call("reserve", [0, 1, 2, 3], [1, 15, 17, 11])  # 1, 0, 2, 0: the third passes the two free pages
    p.call("reserve", [3, 2, 1], [129, 0, 0])         # past max_pages: refused, the rest as asked
    p.call("truncate", [1, 2], [3, 0])
    p.call("compact")


def test_fork_takes_parents_as_they_stand_and_refuses_what_is_not_empty():
    p = Pair(pages=40, page=16, seqs=8)
    p.call("reserve", [0, 1], [37, 32])
    p.append(0, [0], [37])
    p.append(1, [1], [32])
    p.call("fork", [0, 0, 1, 3, 0, 2], [2, 3, 4, 5, 2, 6])  # 3 -> 5 and 2 -> 6: empty at the start; 2 listed twice
    p.call("fork", [0, 7, 9, 0], [1, 7, 6, -1])             # not empty, itself, no slot
    p.call("reserve", [0, 2, 3], [1, 1, 12])
    p.append(1, [2, 3], [1, 12])
    p.call("truncate", [0, 2, 4], [0, 0, 0])
    p.call("truncate", [3, 1], [20, 10])
    p.call("fork", [3, 3], [0, 2])
    p.call("truncate", [0, 2], [12, 3])       # into shared pages
    p.call("reserve", [0, 3, 2], [1, 1, 20])  # copies of their own
    p.append(0, [0, 3, 2], [1, 1, 20])


def test_append_edges():
    p = Pair(pages=30, page=16, seqs=6, max_pages=5)
    p.call("reserve", [0, 1, 2, 3], [40, 1, 0, 16])
    p.append(0, [3, 0, 1, 2], [16, 40, 1, 0])
    p.append(1, [0, 1, 0, 9], [3, 1, 2, 1])      # listed before, no slot: refused
    p.append(1, [1, 3], [2, 1])                   # more rows than tokens: refused
    p.append(0, [0, 1], [7, 1], ids=False)
    p.call("fork", [0], [4])
    p.append(0, [0], [30])                        # its first rows lie in pages that slot 4 shares: not written
    for cu in ([5, 3, 4], [0, 4, 2], [0, -4, 2], [0, 2, 99], [2 ** 31 - 1, -2 ** 31, 3]):  # no bounds: nothing is read or written outside
        before = p.cache.k.clone()
        rows = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
        kda.kda_kv_append(p.cache, 0, rows, rows, _i32(cu), _i32([5, 5]), 2, 4)
        kda.device_status(clear=True)
        assert torch.equal(p.cache.k, before)


def test_append_with_decreasing_bounds_writes_nothing_it_has_not_read():
    p = Pair(pages=10, page=16, seqs=3, max_pages=4)
    p.call("reserve", [0, 1], [16, 16])
    before = p.cache.k.clone()
    rows = torch.ones((6, 128), dtype=torch.bfloat16, device="cuda")
    kda.kda_kv_append(p.cache, 0, rows, rows, _i32([0, 6, 2]), _i32([0, 1]), 2, 6)
    assert kda.device_status(clear=True) == 1 and torch.equal(p.cache.k, before)


def test_append_of_many_sequences():
    """More sequences than the rows' blocks mark one by one, empty ones among them."""
    n = 1500
    p = Pair(pages=n + 40, page=16, heads=1, seqs=n, max_pages=2, layers=1)
    rows = [(i * 7) % 3 for i in range(n)]
    kda.kda_kv_reserve(p.cache, None, _i32(rows), n)
    p.model.reserve(range(n), rows)
    p.append(0, list(range(n)), rows, ids=False)
    order = [int(x) for x in np.random.default_rng(3).permutation(n)]
    p.append(0, order, [rows[i] for i in order])


def test_large_pools_and_many_slots():
    """More pages than one round of the scan, more pairs than one block has threads, far offsets: pages
    past the 2^32nd byte of a pool."""
    pages, seqs = 33000, 1500
    c = kda.KVCache.empty(pages, 64, 8, 128, seqs, 40)
    add = [(37 * i) % 1300 for i in range(seqs)]
    kda.kda_kv_reserve(c, None, _i32(add), seqs)
    need = [-(-a // 64) for a in add]
    assert kda.device_status() == 0 and c.seq_len.tolist() == add
    table, first = c.page_table.cpu().numpy(), np.concatenate([[0], np.cumsum(need)])
    for i in range(seqs):
        assert table[i, :need[i]].tolist() == list(range(first[i], first[i + 1])) and (table[i, need[i]:] == -1).all()
    # all but the last slots leave; what remains moves down from the far end
    kda.kda_kv_reserve(c, _i32([0]), _i32([2500 - add[0]]), 1)
    full = int((c.ref > 0).sum())
    keep = _i32(range(1400, 1500))
    probe = torch.randn((1, 8 * 128), device="cuda").bfloat16()
    last = int(c.page_table[0, 39])
    assert last == full - 1
    c.ref[last], c.ref[pages - 1] = 0, 1
    c.page_table[0, 39] = pages - 1
    kda.kda_kv_append(c, 0, probe, -probe, _i32([0, 1]), _i32([0]), 1, 1)
    assert torch.equal(c.k[0, pages - 1, :, 3].reshape(-1), probe[0])  # token 2499: row 3 of its page
    kda.kda_kv_truncate(c, _i32(range(1, 1400)), _i32([0] * 1399), 1399)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_kv_compact(c, live)
    assert int(live) == 40 + sum(need[1400:]) == int((c.ref[:int(live)] > 0).sum()) == int((c.ref > 0).sum())
    got = c.page_table[0, 39]
    assert torch.equal(c.k[0, got, :, 3].reshape(-1), probe[0]) and torch.equal(c.v[0, got, :, 3].reshape(-1), -probe[0])
    assert int(c.page_table.max()) == int(live) - 1 and len(keep) == 100


def _append_with_bounds(p, cu, slots, total):
    """kda_kv_append with any bounds, against the rows that its description lets through: of a sequence whose bounds are
    0 <= cu[b] <= cu[b + 1] <= min(total, cu[B]); where cu decreases these may stay as they were too."""
    c, m = p.cache, p.model
    before = m.k.copy(), m.v.copy()
    w = c.k.shape[2] * c.k.shape[4]
    k_new, v_new = (torch.from_numpy(p.rng.standard_normal((total, w), dtype=np.float32)).cuda().bfloat16() for _ in range(2))
    kda.kda_kv_append(c, 0, k_new, v_new, _i32(cu), _i32(slots), len(slots), total)
    kb, vb = (_bits(t).reshape(-1, c.k.shape[2], c.k.shape[4]) for t in (k_new, v_new))
    for b, s in enumerate(slots):
        if 0 <= cu[b] <= cu[b + 1] <= min(total, cu[-1]):
            m.append(0, kb[cu[b]:cu[b + 1]], vb[cu[b]:cu[b + 1]], [0, cu[b + 1] - cu[b]], [s])
        else:
            m.status = 1
    if any(b < a for a, b in zip(cu, cu[1:])):
        assert m.status == 1
        m.k, m.v = (np.where((new == got).all(-1, keepdims=True), new, old) for new, old, got in
                    ((m.k, before[0], _bits(c.k)), (m.v, before[1], _bits(c.v))))
    p.check()


@pytest.mark.parametrize("cu", [[0, 4, 2, 6], [0, -4, 2, 6], [0, 2, 99, 6], [-1, 2, 4, 6], [2 ** 31 - 1, -2 ** 31, 3, 6], [0, 2, 4, 99],
                                [0, 2, 4, -1], [6, 4, 2, 0], [0, 0, 6, 3], [3, 5, 4, 6]])
def test_append_bad_bounds_of_sequences_with_room(cu):
    """Slots that hold enough tokens in pages of their own, so that only the bounds can refuse a row."""
    p = Pair(pages=12, page=16, seqs=3, max_pages=4)
    p.call("reserve", [0, 1, 2], [32, 32, 32])
    _append_with_bounds(p, cu, [2, 0, 1], 6)


@pytest.mark.parametrize("wrong", [{700: -5}, {700: 2 ** 31 - 1}, {3: 900, 1400: 2}, {0: -1}, {i: -i for i in range(1, 1500, 2)}, {1500: 40}])
def test_append_bad_bounds_among_many_sequences(wrong):
    """More sequences than the rows' blocks mark one by one."""
    n = 1500
    p = Pair(pages=n + 20, page=16, heads=1, seqs=n, max_pages=1, layers=1)
    kda.kda_kv_reserve(p.cache, None, _i32([3] * n), n)
    p.model.reserve(range(n), [3] * n)
    rows = [(i * 7) % 3 for i in range(n)]
    cu = [0] + np.cumsum(rows).tolist()
    total = cu[-1]
    for i, x in wrong.items():
        cu[i] = x
    order = [int(x) for x in np.random.default_rng(5).permutation(n)]
    _append_with_bounds(p, cu, order, total)


def test_fork_and_truncate_of_many_slots():
    """More pairs than one block has threads, refused ones among them, and pages that many slots share."""
    n = 1300
    p = Pair(pages=4000, page=16, heads=1, seqs=2 * n + 1, max_pages=3, layers=1)
    p.call("reserve", list(range(n)), [(i * 11) % 49 for i in range(n)])
    order = [int(x) for x in np.random.default_rng(8).permutation(n)]
    p.call("fork", [x if x % 50 else -1 for x in order], [n + i for i in range(n)])
    p.call("fork", [order[0]] * 4, [2 * n, 2 * n, 0, n])  # free, listed before, not empty, not empty or no pair's child
    slots = list(range(2 * n))
    lens = [int(x) for x in p.model.seq_len[:2 * n]]
    p.call("truncate", slots[::-1], [x // 2 for x in lens[::-1]])
    p.call("reserve", slots, [3] * (2 * n))  # copies of shared last pages, until the pages run out
    p.call("compact")


def test_a_captured_step_replayed():
    """Reserve, append, attention, truncate, fork and compaction in one graph, replayed on changing inputs."""
    page, H, D, seqs = 16, 2, 64, 5
    p = Pair(pages=30, page=page, heads=1, dim=D, seqs=seqs, max_pages=6, layers=2, seed=4)
    c, gen = p.cache, torch.Generator().manual_seed(9)
    p.call("reserve", [0, 1, 2], [13, 30, 1])
    slots, add, cu = _i32([2, 0, 1]), _i32([1, 1, 1]), _i32([0, 1, 2, 3])
    parent, child, gone, none = _i32([1]), _i32([3]), _i32([3]), _i32([0])
    k_new, v_new = (torch.zeros((3, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, out = (torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, d = torch.zeros((3, H), device="cuda"), kda.dims(H, D, scale=0.125)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kda.kda_kv_reserve(c, slots, add, 3)
        for layer in range(2):
            kda.kda_kv_append(c, layer, k_new, v_new, cu, slots, 3, 3)
            kda.kda_attn_decode(c, layer, q, slots, 3, 1, out, d, lse=lse)
        kda.kda_kv_truncate(c, gone, none, 1)
        kda.kda_kv_fork(c, parent, child, 1)
        kda.kda_kv_compact(c)
    p.check()  # capture alone changes nothing
    m = p.model
    for step in range(25):
        new = torch.randn((2, 3, D), generator=gen).bfloat16()
        qs = torch.randn((3, H, D), generator=gen).bfloat16()
        k_new.copy_(new[0]), v_new.copy_(new[1]), q.copy_(qs)
        g.replay()
        m.reserve([2, 0, 1], [1, 1, 1])
        for layer in range(2):
            m.append(layer, *[_bits(x).reshape(3, 1, D) for x in (k_new, v_new)], [0, 1, 2, 3], [2, 0, 1])
        for i, s in enumerate([2, 0, 1]):
            n = int(m.seq_len[s])
            kv = [torch.from_numpy(np.stack([x[1, m.table[s, j // page], 0, j % page] for j in range(n)]).view(np.int16)).view(
                torch.bfloat16).double().numpy() for x in (m.k, m.v)]
            o, l, sp = zip(*[oracle.attention(qs[i, h:h + 1].double().numpy(), kv[0], kv[1], [n - 1], 0.125) for h in range(H)])
            check(out[i:i + 1], lse[i:i + 1], (np.stack(o, 1), np.stack(l, 1), np.stack(sp, 1)))
        m.truncate([3], [0])
        m.fork([1], [3])
        m.compact()
        p.check()
