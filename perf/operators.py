"""The paged key-value cache operators and the attention that reads it: cases, plain forms and the library's calls.

Five operators over one cache (K and V pools [layers, pages, kv_heads, page_size, D] BF16, a page table
[max_seqs, max_pages] with -1 for no page, sequence lengths and page reference counts):

  decode   K query rows of each of N sequences against the sequence's cached rows
  prefill  packed prompt (or draft) rows of B sequences against the cache they were appended to
  append   packed K and V rows into the pages of their sequences
  beam     dropping, forking and extending sequences (page bookkeeping and the copy of each partly filled last page)
  compact  moving the live pages to the front of the pools

Query row t of the n rows of a sequence of length len stands at position p = len - n + t and sees the cached rows
j <= p with window == 0 or j > p - window or j < sinks: o = sum_j softmax_j(scale q.k_j) v_j, lse = log sum_j
exp(scale q.k_j); a row that sees nothing has o = 0 and lse = -inf.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one interactive sequence, 4096 cached tokens: a step whose latency counts
        dict(name="decode 1 x 4096", op="decode", seqs=1, rows=1, heads=32, kv_heads=8, dim=128, page=64, max_len=4096,
             ragged=False, window=0, sinks=0),
        # a serving batch of unequal sequences on small pages, four draft rows each (a speculative step)
        dict(name="decode 64 ragged, 4 rows", op="decode", seqs=64, rows=4, heads=32, kv_heads=8, dim=128, page=16,
             max_len=8000, ragged=True, window=0, sinks=0),
        # a few very long contexts
        dict(name="decode 8 x 65500", op="decode", seqs=8, rows=1, heads=32, kv_heads=8, dim=128, page=64,
             max_len=65500, ragged=False, window=0, sinks=0),
        # the draft rows of eight sequences, 1 to 4 each
        dict(name="prefill 8 drafts", op="prefill", seqs=8, max_rows=4, cached=2000, heads=32, kv_heads=8, dim=128,
             page=64, ragged=True, window=0, sinks=0),
        # a packed batch of unequal prompts, some behind cached tokens, with window and sinks, small heads
        dict(name="prefill 6 packed, windowed", op="prefill", seqs=6, max_rows=2341, cached=1000, heads=16, kv_heads=4,
             dim=64, page=16, ragged=True, window=512, sinks=4),
        # one long prompt, every earlier token visible
        dict(name="prefill 1 x 8192", op="prefill", seqs=1, max_rows=8192, cached=0, heads=32, kv_heads=8, dim=128,
             page=64, ragged=False, window=0, sinks=0),
        # one token of each of 256 sequences
        dict(name="append 256 x 1", op="append", seqs=256, max_rows=1, cached=1000, kv_heads=8, dim=128, page=16,
             ragged=False),
        # the rows of a packed prefill
        dict(name="append 8 packed", op="append", seqs=8, max_rows=8192, cached=500, kv_heads=8, dim=128, page=64,
             ragged=True),
        # one prompt forked into four samples
        dict(name="beam 1 to 4", op="beam", seqs=1, width=4, max_len=1000, layers=4, kv_heads=8, dim=128, page=16),
        # a beam search of 64 requests
        dict(name="beam 64 to 256", op="beam", seqs=64, width=4, max_len=1000, layers=8, kv_heads=8, dim=128, page=64),
        # a small pool with a few holes
        dict(name="compact 256 pages", op="compact", pages=256, live_percent=80, seqs=16, layers=4, kv_heads=8, dim=128,
             page=16),
        # a pool that half of its sequences have left
        dict(name="compact 4096 pages", op="compact", pages=4096, live_percent=50, seqs=64, layers=4, kv_heads=8,
             dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "beam", "compact"])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, kv_heads=kv_heads, dim=dim, page=page)
    if op in ("decode", "prefill"):
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        c.update(heads=kv_heads * group, ragged=rng.random() < 0.7, window=0, sinks=0)
        if rng.random() < 0.5:
            c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 5, 64, 130]))
    if op == "decode":
        seqs = _log(rng, 1, 256)
        rows = rng.randint(1, max(1, min(8, 64 // group)))
        room = 8 * 65500 * 8 * 128 // (seqs * kv_heads * dim)
        c.update(seqs=seqs, rows=rows, max_len=_log(rng, 1, min(65500, room)))
    elif op == "prefill":
        seqs = _log(rng, 1, 16)
        room = int(math.sqrt(8192 * 8192 * 32 / (2 * seqs * c["heads"])))
        rows = _log(rng, 1, min(8192, room))
        c.update(seqs=seqs, max_rows=rows, cached=rng.choice([0, _log(rng, 1, min(16000, 8192 * 8192 * 16 // (seqs * c["heads"] * rows)))]))
    elif op == "append":
        seqs = _log(rng, 1, 256)
        c.update(seqs=seqs, max_rows=_log(rng, 1, max(1, 60000 // seqs)), cached=rng.choice([0, _log(rng, 1, 1000)]),
                 ragged=rng.random() < 0.7)
    elif op == "beam":
        c.update(seqs=_log(rng, 1, 64), width=rng.randint(1, 4), max_len=_log(rng, 1, 1000), layers=rng.randint(1, 8))
    else:
        seqs = _log(rng, 1, 64)
        c.update(pages=max(2 * seqs, _log(rng, 16, 4096 * 16 // page)), live_percent=rng.randint(20, 95), seqs=seqs,
                 layers=rng.randint(1, 4))
    return c


# ------------------------------------------------------------------------------------------- sizes of a case

def _lens(case):
    """Per sequence, before shuffling: (rows, length with them)."""
    n = case["seqs"]
    if case["op"] == "decode":
        return [(case["rows"], case["max_len"] * (i + 1) // n if case["ragged"] else case["max_len"]) for i in range(n)]
    if case["op"] in ("prefill", "append"):
        r = [case["max_rows"] * (i + 1) // n if case["ragged"] else case["max_rows"] for i in range(n)]
        c = [case["cached"] * ((7 * i + 3) % n + 1) // n if case["ragged"] else case["cached"] for i in range(n)]
        return [(a, a + b) for a, b in zip(r, c)]
    return [(0, max(1, case["max_len"] * (i + 1) // n)) for i in range(n)]


def _visible(p, window, sinks):
    if p < 0:
        return 0
    return p + 1 if not window or p < window else window + min(sinks, p + 1 - window)


def work(case):
    """What a pass cannot do without: every visible cached row, the queries and the outputs once."""
    op, d, hk = case["op"], case["dim"], case["kv_heads"]
    if op in ("decode", "prefill"):
        h, w, s = case["heads"], case["window"], case["sinks"]
        pairs = kv = total = 0
        for n, ln in _lens(case):
            pairs += sum(_visible(ln - n + t, w, s) for t in range(n))
            first = ln - n - w + 1  # the first row in some query's window
            kv += (ln if not w or first <= s else ln - first + s) if n and ln > 0 else 0
            total += n
        return {"bytes": kv * hk * d * 4 + total * h * (d * 4 + 4), "flops": 4 * pairs * h * d}
    if op == "append":
        return {"bytes": sum(n for n, _ in _lens(case)) * hk * d * 8, "flops": 0}
    if op == "beam":
        rows = sum(ln % case["page"] for _, ln in _lens(case)) * case["width"]
        entries = sum(-(-ln // case["page"]) for _, ln in _lens(case)) * case["width"]
        return {"bytes": rows * case["layers"] * hk * d * 8 + entries * 12, "flops": 0}
    live = case["pages"] * case["live_percent"] // 100
    moved = live * (case["pages"] - live) // case["pages"]  # the expected number past the live count
    return {"bytes": moved * case["layers"] * hk * case["page"] * d * 8 + 8 * live + 8 * case["pages"], "flops": 0}


# ------------------------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(shape, dtype=torch.bfloat16, device=DEV, generator=gen)


def _pool(gen, case, num_pages, layers=1):
    shape = (layers, num_pages, case["kv_heads"], case["page"], case["dim"])
    return _randn(gen, *shape), _randn(gen, *shape)


def _table(lens, page, max_seqs, max_pages, order):
    """A page table whose sequences take their pages from `order`, one after the other."""
    table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32)
    at = 0
    for i, ln in enumerate(lens):
        n = -(-ln // page)
        table[i, :n] = order[at:at + n]
        at += n
    return table, at


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op, page = case["op"], case["page"]
    s = {"case": case}
    if op == "compact":
        live = case["pages"] * case["live_percent"] // 100
        each = [live * (i + 1) // case["seqs"] - live * i // case["seqs"] for i in range(case["seqs"])]
        lens = [n * page for n in each]
        order = torch.randperm(case["pages"], generator=host, dtype=torch.int64).to(torch.int32)
        table, used = _table(lens, page, case["seqs"], max(each), order)
        ref = torch.zeros(case["pages"], dtype=torch.int32)
        ref[order[:used].long()] = 1
        s["k"], s["v"] = _pool(gen, case, case["pages"], case["layers"])
        s.update(table0=table.to(DEV), ref0=ref.to(DEV), seq_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 live=torch.zeros(1, dtype=torch.int32, device=DEV))
        s.update(table=s["table0"].clone(), ref=s["ref0"].clone())
        return s
    sizes = _lens(case)
    sizes = [sizes[i] for i in torch.randperm(len(sizes), generator=host).tolist()]
    rows, lens = [r for r, _ in sizes], [n for _, n in sizes]
    n = case["seqs"]
    if op == "beam":
        children = n * case["width"]
        lens = lens + [1 + (i * 37) % page for i in range(children)]  # what the children's slots held before
        max_seqs, max_pages = n + children, -(-(max(lens) + 1) // page)
        pages = sum(-(-ln // page) for ln in lens) + 2 * children + 8
    else:
        max_seqs, max_pages = n, max(1, -(-max(lens) // page))
        pages = sum(-(-ln // page) for ln in lens) + 8
    order = torch.randperm(pages, generator=host, dtype=torch.int64).to(torch.int32)
    table, used = _table(lens, page, max_seqs, max_pages, order)
    ref = torch.zeros(pages, dtype=torch.int32)
    ref[order[:used].long()] = 1
    s["k"], s["v"] = _pool(gen, case, pages, case.get("layers", 1))
    s.update(table=table.to(DEV), ref=ref.to(DEV), seq_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if op == "beam":
        s["parent"] = torch.arange(n, dtype=torch.int32, device=DEV).repeat_interleave(case["width"])
        s["child"] = torch.arange(n, n + children, dtype=torch.int32, device=DEV)
        s["zero"] = torch.zeros(children, dtype=torch.int32, device=DEV)
        s["one"] = torch.ones(children, dtype=torch.int32, device=DEV)
        return s
    total = sum(rows)
    s.update(total=total, max_rows=max(rows), max_len=max(lens), slots=torch.arange(n, dtype=torch.int32, device=DEV),
             cu=torch.tensor([sum(rows[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV))
    if op == "append":  # the k and v columns of packed q|k|v projection rows
        w = case["kv_heads"] * case["dim"]
        qkv = _randn(gen, total, 6 * w)
        s["k_new"], s["v_new"] = qkv[:, 4 * w:5 * w], qkv[:, 5 * w:]
        return s
    # queries with twice the keys' spread, so that a row attends to few keys, as trained heads do
    s["q"] = _randn(gen, total, case["heads"], case["dim"]) * 2
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((total, case["heads"]), dtype=torch.float32, device=DEV)
    s["scale"] = case["dim"] ** -0.5
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _gather(pool, table):
    """[pages, Hk, page, D] and [B, n] page indices -> [B, Hk, n * page, D] in 32 bits."""
    got = pool[table.clamp(min=0).long()]
    b, n, hk, page, d = got.shape
    return got.permute(0, 2, 1, 3, 4).reshape(b, hk, n * page, d).float()


def _plain_attention(s):
    case = s["case"]
    hk, d, h = case["kv_heads"], case["dim"], case["heads"]
    b, r, g = case["seqs"], s["max_rows"], h // hk
    k, v = _gather(s["k"][0], s["table"]), _gather(s["v"][0], s["table"])
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    t = torch.arange(r, device=DEV)
    real = t < n[:, None]                                                   # [b, r]
    row = torch.where(real, s["cu"][:-1, None].long() + t, 0)
    q = s["q"][row].float().reshape(b, r, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, r * g, d)
    p = (s["seq_len"].long() - n)[:, None] + t
    j = torch.arange(k.shape[2], device=DEV)
    seen = j <= p[..., None]
    if case["window"]:
        seen &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    seen = seen.repeat_interleave(g, dim=1)[:, None]                        # [b, 1, r * g, keys]
    x = torch.where(seen, q @ k.transpose(2, 3) * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, e @ v / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.reshape(b, hk, r, g, d).permute(0, 2, 1, 3, 4).reshape(b, r, h, d)
    lse = lse.reshape(b, hk, r, g).permute(0, 2, 1, 3).reshape(b, r, h)
    return o[real].to(torch.bfloat16), lse[real]


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), n, output_size=s["total"])
    t = torch.arange(s["total"], device=DEV) - s["cu"][:-1].long()[seq]
    at = (s["seq_len"].long() - n)[seq] + t
    to = s["table"][seq, at // page].long()
    shape = (s["total"], case["kv_heads"], case["dim"])
    s["k"][0][to, :, at % page] = s["k_new"].reshape(shape)
    s["v"][0][to, :, at % page] = s["v_new"].reshape(shape)
    return s["k"], s["v"]


def _take_free(ref, count):
    """The `count` lowest pages with no reference, now with one."""
    got = torch.nonzero(ref == 0)[:count, 0]
    ref[got] = 1
    return got


def _plain_truncate(s, slots, new_len):
    slots, page = slots.long(), s["case"]["page"]
    rows = s["table"][slots]
    gone = (torch.arange(rows.shape[1], device=DEV) >= (new_len.long()[:, None] + page - 1) // page) & (rows >= 0)
    s["ref"].index_add_(0, rows[gone].long(), torch.full((1,), -1, dtype=torch.int32, device=DEV).expand(int(gone.sum())))
    s["table"][slots] = torch.where(gone, -1, rows)
    s["seq_len"][slots] = new_len


def _plain_fork(s, parent, child):
    parent, child, page = parent.long(), child.long(), s["case"]["page"]
    ln = s["seq_len"][parent].long()
    full, rest = ln // page, ln % page
    rows = s["table"][parent]
    shared = torch.arange(rows.shape[1], device=DEV) < full[:, None]
    pages = rows[shared].long()
    s["ref"].index_add_(0, pages, torch.ones(1, dtype=torch.int32, device=DEV).expand(pages.numel()))
    s["table"][child] = torch.where(shared, rows, -1)
    part = torch.nonzero(rest > 0)[:, 0]
    dst = _take_free(s["ref"], part.numel())
    src = rows[part, full[part]].long()
    s["table"][child[part], full[part]] = dst.to(torch.int32)
    keep = (torch.arange(page, device=DEV) < rest[part, None])[None, :, None, :, None]
    for pool in (s["k"], s["v"]):
        pool[:, dst] = torch.where(keep, pool[:, src], pool[:, dst])
    s["seq_len"][child] = ln.to(torch.int32)


def _plain_reserve_one(s, slots):
    """Room for one more token in each slot."""
    slots, page = slots.long(), s["case"]["page"]
    ln = s["seq_len"][slots].long()
    need = torch.nonzero(ln % page == 0)[:, 0]
    got = _take_free(s["ref"], need.numel())
    s["table"][slots[need], ln[need] // page] = got.to(torch.int32)
    s["seq_len"][slots] = (ln + 1).to(torch.int32)


def _plain_compact(s):
    ref = s["ref"]
    used = ref > 0
    live = int(used.sum())
    dst = torch.nonzero(~used[:live])[:, 0]
    src = torch.nonzero(used[live:])[:, 0] + live
    for pool in (s["k"], s["v"]):
        pool[:, dst] = pool[:, src]
    to = torch.arange(ref.numel(), device=DEV, dtype=torch.int32)
    to[src] = dst.to(torch.int32)
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], -1))
    ref[dst] = ref[src]
    ref[src] = 0
    s["live"].fill_(live)


# ------------------------------------------------------------------------------------------- the calls

def _handles(s):
    """The cache handle and dimensions that a user's program makes once and keeps."""
    if "cache" not in s:
        import kda_gated_delta_gate_b200 as kda
        case = s["case"]
        s["kda"] = kda
        s["cache"] = kda.KVCache(s["k"], s["v"], s["table"], s["seq_len"], s["ref"])
        if "heads" in case:
            s["dims"] = kda.dims(case["heads"], case["dim"], scale=s["scale"])
    return s["kda"], s["cache"]


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "compact":  # the scheduler's own tables go up first, as after each of its steps
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
    if own:
        kda, cache = _handles(s)
        if op == "decode":
            kda.kda_attn_decode(cache, 0, s["q"], s["slots"], case["seqs"], case["rows"], s["out"], s["dims"],
                                window=case["window"], sinks=case["sinks"], lse=s["lse"])
        elif op == "prefill":
            kda.kda_attn_prefill(cache, 0, s["q"], s["cu"], s["slots"], case["seqs"], s["max_rows"], s["total"],
                                 s["out"], s["dims"], window=case["window"], sinks=case["sinks"], lse=s["lse"])
        elif op == "append":
            kda.kda_kv_append(cache, 0, s["k_new"], s["v_new"], s["cu"], s["slots"], case["seqs"], s["total"])
        elif op == "beam":
            n = s["child"].numel()
            kda.kda_kv_truncate(cache, s["child"], s["zero"], n)
            kda.kda_kv_fork(cache, s["parent"], s["child"], n)
            kda.kda_kv_reserve(cache, s["child"], s["one"], n)
        else:
            kda.kda_kv_compact(cache, s["live"])
    elif op in ("decode", "prefill"):
        return dict(zip(("out", "lse"), _plain_attention(s)))
    elif op == "append":
        _plain_append(s)
    elif op == "beam":
        _plain_truncate(s, s["child"], s["zero"])
        _plain_fork(s, s["parent"], s["child"])
        _plain_reserve_one(s, s["child"])
    else:
        _plain_compact(s)
    if op in ("decode", "prefill"):
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        return {"k": s["k"], "v": s["v"]}
    got = {"k": s["k"], "v": s["v"], "table": s["table"], "seq_len": s["seq_len"], "ref": s["ref"]}
    return {**got, "live": s["live"]} if op == "compact" else got


def exact(case, seed):
    """The attention of each sequence and kv head by itself, in 64 bits; the other operators move data unchanged."""
    if case["op"] not in ("decode", "prefill"):
        return None
    s = prepare(case, seed)
    hk, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    cu, lens, table = s["cu"].tolist(), s["seq_len"].tolist(), s["table"].tolist()
    for i in range(case["seqs"]):
        n, ln = cu[i + 1] - cu[i], lens[i]
        pages = torch.tensor(table[i][:-(-ln // case["page"])], device=DEV, dtype=torch.int64)
        place = torch.arange(ln - n, ln, device=DEV)
        key = torch.arange(max(ln, 0), device=DEV)
        hidden = key[None, :] > place[:, None]
        if case["window"]:
            hidden |= (place[:, None] - key[None, :] >= case["window"]) & (key[None, :] >= case["sinks"])
        if ln <= 0 or n == 0:
            continue
        for hh in range(hk):
            keys = s["k"][0, pages, hh].reshape(-1, case["dim"])[:ln].double()
            vals = s["v"][0, pages, hh].reshape(-1, case["dim"])[:ln].double()
            for a in range(hh * g, hh * g + g):
                logit = (s["q"][cu[i]:cu[i + 1], a].double() @ keys.T) * s["scale"]
                logit.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(logit, dim=1)
                lse[cu[i]:cu[i + 1], a] = z
                weight = torch.exp(logit - torch.where(z == -math.inf, 0.0, z)[:, None])
                out[cu[i]:cu[i + 1], a] = weight @ vals
    return {"out": out, "lse": lse}
