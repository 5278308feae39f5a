"""The shared-prefix decode attention and the page operations, as a user calls them, with plain forms beside them.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program has in hand, ``run()`` one pass: in elementary
torch operations (``own`` false) or by the library's calls (``own`` true).  ``exact()`` is the attention in 64 bits.

Layouts: q and out fp16 [B][nq][Hq][128]; fp16 cache [blocks][Hkv][bs][128]; q8_0 and int8-row cache bytes
[blocks][Hkv][tile], the int8 values of a tile first, then its scales (fp16 per 32 values, or fp32 per row);
block_table int32 [rows][entries]; lengths int32 [rows].
"""
import random

import numpy as np
import torch

own = False

D = 128
SCALE = float(np.float32(D ** -0.5))
KV = {"fp16": 0, "q8_0": 1, "int8_row": 2}


# ------------------------------------------------------------------ cases
def _attend(name, kv, batch, n_query, q_heads, kv_heads, block, prefix, suffix, causal=1, window=0):
    case = dict(op="attend", kv=kv, batch=batch, n_query=n_query, q_heads=q_heads, kv_heads=kv_heads, block=block,
                prefix=prefix, suffix=suffix, causal=causal, window=window)
    return dict(case, name=name) if name else case


def _copy(name, kv, kv_heads, block, blocks, pairs):
    case = dict(op="copy", kv=kv, kv_heads=kv_heads, block=block, blocks=blocks, pairs=pairs)
    return dict(case, name=name) if name else case


def _fork(name, kv, kv_heads, block, blocks, parents, children, longest, grow):
    case = dict(op="fork", kv=kv, kv_heads=kv_heads, block=block, blocks=blocks, parents=parents, children=children,
                longest=longest, grow=grow)
    return dict(case, name=name) if name else case


def _compact(name, kv, kv_heads, block, blocks, live, moves, rows):
    case = dict(op="compact", kv=kv, kv_heads=kv_heads, block=block, blocks=blocks, live=live, moves=moves, rows=rows)
    return dict(case, name=name) if name else case


def listed():
    return [
        # four answers to one short prompt, the first tokens: a call that is all latency
        _attend("attend-few-short", "fp16", 4, 1, 32, 8, 16, 1024, 48),
        # a batch behind one system prompt of 16k tokens, plain decode steps
        _attend("attend-batch", "fp16", 32, 1, 32, 8, 16, 16384, 700),
        # the same with speculative verify steps of 8 tokens over a 32k prompt in larger pages
        _attend("attend-verify", "fp16", 16, 8, 32, 8, 64, 32768, 1500),
        # verify steps of 4 tokens over a q8_0 cache, odd page size
        _attend("attend-q8_0", "q8_0", 24, 4, 32, 8, 48, 24576, 900),
        # 24 query rows a sequence (4 tokens x 6 heads) over int8 rows, 61k tokens in common
        _attend("attend-int8-row", "int8_row", 8, 4, 24, 4, 16, 61440, 1200),
        # many answers over a 128k document: the largest call
        _attend("attend-long", "fp16", 64, 1, 64, 8, 16, 131072, 1000),
        # a handful of pages of a small cache: latency
        _copy("copy-few", "fp16", 2, 16, 128, 7),
        # a long sequence's pages moved at once
        _copy("copy-many", "q8_0", 8, 32, 12289, 5001),
        # one prompt, seven answers, one new token each
        _fork("fork-one", "fp16", 8, 16, 4096, 1, 7, 8192, 1),
        # a round of parallel sampling for 32 prompts, 4 new tokens each
        _fork("fork-round", "fp16", 8, 16, 24576, 32, 7, 9000, 4),
        # a small pool closed up after a few sequences ended
        _compact("compact-small", "fp16", 2, 16, 400, 150, 37, 6),
        # a large pool, two thirds live, closed up
        _compact("compact-large", "fp16", 8, 16, 16384, 11000, 3300, 64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "copy", "fork", "compact"])
    kv = rng.choice(["fp16", "fp16", "q8_0", "int8_row"])
    if op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 6, 8])
        n_query = rng.choice([1, 1, 2, 3, 4, 8, 12])
        block = 16 * rng.choice([1, 1, 2, 3, 4, 7])
        batch = _log(rng, 1, 64)
        prefix = _log(rng, 16, 131072)
        while batch * n_query * group * kv_heads * prefix > 300_000_000:  # no more than the largest listed one
            prefix //= 2
        prefix = max(1, prefix // block) * block
        suffix = _log(rng, n_query + 1, 2000)
        window = rng.choice([0, 0, 0, _log(rng, 64, 4096)])
        return _attend(None, kv, batch, n_query, group * kv_heads, kv_heads, block, prefix, suffix,
                       rng.choice([1, 1, 1, 0]), window)
    kv_heads, block = rng.choice([1, 2, 4, 8]), 16 * rng.choice([1, 2, 3, 4])
    most = 12000 * 16 // (block * kv_heads // 8 or 1)
    most = min(most, 40000)
    if op == "copy":
        pairs = _log(rng, 1, most // 2 - 8)
        return _copy(None, kv, kv_heads, block, 2 * pairs + rng.randrange(1, 9), pairs)
    if op == "fork":
        parents, children, longest, grow = _log(rng, 1, 24), rng.randrange(1, 9), _log(rng, 40, 6000), rng.randrange(1, 40)
        need = parents * (-(-longest // block) + children * (2 + -(-grow // block)) + 2 + -(-grow // block))
        return _fork(None, kv, kv_heads, block, need + rng.randrange(0, 500), parents, children, longest, grow)
    blocks = _log(rng, 8, most)
    live = rng.randrange(2, max(3, blocks - 1))
    moves = rng.randrange(1, max(2, min(live, blocks - live)))
    return _compact(None, kv, kv_heads, block, blocks, live, moves, rng.randrange(1, 65))


def _token_bytes(kv):
    """Bytes of one key or value row of one KV head."""
    return {"fp16": 256, "q8_0": 136, "int8_row": 132}[kv]


def _lengths(case):
    """Context lengths: the prefix, then between n_query and `suffix` tokens of a sequence's own, all different."""
    batch, low = case["batch"], case["n_query"]
    span = max(0, case["suffix"] - low)
    return [case["prefix"] + low + (span * ((s * 37 + 11) % batch) // max(1, batch - 1) if batch > 1 else span)
            for s in range(batch)]


def work(case):
    page = case["kv_heads"] * case["block"] * _token_bytes(case["kv"])
    if case["op"] == "attend":
        rows, flops, own_keys, low_all, high_all = case["n_query"] * case["q_heads"], 0, 0, case["prefix"], 0
        for length in _lengths(case):
            lows = []
            for i in range(case["n_query"]):
                high = length - case["n_query"] + i if case["causal"] else length - 1
                low = max(0, high - case["window"] + 1) if case["window"] else 0
                lows.append(low)
                flops += 4 * D * case["q_heads"] * (high - low + 1)
            own_keys += length - max(case["prefix"], min(lows))
            low_all, high_all = min(low_all, min(lows)), case["prefix"]
        keys = max(0, high_all - low_all) + own_keys
        data = keys * case["kv_heads"] * 2 * _token_bytes(case["kv"])
        return {"bytes": data + 4 * case["batch"] * rows * D, "flops": flops}
    if case["op"] == "copy":
        return {"bytes": 4 * page * case["pairs"] + 8 * case["pairs"], "flops": 0}
    if case["op"] == "fork":
        rows = case["parents"] * (1 + case["children"])
        copies = case["parents"] * case["children"]
        return {"bytes": 4 * page * copies + 4 * rows * 8 + 4 * rows * (case["longest"] // case["block"]), "flops": 0}
    return {"bytes": 4 * page * case["moves"] + 8 * case["blocks"] + 8 * case["live"], "flops": 0}


# ------------------------------------------------------------------ inputs
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _generator(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    return g


def _cache(kv, x):
    """fp16 values [blocks][Hkv][bs][128] as a cache of this type."""
    if kv == "fp16":
        return x
    blocks, heads, bs, _ = x.shape
    parts = []
    for piece in x.split(2048):  # in pieces: the 32-bit copies are large
        f = piece.float()
        if kv == "q8_0":
            g = f.view(-1, heads, bs, 4, 32)
            d = (g.abs().amax(-1) / 127).half()
            q = (g / d.float().clamp_min(1e-30).unsqueeze(-1)).round().clamp(-127, 127)
        else:
            d = f.abs().amax(-1) / 127
            q = (f / d.clamp_min(1e-30).unsqueeze(-1)).round().clamp(-127, 127)
        values = q.to(torch.int8).reshape(len(piece), heads, bs * D).view(torch.uint8)
        scales = d.contiguous().reshape(len(piece), heads, -1).view(torch.uint8)
        parts.append(torch.cat([values, scales], -1))
    return torch.cat(parts).contiguous()


def _inputs(case, seed):
    g, dev = _generator(seed), _device()
    host = np.random.RandomState(seed % (2 ** 31))
    half = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.float16)  # noqa: E731
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)       # noqa: E731
    bs, heads = case["block"], case["kv_heads"]
    if case["op"] == "attend":
        lens = _lengths(case)
        shared = case["prefix"] // bs
        rest = [-(-n // bs) - shared for n in lens]
        blocks = shared + sum(rest) + 3
        order = host.permutation(blocks)
        width = shared + max(rest) + 1
        table = np.full((case["batch"], width), -1)
        table[:, :shared] = order[:shared]
        at = shared
        for s, n in enumerate(rest):
            table[s, shared:shared + n] = order[at:at + n]
            at += n
        k, v = half(blocks, heads, bs, D), half(blocks, heads, bs, D)
        # one key in a hundred stands out, so that some rows have a few heavy weights
        k *= torch.where(torch.rand(blocks, heads, bs, 1, generator=g, device=dev) < 0.01, 4.0, 1.0).half()
        return dict(case=case, q=half(case["batch"], case["n_query"], case["q_heads"], D), k=_cache(case["kv"], k),
                    v=_cache(case["kv"], v), table=ints(table), lens=ints(lens), prefix_table=ints(order[:shared]),
                    prefix_len=ints([case["prefix"]]))
    blocks = case["blocks"]
    if case["kv"] == "fp16":
        k, v = half(blocks, heads, bs, D), half(blocks, heads, bs, D)
    else:
        shape = (blocks, heads, bs * _token_bytes(case["kv"]))
        k, v = (torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8) for _ in range(2))
    state = dict(case=case, k=k, v=v)
    if case["op"] == "copy":
        order = host.permutation(blocks)[:2 * case["pairs"]]
        return dict(state, src=ints(order[:case["pairs"]]), dst=ints(order[case["pairs"]:]))
    if case["op"] == "fork":
        parents, children = case["parents"], case["children"]
        rows = parents * (1 + children)
        lens = np.zeros(rows, dtype=np.int64)
        low = max(1, case["longest"] // 2 // bs)
        high = max(low + 1, case["longest"] // bs)
        lens[:parents] = bs * host.randint(low, high, parents) - host.randint(1, bs, parents)  # a ragged last page
        width = -(-(case["longest"] + case["grow"] + bs) // bs)
        order = host.permutation(blocks)
        table, refs, at = np.full((rows, width), -1), np.zeros(blocks), 0
        for s in range(parents):
            n = -(-lens[s] // bs)
            table[s, :n] = order[at:at + n]
            refs[order[at:at + n]] = 1
            at += n
        kids = np.arange(parents, rows)
        return dict(state, table=ints(table), lens=ints(lens), refs=ints(refs), parents=ints((kids - parents) // children),
                    children=ints(kids), rows=ints(np.concatenate([kids, np.arange(parents)])),
                    base=ints(np.concatenate([np.zeros(len(kids)), lens[:parents]])),
                    grown=ints(np.concatenate([np.repeat(lens[:parents], children), lens[:parents]]) + case["grow"]))
    # compact: `moves` live pages lie behind the first `live` slots
    live, moves, rows = case["live"], case["moves"], case["rows"]
    alive = np.zeros(blocks, dtype=bool)
    alive[:live] = True
    alive[host.permutation(live)[:moves]] = False
    alive[live + host.permutation(blocks - live)[:moves]] = True
    pages = host.permutation(np.flatnonzero(alive))
    common = pages[:live // 4]  # a prefix that every row shares
    each = np.array_split(pages[live // 4:], rows)
    width = len(common) + max(len(e) for e in each) + 1
    table, refs, lens = np.full((rows, width), -1), np.zeros(blocks), np.zeros(rows)
    refs[common] = rows
    for s, e in enumerate(each):
        row = np.concatenate([common, e])
        table[s, :len(row)] = row
        refs[e] = 1
        lens[s] = max(0, len(row) * bs - host.randint(0, bs))
    meta = ints(np.concatenate([table.ravel(), refs, lens]))  # one buffer: the pass starts from the same books
    state.update(meta0=meta.clone(), meta=meta, table=meta[:rows * width].view(rows, width),
                 refs=meta[rows * width:rows * width + blocks], lens=meta[rows * width + blocks:])
    return state


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        from paged_kv_decode_flash_b200 import pages, shared_prefix
        if case["op"] == "attend":
            state["decode"] = shared_prefix.SharedPrefixDecode(
                num_seqs=case["batch"], num_q_heads=case["q_heads"], num_kv_heads=case["kv_heads"], head_dim=D,
                block_size=case["block"], max_blocks_per_seq=state["table"].shape[1], num_blocks=len(state["k"]),
                n_query=case["n_query"], prefix_blocks=len(state["prefix_table"]))
        elif case["op"] == "copy":
            state["pool"] = pages.PagePool(num_seqs=1, num_kv_heads=case["kv_heads"], head_dim=D,
                                           block_size=case["block"], max_blocks_per_seq=1, num_blocks=case["blocks"])
        else:
            state["pool"] = pages.PagePool(num_seqs=len(state["lens"]), num_kv_heads=case["kv_heads"], head_dim=D,
                                           block_size=case["block"], max_blocks_per_seq=state["table"].shape[1],
                                           num_blocks=case["blocks"], block_table=state["table"],
                                           context_lens=state["lens"], ref_counts=state["refs"])
    return state


# ------------------------------------------------------------------ plain forms
def _values(kv, tiles, bs):
    """Tiles [...][Hkv][tile] of a cache as 32-bit values [...][Hkv][bs][128]."""
    if kv == "fp16":
        return tiles.float()
    lead = tiles.shape[:-1]
    q = tiles[..., :bs * D].contiguous().view(torch.int8).view(*lead, bs, D).float()
    raw = tiles[..., bs * D:].contiguous()
    if kv == "q8_0":
        d = raw.view(torch.float16).view(*lead, bs, 4).float()
        return (q.view(*lead, bs, 4, 32) * d.unsqueeze(-1)).view(*lead, bs, D)
    return q * raw.view(torch.float32).view(*lead, bs, 1)


def _plain_attend(st):
    c = st["case"]
    b, nq, hq, hkv, bs = c["batch"], c["n_query"], c["q_heads"], c["kv_heads"], c["block"]
    group, prefix = hq // hkv, c["prefix"]
    dev = st["q"].device
    q = st["q"].float().view(b, nq, hkv, group, D).permute(2, 0, 1, 3, 4)             # [Hkv][B][nq][G][D]
    high = st["lens"].view(b, 1) - (nq - torch.arange(nq, device=dev) if c["causal"] else
                                    torch.ones(nq, dtype=torch.int64, device=dev))    # the last visible key [B][nq]
    low = high - c["window"] + 1 if c["window"] else torch.zeros_like(high)
    # the prefix once, for all rows of a KV head
    pk, pv = (_values(c["kv"], st[n][st["prefix_table"]], bs).transpose(0, 1).reshape(hkv, prefix, D) for n in "kv")
    zp = torch.matmul(q.reshape(hkv, -1, D), pk.transpose(1, 2)).view(hkv, b, nq, group, prefix) * SCALE
    at = torch.arange(prefix, device=dev)
    see = (at >= low.unsqueeze(-1)) & (at <= high.unsqueeze(-1))                       # [B][nq][P]
    zp = zp.masked_fill(~see.view(1, b, nq, 1, prefix), float("-inf"))
    # every sequence's own keys, padded to the longest
    tail = st["table"][:, prefix // bs:]
    size = tail.shape[1] * bs
    sk, sv = (_values(c["kv"], st[n][tail.clamp_min(0)], bs).transpose(1, 2).reshape(b, hkv, size, D) for n in "kv")
    qs = q.transpose(0, 1).reshape(b, hkv, nq * group, D)
    zs = torch.matmul(qs, sk.transpose(2, 3)).view(b, hkv, nq, group, size) * SCALE
    at = torch.arange(prefix, prefix + size, device=dev)
    see = (at >= low.unsqueeze(-1)) & (at <= high.unsqueeze(-1))
    zs = zs.masked_fill(~see.view(b, 1, nq, 1, size), float("-inf")).transpose(0, 1)   # [Hkv][B][nq][G][S]
    top = torch.maximum(zp.amax(-1, keepdim=True), zs.amax(-1, keepdim=True))
    ep, es = torch.exp(zp - top), torch.exp(zs - top)
    total = ep.sum(-1, keepdim=True) + es.sum(-1, keepdim=True)
    out = torch.matmul(ep.view(hkv, -1, prefix), pv).view(hkv, b, nq, group, D)
    out = out + torch.matmul(es.transpose(0, 1).reshape(b, hkv, nq * group, size), sv).view(
        b, hkv, nq, group, D).transpose(0, 1)
    return (out / total).permute(1, 2, 0, 3, 4).reshape(b, nq, hq, D).half()


def _plain_copy(st, src, dst):
    st["k"][dst] = st["k"][src]
    st["v"][dst] = st["v"][src]


def _plain_fork(st):
    bs, table, lens, refs = st["case"]["block"], st["table"], st["lens"], st["refs"]
    parents, children = st["parents"].long(), st["children"].long()
    held = (lens[parents] + bs - 1) // bs
    cols = torch.arange(table.shape[1], device=table.device)
    take = cols < held.unsqueeze(1)
    rows = table[parents]
    table[children] = torch.where(take, rows, table[children])
    refs.index_add_(0, rows.clamp_min(0).reshape(-1), take.reshape(-1).int())
    lens[children] = lens[parents]


def _plain_resize(st, rows, new):
    """Rows set to new lengths.  Fresh pages are the lowest free ones, in the order of the requests; a ragged last page
    that others hold too is copied before it is written, but its last holder in the order keeps it."""
    bs, table, lens, refs = st["case"]["block"], st["table"], st["lens"], st["refs"]
    rows, n, dev = rows.long(), len(rows), table.device
    old, index = lens[rows], torch.arange(n, device=dev)
    have, want = (old + bs - 1) // bs, (new + bs - 1) // bs
    page = table[rows, (old // bs).clamp_max(table.shape[1] - 1).long()].clamp_min(0).long()
    ragged = (new > old) & (old % bs != 0)
    holders = torch.zeros_like(refs).index_add_(0, page, ragged.int())
    last = torch.full_like(refs, -1).scatter_reduce_(0, page, torch.where(ragged, index, -1).int(), "amax")
    keeps = (holders[page] == refs[page]) & (last[page] == index)
    split = ragged & (refs[page] > 1) & ~keeps
    need = (want - have).clamp_min(0) + split.int()
    start = torch.cumsum(need, 0) - need
    free = torch.argsort((refs != 0).int(), stable=True)
    fresh = free[start.clamp_max(len(free) - 1)].int()
    src, dst = torch.where(split, page.int(), -1), torch.where(split, fresh, -1)
    cols = torch.arange(table.shape[1], device=dev)
    mine = table[rows]
    added = (cols >= have.unsqueeze(1)) & (cols < want.unsqueeze(1))
    dropped = (cols >= want.unsqueeze(1)) & (cols < have.unsqueeze(1))
    which = (start + split.int() - have).unsqueeze(1) + cols
    new_pages = free[which.clamp(0, len(free) - 1)].int()
    refs.index_add_(0, mine.clamp_min(0).reshape(-1), -dropped.reshape(-1).int())
    refs.index_add_(0, page, -split.int())
    refs.index_add_(0, fresh.long(), split.int())
    refs.index_add_(0, new_pages.reshape(-1).long(), added.reshape(-1).int())
    mine = torch.where(added, new_pages, mine)
    table[rows] = torch.where(split.unsqueeze(1) & (cols == (old // bs).unsqueeze(1)), fresh.unsqueeze(1), mine)
    lens[rows] = new
    return src, dst


def _plain_compact(st):
    bs, table, lens, refs = st["case"]["block"], st["table"], st["lens"], st["refs"]
    n, dev = len(refs), refs.device
    index, live = torch.arange(n, device=dev), refs > 0
    count = live.sum()
    gaps = torch.nonzero(~live & (index < count)).view(-1)
    tail = torch.nonzero(live & (index >= count)).view(-1)
    remap = torch.where(live, index, -1).int()
    remap[tail] = gaps.int()
    room = max(1, n // 2)
    src, dst = (torch.full((room,), -1, dtype=torch.int32, device=dev) for _ in range(2))
    src[:len(tail)] = tail.int()
    dst[:len(gaps)] = gaps.int()
    refs[gaps] = refs[tail]
    refs[tail] = 0
    held = ((lens + bs - 1) // bs).unsqueeze(1)
    cols = torch.arange(table.shape[1], device=dev)
    table.copy_(torch.where(cols < held, remap[table.clamp_min(0).long()], table))
    return tail, gaps, src, dst, torch.full((1,), len(tail), dtype=torch.int32, device=dev), remap


def _bits(cache):
    """A cache that was moved, not computed: its bits, as whole numbers."""
    return cache.view(torch.int16) if cache.dtype == torch.float16 else cache


def run(state):
    op = state["case"]["op"]
    if op == "attend":
        if own:
            return state["decode"](state["q"], state["k"], state["v"], state["table"], state["lens"],
                                   state["prefix_table"], state["prefix_len"], causal=state["case"]["causal"],
                                   window=state["case"]["window"], scale=SCALE, kv_dtype=KV[state["case"]["kv"]])
        return _plain_attend(state)
    kind = KV[state["case"]["kv"]]
    if op == "copy":
        if own:
            state["pool"].copy(state["k"], state["v"], state["src"], state["dst"], kv_dtype=kind)
        else:
            _plain_copy(state, state["src"], state["dst"])
        return dict(k=_bits(state["k"]), v=_bits(state["v"]))
    if op == "fork":
        # a round of parallel sampling: the last round's answers dropped, every prompt forked, all rows grown for their
        # new tokens, the pages that they would write in common copied
        if own:
            pool = state["pool"]
            pool.resize(state["rows"], state["base"])
            pool.fork(state["parents"], state["children"])
            src, dst = pool.resize(state["rows"], state["grown"])
            pool.copy(state["k"], state["v"], src, dst, kv_dtype=kind)
        else:
            _plain_resize(state, state["rows"], state["base"])
            _plain_fork(state)
            src, dst = _plain_resize(state, state["rows"], state["grown"])
            some = torch.nonzero(src >= 0).view(-1)
            _plain_copy(state, src[some], dst[some])
        return dict(table=state["table"], lens=state["lens"], refs=state["refs"], src=src, dst=dst,
                    k=_bits(state["k"]), v=_bits(state["v"]))
    state["meta"].copy_(state["meta0"])
    if own:
        moved = state["pool"].compact()
        state["pool"].copy(state["k"], state["v"], moved.src, moved.dst, kv_dtype=kind, count=moved.count)
        src, dst, count, remap = moved.src, moved.dst, moved.count, moved.remap
    else:
        tail, gaps, src, dst, count, remap = _plain_compact(state)
        _plain_copy(state, tail, gaps)
    return dict(table=state["table"], lens=state["lens"], refs=state["refs"], src=src, dst=dst, count=count, remap=remap,
                k=_bits(state["k"]), v=_bits(state["v"]))


# ------------------------------------------------------------------ the definition in 64 bits
def _rows64(kv, tiles, bs):
    """Tiles [n][tile] of one KV head as 64-bit rows [n * bs][128]."""
    if kv == "fp16":
        return tiles.reshape(-1, D).double()
    q = tiles[:, :bs * D].contiguous().view(torch.int8).reshape(-1, D).double()
    raw = tiles[:, bs * D:].contiguous()
    if kv == "q8_0":
        return q * raw.view(torch.float16).reshape(-1, 4).double().repeat_interleave(32, dim=1)
    return q * raw.view(torch.float32).reshape(-1, 1).double()


def exact(case, seed):
    if case["op"] != "attend":
        return None  # pages are moved and counted: nothing is computed in floating point
    st = _inputs(case, seed)
    q, nq, bs = st["q"].double(), case["n_query"], case["block"]
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros_like(q)
    for s, length in enumerate(_lengths(case)):
        pages = st["table"][s, :-(-length // bs)].long()
        for h in range(case["kv_heads"]):
            k = _rows64(case["kv"], st["k"][pages, h], bs)[:length]
            v = _rows64(case["kv"], st["v"][pages, h], bs)[:length]
            for i in range(nq):
                last = length - nq + i if case["causal"] else length - 1
                first = max(0, last - case["window"] + 1) if case["window"] else 0
                z = SCALE * (q[s, i, h * group:(h + 1) * group] @ k[first:last + 1].T)
                w = torch.exp(z - z.max(dim=1, keepdim=True).values)
                out[s, i, h * group:(h + 1) * group] = (w @ v[first:last + 1]) / w.sum(dim=1, keepdim=True)
    return out


if __name__ == "__main__":
    for shown in listed() + [draw(random.Random(n)) for n in range(8)]:
        print(shown, work(shown))
