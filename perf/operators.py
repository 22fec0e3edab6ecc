"""The paged 4-bit cache's operators as they are measured: what each case is, its inputs, and one pass through it.

``own`` false: every operator in elementary torch operations, on the documented bytes of the cache (pages of 64
positions, each KV head's block in the tile format of include/hyq.h).  ``own`` true: the calls a user makes.

Operators (``case["op"]``):

  append   rows of new keys and values, quantised into their sequences' pages (and the key bounds of those pages)
  attend   attention of the last n_q tokens of every sequence over all of its positions, causal
  sparse   the same over the k blocks that the key bounds score highest for each token and KV head: the selection,
           then the attention
  branch   one step of sampling several continuations of shared prompts: the last step's branches are freed, the
           parents forked again, and room for one token reserved in each branch (shared last pages are copied)
  compact  the pages in use moved to the front of the pool
"""
import math

import torch

own = False

D, G, ROWS = 128, 4, 64          # head_dim, quantisation groups of 32, positions per page
EMIN = -40                       # smallest exponent of a bound or query step
REC = 272                        # bytes of a bound record: lo[128], hi[128], exponent int32, 12 unused


# --- cases ---------------------------------------------------------------------------------------------------------

def _case(name, op, **kw):
    c = {"name": name, "op": op, "hq": 32, "hkv": 8, "bits_k": 4, "bits_v": 4}
    c.update(kw)
    return c


def listed():
    return [
        # every running request appends its newest token
        _case("append 64 x 1", "append", batch=64, rows=1, length=2000, hats=False),
        # a batch of prompts of unlike lengths behind a shared start, with the rows read back for the prompt's own pass
        _case("append prompts 8 x 8192", "append", batch=8, rows=8192, length=1000, hats=True),
        # one short chat, the smallest call
        _case("attend 1 x 1000", "attend", batch=1, n_q=1, length=1000),
        # one long document
        _case("attend 1 x 32768", "attend", batch=1, n_q=1, length=32768),
        # a full server: many requests of unlike lengths
        _case("attend 64 x 32768", "attend", batch=64, n_q=1, length=32768),
        # four drafted tokens are verified at once, wide GQA groups, 8-bit codes
        _case("attend drafts 8 x 16001", "attend", batch=8, n_q=4, length=16001, hq=64, bits_k=8, bits_v=8),
        # one long document, an eighth of it read
        _case("sparse 1 x 32768", "sparse", batch=1, n_q=1, length=32768, blocks=64),
        # long contexts served together, two tokens a sequence
        _case("sparse 16 x 65536", "sparse", batch=16, n_q=2, length=65536, blocks=128),
        # two branches of four short prompts in a small model
        _case("branch 4 x 2", "branch", parents=4, children=2, length=300, layers=2, hkv=4, hq=4),
        # eight samples for each of eight prompts, a model of 32 layers
        _case("branch 8 x 8", "branch", parents=8, children=8, length=2000, layers=32),
        # a small pool
        _case("compact 96", "compact", pages=96, live=0.5, seqs=6, layers=2),
        # a large one, after many requests have come and gone
        _case("compact 1024", "compact", pages=1024, live=0.6, seqs=40, layers=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "sparse", "sparse", "branch", "compact"])
    hq, hkv = rng.choice([(4, 4), (8, 2), (10, 2), (32, 8), (32, 8), (64, 8), (14, 2)])
    bits = rng.choice([(4, 4), (4, 4), (4, 4), (8, 8), (8, 4), (4, 8)])
    c = {"op": op, "hq": hq, "hkv": hkv, "bits_k": bits[0], "bits_v": bits[1]}
    if op == "append":
        if rng.random() < 0.5:
            c.update(batch=_log(rng, 1, 128), rows=1, length=_log(rng, 1, 2500), hats=False)
        else:
            b = _log(rng, 1, 16)
            c.update(batch=b, rows=_log(rng, 2, 30000 // b), length=_log(rng, 1, 2500), hats=rng.random() < 0.5)
    elif op == "attend":
        b = _log(rng, 1, 64)
        c.update(batch=b, n_q=rng.choice([1, 1, 1, 2, 3, 5]), length=_log(rng, 20, min(131072, 700000 // b)))
    elif op == "sparse":
        b = _log(rng, 1, 32)
        c.update(batch=b, n_q=rng.choice([1, 1, 2, 3]), length=_log(rng, 500, min(131072, 700000 // b)),
                 blocks=_log(rng, 4, 128))
    elif op == "branch":
        c.update(parents=_log(rng, 1, 8), children=_log(rng, 1, 8), length=_log(rng, 30, 2000), layers=_log(rng, 1, 32))
    else:
        c.update(pages=_log(rng, 40, 1000), live=round(rng.uniform(0.2, 0.9), 3), seqs=_log(rng, 2, 40),
                 layers=_log(rng, 1, 32))
    return c


def _spread(n, top, low=0.25):
    """n lengths between low * top and top, unlike one another, the first one top."""
    return [top if i == 0 else max(1, int(top * (1 - (1 - low) * math.modf(i * 0.6180339887498949)[0]))) for i in range(n)]


def _lens(case):
    """(positions present before the call, new rows) of every row of the call, for append; (length, None) else."""
    n = case["batch"]
    lens = _spread(n, case["length"])
    if case["op"] != "append":
        if n >= 8:
            lens[1] = 1           # a request that has just begun: with n_q > 1 its first tokens see nothing
        return lens, None
    rows = [1] * n if case["rows"] == 1 else _spread(n, case["rows"], 0.05)
    if case["rows"] > 1 and n >= 4:
        rows[2] = 0               # a request that brings nothing this time
    if n >= 2:
        lens[1] = 0               # a new request: its first page is begun by this call
    return lens, rows


def _blocks(n):
    return -(-n // ROWS)


def _tile(case):
    return 256 * (case["bits_k"] + case["bits_v"]) + 512


def work(case):
    op, hkv, hq, tile = case["op"], case["hkv"], case["hq"], _tile(case)
    row = tile / 16               # bytes of one position of one KV head
    if op == "append":
        start, rows = _lens(case)
        n = sum(rows) * hkv
        touched = sum(_blocks(s + r) - s // ROWS for s, r in zip(start, rows) if r)
        again = sum(1 for s, r in zip(start, rows) if r and s % ROWS)
        return {"bytes": n * (2 * D * 2 + row + (2 * D * 2 if case["hats"] else 0)) + (touched + again) * hkv * 260,
                "flops": n * 2 * D * 6}
    if op == "attend":
        lens, _ = _lens(case)
        seen = sum(max(0, n - case["n_q"] + 1 + i) for n in lens for i in range(case["n_q"]))
        return {"bytes": sum(lens) * hkv * row + case["batch"] * case["n_q"] * hq * D * 4, "flops": 4 * D * hq * seen}
    if op == "sparse":
        lens, _ = _lens(case)
        score = take = pages = 0
        for n in lens:
            score += _blocks(n)
            for i in range(case["n_q"]):
                lim = max(0, n - case["n_q"] + 1 + i)
                take += min(_blocks(lim), case["blocks"]) * ROWS if lim >= ROWS * case["blocks"] else lim
            pages += min(n, case["blocks"] * ROWS)       # one token's choice at least has to be read
        return {"bytes": score * hkv * 260 + pages * hkv * row + case["batch"] * case["n_q"] * (hq * D * 4 + hkv * case["blocks"] * 4),
                "flops": 4 * D * hq * take + 2 * 2 * D * hkv * score * case["n_q"]}
    if op == "branch":
        lens = _spread(case["parents"], case["length"])
        tiles = sum(-(-(n % ROWS) // 16) for n in lens) * case["children"]
        cow = sum(1 for n in lens if n % ROWS) * case["children"]
        tables = sum(_blocks(n) for n in lens) * case["children"]
        return {"bytes": 2 * case["layers"] * hkv * (tiles * tile + cow * 260) + tables * 4 * 6 + _branch_pages(case) * 4, "flops": 0}
    n, live = case["pages"], _live(case)
    moves = _moves(case)
    return {"bytes": 2 * case["layers"] * hkv * moves * (4 * tile + 260) + 8 * n + 8 * live, "flops": 0}


# --- the cache's bytes ---------------------------------------------------------------------------------------------

_MAPS = {}


def _map(kind, bits, device):
    """Index of the code of (row, element) = (i // 128, i % 128) among the slots of a tile's code region, and the inverse
    (slot -> 128 row + element).  Slots are the nibbles (low first) or the bytes of the region, in order."""
    key = (kind, bits, str(device))
    if key not in _MAPS:
        s = torch.arange(2048)
        if bits == 4:
            word, n = s // 8, s % 8
            a, b, c = n & 1, (n >> 1) & 1, n >> 2
            u = 4 * (word // 128) + word % 4
            lane = (word // 4) % 32
            g, t = lane // 4, lane % 4
            if kind == "k":
                row, el = g + 8 * a, 8 * (t + 4 * (u // 2)) + 4 * (u % 2) + 2 * b + c
            else:
                row, el = 2 * t + 8 * b + c, 32 * (u // 2) + 4 * g + 2 * (u % 2) + a
        else:
            word, j = s // 4, s % 4
            u = 4 * (word // 128) + word % 4
            lane = (word // 4) % 32
            g, t = lane // 4, lane % 4
            if kind == "k":
                row, el = g + 8 * (u % 2), 16 * (u // 2) + 4 * t + torch.tensor([0, 2, 1, 3])[j]
            else:
                row, el = 2 * t + torch.tensor([0, 8, 1, 9])[j], 32 * (u // 4) + 4 * g + 2 * ((u // 2) % 2) + u % 2
        src = row * D + el                       # slot -> element
        inv = torch.empty_like(src)
        inv[src] = s                             # element -> slot
        _MAPS[key] = (inv.to(device), src.to(device))
    return _MAPS[key]


def _codes(tiles, kind, bits, off):
    """Codes uint8 [..., 16, 128] of the region at byte ``off`` of tiles uint8 [..., tile bytes]."""
    reg = tiles[..., off:off + 256 * bits]
    if bits == 4:
        reg = torch.stack([reg & 15, reg >> 4], -1).flatten(-2)
    inv, _ = _map(kind, bits, tiles.device)
    return reg[..., inv].unflatten(-1, (16, D))


def _region(codes, kind, bits):
    """The inverse: bytes [..., 256 bits] of codes [..., 16, 128]."""
    _, src = _map(kind, bits, codes.device)
    s = codes.flatten(-2)[..., src]
    return s if bits == 8 else s[..., 0::2] | (s[..., 1::2] << 4)


def _meta(tiles, kind, off):
    """FP16 step and zero [..., 16, 4] of the 256-byte region at ``off``."""
    h = tiles[..., off:off + 256].contiguous().view(torch.float16)
    if kind == "k":
        h = h.unflatten(-1, (16, 2, G))
        return h[..., 0, :], h[..., 1, :]
    h = h.unflatten(-1, (2, 8, G, 2)).transpose(-1, -2)          # scales | zeros, row pair, row in the pair, group
    return h[..., 0, :, :, :].flatten(-3, -2), h[..., 1, :, :, :].flatten(-3, -2)


def _meta_bytes(s, z, kind):
    if kind == "k":
        h = torch.stack([s, z], -2)
    else:
        h = torch.stack([s.unflatten(-2, (8, 2)), z.unflatten(-2, (8, 2))], -4).transpose(-1, -2)
    return h.flatten(-3 if kind == "k" else -4).contiguous().view(torch.uint8)


def _unpack(blocks, bk, bv):
    """Keys and values float32 [..., 64, 128] of page blocks uint8 [..., block bytes]."""
    t = blocks.unflatten(-1, (4, -1))
    ck, cv = 256 * bk, 256 * bv
    out = []
    for kind, bits, co, mo in (("k", bk, 0, ck + cv), ("v", bv, ck, ck + cv + 256)):
        c = _codes(t, kind, bits, co).float().unflatten(-1, (G, 32))
        s, z = _meta(t, kind, mo)
        out.append((c * s.float()[..., None] + z.float()[..., None]).flatten(-2).flatten(-3, -2))
    return out


def _pack(kc, ks, kz, vc, vs, vz, bk, bv):
    """Page blocks uint8 [..., block bytes] of codes [..., 64, 128] and metadata [..., 64, 4]."""
    f = lambda x: x.unflatten(-2, (4, 16))  # noqa: E731
    parts = [_region(f(kc), "k", bk), _region(f(vc), "v", bv), _meta_bytes(f(ks), f(kz), "k"), _meta_bytes(f(vs), f(vz), "v")]
    return torch.cat(parts, -1).flatten(-2)


def _quantise(x, bits):
    """Codes uint8, step and zero FP16 of rows [..., 128]: the smallest FP16 step s with qmax s >= max - min of a group of
    32, the zero min in FP16, the code nearest to (x - z) / s with ties to the even one, decided exactly."""
    qmax = float((1 << bits) - 1)
    g = x.unflatten(-1, (G, 32)).double()
    mn, mx = g.amin(-1), g.amax(-1)
    d = mx - mn
    b = (d / qmax).to(torch.float16).view(torch.int16)
    val = lambda i: i.view(torch.float16).double()  # noqa: E731
    lo = (b - 1).clamp_min(0)
    s = torch.where(val(lo) * qmax >= d, lo, torch.where(val(b) * qmax >= d, b, b + 1)).view(torch.float16)
    z = mn.float().to(torch.float16)
    sd, zd = s.double()[..., None], z.double()[..., None]
    live = sd > 0
    c = torch.where(live, torch.round((g - zd) / torch.where(live, sd, 1.0)).clamp(0, qmax), 0.0)
    for step in (1.0, -1.0):                                     # the sign of x minus a midpoint is exact
        dist = (g - (zd + (c + 0.5 * step) * sd)) * step
        move = live & (c + step >= 0) & (c + step <= qmax) & ((dist > 0) | ((dist == 0) & (c % 2 == 1)))
        c = torch.where(move, c + step, c)
    return c.to(torch.uint8).flatten(-2), s, z


def _step_exp(amax):
    """Smallest integer e >= -40 with amax <= 127 * 2^e."""
    m, x = torch.frexp(amax.double())
    return torch.where(amax > 0, x - 7 + (m > 127 / 128), torch.full_like(x, EMIN)).clamp_min(EMIN).to(torch.int32)


def _bounds(k, valid, old=None, merge=None):
    """Bound records uint8 [..., 272] of keys [..., 64, 128] with rows ``valid`` [..., 64]; where ``merge``, joined with the
    record ``old``."""
    v = valid[..., None]
    k = k.double()
    mn = torch.where(v, k, math.inf).amin(-2)
    mx = torch.where(v, k, -math.inf).amax(-2)
    e = _step_exp(torch.where(v, k.abs(), 0.0).amax((-2, -1)))
    if old is not None:
        oe = old[..., 256:260].contiguous().view(torch.int32)[..., 0]
        ol, oh = old[..., :D].view(torch.int8).double(), old[..., D:2 * D].view(torch.int8).double()
        p = torch.exp2(oe.double())[..., None]
        m = merge[..., None]
        mn, mx = torch.where(m, torch.minimum(mn, ol * p), mn), torch.where(m, torch.maximum(mx, oh * p), mx)
        e = torch.where(merge, torch.maximum(e, oe), e)
    inv = torch.exp2(-e.double())[..., None]
    rec = [torch.floor(mn * inv).to(torch.int8).view(torch.uint8), torch.ceil(mx * inv).to(torch.int8).view(torch.uint8),
           e[..., None].contiguous().view(torch.uint8), torch.zeros(e.shape + (12,), dtype=torch.uint8, device=k.device)]
    return torch.cat(rec, -1)


# --- inputs --------------------------------------------------------------------------------------------------------

def _rows_like_keys(shape, u, gen, dev):
    """Keys as a model's: a few channels of large values, and 2% of positions that every query looks at.
    shape [..., HKV, 64 or any, 128] with u [HKV, 1, 128]."""
    k = torch.randn(shape, generator=gen, device=dev)
    k[..., [5, 64, 101]] *= 8
    sink = torch.rand(shape[:-1] + (1,), generator=gen, device=dev) < 0.02
    return torch.where(sink, k + 4 * u, k).to(torch.bfloat16)


def _fill(pool, bounds, pages, rows, case, u, gen, with_bounds):
    """Random content of the listed pages of layer 0, their first ``rows`` positions filled."""
    hkv, dev = case["hkv"], pool.device
    step = max(1, 4096 // hkv)
    for at in range(0, len(pages), step):
        p = pages[at:at + step]
        k = _rows_like_keys((len(p), hkv, ROWS, D), u, gen, dev)
        v = torch.randn(len(p), hkv, ROWS, D, generator=gen, device=dev).to(torch.bfloat16)
        pool[0, p] = _pack(*_quantise(k, case["bits_k"]), *_quantise(v, case["bits_v"]), case["bits_k"], case["bits_v"])
        if with_bounds:
            valid = (torch.arange(ROWS, device=dev) < rows[at:at + step, None])[:, None].expand(-1, hkv, -1)
            bounds[0, p] = _bounds(k, valid)


def _tables(lens, gen, dev, spare):
    """A table that gives every sequence pages of its own at random places of the pool."""
    need = [_blocks(n) for n in lens]
    total, width = sum(need), max(max(need), 1)
    n_pages = total + spare
    perm = torch.randperm(n_pages, generator=gen, device=dev)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(need))
    first = torch.tensor([0] + need).cumsum(0)[:-1]
    blk = torch.arange(total) - first[seq]
    table = table.to(dev)
    table[seq.to(dev), blk.to(dev)] = perm[:total].to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[perm[:total]] = 1
    return table, refs, seq.to(dev), blk.to(dev), perm[:total]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    if case["op"] in ("branch", "compact"):
        return (_prepare_branch if case["op"] == "branch" else _prepare_compact)(case, gen, dev)
    hq, hkv, n = case["hq"], case["hkv"], case["batch"]
    lens, rows = _lens(case)
    total = [a + b for a, b in zip(lens, rows)] if rows else lens
    table, refs, seq, blk, pages = _tables(total, gen, dev, max(4, sum(map(_blocks, total)) // 10))
    size = 4 * _tile(case)
    pool = torch.zeros(1, len(refs), hkv, size, dtype=torch.uint8, device=dev)
    bounds = torch.zeros(1, len(refs), hkv, REC, dtype=torch.uint8, device=dev)
    u = torch.randn(hkv, 1, D, generator=gen, device=dev)
    u /= u.norm(dim=-1, keepdim=True)
    st = {"case": case, "pool": pool, "bounds": bounds, "table": table, "refs": refs,
          "lens": torch.tensor(total, dtype=torch.int32, device=dev)}
    before = torch.tensor(lens, device=dev)
    filled = (before[seq] - blk * ROWS).clamp(0, ROWS)
    # a call lists its sequences in an order of its own
    order = torch.randperm(n, generator=gen, device=dev)
    st["seqs"] = order.to(torch.int32)
    if rows:
        part = (filled > 0) & (filled < ROWS)
        _fill(pool, bounds, pages[part], filled[part], case, u, gen, True)
        cnt = torch.tensor(rows)[order.cpu()]
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), cnt.cumsum(0)])
        t = int(cu[-1])
        k = torch.empty(t, hkv, D, dtype=torch.bfloat16, device=dev)
        for at in range(0, t, 16384):
            k[at:at + 16384] = _rows_like_keys((hkv, min(16384, t - at), D), u, gen, dev).transpose(0, 1)
        v = torch.randn(t, hkv, D, generator=gen, device=dev).to(torch.bfloat16)
        st.update(k=k, v=v, cu=None if case["rows"] == 1 else cu.to(torch.int32).to(dev),
                  k_hat=torch.empty_like(k) if case["hats"] else None, v_hat=torch.empty_like(v) if case["hats"] else None)
        return st
    _fill(pool, bounds, pages, filled, case, u, gen, case["op"] == "sparse")
    q = torch.randn(n, case["n_q"], hkv, hq // hkv, D, generator=gen, device=dev) + 2 * u
    st["q"] = q.to(torch.bfloat16).view(n, case["n_q"], hq, D)
    st["out"] = torch.empty_like(st["q"])
    if case["op"] == "sparse":
        st["sel"] = torch.empty(n, case["n_q"], hkv, case["blocks"], dtype=torch.int32, device=dev)
    return st


def _branch_pages(case):
    lens = _spread(case["parents"], case["length"])
    return sum(_blocks(n) for n in lens) + 2 * len(lens) * case["children"] + 8


def _prepare_branch(case, gen, dev):
    """The state after one such step: every branch holds its parent's pages, and a last page of its own."""
    p, f, hkv = case["parents"], case["children"], case["hkv"]
    lens = _spread(p, case["length"])
    n_pages, width = _branch_pages(case), _blocks(case["length"]) + 1
    perm = torch.randperm(n_pages, generator=gen, device=dev).cpu().tolist()
    table = torch.full((p + p * f, width), -1, dtype=torch.int32)
    refs = [0] * n_pages
    take = iter(perm)
    for i, n in enumerate(lens):
        ids = [next(take) for _ in range(_blocks(n))]
        table[i, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        for x in ids[:n // ROWS]:
            refs[x] += 1 + f
        for x in ids[n // ROWS:]:
            refs[x] += 1
    for j in range(p * f):
        n = lens[j // f]
        table[p + j] = table[j // f]
        x = next(take)
        table[p + j, n // ROWS] = x
        refs[x] += 1
    pool = torch.randint(0, 256, (case["layers"], n_pages, hkv, 4 * _tile(case)), generator=gen, device=dev, dtype=torch.uint8)
    bounds = torch.randint(0, 256, (case["layers"], n_pages, hkv, REC), generator=gen, device=dev, dtype=torch.uint8)
    dst = torch.arange(p, p + p * f, dtype=torch.int32, device=dev)
    return {"case": case, "pool": pool, "bounds": bounds, "table": table.to(dev), "refs": torch.tensor(refs, dtype=torch.int32, device=dev),
            "lens": torch.tensor(lens + [lens[j // f] + 1 for j in range(p * f)], dtype=torch.int32, device=dev),
            "src": (torch.arange(p * f, device=dev) // f).to(torch.int32), "dst": dst}


def _live(case):
    return max(1, min(case["pages"], round(case["pages"] * case["live"])))


def _moves(case):
    n, live = case["pages"], _live(case)
    return min(live, n - live, round(live * (n - live) / n))


def _prepare_compact(case, gen, dev):
    """A pool in which ``live`` of the pages are held, scattered; every eighth of a sequence's pages is shared with the next one."""
    n, live, moves, hkv = case["pages"], _live(case), _moves(case), case["hkv"]
    front = torch.randperm(live, generator=gen, device=dev)[:live - moves]
    back = live + torch.randperm(n - live, generator=gen, device=dev)[:moves]
    ids = torch.cat([front, back])[torch.randperm(live, generator=gen, device=dev)].cpu()
    s = min(case["seqs"], live)
    per = [len(range(i, live, s)) for i in range(s)]
    own_ids = [ids[i::s] for i in range(s)]
    rows = [torch.cat([own_ids[i], own_ids[(i + 1) % s][::8]]) if s > 1 else own_ids[i] for i in range(s)]
    table = torch.full((s, max(map(len, rows))), -1, dtype=torch.int32)
    refs = torch.zeros(n, dtype=torch.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r.to(torch.int32)
        refs.index_add_(0, r, torch.ones(len(r), dtype=torch.int32))
    assert sum(per) == live
    pool = torch.randint(0, 256, (case["layers"], n, hkv, 4 * _tile(case)), generator=gen, device=dev, dtype=torch.uint8)
    bounds = torch.randint(0, 256, (case["layers"], n, hkv, REC), generator=gen, device=dev, dtype=torch.uint8)
    table = table.to(dev)
    return {"case": case, "pool": pool, "bounds": bounds, "table": table, "refs": refs.to(dev),
            "lens": torch.tensor([len(r) * ROWS - (7 * i) % ROWS for i, r in enumerate(rows)], dtype=torch.int32, device=dev),
            "table_out": torch.empty_like(table), "refs_out": torch.empty(n, dtype=torch.int32, device=dev)}


# --- one pass ------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"append": _append, "attend": _attend, "sparse": _sparse, "branch": _branch, "compact": _compact}[st["case"]["op"]](st)


def _cache(st):
    """The handle that a program makes once for its pool."""
    if "cache" not in st:
        import hybrid_precision_quantized_gb300 as hyq
        c = st["case"]
        cfg = hyq.make_config(1, c["hq"], c["hkv"], capacity=ROWS, bits_k=c["bits_k"], bits_v=c["bits_v"])
        st["cache"] = hyq.PagedCache(cfg, n_pages=st["pool"].shape[1], n_seqs=st["table"].shape[0], max_blocks=st["table"].shape[1],
                                     n_layers=st["pool"].shape[0], device=st["pool"].device,
                                     buffers={k: st[k] for k in ("pool", "bounds", "table", "lens", "refs")})
    return st["cache"]


def _own(st):
    c, cache = st["case"], _cache(st)
    if c["op"] == "append":
        cache.append(0, st["k"], st["v"], seqs=st["seqs"], cu_rows=st["cu"], k_hat=st["k_hat"], v_hat=st["v_hat"])
        return _append_outputs(st)
    if c["op"] == "attend":
        cache.attention(0, st["q"], st["out"], seqs=st["seqs"])
        return {"out": st["out"]}
    if c["op"] == "sparse":
        cache.select(0, st["q"], st["sel"], seqs=st["seqs"], n_first=1, n_last=2)
        cache.attention_blocks(0, st["q"], st["sel"], st["out"], seqs=st["seqs"])
        return {"out": st["out"], "sel": st["sel"]}
    if c["op"] == "branch":
        cache.truncate(st["dst"])
        cache.fork(st["src"], st["dst"])
        cache.reserve(st["dst"])
        return {k: st[k] for k in ("pool", "bounds", "table", "lens", "refs")}
    cache.compact(st["table_out"], st["refs_out"])
    return {k: st[k] for k in ("pool", "bounds", "table_out", "refs_out")}


def _append_outputs(st):
    out = {"pool": st["pool"], "bounds": st["bounds"]}
    if st["k_hat"] is not None:
        out.update(k_hat=st["k_hat"], v_hat=st["v_hat"])
    return out


def _append(st):
    c, dev = st["case"], st["pool"].device
    bk, bv = c["bits_k"], c["bits_v"]
    seqs, t, b = st["seqs"].long(), st["k"].shape[0], st["seqs"].shape[0]
    cu = st["cu"].long() if st["cu"] is not None else torch.arange(b + 1, device=dev)
    rows, end = cu[1:] - cu[:-1], st["lens"].long()[seqs]
    start = end - rows
    # the pages that get rows: one slot each, the last one again in the slots that are left over
    first = start // ROWS
    count = torch.where(rows > 0, (end - 1) // ROWS - first + 1, 0)
    upto = count.cumsum(0)
    slot = torch.minimum(torch.arange(t // ROWS + 2 * min(b, t), device=dev), upto[-1] - 1)
    i = torch.searchsorted(upto, slot, right=True)
    blk = first[i] + slot - (upto - count)[i]
    page = st["table"].long()[seqs[i], blk]
    pos = blk[:, None] * ROWS + torch.arange(ROWS, device=dev)
    new = (pos >= start[i][:, None]) & (pos < end[i][:, None])
    tok = torch.where(new, cu[i][:, None] + pos - start[i][:, None], 0)
    k, v = (x[tok].transpose(1, 2) for x in (st["k"], st["v"]))                   # [slots, HKV, 64, 128]
    (kc, ks, kz), (vc, vs, vz) = _quantise(k, bk), _quantise(v, bv)
    old = st["pool"][0, page]
    tiles = old.unflatten(-1, (4, -1))
    ck, cv = 256 * bk, 256 * bv
    m = new[:, None, :, None]
    keep = lambda x, y: torch.where(m, x, y)  # noqa: E731
    rows64 = lambda x: x.flatten(-3, -2)  # noqa: E731
    (ok, oz), (pk, pz) = _meta(tiles, "k", ck + cv), _meta(tiles, "v", ck + cv + 256)
    h16 = lambda x, y: keep(x.view(torch.int16), rows64(y).contiguous().view(torch.int16)).view(torch.float16)  # noqa: E731
    st["pool"][0, page] = _pack(keep(kc, rows64(_codes(tiles, "k", bk, 0))), h16(ks, ok), h16(kz, oz),
                                keep(vc, rows64(_codes(tiles, "v", bv, ck))), h16(vs, pk), h16(vz, pz), bk, bv)
    merge = (start[i] > blk * ROWS)[:, None].expand(-1, c["hkv"])
    st["bounds"][0, page] = _bounds(k, new[:, None].expand(-1, c["hkv"], -1), st["bounds"][0, page], merge)
    if st["k_hat"] is not None:
        for name, x, bits in (("k_hat", st["k"], bk), ("v_hat", st["v"], bv)):
            cc, s, z = _quantise(x, bits)
            st[name].copy_((cc.float().unflatten(-1, (G, 32)) * s.float()[..., None] + z.float()[..., None]).flatten(-2))
    return _append_outputs(st)


def _softmax_v(x, seen, v):
    """softmax of logits x [..., R, L] over the places ``seen`` [..., R, L] times v [..., L, 128]; zeros where none is."""
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    s = p.sum(-1, keepdim=True)
    return torch.where(s > 0, torch.matmul(p, v) / torch.where(s > 0, s, 1.0), 0.0)


def _attend(st):
    c, dev = st["case"], st["pool"].device
    hkv, nq = c["hkv"], c["n_q"]
    g = c["hq"] // hkv
    seqs = st["seqs"].long()
    end, table = st["lens"].long()[seqs], st["table"].long()[seqs].clamp_min(0)
    k, v = _unpack(st["pool"][0, table], c["bits_k"], c["bits_v"])               # [B, blocks, HKV, 64, 128]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))                     # [B, HKV, L, 128]
    q = st["q"].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, HKV, n_q g, 128]
    lim = end[:, None] - nq + 1 + torch.arange(nq, device=dev)                   # positions that a token sees
    seen = torch.arange(k.shape[2], device=dev) < lim.repeat_interleave(g, 1)[:, None, :, None]
    v = torch.where((torch.arange(k.shape[2], device=dev) < end[:, None])[:, None, :, None], v, 0.0)
    o = _softmax_v(torch.matmul(q, k.transpose(2, 3)) * D ** -0.5, seen, v)
    return {"out": o.unflatten(2, (nq, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(torch.bfloat16)}


def _select(st, n_first=1, n_last=2):
    c, dev = st["case"], st["pool"].device
    hkv, nq, kb = c["hkv"], c["n_q"], c["blocks"]
    seqs = st["seqs"].long()
    table = st["table"].long()[seqs].clamp_min(0)
    rec = st["bounds"][0, table].transpose(1, 2)                                  # [B, HKV, blocks, 272]
    lo, hi = rec[..., :D].view(torch.int8).double(), rec[..., D:2 * D].view(torch.int8).double()
    e = rec[..., 256:260].contiguous().view(torch.int32)[..., 0].double()
    q = st["q"].double().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)           # [B, HKV, n_q, g, 128]
    code = torch.round(q * torch.exp2(-_step_exp(q.abs().amax((-2, -1))).double())[..., None, None])
    a, n = code.clamp_min(0).sum(-2), code.clamp_max(0).sum(-2)                   # [B, HKV, n_q, 128]
    score = (torch.matmul(a, hi.transpose(2, 3)) + torch.matmul(n, lo.transpose(2, 3))) * torch.exp2(e)[:, :, None]
    lim = st["lens"].long()[seqs][:, None] - nq + 1 + torch.arange(nq, device=dev)
    nb = ((lim.clamp_min(0) + ROWS - 1) // ROWS)[:, None, :, None]
    j = torch.arange(table.shape[1], device=dev)
    score = torch.where((j < n_first) | (j >= nb - n_last), math.inf, score)
    score = torch.where(j < nb, score, -math.inf)
    at = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :kb]
    at = torch.where(torch.arange(at.shape[-1], device=dev) < nb, at, 1 << 30).sort(-1).values
    sel = torch.full(at.shape[:-1] + (kb,), -1, dtype=torch.int32, device=dev)
    sel[..., :at.shape[-1]] = torch.where(at < 1 << 30, at, -1)
    return sel.transpose(1, 2).contiguous(), lim


def _sparse(st):
    c, dev = st["case"], st["pool"].device
    hkv, nq = c["hkv"], c["n_q"]
    seqs = st["seqs"].long()
    sel, lim = _select(st)                                                        # [B, n_q, HKV, k]
    at = sel.long().clamp_min(0)
    page = torch.gather(st["table"].long()[seqs][:, None, None].expand(-1, nq, hkv, -1), 3, at).clamp_min(0)
    k, v = _unpack(st["pool"][0, page, torch.arange(hkv, device=dev)[:, None]], c["bits_k"], c["bits_v"])
    k, v = k.flatten(3, 4), v.flatten(3, 4)                                       # [B, n_q, HKV, 64 k, 128]
    pos = (at[..., None] * ROWS + torch.arange(ROWS, device=dev)).flatten(3)
    seen = (pos < lim[:, :, None, None]) & (sel >= 0).repeat_interleave(ROWS, 3)
    v = torch.where(seen[..., None], v, 0.0)
    q = st["q"].float().unflatten(2, (hkv, -1))
    o = _softmax_v(torch.matmul(q, k.transpose(3, 4)) * D ** -0.5, seen[..., None, :], v)
    return {"out": o.flatten(2, 3).to(torch.bfloat16), "sel": sel}


def _held(st, seqs):
    """Which entries of the table rows ``seqs`` hold a page, and the pages."""
    nb = (st["lens"].long()[seqs] + ROWS - 1) // ROWS
    held = torch.arange(st["table"].shape[1], device=nb.device) < nb[:, None]
    return held, st["table"].long()[seqs].clamp_min(0)


def _branch(st):
    dev, table, lens, refs = st["pool"].device, st["table"], st["lens"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    held, page = _held(st, dst)                                                   # free the last branches
    refs.index_add_(0, page.flatten(), -held.flatten().to(torch.int32))
    lens[dst] = 0
    held, page = _held(st, src)                                                   # fork the parents
    table[dst] = torch.where(held, table[src], table[dst])
    refs.index_add_(0, page.flatten(), held.flatten().to(torch.int32))
    lens[dst] = lens[src]
    n = lens.long()[dst]                                                          # room for one token in each
    part = n % ROWS
    last = torch.gather(table.long()[dst], 1, ((n - 1) // ROWS).clamp_min(0)[:, None])[:, 0].clamp_min(0)
    cand = (part > 0) & (refs[last] > 1)
    before = ((last[:, None] == last) & cand).tril(-1).sum(1)
    copy = cand & (refs[last] - before > 1)
    new = copy | (part == 0)
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)[:len(dst)]
    to = torch.where(new, free[(new.cumsum(0) - 1).clamp_min(0)], last)
    refs.index_add_(0, last, -copy.to(torch.int32))
    refs.index_add_(0, to, new.to(torch.int32))
    table[dst, n // ROWS] = to.to(torch.int32)
    lens[dst] += 1
    tiles = (torch.arange(4, device=dev) * 16 < part[:, None]) & copy[:, None]    # tiles that hold rows
    pool = st["pool"].unflatten(-1, (4, -1))
    pool[:, to] = torch.where(tiles[:, None, :, None], pool[:, last], pool[:, to])
    st["bounds"][:, to] = torch.where(copy[:, None, None], st["bounds"][:, last], st["bounds"][:, to])
    return {k: st[k] for k in ("pool", "bounds", "table", "lens", "refs")}


def _compact(st):
    dev, refs, table = st["pool"].device, st["refs"], st["table"]
    n = refs.shape[0]
    ids = torch.arange(n, device=dev)
    live = refs > 0
    count = live.sum()
    high, gap = live & (ids >= count), ~live & (ids < count)
    # the r-th live page past the end goes to the r-th gap
    gaps, highs = (torch.argsort((~x).to(torch.int32), stable=True) for x in (gap, high))
    to = torch.where(high, gaps[(high.cumsum(0) - 1).clamp_min(0)], ids)
    came = torch.where(gap, highs[(gap.cumsum(0) - 1).clamp_min(0)], ids)
    held, page = _held(st, torch.arange(table.shape[0], device=dev))
    st["table_out"].copy_(torch.where(held, to[page].to(torch.int32), table))
    st["refs_out"].copy_(torch.where(ids < count, refs[came], 0))
    st["pool"].copy_(st["pool"][:, came])
    st["bounds"].copy_(st["bounds"][:, came])
    return {k: st[k] for k in ("pool", "bounds", "table_out", "refs_out")}


# --- the definitions in 64 bits ------------------------------------------------------------------------------------

def _value(block, r, bits_k, bits_v, kind):
    """Dequantised rows r (tensor of row numbers below 64) of page blocks uint8 [n, block bytes], float64 [n, 128], element by
    element from the tile format."""
    bits = bits_k if kind == "k" else bits_v
    code_at = 0 if kind == "k" else 256 * bits_k
    meta_at = 256 * (bits_k + bits_v) + (0 if kind == "k" else 256)
    e = torch.arange(D, device=block.device)
    base = (r // 16 * (256 * (bits_k + bits_v) + 512))[:, None]
    i, q = (r % 16)[:, None], e // 32
    if kind == "k" and bits == 4:
        g, a, t = i % 8, i // 8, (e // 8) % 4
        u = 2 * (e // 32) + (e // 4) % 2
        byte, high = 4 * (u % 4) + 512 * (u // 4) + 16 * (4 * g + t) + (e // 2) % 2 + 2 * (e % 2), a + 0 * e
    elif kind == "k":
        g, t, u = i % 8, (e // 4) % 4, 2 * (e // 16) + i // 8
        byte = 512 * (u // 4) + 16 * (4 * g + t) + 4 * (u % 4) + (e // 2) % 2 + 2 * (e % 2)
    elif bits == 4:
        t, b, c, g = (i % 8) // 2, i // 8, i % 2, (e // 4) % 8
        u = 2 * (e // 32) + (e // 2) % 2
        byte, high = 512 * (u // 4) + 16 * (4 * g + t) + 4 * (u % 4) + b + 2 * c, e % 2 + 0 * i
    else:
        t, g, j = (i % 8) // 2, (e // 4) % 8, 2 * (i % 2) + i // 8
        u = 4 * (e // 32) + 2 * ((e // 2) % 2) + e % 2
        byte = 512 * (u // 4) + 16 * (4 * g + t) + 4 * (u % 4) + j
    code = torch.gather(block, 1, base + code_at + byte).long()
    if bits == 4:
        code = (code >> (4 * high)) & 15
    s_at = 16 * i + 2 * q if kind == "k" else 16 * (i // 2) + 4 * q + 2 * (i % 2)
    half = block.view(torch.int16) if block.is_contiguous() else block.contiguous().view(torch.int16)
    s = torch.gather(half, 1, (base + meta_at + s_at) // 2).view(torch.float16).double()
    z = torch.gather(half, 1, (base + meta_at + s_at + (8 if kind == "k" else 128)) // 2).view(torch.float16).double()
    return code * s + z


def _group64(x, bits):
    """One tensor of rows in 64 bits: c s + z with the step by search over the FP16 values and the code by comparison of
    the distances to its two neighbours."""
    steps = torch.arange(0x7c00, dtype=torch.int32, device=x.device).to(torch.int16).view(torch.float16).double()
    qmax = (1 << bits) - 1
    out = []
    for part in x.double().unflatten(-1, (G, 32)).flatten(0, -2).split(1 << 18):
        low, top = part.min(1).values, part.max(1).values
        s = steps[torch.searchsorted(steps * qmax, top - low)]
        z = low.float().to(torch.float16).double()
        y = part - z[:, None]
        c = torch.where(s[:, None] > 0, torch.floor(y / s[:, None].clamp_min(1e-30)).clamp(0, qmax), 0.0)
        d0, d1 = (y - c * s[:, None]).abs(), ((c + 1) * s[:, None] - y).abs()
        c = torch.where((s[:, None] > 0) & (c < qmax) & ((d1 < d0) | ((d1 == d0) & (c % 2 == 1))), c + 1, c)
        out.append(c * s[:, None] + z[:, None])
    return torch.cat(out).view(x.shape[:-1] + (D,))


def exact(case, seed):
    if case["op"] in ("branch", "compact"):
        return None
    st = prepare(case, seed)
    hkv, dev = case["hkv"], st["pool"].device
    if case["op"] == "append":
        if not case["hats"]:
            return None
        return {"pool": None, "bounds": None, "k_hat": _group64(st["k"], case["bits_k"]), "v_hat": _group64(st["v"], case["bits_v"])}
    nq, g = case["n_q"], case["hq"] // hkv
    out = torch.zeros(case["batch"], nq, case["hq"], D, dtype=torch.float64, device=dev)
    lens, seqs = st["lens"].tolist(), st["seqs"].tolist()
    for b, s in enumerate(seqs):
        n = lens[s]
        pos = torch.arange(n, device=dev)
        pages = st["table"][s].long()[pos // ROWS]
        for h in range(hkv):
            q = st["q"][b, :, h * g:(h + 1) * g].double()
            if case["op"] == "attend":
                blocks = st["pool"][0, st["table"][s].long()[:_blocks(n)], h]
                keys, vals = (torch.cat([_value(x.repeat_interleave(ROWS, 0), torch.arange(ROWS, device=dev).repeat(len(x)),
                                                case["bits_k"], case["bits_v"], kind) for x in blocks.split(64)])[:n] for kind in "kv")
            for i in range(nq):
                lim = n - nq + 1 + i
                if lim <= 0:
                    continue
                if case["op"] == "attend":
                    kk, vv = keys[:lim], vals[:lim]
                else:
                    mine = _choice(st["bounds"][0, pages[:lim:ROWS], h], q[i], case["blocks"])
                    x = st["pool"][0, pages[mine * ROWS], h]
                    r = torch.arange(ROWS, device=dev).repeat(len(mine))
                    keep = mine.repeat_interleave(ROWS) * ROWS + r < lim
                    kk, vv = (_value(x.repeat_interleave(ROWS, 0), r, case["bits_k"], case["bits_v"], kind)[keep] for kind in "kv")
                w = torch.softmax((q[i] @ kk.T) / math.sqrt(D), -1)
                out[b, i, h * g:(h + 1) * g] = w @ vv
    return {"out": out} if case["op"] == "attend" else {"out": out, "sel": None}


def _choice(rec, q, k):
    """The blocks that one token's heads q [g, 128] read, ascending, from the records [blocks, 272] of its blocks."""
    n = rec.shape[0]
    if n <= k:
        return torch.arange(n, device=rec.device)
    lo, hi = rec[:, :D].view(torch.int8).double(), rec[:, D:2 * D].view(torch.int8).double()
    e = rec[:, 256:260].contiguous().view(torch.int32)[:, 0].double()
    step = 2.0 ** EMIN
    top = float(q.abs().max())
    while 127 * step < top:
        step *= 2
    c = torch.round(q / step)
    score = torch.maximum(c[:, None] * lo, c[:, None] * hi).sum((0, 2)) * 2.0 ** e
    score[0] = score[-2:] = math.inf
    return score.sort(descending=True, stable=True).indices[:k].sort().values
