"""More of the paged cache's operators as they are measured: what each case is, its inputs, and one pass through it.

``own`` false: every operator in elementary torch operations, on the documented bytes of the cache (pages of 64
positions, each KV head's block in the tile format of include/hyq.h).  ``own`` true: the calls a user makes.

Operators (``case["op"]``):

  shared   attention of the last n_q tokens of every sequence, causal, in groups of sequences that begin with the same
           pages: those are read once for a group
  cross    attention of any number of tokens a sequence (a decoder's) over all positions of the sequence (an encoder's
           states), not causal
  weigh    the attention weights that the last n_q tokens give to every position, added to what each position has
           received so far, per KV head
  evict    one step of a cache held at a budget: room for new positions, then every layer and KV head drops the positions
           that received least, keeping the first ones and the latest
"""
import math

import torch

own = False

D, G, ROWS = 128, 4, 64          # head_dim, quantisation groups of 32, positions per page
EMIN = -40                       # smallest exponent of a bound's step
REC = 272                        # bytes of a bound record: lo[128], hi[128], exponent int32, 12 unused


# --- cases ---------------------------------------------------------------------------------------------------------

def _case(name, op, **kw):
    c = {"name": name, "op": op, "hq": 32, "hkv": 8, "bits_k": 4, "bits_v": 4}
    c.update(kw)
    return c


def listed():
    return [
        # four samples of one short prompt
        _case("shared 4 x 1000", "shared", groups=1, members=4, n_q=1, prefix=960, suffix=100),
        # three system prompts of unlike lengths, four drafted tokens a request, wide GQA groups, 8-bit codes
        _case("shared drafts 3 x 8", "shared", groups=3, members=8, n_q=4, prefix=8192, suffix=700, hq=64, bits_k=8, bits_v=8),
        # many questions about one long document
        _case("shared 64 x 32768", "shared", groups=1, members=64, n_q=1, prefix=32768, suffix=500),
        # five beams of a small decoder over one encoded input
        _case("cross 1 x 1500", "cross", batch=1, tokens=5, length=1500, hq=8, hkv=8),
        # a batch of decoder prompts of unlike lengths
        _case("cross 16 x 1500", "cross", batch=16, tokens=448, length=1500),
        # long targets over long sources, 8-bit codes
        _case("cross 4 x 16001", "cross", batch=4, tokens=2000, length=16001, bits_k=8, bits_v=8),
        # one short chat's newest token
        _case("weigh 1 x 1000", "weigh", batch=1, n_q=1, length=1000),
        # the last queries of a batch of prompts, which look back over them
        _case("weigh prompts 8 x 8192", "weigh", batch=8, n_q=64, length=8192),
        # a full server: many requests of unlike lengths
        _case("weigh 64 x 32768", "weigh", batch=64, n_q=1, length=32768),
        # two layers of one small chat held at 512 positions
        _case("evict 1 x 512", "evict", seqs=1, keep=512, new=64, layers=2, n_first=4, n_last=32),
        # a running batch held at 4096 positions, a page at a time, a model of 32 layers
        _case("evict 16 x 4096", "evict", seqs=16, keep=4096, new=64, layers=32, n_first=4, n_last=128),
        # long prompts cut down to 4096 positions
        _case("evict prompts 8 x 32768", "evict", seqs=8, keep=4096, new=28672, layers=8, n_first=4, n_last=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "cross", "cross", "weigh", "weigh", "evict"])
    hq, hkv = rng.choice([(4, 4), (8, 2), (10, 2), (32, 8), (32, 8), (64, 8), (14, 2)])
    bits = rng.choice([(4, 4), (4, 4), (4, 4), (8, 8), (8, 4), (4, 8)])
    c = {"op": op, "hq": hq, "hkv": hkv, "bits_k": bits[0], "bits_v": bits[1]}
    room = 32 / hq                # the largest cases have 32 query heads
    if op == "shared":
        g, nq = _log(rng, 1, 6), rng.choice([1, 1, 1, 2, 3, 5])
        m = _log(rng, 1, 64 // g)
        c.update(groups=g, members=m, n_q=nq, prefix=_log(rng, 30, min(65536, int(64 * 32768 * room / (g * m * nq)))),
                 suffix=_log(rng, 1, 1500))
    elif op == "cross":
        b = _log(rng, 1, 16)
        t = _log(rng, 1, 2000)
        c.update(batch=b, tokens=t, length=_log(rng, 20, min(32768, int(4 * 2000 * 16001 * room / (b * t)))))
    elif op == "weigh":
        b, nq = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5, 16, 64])
        c.update(batch=b, n_q=nq, length=_log(rng, 20, min(131072, int(64 * 32768 * min(1.0, 2 * room / nq) / b))))
    else:
        s, layers = _log(rng, 1, 16), _log(rng, 1, 16)
        top = 1000000 // (s * layers)
        k = _log(rng, 40, min(8192, top))
        first = rng.choice([0, 1, 4])
        c.update(seqs=s, keep=k, new=_log(rng, 1, max(1, min(32768, top - k))), layers=layers, n_first=first,
                 n_last=min(k - first, _log(rng, 1, 300)))
    return c


def _spread(n, top, low=0.25):
    """n lengths between low * top and top, unlike one another, the first one top."""
    return [top if i == 0 else max(1, int(top * (1 - (1 - low) * math.modf(i * 0.6180339887498949)[0]))) for i in range(n)]


def _blocks(n):
    return -(-n // ROWS)


def _tile(case):
    return 256 * (case["bits_k"] + case["bits_v"]) + 512


def _groups(case):
    """Per group (positions shared, lengths of its sequences): the shared part whole pages, behind it at least n_q positions."""
    sizes = _spread(case["groups"], case["members"])
    shared = [n // ROWS * ROWS for n in _spread(case["groups"], case["prefix"], 0.5)]
    tails = iter(_spread(sum(sizes), case["suffix"], 0.02))
    return [(p, [p + next(tails) + case["n_q"] - 1 for _ in range(m)]) for p, m in zip(shared, sizes)]


def _cross(case):
    """(positions, tokens) of every sequence."""
    lens, toks = _spread(case["batch"], case["length"]), _spread(case["batch"], case["tokens"], 0.05)
    if case["batch"] >= 4:
        toks[2] = 0               # a request that has nothing to ask this time
        lens[3] = 0               # one whose input has not been encoded yet
    return lens, toks


def _weigh_lens(case):
    lens = _spread(case["batch"], case["length"])
    if case["batch"] >= 8:
        lens[1] = 1               # a request that has just begun: with n_q > 1 its first tokens see nothing
    return lens


def _evict_lens(case):
    """(positions kept, new ones) of every sequence."""
    least = case["n_first"] + case["n_last"]
    keep = [max(least, n) for n in _spread(case["seqs"], case["keep"], 0.7)]
    new = _spread(case["seqs"], case["new"], 0.5)
    if case["seqs"] >= 4:
        new[2] = 0                # a sequence that did not grow
    return keep, new


def work(case):
    op, hkv, hq, tile = case["op"], case["hkv"], case["hq"], _tile(case)
    row = tile / 16               # bytes of one position of one KV head
    key = 16 * case["bits_k"] + 16
    if op == "shared":
        cells = n_rows = seen = 0
        for p, lens in _groups(case):
            cells += p + sum(n - p for n in lens)
            n_rows += len(lens) * case["n_q"]
            seen += sum(n - case["n_q"] + 1 + i for n in lens for i in range(case["n_q"]))
        return {"bytes": cells * hkv * row + n_rows * hq * D * 4, "flops": 4 * D * hq * seen}
    if op == "cross":
        lens, toks = _cross(case)
        return {"bytes": sum(n for n, t in zip(lens, toks) if t) * hkv * row + sum(toks) * hq * D * 4,
                "flops": 4 * D * hq * sum(n * t for n, t in zip(lens, toks))}
    if op == "weigh":
        lens = _weigh_lens(case)
        seen = sum(max(0, n - case["n_q"] + 1 + i) for n in lens for i in range(case["n_q"]))
        return {"bytes": sum(lens) * hkv * (key + 8) + case["batch"] * case["n_q"] * hq * (D * 2 + 4), "flops": 2 * D * hq * seen}
    nbytes = 0
    for k, m in zip(*_evict_lens(case)):
        if m == 0:
            continue
        n, w = k + m, k - case["n_last"]
        free = (w - case["n_first"]) * m / max(1, n - case["n_first"] - case["n_last"])      # places that rows move to, on average
        pages = min(_blocks(w), free) + _blocks(k) - w // ROWS
        nbytes += 4 * n + (free + case["n_last"]) * (2 * row + 4) + pages * (64 * key + 260)
    return {"bytes": nbytes * case["layers"] * hkv, "flops": 0}


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
    """FP16 step and zero [..., 16, 4] of the 256-byte region at ``off``, as they are held (int16)."""
    h = tiles[..., off:off + 256].contiguous().view(torch.int16)
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


def _layout(case):
    """(kind, bits, byte of the codes, byte of the metadata) of the two halves of a tile."""
    bk, bv = case["bits_k"], case["bits_v"]
    return ("k", bk, 0, 256 * (bk + bv)), ("v", bv, 256 * bk, 256 * (bk + bv) + 256)


def _held_rows(blocks, case, kinds="kv"):
    """Per kind the codes [..., 64, 128], steps and zeros [..., 64, 4] (int16) of page blocks uint8 [..., block bytes]."""
    t = blocks.unflatten(-1, (4, -1))
    out = []
    for kind, bits, co, mo in _layout(case):
        if kind in kinds:
            s, z = _meta(t, kind, mo)
            out.append([x.flatten(-3, -2) for x in (_codes(t, kind, bits, co), s, z)])
    return out


def _values(codes, s, z):
    """c s + z in float32."""
    h = lambda x: x.contiguous().view(torch.float16).float()[..., None]  # noqa: E731
    return (codes.float().unflatten(-1, (G, 32)) * h(s) + h(z)).flatten(-2)


def _unpack(blocks, case, kinds="kv"):
    """Keys and values float32 [..., 64, 128] of page blocks."""
    return [_values(*x) for x in _held_rows(blocks, case, kinds)]


def _pack(rows, case):
    """The inverse of _held_rows."""
    f = lambda x: x.unflatten(-2, (4, 16))  # noqa: E731
    codes = [_region(f(c), kind, bits) for (c, _, _), (kind, bits, _, _) in zip(rows, _layout(case))]
    metas = [_meta_bytes(f(s), f(z), kind) for (_, s, z), kind in zip(rows, "kv")]
    return torch.cat(codes + metas, -1).flatten(-2)


def _quantise(x, bits):
    """Codes uint8, step and zero (FP16, as int16) of rows [..., 128]."""
    qmax = float((1 << bits) - 1)
    g = x.unflatten(-1, (G, 32)).double()
    mn, mx = g.amin(-1), g.amax(-1)
    s = ((mx - mn) / qmax * (1 + 2 ** -10)).to(torch.float16)
    z = mn.float().to(torch.float16)
    sd, zd = s.double()[..., None], z.double()[..., None]
    c = torch.where(sd > 0, torch.round((g - zd) / torch.where(sd > 0, sd, 1.0)).clamp(0, qmax), 0.0)
    return c.to(torch.uint8).flatten(-2), s.view(torch.int16), z.view(torch.int16)


def _record(k, valid):
    """Bound records uint8 [..., 272] of keys [..., 64, 128] over the rows ``valid`` [..., 64]."""
    v = valid[..., None]
    mn = torch.where(v, k, math.inf).amin(-2).double()
    mx = torch.where(v, k, -math.inf).amax(-2).double()
    amax = torch.where(v, k.abs(), 0.0).amax((-2, -1))
    m, x = torch.frexp(amax.double())            # smallest integer e >= -40 with amax <= 127 * 2^e
    e = torch.where(amax > 0, x - 7 + (m > 127 / 128), torch.full_like(x, EMIN)).clamp_min(EMIN).to(torch.int32)
    inv = torch.exp2(-e.double())[..., None]
    rec = [torch.floor(mn * inv).to(torch.int8).view(torch.uint8), torch.ceil(mx * inv).to(torch.int8).view(torch.uint8),
           e[..., None].contiguous().view(torch.uint8), torch.zeros(e.shape + (12,), dtype=torch.uint8, device=k.device)]
    return torch.cat(rec, -1)


# --- inputs --------------------------------------------------------------------------------------------------------

def _rows_like_keys(shape, u, gen, dev):
    """Keys as a model's: a few channels of large values, and 2% of positions that every query looks at.
    shape [..., HKV, 64, 128] with u [HKV, 1, 128]."""
    k = torch.randn(shape, generator=gen, device=dev)
    k[..., [5, 64, 101]] *= 8
    sink = torch.rand(shape[:-1] + (1,), generator=gen, device=dev) < 0.02
    return torch.where(sink, k + 4 * u, k).to(torch.bfloat16)


def _random_blocks(n, case, u, gen, dev):
    """n pages of rows, quantised: uint8 [n, HKV, block bytes]."""
    hkv, out = case["hkv"], []
    for at in range(0, n, max(1, 4096 // hkv)):
        m = min(n - at, max(1, 4096 // hkv))
        k = _rows_like_keys((m, hkv, ROWS, D), u, gen, dev)
        v = torch.randn(m, hkv, ROWS, D, generator=gen, device=dev).to(torch.bfloat16)
        out.append(_pack([_quantise(k, case["bits_k"]), _quantise(v, case["bits_v"])], case))
    return torch.cat(out)


def _place(need, n_pages, width, gen, dev):
    """A table in which sequence i holds need[i] pages of its own, at random places of the pool, and the pages."""
    perm = torch.randperm(n_pages, generator=gen, device=dev)
    seq = torch.repeat_interleave(torch.arange(len(need)), torch.tensor(need))
    first = torch.tensor([0] + need).cumsum(0)[:-1]
    total = sum(need)
    blk = torch.arange(total) - first[seq]
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=dev)
    table[seq.to(dev), blk.to(dev)] = perm[:total].to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[perm[:total]] = 1
    return table, refs, perm[:total]


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    hkv, hq = case["hkv"], case["hq"]
    u = torch.randn(hkv, 1, D, generator=gen, device=dev)
    u /= u.norm(dim=-1, keepdim=True)
    st = {"case": case}
    if case["op"] == "evict":
        return _prepare_evict(st, u, gen, dev)
    if case["op"] == "shared":
        groups = _groups(case)
        lens = [n for _, ns in groups for n in ns]
        own_need = [_blocks(n - p) for p, ns in groups for n in ns]
        need = [p // ROWS for p, _ in groups] + own_need           # the shared parts first, as sequences of their own
    else:
        lens = _weigh_lens(case) if case["op"] == "weigh" else _cross(case)[0]
        need = [_blocks(n) for n in lens]
    n_pages = sum(need) + max(4, sum(need) // 10)
    width = max(1, *need) if case["op"] != "shared" else max(_blocks(n) for n in lens)
    table, refs, pages = _place(need, n_pages, width, gen, dev)
    if case["op"] == "shared":
        parts, ng, i = table, len(groups), 0
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
        for j, (p, ns) in enumerate(groups):
            nb = p // ROWS
            refs[parts[j, :nb].long()] = len(ns)
            for _ in ns:
                table[i, :nb] = parts[j, :nb]
                m = own_need[i]
                table[i, nb:nb + m] = parts[ng + i, :m]
                i += 1
    size = 4 * _tile(case)
    st["pool"] = torch.zeros(1, n_pages, hkv, size, dtype=torch.uint8, device=dev)
    st["pool"][0, pages] = _random_blocks(len(pages), case, u, gen, dev)
    n = len(lens)
    # the sequences' numbers are not those of the call's rows; a group's rows stand together
    order = torch.randperm(n, generator=gen, device=dev)
    back = torch.argsort(order)
    st.update(table=table[back].contiguous(), lens=_ints(lens, dev)[back].contiguous(), refs=refs, seqs=order.to(torch.int32))
    toks = _cross(case)[1] if case["op"] == "cross" else [case["n_q"]] * n
    t = sum(toks)
    q = torch.randn(t, hkv, hq // hkv, D, generator=gen, device=dev) + 2 * u
    q = q.to(torch.bfloat16).flatten(1, 2)
    if case["op"] == "cross":
        st.update(q=q, out=torch.empty_like(q), host=list(zip(lens, toks)),
                  cu=torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(toks).cumsum(0).to(torch.int32)]).to(dev))
        return st
    st["q"] = q.unflatten(0, (n, case["n_q"])).contiguous()
    if case["op"] == "shared":
        st["out"] = torch.empty_like(st["q"])
        sizes = [len(ns) for _, ns in groups]
        st.update(cu=torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(sizes).cumsum(0).to(torch.int32)]).to(dev),
                  n_shared=_ints([p for p, _ in groups], dev), host=groups)
        return st
    # what the positions have received so far, and the logarithms of the softmax sums that the attention has left
    st["mass"] = torch.rand(1, n_pages, hkv, ROWS, generator=gen, device=dev)
    st["lse"] = _lse(st)
    return st


def _lse(st):
    """float32 [batch, n_q, HQ], a sequence at a time."""
    c = st["case"]
    g, nq = c["hq"] // c["hkv"], c["n_q"]
    out = torch.empty(c["batch"], nq, c["hq"], device=st["q"].device)
    lens = _weigh_lens(c)
    for b in range(c["batch"]):
        n = lens[b]
        page = st["table"][st["seqs"][b]].long()[:_blocks(n)]
        (k,) = _unpack(st["pool"][0, page], c, "k")                                # [blocks, HKV, 64, 128]
        k = k.transpose(0, 1).flatten(1, 2)[:, :n]
        q = st["q"][b].float().unflatten(1, (c["hkv"], g)).permute(1, 0, 2, 3).flatten(1, 2)
        x = torch.matmul(q, k.transpose(1, 2)) * D ** -0.5                         # [HKV, n_q g, n]
        lim = (n - nq + 1 + torch.arange(nq, device=x.device)).repeat_interleave(g)
        x = torch.where(torch.arange(n, device=x.device) < lim[:, None], x, -math.inf)
        out[b] = torch.logsumexp(x.double(), -1).float().unflatten(1, (nq, g)).transpose(0, 1).flatten(1)
    return out


def _prepare_evict(st, u, gen, dev):
    c = st["case"]
    keep, new = _evict_lens(c)
    need = [_blocks(k) for k in keep]
    full = [_blocks(k + m) for k, m in zip(keep, new)]
    n_pages = sum(full) + max(4, sum(full) // 10)
    table, refs, _ = _place(need, n_pages, max(full), gen, dev)
    # pages of valid rows, most of them met more than once
    some = _random_blocks(max(1, 1024 // c["hkv"]), c, u, gen, dev).flatten(0, 1)
    shape = (c["layers"], n_pages, c["hkv"])
    st["pool"] = some[torch.randint(0, len(some), shape, generator=gen, device=dev)]
    st["bounds"] = torch.randint(0, 256, shape + (REC,), generator=gen, device=dev, dtype=torch.uint8)
    # a few positions receive most of the weight, some nothing at all
    m = torch.exp(3 * torch.randn(shape + (ROWS,), generator=gen, device=dev))
    st["mass"] = torch.where(torch.rand(m.shape, generator=gen, device=dev) < 0.1, 0.0, m)
    order = torch.randperm(c["seqs"], generator=gen, device=dev)
    back = torch.argsort(order)
    st.update(table=table[back].contiguous(), lens=_ints(keep, dev)[back].contiguous(), refs=refs, seqs=order.to(torch.int32),
              keep=_ints(keep, dev), new=_ints(new, dev), host=list(zip(keep, new)))
    return st


# --- one pass ------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"shared": _shared, "cross": _cross_plain, "weigh": _weigh, "evict": _evict}[st["case"]["op"]](st)


def _cache(st):
    """The handle that a program makes once for its pool."""
    if "cache" not in st:
        import hybrid_precision_quantized_gb300 as hyq
        c = st["case"]
        cfg = hyq.make_config(1, c["hq"], c["hkv"], capacity=ROWS, bits_k=c["bits_k"], bits_v=c["bits_v"])
        given = {k: st[k] for k in ("pool", "bounds", "table", "lens", "refs") if k in st}
        st["cache"] = hyq.PagedCache(cfg, n_pages=st["pool"].shape[1], n_seqs=st["table"].shape[0], max_blocks=st["table"].shape[1],
                                     n_layers=st["pool"].shape[0], device=st["pool"].device, buffers=given)
    return st["cache"]


def _evicted(st):
    return {k: st[k] for k in ("pool", "bounds", "table", "lens", "refs", "mass")}


def _own(st):
    c, cache = st["case"], _cache(st)
    if c["op"] == "shared":
        cache.attention_shared(0, st["q"], st["out"], st["cu"], st["n_shared"], seqs=st["seqs"])
        return {"out": st["out"]}
    if c["op"] == "cross":
        cache.cross_attention(0, st["q"], st["out"], seqs=st["seqs"], cu_q=st["cu"])
        return {"out": st["out"]}
    if c["op"] == "weigh":
        cache.accumulate(0, st["q"], st["lse"], st["mass"], seqs=st["seqs"])
        return {"mass": st["mass"]}
    cache.reserve(st["seqs"], st["new"])
    cache.evict(st["mass"], st["keep"], seqs=st["seqs"], n_first=c["n_first"], n_last=c["n_last"])
    return _evicted(st)


def _softmax(x):
    """Softmax of logits over the last axis, -inf where a place is not seen; zeros where none is."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    s = p.sum(-1, keepdim=True)
    return torch.where(s > 0, p / torch.where(s > 0, s, 1.0), 0.0)


def _shared(st):
    c, dev = st["case"], st["pool"].device
    hkv, nq = c["hkv"], c["n_q"]
    g = c["hq"] // hkv
    table, out, at = st["table"].long()[st["seqs"].long()], [], 0
    for p, lens in st["host"]:
        m, nb = len(lens), p // ROWS
        mine = table[at:at + m]
        end = st["lens"].long()[st["seqs"].long()[at:at + m]]
        k0, v0 = (x.transpose(0, 1).flatten(1, 2) for x in _unpack(st["pool"][0, mine[0, :nb]], c))          # [HKV, p, 128]
        k1, v1 = (x.transpose(1, 2).flatten(2, 3) for x in _unpack(st["pool"][0, mine[:, nb:].clamp_min(0)], c))  # [m, HKV, L, 128]
        q = st["q"][at:at + m].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)            # [m, HKV, n_q g, 128]
        qh = q.transpose(0, 1).flatten(1, 2)                                                                  # [HKV, m n_q g, 128]
        x0 = torch.matmul(qh, k0.transpose(1, 2)).unflatten(1, (m, nq * g)).transpose(0, 1)
        pos = p + torch.arange(k1.shape[2], device=dev)
        lim = end[:, None] - nq + 1 + torch.arange(nq, device=dev)                                            # positions that a token sees
        seen = pos < lim.repeat_interleave(g, 1)[:, None, :, None]
        v1 = torch.where((pos < end[:, None])[:, None, :, None], v1, 0.0)
        x1 = torch.where(seen, torch.matmul(q, k1.transpose(2, 3)), -math.inf)
        w = _softmax(torch.cat([x0, x1], -1) * D ** -0.5)
        o = torch.matmul(w[..., :p].transpose(0, 1).flatten(1, 2), v0).unflatten(1, (m, nq * g)).transpose(0, 1)
        o = o + torch.matmul(w[..., p:], v1)
        out.append(o.unflatten(2, (nq, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(torch.bfloat16))
        at += m
    return {"out": torch.cat(out)}


def _cross_plain(st):
    c = st["case"]
    hkv, g = c["hkv"], c["hq"] // c["hkv"]
    table, out, at = st["table"].long()[st["seqs"].long()], [], 0
    for i, (n, t) in enumerate(st["host"]):
        if t == 0:
            continue
        k, v = (x.transpose(0, 1).flatten(1, 2)[:, :n] for x in _unpack(st["pool"][0, table[i, :_blocks(n)]], c))
        q = st["q"][at:at + t].float().unflatten(1, (hkv, g)).transpose(0, 1).flatten(1, 2)                   # [HKV, t g, 128]
        o = torch.matmul(_softmax(torch.matmul(q, k.transpose(1, 2)) * D ** -0.5), v) if n else torch.zeros_like(q)
        out.append(o.unflatten(1, (t, g)).transpose(0, 1).flatten(1, 2).to(torch.bfloat16))
        at += t
    return {"out": torch.cat(out)}


def _weigh(st):
    c, dev = st["case"], st["pool"].device
    hkv, nq = c["hkv"], c["n_q"]
    g = c["hq"] // hkv
    seqs = st["seqs"].long()
    end, table = st["lens"].long()[seqs], st["table"].long()[seqs].clamp_min(0)
    (k,) = _unpack(st["pool"][0, table], c, "k")                                  # [B, blocks, HKV, 64, 128]
    k = k.transpose(1, 2).flatten(2, 3)                                           # [B, HKV, L, 128]
    q = st["q"].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = st["lse"].unflatten(2, (hkv, g)).permute(0, 2, 1, 3).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    lim = (end[:, None] - nq + 1 + torch.arange(nq, device=dev)).repeat_interleave(g, 1)[:, None, :, None]
    pos = torch.arange(k.shape[2], device=dev)
    add = torch.where(pos < lim, torch.exp(x - lse[..., None]), 0.0).sum(2)       # [B, HKV, L]
    old = st["mass"][0, table].transpose(1, 2).flatten(2, 3)
    fresh = pos >= end[:, None, None] - nq                                        # the new positions begin at zero
    add = (torch.where(fresh, 0.0, old) + add).unflatten(2, (-1, ROWS)).transpose(1, 2)
    here = (pos < end[:, None]).unflatten(1, (-1, ROWS))                          # [B, blocks, 64]
    b, blk, r = here.nonzero(as_tuple=True)
    st["mass"][0, table[b, blk], :, r] = add[b, blk, :, r]
    return {"mass": st["mass"]}


def _reserve(st):
    """Room for the new positions; the sequences hold pages of their own."""
    dev, table, refs = st["pool"].device, st["table"], st["refs"]
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    at = 0
    for i, (k, m) in enumerate(st["host"]):
        a, b = _blocks(k), _blocks(k + m)
        table[st["seqs"].long()[i], torch.arange(a, b, device=dev)] = free[at:at + b - a].to(torch.int32)
        at += b - a
    refs[free[:at]] = 1
    st["lens"][st["seqs"].long()] += st["new"]


def _evict(st):
    c, dev = st["case"], st["pool"].device
    first, last = c["n_first"], c["n_last"]
    _reserve(st)
    for i, (k, m) in enumerate(st["host"]):
        if m == 0:
            continue
        n, w = k + m, k - last
        page = st["table"][st["seqs"].long()[i]].long()[:_blocks(n)]
        mass = st["mass"][:, page].transpose(1, 2).flatten(2, 3)                  # [layers, HKV, 64 blocks]
        key = mass[..., :n - last].clone()
        key[..., :first] = math.inf
        best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :w]
        kept = torch.zeros(key.shape, dtype=torch.bool, device=dev).scatter_(2, best, True)
        # a kept position from w on goes to the free place of the same rank before w
        place = torch.argsort(kept[..., :w].to(torch.int32), dim=-1, stable=True)
        come = w + torch.argsort((~kept[..., w:]).to(torch.int32), dim=-1, stable=True)
        src = torch.arange(k, device=dev).expand(key.shape[:2] + (k,)).clone()
        free = (~kept[..., :w]).sum(-1, keepdim=True)
        r = min(w, n - last - w)
        hit = torch.arange(r, device=dev) < free
        src.scatter_(2, place[..., :r], torch.where(hit, come[..., :r], place[..., :r]))
        src[..., w:] = torch.arange(n - last, n, device=dev)
        nb = _blocks(k)
        rows = _held_rows(st["pool"][:, page].transpose(1, 2), c)                 # [layers, HKV, blocks, 64, ..]
        moved = []
        for part in rows:
            part = [x.flatten(2, 3) for x in part]
            moved.append([torch.cat([x.gather(2, src[..., None].expand(-1, -1, -1, x.shape[-1])), x[:, :, k:nb * ROWS]], 2)
                          .unflatten(2, (nb, ROWS)) for x in part])
        st["pool"][:, page[:nb]] = _pack(moved, c).transpose(1, 2)
        mass = torch.cat([mass.gather(2, src), mass[..., k:nb * ROWS]], 2).unflatten(2, (nb, ROWS))
        st["mass"][:, page[:nb]] = mass.transpose(1, 2)
        # records of the pages that received a row
        new = torch.zeros(src.shape[:2] + (nb * ROWS,), dtype=torch.bool, device=dev)
        new[..., :k] = src != torch.arange(k, device=dev)
        got = new.unflatten(2, (nb, ROWS)).any(-1)
        valid = (torch.arange(nb * ROWS, device=dev) < k).unflatten(0, (nb, ROWS)).expand(got.shape + (ROWS,))
        rec = _record(_values(*moved[0]), valid).transpose(1, 2)
        st["bounds"][:, page[:nb]] = torch.where(got.transpose(1, 2)[..., None], rec, st["bounds"][:, page[:nb]])
        st["refs"][page[nb:]] -= 1
        st["lens"][st["seqs"].long()[i]] = k
    return _evicted(st)


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


def _sequence64(st, page, n, h, kind):
    """Keys or values float64 [n, 128] of KV head h of the sequence that lies in the pages ``page``."""
    c, out = st["case"], []
    for x in st["pool"][0, page, h].split(64):
        r = torch.arange(ROWS, device=x.device).repeat(len(x))
        out.append(_value(x.repeat_interleave(ROWS, 0), r, c["bits_k"], c["bits_v"], kind))
    return torch.cat(out)[:n]


def exact(case, seed):
    if case["op"] == "evict":
        return None
    st = prepare(case, seed)
    hkv, g, dev = case["hkv"], case["hq"] // case["hkv"], st["pool"].device
    lens, seqs = st["lens"].tolist(), st["seqs"].tolist()
    if case["op"] == "weigh":
        mass, nq = st["mass"].double(), case["n_q"]
    else:
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=dev)
    starts = st["cu"].tolist() if case["op"] == "cross" else None
    for b, s in enumerate(seqs):
        n = lens[s]
        if n == 0 or (starts and starts[b] == starts[b + 1]):
            continue
        page = st["table"][s].long()[:_blocks(n)]
        pos = torch.arange(n, device=dev)
        for h in range(hkv):
            heads = slice(h * g, (h + 1) * g)
            keys = _sequence64(st, page, n, h, "k")
            if case["op"] == "weigh":
                got = mass[0, page[pos // ROWS], h, pos % ROWS]
                got[max(0, n - nq):] = 0.0
                for i in range(nq):
                    lim = n - nq + 1 + i
                    if lim > 0:
                        x = (st["q"][b, i, heads].double() @ keys[:lim].T) / math.sqrt(D)
                        got[:lim] += torch.exp(x - st["lse"][b, i, heads].double()[:, None]).sum(0)
                mass[0, page[pos // ROWS], h, pos % ROWS] = got
                continue
            vals = _sequence64(st, page, n, h, "v")
            if case["op"] == "cross":
                for at in range(starts[b], starts[b + 1], 256):
                    rows = slice(at, min(at + 256, starts[b + 1]))
                    x = (st["q"][rows, heads].double() @ keys.T) / math.sqrt(D)
                    out[rows, heads] = torch.softmax(x, -1) @ vals
            else:
                for i in range(case["n_q"]):
                    lim = n - case["n_q"] + 1 + i
                    x = (st["q"][b, i, heads].double() @ keys[:lim].T) / math.sqrt(D)
                    out[b, i, heads] = torch.softmax(x, -1) @ vals[:lim]
    return {"mass": mass} if case["op"] == "weigh" else {"out": out}
