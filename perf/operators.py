"""The 4-bit window cache's operators, as a user's program calls them, beside
their plain forms in elementary torch operations.

A paged cache of K and V in 4 bits holds the tokens that a serving loop still
appends to and drops from; the lattice streams hold what no longer changes.
A token of one KV head is one 128-wide tile: y = H D x / sqrt(128) (Hadamard
transform after a diagonal of signs), 16 uniform levels (c - 7.5) s with one
bf16 scale s = max|y| / 7.5 a tile.  16 tokens of one head form a unit of 2112
bytes: K codes [16][64], V codes as [8 token pairs][8 chunks of 16 dimensions]
[2 tokens][8 bytes], K scales [16], V scales [16]; a page is [KV heads][page
tokens / 16] units.

Operators:
  append  writes new K and V rows (prompt rows or one token a sequence);
  read    gives rows back as the values that they stand for;
  attend  softmax(scale q K^T, capped on request) V for one or several new
          tokens a sequence, with the log of each row's sum and, on request,
          every token's weight added to its accumulated mass;
  evict   keeps the most recent tokens and those of the largest accumulated
          mass, in order, on pages of their own.
An append or an evict is followed by the read of the rows that it wrote, so
that what the cache holds comes back as values.
"""
import math

import torch

own = False

TILE = 128
UNIT = 16
UNIT_BYTES = 2112
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of a few chat sessions: the smallest write
        dict(name="append_one_token", op="append", batch=4, new=1, ragged=0.0, past=700, heads=8,
             page=16, dtype="bf16"),
        # prompts of several users, ragged, out of the fused projection's rows
        dict(name="append_prompts", op="append", batch=8, new=6001, ragged=0.6, past=0, heads=8,
             page=64, dtype="bf16"),
        # fp32 rows of a smaller model, appended behind an odd past
        dict(name="append_f32_odd", op="append", batch=3, new=517, ragged=0.3, past=45, heads=2,
             page=48, dtype="f32"),
        # a full window handed to the lattice encoder, head by head
        dict(name="read_window", op="read", batch=1, len=32768, ragged=0.0, heads=8, page=64,
             dtype="bf16"),
        # a few odd sequences read as fp16
        dict(name="read_odd", op="read", batch=5, len=333, ragged=0.8, heads=3, page=16,
             dtype="f16"),
        # one session at the start of its answer: latency alone
        dict(name="attend_short", op="attend", batch=1, len=77, ragged=0.0, heads=8, group=4,
             new=1, page=16, cap=0.0, mass=False, dtype="bf16", out="bf16"),
        # one session at the length of the long-context layer
        dict(name="attend_long_one", op="attend", batch=1, len=131072, ragged=0.0, heads=8,
             group=4, new=1, page=64, cap=0.0, mass=False, dtype="bf16", out="bf16"),
        # the decode-attention batch: 16 sessions of 32768 tokens, 32 query heads
        dict(name="attend_batch", op="attend", batch=16, len=32768, ragged=0.0, heads=8, group=4,
             new=1, page=64, cap=0.0, mass=False, dtype="bf16", out="bf16"),
        # four proposed tokens verified at once, capped scores, ragged sessions
        dict(name="attend_verify_cap", op="attend", batch=24, len=4093, ragged=0.9, heads=8,
             group=4, new=4, page=32, cap=30.0, mass=False, dtype="f16", out="f32"),
        # a decoding step that also accumulates each token's weight
        dict(name="attend_mass", op="attend", batch=16, len=8192, ragged=0.3, heads=8, group=4,
             new=1, page=16, cap=0.0, mass=True, dtype="bf16", out="bf16"),
        # a few sessions just over their budget
        dict(name="evict_small", op="evict", batch=4, len=300, ragged=0.1, heads=8, page=16,
             budget=256, recent=32),
        # long sessions cut down to an eighth
        dict(name="evict_long", op="evict", batch=16, len=32768, ragged=0.2, heads=8, page=64,
             budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "evict"])
    heads = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    c = dict(op=op, heads=heads, page=page, ragged=round(rng.uniform(0.0, 0.95), 3))
    if op == "append":
        c.update(batch=_log(rng, 1, 16), new=_log(rng, 1, 2500), past=rng.randrange(0, 2000),
                 dtype=rng.choice(["bf16", "f16", "f32"]))
    elif op == "read":
        c.update(batch=_log(rng, 1, 8), len=_log(rng, 1, 8000),
                 dtype=rng.choice(["bf16", "f16", "f32"]))
    elif op == "attend":
        batch, group = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8, 16])
        new = rng.choice([1, 1, 1, 2, 3, 4, 8])
        most = 524288 * 4 // (max(4, group * new) * batch)
        c.update(batch=batch, len=_log(rng, 1, min(131072, most)), group=group, new=new,
                 cap=rng.choice([0.0, 0.0, 20.0, 50.0]), mass=rng.random() < 0.3,
                 dtype=rng.choice(["bf16", "f16", "f32"]),
                 out=rng.choice(["bf16", "f16", "f32"]))
    else:
        batch = _log(rng, 1, 32)
        length = _log(rng, 64, 524288 // batch)
        budget = max(1, int(length * rng.uniform(0.05, 1.1)))
        c.update(batch=batch, len=length, budget=budget, recent=rng.randrange(0, budget + 1))
    return c


def _spread(batch, longest, ragged):
    """Lengths of a batch: the longest one first, the others down to (1 - ragged) of it."""
    less = int(longest * ragged)
    return [max(1, longest - ((b * 2654435761) % (1 << 32)) * less // (1 << 32))
            for b in range(batch)]


def _lengths(case):
    if case["op"] == "append":
        return [case["past"] + n for n in _spread(case["batch"], case["new"], case["ragged"])]
    return _spread(case["batch"], case["len"], case["ragged"])


# ------------------------------------------------------------------ the format, in torch
def _hadamard(device, dtype=torch.float32):
    """H / sqrt(128), Sylvester's order."""
    i = torch.arange(TILE, device=device)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = (x ^ (x >> 1)) & 1
    return (1.0 - 2.0 * x.to(dtype)) / math.sqrt(TILE)


def _diagonal(signs):
    """The +-1 diagonal of a 128-bit mask, int32 [4]."""
    i = torch.arange(TILE, device=signs.device)
    bit = (signs.to(torch.int64)[i // 32] >> (i % 32)) & 1
    return 1.0 - 2.0 * bit.to(torch.float32)


def _quantize(x, diag, had):
    """Rows [..., 128] -> codes uint8 [..., 128] and bf16 scales [...]."""
    y = (x.to(torch.float32) * diag) @ had
    s = (y.abs().amax(-1) / 7.5).to(torch.bfloat16)
    sf = s.to(torch.float32)[..., None]
    t = torch.floor(y / sf.clamp_min(1e-38) + 8.0)
    return torch.where(sf > 0, t.clamp(0, 15), torch.full_like(t, 8.0)).to(torch.uint8), s


def _pack_k(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _units(k, v, ks, vs):
    """Codes [..., T, 128] and scales [..., T] (T a multiple of 16) -> units [..., T / 16, 2112]."""
    lead, n = k.shape[:-2], k.shape[-2] // UNIT
    kb = _pack_k(k).reshape(*lead, n, 1024)
    vb = _pack_k(v).reshape(*lead, n, 8, 2, 8, 8).transpose(-2, -3).reshape(*lead, n, 1024)
    sb = [s.contiguous().view(torch.uint8).reshape(*lead, n, 32) for s in (ks, vs)]
    return torch.cat([kb, vb] + sb, -1)


def _unpack(b):
    """Bytes [..., n] -> codes [..., 2 n] as fp32."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2).to(torch.float32)


def _values(units):
    """Units [..., 2112] -> K and V rows [..., 16, 128] fp32 in the transformed domain."""
    lead = units.shape[:-1]
    s = units[..., 2048:].contiguous().view(torch.bfloat16).to(torch.float32)
    k = _unpack(units[..., :1024].reshape(*lead, UNIT, 64))
    v = units[..., 1024:2048].reshape(*lead, 8, 8, 2, 8).transpose(-2, -3)
    v = _unpack(v.reshape(*lead, UNIT, 64))
    return (k - 7.5) * s[..., :UNIT, None], (v - 7.5) * s[..., UNIT:, None]


def _rows(pages, table, diag, had):
    """The whole cache as K and V [n_seqs][heads][table width * page][128] fp32."""
    u = pages[table.to(torch.int64)]                       # [B][W][heads][P / 16][2112]
    B, W, nh, pu, _ = u.shape
    u = u.permute(0, 2, 1, 3, 4).reshape(B, nh, W * pu, UNIT_BYTES)
    return tuple((x.reshape(B, nh, W * pu * UNIT, TILE) @ had) * diag for x in _values(u))


# ------------------------------------------------------------------ states
def _tokens(shape, g, scale):
    """K or V rows: heavy-tailed noise under per-channel scales."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x.mul_(scale)


def _fill(n_pages, heads, page, g, signs):
    """Pages of a cache in use: rows drawn a few pages at a time, transformed and quantized."""
    had, diag = _hadamard("cuda"), _diagonal(signs)
    chan = [torch.exp(0.4 * torch.randn((heads, 1, TILE), generator=g, device="cuda"))
            for _ in range(2)]
    pages = torch.empty((n_pages, heads, page // UNIT, UNIT_BYTES), dtype=torch.uint8,
                        device="cuda")
    step = max(1, (1 << 19) // (heads * page))
    for lo in range(0, n_pages, step):
        n = min(step, n_pages - lo)
        q = [_quantize(_tokens((n, heads, page, TILE), g, c), diag, had) for c in chan]
        pages[lo:lo + n] = _units(q[0][0], q[1][0], q[0][1], q[1][1])
    return pages


def _table(batch, width, spare, g):
    n = batch * width
    order = torch.randperm(n + spare, generator=g, device="cuda").to(torch.int32)
    return order[:n].reshape(batch, width).contiguous(), order[n:]


def _ids(lens, first):
    """Sequence and position of every token of ragged runs that start at `first`."""
    seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(lens)])
    pos = torch.cat([torch.arange(f, f + n, dtype=torch.int32) for f, n in zip(first, lens)])
    return seq.cuda(), pos.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    op, B, nh, P = case["op"], case["batch"], case["heads"], case["page"]
    lens = _lengths(case)
    width = -(-max(lens) // P)
    signs = torch.randint(-2**31, 2**31 - 1, (4,), generator=g, device="cuda").to(torch.int32)
    s = dict(case=case, lens=lens, signs=signs, width=width, had=_hadamard("cuda"),
             diag=_diagonal(signs), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op == "append":
        past = [case["past"]] * B
        news = [n - p for n, p in zip(lens, past)]
        s["seq"], s["pos"] = _ids(news, past)
        n = sum(news)
        # rows of a fused projection: 2 query heads a KV head, then K, then V
        qkv = _tokens((n, 4 * nh, TILE), g, torch.exp(0.4 * torch.randn(
            (4 * nh, TILE), generator=g, device="cuda"))).to(DTYPES[case["dtype"]])
        s["k"], s["v"] = qkv[:, 2 * nh:3 * nh], qkv[:, 3 * nh:]
        s["table"], _ = _table(B, width, 3, g)
        s["pages"] = torch.zeros((B * width + 3, nh, P // UNIT, UNIT_BYTES), dtype=torch.uint8,
                                 device="cuda")
        s["rows"] = [torch.empty((n, nh, TILE), dtype=torch.bfloat16, device="cuda")
                     for _ in range(2)]
    else:
        spare = 3
        if op == "evict":
            new_width = -(-min(case["budget"], max(lens)) // P)
            spare += B * new_width
        s["table"], rest = _table(B, width, spare, g)
        s["pages"] = _fill(B * width + spare, nh, P, g, signs)
    if op == "read":
        s["seq"], s["pos"] = _ids(lens, [0] * B)
        n = sum(lens)
        # head by head, as the lattice encoder takes a slab
        s["rows"] = [torch.empty((nh, n, TILE), dtype=DTYPES[case["dtype"]],
                                 device="cuda").transpose(0, 1) for _ in range(2)]
    if op == "attend":
        Hq, new, dt = nh * case["group"], case["new"], DTYPES[case["dtype"]]
        qkv = 1.5 * torch.randn((B, new, Hq + 2 * nh, TILE), generator=g, device="cuda")
        s["q"] = qkv.to(dt)[:, :, :Hq]
        s["out"] = torch.empty((B, new, Hq, TILE), dtype=DTYPES[case["out"]], device="cuda")
        s["lse"] = torch.empty((B, new, Hq), dtype=torch.float32, device="cuda")
        s["scale"] = TILE ** -0.5
        s["mass"] = s["mass_out"] = None
        if case["mass"]:
            s["mass"] = torch.rand((B, nh, width * P), generator=g, device="cuda")
            s["mass_out"] = torch.zeros_like(s["mass"])
    if op == "evict":
        # accumulated weights: heavy-tailed, many of them equal (quantized sums)
        m = torch.rand((B, nh, width * P), generator=g, device="cuda").clamp_min(1e-6)
        s["mass"] = (m ** -0.5 * 64.0).floor() / 64.0
        s["new_table"] = rest[:B * new_width].reshape(B, new_width).contiguous()
        s["kept"] = torch.empty((B, nh, case["budget"]), dtype=torch.int32, device="cuda")
        s["new_lengths"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["new_mass"] = torch.zeros((B, nh, new_width * P), dtype=torch.float32, device="cuda")
        new_lens = [min(n, case["budget"]) for n in lens]
        s["seq"], s["pos"] = _ids(new_lens, [0] * B)
        s["rows"] = [torch.empty((sum(new_lens), nh, TILE), dtype=torch.bfloat16, device="cuda")
                     for _ in range(2)]
    if own:
        from weights_hq_encode_gb300 import hq
        s["cache"] = hq.make_kv4_cache(s["pages"], s["table"], P, nh, signs)
        if op == "evict":
            s["new_cache"] = hq.make_kv4_cache(s["pages"], s["new_table"], P, nh, signs)
        if op == "attend":
            s["ws"] = torch.empty(hq.hq_kv4_attention_workspace_bytes(
                s["cache"], new, Hq, case["mass"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _done(code):
    """A call that the library refused, or could not launch, is no pass."""
    if code != 0:
        raise RuntimeError(f"the library returned {code}")


def _run_own(s):
    from weights_hq_encode_gb300 import hq
    op = s["case"]["op"]
    if op == "append":
        _done(hq.hq_kv4_append(s["cache"], s["k"], s["v"], s["seq"], s["pos"], s["status"]))
        _done(hq.hq_kv4_read(s["cache"], s["seq"], s["pos"], *s["rows"], s["status"]))
        return s["rows"]
    if op == "read":
        _done(hq.hq_kv4_read(s["cache"], s["seq"], s["pos"], *s["rows"], s["status"]))
        return s["rows"]
    if op == "attend":
        _done(hq.hq_kv4_attention(s["cache"], s["lengths"], s["q"], s["scale"], s["case"]["cap"],
                                  s["out"], s["lse"], s["mass"], s["mass_out"], s["ws"],
                                  s["status"]))
        return [s["out"], s["lse"]] + ([s["mass_out"]] if s["mass"] is not None else [])
    _done(hq.hq_kv4_evict(s["cache"], s["lengths"], s["mass"], s["new_cache"], s["case"]["recent"],
                          s["kept"], s["new_lengths"], s["new_mass"], s["status"]))
    _done(hq.hq_kv4_read(s["new_cache"], s["seq"], s["pos"], *s["rows"], s["status"]))
    return [s["kept"], s["new_lengths"], s["new_mass"], *s["rows"]]


def _run_plain(s):
    case, nh, P = s["case"], s["case"]["heads"], s["case"]["page"]
    had, diag, table = s["had"], s["diag"], s["table"].to(torch.int64)
    if case["op"] == "append":
        seq, pos = s["seq"].to(torch.int64), s["pos"].to(torch.int64)
        (k, ks), (v, vs) = _quantize(s["k"], diag, had), _quantize(s["v"], diag, had)
        at = (table[seq, pos // P], (pos % P) // UNIT, pos % UNIT)
        _write(s["pages"], at, k, v, ks, vs)
        return _read_plain(s["pages"], at, diag, had, torch.bfloat16)
    if case["op"] == "read":
        seq, pos = s["seq"].to(torch.int64), s["pos"].to(torch.int64)
        at = (table[seq, pos // P], (pos % P) // UNIT, pos % UNIT)
        return _read_plain(s["pages"], at, diag, had, DTYPES[case["dtype"]])
    if case["op"] == "attend":
        return _attend_plain(s, diag, had)
    return _evict_plain(s, table, diag, had)


def _views(pages):
    """K codes, V codes and scales of all pages as views indexed by token."""
    lead = pages.shape[:-1]
    k = pages[..., :1024].view(*lead, UNIT, 64)
    v = pages[..., 1024:2048].view(*lead, 8, 8, 2, 8)
    return k, v, pages[..., 2048:].view(torch.bfloat16)


def _write(pages, at, k, v, ks, vs):
    """Rows [n][heads][128] into the units at (page, unit, token)."""
    page, unit, tok = at
    K, V, S = _views(pages)
    K[page, :, unit, tok] = _pack_k(k)
    V[page, :, unit, tok // 2, :, tok % 2] = _pack_k(v).unflatten(-1, (8, 8))
    S[page, :, unit, tok] = ks
    S[page, :, unit, UNIT + tok] = vs


def _read_plain(pages, at, diag, had, dtype):
    page, unit, tok = at
    K, V, S = _views(pages)
    k = (_unpack(K[page, :, unit, tok]) - 7.5) * S[page, :, unit, tok][..., None]
    v = _unpack(V[page, :, unit, tok // 2, :, tok % 2].flatten(-2))
    v = (v - 7.5) * S[page, :, unit, UNIT + tok][..., None]
    return [((x @ had) * diag).to(dtype) for x in (k, v)]


def _attend_plain(s, diag, had):
    case, lengths = s["case"], s["lengths"].to(torch.int64)
    B, new, Hq, _ = s["q"].shape
    nh = case["heads"]
    G = Hq // nh
    k, v = _rows(s["pages"], s["table"], diag, had)            # [B][heads][T][128]
    T = k.shape[2]
    q = s["q"].to(torch.float32).unflatten(2, (nh, G)).permute(0, 2, 1, 3, 4)
    z = q.reshape(B, nh, new * G, TILE) @ k.transpose(2, 3) * s["scale"]
    if case["cap"] > 0:
        z = case["cap"] * torch.tanh(z / case["cap"])
    t = torch.arange(T, device="cuda")
    last = lengths[:, None] - new + torch.arange(new, device="cuda")      # last visible token
    seen = (t <= last[:, :, None])[:, None, :, None]                      # [B][1][new][1][T]
    z = z.unflatten(2, (new, G)).masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp_min(1e-38)
    out = (p.reshape(B, nh, new * G, T) @ v).unflatten(2, (new, G))
    out = out.permute(0, 2, 1, 3, 4).reshape(B, new, Hq, TILE).to(DTYPES[case["out"]])
    lse = (torch.log(total) + top).squeeze(-1).permute(0, 2, 1, 3).reshape(B, new, Hq)
    if s["mass"] is None:
        return [out, lse]
    live = (t < lengths[:, None])[:, None]
    return [out, lse, torch.where(live, s["mass"] + p.sum((2, 3)), torch.zeros_like(s["mass"]))]


def _evict_plain(s, table, diag, had):
    case, P = s["case"], s["case"]["page"]
    mass, n = s["mass"], s["lengths"].to(torch.int64)[:, None, None]
    budget, recent = case["budget"], case["recent"]
    t = torch.arange(mass.shape[2], device="cuda")
    # the recent tokens first, then by mass, then those behind the end; ties to the lower index
    key = torch.where(t >= n, -math.inf, torch.where(t >= n - recent, math.inf, mass))
    order = torch.argsort(key, dim=-1, descending=True, stable=True)[..., :budget]
    short = budget - order.shape[-1]
    new = n.clamp_max(budget)
    i = torch.arange(order.shape[-1], device="cuda")
    big = mass.shape[2]
    kept = torch.sort(torch.where(i < new, order, big), dim=-1).values
    live = kept < big
    new_mass = torch.zeros_like(s["new_mass"])
    m = torch.where(live, torch.gather(mass, 2, kept.clamp_max(big - 1)), 0.0)
    new_mass[..., :m.shape[-1]] = m[..., :new_mass.shape[-1]]
    # the kept rows as values, token by token and head by head
    seq, pos = s["seq"].to(torch.int64), s["pos"].to(torch.int64)
    src = kept[seq, :, pos]                                               # [n][heads]
    h = torch.arange(case["heads"], device="cuda")
    page, unit, tok = table[seq[:, None], src // P], (src % P) // UNIT, src % UNIT
    K, V, S = _views(s["pages"])
    k = (_unpack(K[page, h, unit, tok]) - 7.5) * S[page, h, unit, tok][..., None]
    v = _unpack(V[page, h, unit, tok // 2, :, tok % 2].flatten(-2))
    v = (v - 7.5) * S[page, h, unit, UNIT + tok][..., None]
    kept = torch.nn.functional.pad(torch.where(live, kept, -1), (0, short), value=-1)
    return [kept.to(torch.int32), new.flatten().to(torch.int32), new_mass,
            *[((x @ had) * diag).to(torch.bfloat16) for x in (k, v)]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    nh, lens = case["heads"], _lengths(case)
    row = UNIT_BYTES // UNIT                                   # one token and head, K and V
    size = {"bf16": 2, "f16": 2, "f32": 4}
    fwht = 2 * 2 * 7 * TILE                                    # of K and V, in and out alike
    if case["op"] == "append":
        n = sum(lens) - case["past"] * case["batch"]
        b = n * nh * (2 * TILE * size[case["dtype"]] + row + row + 2 * TILE * 2) + n * 8
        return {"bytes": b, "flops": n * nh * 2 * fwht}
    if case["op"] == "read":
        n = sum(lens)
        return {"bytes": n * nh * (row + 2 * TILE * size[case["dtype"]]) + n * 8,
                "flops": n * nh * fwht}
    n = sum(lens)
    if case["op"] == "attend":
        q = case["batch"] * case["new"] * nh * case["group"]
        b = n * nh * (row + (8 if case["mass"] else 0))
        b += q * (TILE * (size[case["dtype"]] + size[case["out"]]) + 4)
        return {"bytes": b, "flops": 4 * TILE * n * nh * case["group"] * case["new"]}
    m = sum(min(x, case["budget"]) for x in lens)
    b = n * nh * 4 + m * nh * (4 + 4 + 2 * row) + m * nh * (row + 2 * TILE * 2)
    return {"bytes": b, "flops": m * nh * fwht}


# ------------------------------------------------------------------ the definition in 64 bits
def _sylvester64():
    h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while h.shape[0] < TILE:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _signs64(signs):
    words = [int(w) & 0xFFFFFFFF for w in signs.tolist()]
    return torch.tensor([-1.0 if words[i >> 5] >> (i & 31) & 1 else 1.0 for i in range(TILE)],
                        dtype=torch.float64, device="cuda")


def _decode64(flat, page, head, pos, P, nh, which, d64):
    """Values of K (0) or V (1) rows by the byte addresses of their codes, in 64 bits; page, head
    and pos are int64 tensors of one shape."""
    base = ((page * nh + head) * (P // UNIT) + (pos % P) // UNIT) * UNIT_BYTES
    t, d = (pos % UNIT)[..., None], torch.arange(TILE, device="cuda")
    byte = t * 64 + d // 2
    if which:
        byte = 1024 + (t // 2) * 128 + (d // 16) * 16 + (t % 2) * 8 + (d % 16) // 2
    code = (flat[base[..., None] + byte].to(torch.int64) >> (4 * (d % 2))) & 15
    at = base + 2048 + which * 32 + (pos % UNIT) * 2
    bits = flat[at].to(torch.int32) | (flat[at + 1].to(torch.int32) << 8)
    s = (bits << 16).view(torch.float32).to(torch.float64)
    y = (code.to(torch.float64) - 7.5) * s[..., None]
    return (y @ _sylvester64()) * d64 / math.sqrt(128.0)


def exact(case, seed):
    if case["op"] == "attend" and sum(_lengths(case)) * case["heads"] > 6_000_000:
        return None
    s = prepare(case, seed)
    nh, P, lens = case["heads"], case["page"], s["lens"]
    d64, flat = _signs64(s["signs"]), s["pages"].flatten()
    table = s["table"].to(torch.int64)
    heads = torch.arange(nh, device="cuda")
    if case["op"] == "append":
        found = []
        for x in (s["k"], s["v"]):
            y = (x.to(torch.float64) * d64) @ _sylvester64() / math.sqrt(128.0)
            sc = (y.abs().amax(-1, keepdim=True) / 7.5).to(torch.bfloat16).to(torch.float64)
            c = torch.floor(y / sc + 8.0).clamp(0, 15)
            found.append((((c - 7.5) * sc) @ _sylvester64()) * d64 / math.sqrt(128.0))
        return found
    if case["op"] == "read":
        seq, pos = s["seq"].to(torch.int64), s["pos"].to(torch.int64)
        page = table[seq, pos // P][:, None].expand(-1, nh)
        where = (page, heads.expand_as(page), pos[:, None].expand_as(page))
        return [_decode64(flat, *where, P, nh, w, d64) for w in (0, 1)]
    if case["op"] == "attend":
        return _attend64(s, flat, table, d64)
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int64)
    new_mass = torch.zeros(s["new_mass"].shape, dtype=torch.float64)
    mass = s["mass"].double().cpu()
    for b, n in enumerate(lens):
        old = max(0, n - case["recent"])
        for h in range(nh):
            m = mass[b, h, :old].numpy()
            best = (-m).argsort(kind="stable")[:max(0, min(n, case["budget"]) - (n - old))]
            keep = torch.cat([torch.from_numpy(best), torch.arange(old, n)]).sort().values
            kept[b, h, :len(keep)] = keep
            new_mass[b, h, :len(keep)] = mass[b, h, keep]
    seq, pos = s["seq"].to(torch.int64), s["pos"].to(torch.int64)
    src = kept.cuda()[seq, :, pos]
    page = table[seq[:, None], src // P]
    rows = [_decode64(flat, page, heads.expand_as(page), src, P, nh, w, d64) for w in (0, 1)]
    return [None, None, new_mass.cuda(), *rows]


def _attend64(s, flat, table, d64):
    case, nh, P = s["case"], s["case"]["heads"], s["case"]["page"]
    B, new, Hq, _ = s["q"].shape
    G = Hq // nh
    out = torch.zeros((B, new, Hq, TILE), dtype=torch.float64, device="cuda")
    lse = torch.full((B, new, Hq), -math.inf, dtype=torch.float64, device="cuda")
    mass = None if s["mass"] is None else torch.zeros(s["mass"].shape, dtype=torch.float64,
                                                      device="cuda")
    for b, n in enumerate(s["lens"]):
        pos = torch.arange(n, device="cuda")
        page = table[b, pos // P]
        for h in range(nh):
            head = torch.full_like(pos, h)
            k = _decode64(flat, page, head, pos, P, nh, 0, d64)
            v = _decode64(flat, page, head, pos, P, nh, 1, d64)
            add = torch.zeros(n, dtype=torch.float64, device="cuda")
            for j in range(max(0, new - n), new):
                m = n - new + j + 1
                z = s["q"][b, j, h * G:(h + 1) * G].to(torch.float64) @ k[:m].T * s["scale"]
                if case["cap"] > 0:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                out[b, j, h * G:(h + 1) * G] = p @ v[:m]
                add[:m] += p.sum(0)
            if mass is not None:
                mass[b, h, :n] = s["mass"][b, h, :n].double() + add
    return [out, lse] if mass is None else [out, lse, mass]
