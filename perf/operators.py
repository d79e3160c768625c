"""KV-cache compression for decode: cases, plain forms and 64-bit definitions of

* ``kv4_write`` / ``kv4_read``: k-hat and v rows into a paged cache held in 4 bits, and back;
* ``decode_kv4`` / ``decode_append_kv4``: decode attention over such a cache;
* ``decode(..., weights=)`` and its paged and append forms: decode that also accumulates, per cached
  row and KV head, the attention weight the row received;
* ``kv_evict`` / ``kv_evict_paged`` / ``kv4_evict``: eviction down to a budget of rows by that weight.

The 4-bit format.  A group is 32 consecutive elements of one head vector.  Its scale s is max|x| / 7
rounded to an unsigned 8-bit float (5 exponent bits, bias 15, 3 mantissa bits; the byte shifted left by
7 is the same number in fp16), at most 7680; an element is c = clamp(round(x / s), -7, 7), stored as
c + 8.  A record of 2176 bytes holds 16 consecutive rows of one KV head:
  bytes    0..1023  K codes: element 16 s + 4 t + 2 n + o of row r in byte 64 r + 16 t + 4 (s / 2) + 2 o + s % 2, nibble n
  bytes 1024..2047  V codes: element 16 g + 2 b + n of row r in byte 512 (r / 8) + 64 g + 16 (r % 8 / 2) + 8 (r % 2) + b, nibble n
  bytes 2048..2111  K scales [row][group]       bytes 2112..2175  V scales [group][row]
and the cache is uint8 [num_pages, Hkv, page_size / 16, 2176].
"""
import math
import random

import torch

own = False

D = 128
GROUP = 32
RECORD = 2176
DEV = "cuda"
THETA = 1.0e6
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a batch of prompts of mixed lengths after their prefill: k-hat and v go into the cache (some already hold rows)
        dict(name="write_prompts_16", op="write", B=16, lo=256, hi=8192, prefix=100, Hkv=8, page=64, len_seed=1),
        # one short prompt, small pages, ending inside a page
        dict(name="write_short", op="write", B=1, lo=37, hi=37, prefix=21, Hkv=2, page=16, len_seed=2),
        # one user, a short conversation: latency
        dict(name="kv4_decode_one_user", op="kv4", B=1, lo=1000, hi=1000, H=32, Hkv=8, page=64, append=False,
             weights=False, pairing="adjacent", len_seed=3),
        # the repository's batched decode, 64 sequences of 1K to 32K rows
        dict(name="kv4_decode_batch_64", op="kv4", B=64, lo=1024, hi=32768, H=32, Hkv=8, page=64, append=False,
             weights=False, pairing="adjacent", len_seed=4),
        # one long context with 8 query heads a KV head: work has to be split along the rows
        dict(name="kv4_decode_long", op="kv4", B=1, lo=32768, hi=32768, H=64, Hkv=8, page=128, append=False,
             weights=False, pairing="adjacent", len_seed=5),
        # a decode step of young sequences (one may be empty), small pages, rotate-half RoPE
        dict(name="kv4_append_young", op="kv4", B=16, lo=0, hi=4096, H=16, Hkv=8, page=16, append=True, weights=False,
             pairing="half", len_seed=6),
        # a decode step that also accumulates the weights an eviction goes by
        dict(name="kv4_append_weights", op="kv4", B=32, lo=1023, hi=8191, H=32, Hkv=8, page=64, append=True, weights=True,
             pairing="adjacent", len_seed=7),
        # the same accumulation on a bf16 cache, contiguous
        dict(name="weights_batch_32", op="bf16", B=32, lo=1024, hi=16384, H=32, Hkv=8, page=0, append=False,
             pairing="adjacent", len_seed=8),
        # ... and on a paged one, few short sequences, one KV head for 16 query heads, with the append
        dict(name="weights_paged_short", op="bf16", B=4, lo=1, hi=700, H=16, Hkv=1, page=16, append=True,
             pairing="adjacent", len_seed=9),
        # prompts cut down to a budget after their prefill
        dict(name="evict_prompts_16", op="evict", kind="rows", B=16, lo=2048, hi=8192, Hkv=8, page=0, budget=1024,
             recent=128, shuffled=False, len_seed=10),
        # the serving loop: every few steps the rows over the budget go
        dict(name="evict_steady_64", op="evict", kind="pages", B=64, lo=2049, hi=2080, Hkv=8, page=64, budget=2048,
             recent=256, shuffled=True, len_seed=11),
        # long contexts in 4 bits cut down to 4096 rows
        dict(name="kv4_evict_long", op="evict", kind="kv4", B=4, lo=8192, hi=32768, Hkv=8, page=64, budget=4096,
             recent=512, shuffled=False, len_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "kv4", "kv4", "bf16", "evict"])
    B = _log(rng, 1, 64)
    top = max(16, min(32768, (1 << 19) // B))     # rows of the longest sequence: at most 2^19 in all
    hi = _log(rng, 16, top)
    lo = rng.randint(1, hi)
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, B=B, lo=lo, hi=hi, Hkv=Hkv, page=rng.choice([16, 32, 48, 64, 128, 256]), len_seed=rng.randrange(1 << 20))
    if op == "write":
        return dict(c, prefix=rng.choice([0, 1, 50, 1000]))
    if op == "evict":
        budget = rng.randint(1, hi)
        return dict(c, kind=rng.choice(["rows", "pages", "kv4"]), budget=budget, recent=rng.randint(0, budget),
                    shuffled=rng.random() < 0.5)
    c = dict(c, H=Hkv * rng.choice([h for h in (1, 2, 3, 4, 5, 8, 16) if h * Hkv <= 64]), append=rng.random() < 0.5,
             pairing=rng.choice(["adjacent", "half"]))
    if op == "kv4":
        return dict(c, weights=rng.random() < 0.5)
    return dict(c, page=rng.choice([0, c["page"]]))


def _lens(case):
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _prefix(case):
    r = random.Random(case["len_seed"] + 1)
    return [r.randint(0, case["prefix"]) for _ in range(case["B"])]


def work(case):
    n, kv = _lens(case), case["Hkv"]
    rows = sum(n)
    if case["op"] == "write":     # read k-hat and v in bf16, write 4-bit rows, return their values
        return dict(bytes=rows * kv * (512 + 136 + 512), flops=0)
    if case["op"] == "evict":
        m, rec, moved, meta = case["budget"], case["recent"], 0.0, 0
        for x in n:
            if x > m:
                free = max(1, x - rec)
                late = min(rec, x - m)                      # recent rows behind the budget, unless rows are shuffled
                part = m * (x - m) / x if case["shuffled"] else late + (m - rec) * (x - m - late) / free
                moved += max(0.0, part)
            meta += 8 * x + 8 * min(x, m)
        row = 272 if case["kind"] == "kv4" else 1024        # read and written
        back = sum(min(x, m) for x in n) * (136 + 512) if case["kind"] == "kv4" else 0
        return dict(bytes=kv * (moved * row + meta + back), flops=0)
    add = 1 if case["append"] else 0
    att = rows + add * case["B"]
    row = 136 if case["op"] == "kv4" else 512
    acc = 8 if case["op"] == "bf16" or case["weights"] else 0
    return dict(bytes=att * kv * (row + acc) + case["B"] * case["H"] * D * 6, flops=4 * D * case["H"] * att)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def _offsets(n):
    o = [0]
    for x in n:
        o.append(o[-1] + x)
    return _i64(o)


def _table(rows, page, g):
    """Pages handed out in random order: table [B, max_pages] (-1 behind a sequence's pages), and their number."""
    need = [(x + page - 1) // page for x in rows]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = _i64([sum(need[:b]) for b in range(len(need))])
    col = torch.arange(max(1, max(need)), device=DEV)
    at = (first[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(col[None] < _i64(need)[:, None], order[at], -1).to(torch.int32).contiguous(), total


def _bytes(num, Hkv, page, g):
    """A 4-bit cache of N(0, 1) rows, filled through the format's definition, some records at a time."""
    records = num * Hkv * (page // 16)
    out = torch.empty((records, RECORD), dtype=torch.uint8, device=DEV)
    step = 1 << 16
    for i in range(0, records, step):
        m = min(step, records - i)
        k, ks = _codes(_normal((m, 16, D), g))
        v, vs = _codes(_normal((m, 16, D), g))
        out[i:i + m] = _records(k, ks, v, vs)
    return out.view(num, Hkv, page // 16, RECORD)


def prepare(case, seed):
    g = _gen(seed)
    n, B, Hkv = _lens(case), case["B"], case["Hkv"]
    s = dict(case=case, n=n, seqlens=_i32(n))
    if case["op"] == "write":
        pre = _prefix(case)
        s["table"], num = _table([p + x for p, x in zip(pre, n)], case["page"], g)
        s.update(k=_normal((sum(n), Hkv, D), g), v=_normal((sum(n), Hkv, D), g), cu=_offsets(n), prefix=_i32(pre),
                 pages=torch.zeros((num, Hkv, case["page"] // 16, RECORD), dtype=torch.uint8, device=DEV), rows=sum(n))
        return s
    if case["op"] == "evict":
        wide = max(n) + 5
        w = torch.exp(1.5 * torch.randn((B, Hkv, wide), generator=g, device=DEV))
        w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.05, 0.0, w)       # rows never looked at: ties
        pos = torch.arange(wide, dtype=torch.int32, device=DEV).expand(B, Hkv, wide)
        if case["shuffled"]:       # earlier evictions have mixed the rows of a sequence
            inside = torch.arange(wide, device=DEV) < s["seqlens"][:, None, None]
            order = torch.where(inside, torch.rand(w.shape, generator=g, device=DEV), 2.0)
            pos = torch.argsort(order, dim=-1).to(torch.int32)
        s.update(w=w.contiguous(), pos=pos.contiguous(), new_w=torch.zeros_like(w), new_pos=torch.zeros_like(w, dtype=torch.int32),
                 max_len=max(n))
        if case["kind"] == "rows":
            s.update(k=_normal((sum(n), Hkv, D), g), v=_normal((sum(n), Hkv, D), g), offsets=_offsets(n))
            return s
        s["table"], num = _table(n, case["page"], g)
        if case["kind"] == "pages":
            s.update(k=_normal((num, case["page"], Hkv, D), g), v=_normal((num, case["page"], Hkv, D), g))
            return s
        left = [min(x, case["budget"]) for x in n]
        s.update(pages=_bytes(num, Hkv, case["page"], g), cu=_offsets(left), zero=_i32([0] * B), rows=sum(left))
        return s
    add = 1 if case["append"] else 0
    s.update(q=_normal((B, case["H"], D), g), wq=torch.rand(D, generator=g, device=DEV) + 0.5,
             wk=torch.rand(D, generator=g, device=DEV) + 0.5, max_len=max(1, max(n) + add))
    if add:
        s.update(k_new=_normal((B, Hkv, D), g), v_new=_normal((B, Hkv, D), g))
    if case["op"] == "bf16" or case["weights"]:
        s["w"] = torch.rand((B, Hkv, s["max_len"] + 3), generator=g, device=DEV)
        s["pos"] = torch.zeros((B, Hkv, s["max_len"] + 3), dtype=torch.int32, device=DEV)
    full = [x + add for x in n]
    if case["page"]:
        s["table"], num = _table(full, case["page"], g)
    if case["op"] == "kv4":
        s.update(pages=_bytes(num, Hkv, case["page"], g), each=_i64(list(range(B + 1))))
    elif case["page"]:
        s.update(k=_normal((num, case["page"], Hkv, D), g), v=_normal((num, case["page"], Hkv, D), g))
    else:
        s.update(k=_normal((sum(full), Hkv, D), g), v=_normal((sum(full), Hkv, D), g), offsets=_offsets(full))
    return s


# ------------------------------------------------------------------ the 4-bit format, plain
def _codes(x):
    """x [..., 128] -> c + 8 [..., 128] and scale bytes [..., 4], uint8."""
    x = x.float().unflatten(-1, (4, GROUP))
    a = x.abs().amax(-1)
    a = a / torch.full_like(a, 7.0)                                     # a division: times 1 / 7 would move what lies on a border
    low = torch.round(a * 2.0 ** 17)                                     # below 2^-14: steps of 2^-17
    man, ex = torch.frexp(a)                                            # a = man 2^ex, man in [0.5, 1)
    eighth = torch.round(man * 16.0)                                    # 8 .. 16 eighths of 2^(ex - 1)
    high = (ex - 1 + 15) * 8 + eighth - 8
    byte = torch.where(a < 2.0 ** -14, low, high).clamp(max=223).to(torch.uint8)
    s = _scale(byte)[..., None]
    c = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)), 0.0).clamp(-7, 7) + 8
    return c.flatten(-2).to(torch.uint8), byte


def _scale(byte):
    return (byte.to(torch.int16) << 7).view(torch.float16).float()


def _records(k, ks, v, vs):
    """Codes [m, 16, 128] and scale bytes [m, 16, 4] -> records [m, 2176]."""
    m = k.shape[0]
    k = k.view(m, 16, 4, 2, 4, 2, 2).permute(0, 1, 4, 2, 6, 3, 5)       # row, t, s/2, o, s%2, n
    v = v.view(m, 2, 4, 2, 8, 8, 2).permute(0, 1, 4, 2, 3, 5, 6)        # row/8, g, row%8/2, row%2, b, n
    parts = [(x[..., 0] | (x[..., 1] << 4)).reshape(m, 1024) for x in (k, v)]
    return torch.cat(parts + [ks.reshape(m, 64), vs.transpose(1, 2).reshape(m, 64)], 1)


def _values(rec):
    """Records [..., 2176] -> K and V [..., 16, 128] in fp32."""
    lead = rec.shape[:-1]
    rec = rec.reshape(-1, RECORD)
    m = rec.shape[0]
    both = torch.stack([rec[:, :2048] & 15, rec[:, :2048] >> 4], -1)
    k = both[:, :1024].reshape(m, 16, 4, 4, 2, 2, 2).permute(0, 1, 3, 5, 2, 6, 4).reshape(m, 16, D)
    v = both[:, 1024:].reshape(m, 2, 8, 4, 2, 8, 2).permute(0, 1, 3, 4, 2, 5, 6).reshape(m, 16, D)
    ks = _scale(rec[:, 2048:2112]).view(m, 16, 4)
    vs = _scale(rec[:, 2112:]).view(m, 4, 16).transpose(1, 2)
    k, v = ((c.float() - 8.0).unflatten(-1, (4, GROUP)) * s[..., None] for c, s in ((k, ks), (v, vs)))
    return k.reshape(*lead, 16, D), v.reshape(*lead, 16, D)


def _rows4(pages, table):
    """K and V [B, Hkv, rows, 128] behind a page table, fp32."""
    B, Hkv = table.shape[0], pages.shape[1]
    rec = pages[table.clamp(min=0).long()].transpose(1, 2)              # [B, Hkv, max_pages, records, 2176]
    k, v = _values(rec)
    return k.reshape(B, Hkv, -1, D), v.reshape(B, Hkv, -1, D)


# ------------------------------------------------------------------ attention, plain
def _rotate(x, pos, pairing):
    """RoPE of x [B, heads, 128] at pos [B], in x's own precision; the angles in 64 bits."""
    i = torch.arange(D // 2, dtype=torch.float64, device=DEV)
    a = pos.double()[:, None] * THETA ** (-2.0 * i / D)
    c, s = torch.cos(a).to(x.dtype)[:, None], torch.sin(a).to(x.dtype)[:, None]
    if pairing == "half":
        u, w = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([u * c - w * s, u * s + w * c], -1)
    u, w = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - w * s, u * s + w * c], -1).flatten(-2)


def _norm(x, w):
    return w * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _attend(s, k, v, n):
    """out [B, H, 128] and the weights of the rows, summed over the query heads of a group [B, Hkv, rows]."""
    B, Hkv = k.shape[0], k.shape[1]
    q = _rotate(_norm(s["q"].float(), s["wq"]), s["seqlens"], s["case"]["pairing"])
    q = q.reshape(B, Hkv, -1, D) / math.sqrt(D)
    sees = torch.arange(k.shape[2], device=DEV) < n[:, None]
    x = torch.matmul(q, k.transpose(-1, -2))
    x = x.masked_fill(~sees[:, None, None], float("-inf"))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    out = torch.matmul(p, v.masked_fill(~sees[:, None, :, None], 0.0))
    return out.reshape(B, -1, D), p.sum(2)


def _new_key(s):
    """k-hat of the appended token in bf16: evaluated in 64 bits, since a quantiser's border may be next to it."""
    k = _rotate(_norm(s["k_new"].double(), s["wk"].double()), s["seqlens"], s["case"]["pairing"])
    return k.to(torch.bfloat16)


def _accumulate(s, got, n):
    w, rows = s["w"], min(got.shape[2], s["w"].shape[2])
    b = torch.arange(w.shape[0], device=DEV)
    if s["case"]["append"]:        # the new row's weight starts from zero, and it gets its position
        w[b, :, s["seqlens"].long()] = 0.0
        s["pos"][b, :, s["seqlens"].long()] = s["seqlens"][:, None].expand(-1, w.shape[1])
    w[..., :rows] += got[..., :rows]


def _plain_kv4(s):
    n = s["seqlens"] + (1 if s["case"]["append"] else 0)
    k, v = _rows4(s["pages"], s["table"])
    out = {}
    if s["case"]["append"]:
        b = torch.arange(len(s["n"]), device=DEV)
        for name, rows, new in (("k_row", k, _new_key(s)), ("v_row", v, s["v_new"])):
            c, byte = _codes(new)
            val = ((c.float() - 8.0).unflatten(-1, (4, GROUP)) * _scale(byte)[..., None]).flatten(-2)
            rows[b, :, s["seqlens"].long()] = val
            out[name] = val.to(torch.bfloat16)
    out["out"], got = _attend(s, k, v, n)
    if s["case"]["weights"]:
        _accumulate(s, got, n)
        out["weights"] = s["w"]
        if s["case"]["append"]:
            out["row_pos"] = s["pos"]
    return out


def _row_index(s):
    """Where row r of sequence b lies in the flat rows [rows, Hkv, 128] of a bf16 cache: [B, rows]."""
    if s["case"]["page"]:
        page = s["case"]["page"]
        r = torch.arange(s["table"].shape[1] * page, device=DEV)
        return s["table"].clamp(min=0).long()[:, r // page] * page + r % page
    r = torch.arange(max(1, s["max_len"]), device=DEV)
    return (s["offsets"][:-1, None] + r[None]).clamp(max=s["k"].shape[0] - 1)


def _plain_bf16(s):
    n = s["seqlens"] + (1 if s["case"]["append"] else 0)
    at = _row_index(s)
    kf, vf = s["k"].view(-1, *s["k"].shape[-2:]), s["v"].view(-1, *s["v"].shape[-2:])
    if s["case"]["append"]:
        b = torch.arange(len(s["n"]), device=DEV)
        new = at[b, s["seqlens"].long()]
        kf[new] = _new_key(s)
        vf[new] = s["v_new"]
    k, v = (x[at].transpose(1, 2).float() for x in (kf, vf))
    out, got = _attend(s, k, v, n)
    _accumulate(s, got, n)
    res = dict(out=out, weights=s["w"])
    if s["case"]["append"]:
        res["row_pos"] = s["pos"]
    return res


def _plain_write(s):
    res = {}
    for name in ("k", "v"):
        c, byte = _codes(s[name])
        res[name] = ((c.float() - 8.0).unflatten(-1, (4, GROUP)) * _scale(byte)[..., None]).flatten(-2).to(torch.bfloat16)
    return res


def _moves(s):
    """For every (sequence, head): which row of the budget takes which row [B, Hkv, budget] (itself where it stays)."""
    m, n = min(s["case"]["budget"], s["max_len"]), s["seqlens"].long()[:, None, None]
    w, pos = s["w"][..., :s["max_len"]], s["pos"][..., :s["max_len"]]
    r = torch.arange(w.shape[-1], device=DEV)
    valid = r < n
    last = torch.where(valid, pos, -2 ** 31).amax(-1, keepdim=True).long()
    key = torch.where(pos.long() > last - s["case"]["recent"], float("inf"), w).masked_fill(~valid, -1.0)
    order = torch.argsort(key, dim=-1, descending=True, stable=True)     # ties: the lowest row first
    rank = torch.empty_like(order).scatter_(-1, order, r.expand_as(order).contiguous())
    keep = valid & (rank < s["case"]["budget"])
    hole, mover = valid[..., :m] & ~keep[..., :m], keep[..., m:]
    at = torch.full(w.shape[:2] + (m + 1,), 0, dtype=torch.int64, device=DEV)
    nth = torch.where(mover, mover.cumsum(-1) - 1, m)                     # the i-th kept row behind the budget ...
    at.scatter_(-1, nth, (r[m:]).expand_as(nth).contiguous())
    src = torch.gather(at, -1, (hole.cumsum(-1) - 1).clamp(min=0))       # ... goes to the i-th free row
    return torch.where(hole, src, r[:m].expand_as(src))


def _plain_evict(s):
    c = s["case"]
    n = s["seqlens"].long()
    left = n.clamp(max=c["budget"])
    src = _moves(s)
    m = src.shape[-1]
    inside = torch.arange(m, device=DEV) < left[:, None, None]
    for new, old in (("new_w", "w"), ("new_pos", "pos")):
        s[new][..., :m] = torch.where(inside, torch.gather(s[old], -1, src), s[new][..., :m])
    res = dict(new_weights=s["new_w"], new_row_pos=s["new_pos"], new_seqlens=left.to(torch.int32))
    b, g, r = torch.where(inside & (src != torch.arange(m, device=DEV)))
    old = src[b, g, r]
    if c["kind"] == "kv4":
        page = c["page"]
        def place(x):
            return s["table"].long()[b, x // page], g, x % page // 16, x % 16
        def bytes_of(x):
            j = torch.arange(64, device=DEV)
            q = torch.arange(4, device=DEV)
            return [64 * x[:, None] + j, 1024 + 512 * (x // 8)[:, None] + 64 * (j // 8) + 16 * (x % 8 // 2)[:, None] + 8 * (x % 2)[:, None] + j % 8,
                    2048 + 4 * x[:, None] + q, 2112 + 16 * q + x[:, None]]
        pf, gf, rf, xf = place(old)
        pt, gt, rt, xt = place(r)
        f, t = torch.cat(bytes_of(xf), 1), torch.cat(bytes_of(xt), 1)
        s["pages"][pt[:, None], gt[:, None], rt[:, None], t] = s["pages"][pf[:, None], gf[:, None], rf[:, None], f]
        k, v = _rows4(s["pages"], s["table"][:, :(m + page - 1) // page])
        take = torch.arange(k.shape[2], device=DEV) < left[:, None]
        res.update(k=k.transpose(1, 2)[take].to(torch.bfloat16), v=v.transpose(1, 2)[take].to(torch.bfloat16))
        return res
    at = _row_index(s)
    for name in ("k", "v"):
        flat = s[name].view(-1, *s[name].shape[-2:])
        flat[at[b, r], g] = flat[at[b, old], g]
        res[name] = s[name]
    return res


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"write": _plain_write, "kv4": _plain_kv4, "bf16": _plain_bf16, "evict": _plain_evict}[c["op"]](s)
    from grouped_query_causal_b200 import binding
    if c["op"] == "write":
        binding.kv4_write(s["k"], s["v"], s["cu"], s["prefix"], s["pages"], s["table"])
        k, v = binding.kv4_read(s["pages"], s["table"], s["cu"], s["prefix"], s["rows"])
        return dict(k=k, v=v)
    if c["op"] == "evict":
        kw = dict(max_len=s["max_len"], recent=c["recent"], row_pos=s["pos"], new_weights=s["new_w"], new_row_pos=s["new_pos"])
        res = dict(new_weights=s["new_w"], new_row_pos=s["new_pos"])
        if c["kind"] == "rows":
            res["new_seqlens"] = binding.kv_evict(s["k"], s["v"], s["offsets"], s["seqlens"], s["w"], c["budget"], **kw)
        elif c["kind"] == "pages":
            res["new_seqlens"] = binding.kv_evict_paged(s["k"], s["v"], s["table"], s["seqlens"], s["w"], c["budget"], **kw)
        else:
            res["new_seqlens"] = binding.kv4_evict(s["pages"], s["table"], s["seqlens"], s["w"], c["budget"], **kw)
            res["k"], res["v"] = binding.kv4_read(s["pages"], s["table"], s["cu"], s["zero"], s["rows"])
            return res
        return dict(res, k=s["k"], v=s["v"])
    rope = binding.RopeConfig.make(theta=THETA, pairing=c["pairing"])
    kw = dict(max_len=s["max_len"], rope=rope, eps=EPS)
    res = {}
    if c["op"] == "kv4":
        if c["weights"]:
            kw["weights"] = res["weights"] = s["w"]
        if not c["append"]:
            res["out"] = binding.decode_kv4(s["q"], s["pages"], s["table"], s["seqlens"], s["wq"], **kw)
            return res
        if c["weights"]:
            kw["row_pos"] = res["row_pos"] = s["pos"]
        res["out"] = binding.decode_append_kv4(s["q"], s["k_new"], s["v_new"], s["pages"], s["table"], s["seqlens"],
                                               s["wq"], s["wk"], **kw)
        k, v = binding.kv4_read(s["pages"], s["table"], s["each"], s["seqlens"], len(s["n"]))
        return dict(res, k_row=k, v_row=v)
    kw["weights"] = res["weights"] = s["w"]
    if c["append"]:
        kw["row_pos"] = res["row_pos"] = s["pos"]
        new = (s["q"], s["k_new"], s["v_new"], s["k"], s["v"])
        if c["page"]:
            res["out"] = binding.decode_append_paged(*new, s["table"], s["seqlens"], s["wq"], s["wk"], **kw)
        else:
            res["out"] = binding.decode_append(*new, s["offsets"], s["seqlens"], s["wq"], s["wk"], **kw)
    elif c["page"]:
        res["out"] = binding.decode_paged(s["q"], s["k"], s["v"], s["table"], s["seqlens"], s["wq"], **kw)
    else:
        res["out"] = binding.decode(s["q"], s["k"], s["v"], s["offsets"], s["seqlens"], s["wq"], **kw)
    return res


# ------------------------------------------------------------------ the definitions in 64 bits, sequence by sequence
_SCALES = [(m / 8.0) * 2.0 ** -14 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 15) for e in range(28) for m in range(8)]


def _exact_quant(x):
    """The value of every element of x [..., 128] (fp64) in the format: the nearest scale of the table, the even one
    of two that are as near, then the nearest multiple."""
    t = torch.tensor(_SCALES, dtype=torch.float64, device=DEV)
    y = x.reshape(-1, 4, 32)
    want, t7 = y.abs().max(dim=2).values, 7 * t           # 7 s is compared, which is exact
    up = torch.searchsorted(t7, want.contiguous()).clamp(1, len(_SCALES) - 1)
    above, below = t7[up] - want, want - t7[up - 1]
    i = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    i = torch.where(want >= t7[-1], len(_SCALES) - 1, i)
    sc = t[i][:, :, None]
    q = torch.where(sc > 0, y / sc.clamp(min=1e-30), 0.0)
    return (torch.round(q).clamp(-7, 7) * sc).reshape(x.shape)


def _exact_rope(x, pos, pairing):
    y = torch.empty_like(x)
    for i in range(64):
        a = float(pos) * THETA ** (-i / 64.0)
        co, si = math.cos(a), math.sin(a)
        lo, hi = (i, i + 64) if pairing == "half" else (2 * i, 2 * i + 1)
        y[:, lo] = x[:, lo] * co - x[:, hi] * si
        y[:, hi] = x[:, lo] * si + x[:, hi] * co
    return y


def _exact_hat(x, w, pos, pairing):
    x = x.double()
    return _exact_rope(x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w.double(), pos, pairing)


def _exact_rows(s, b, n):
    """K and V of the first n rows of sequence b, [n, Hkv, 128] fp64, from the cache's bytes."""
    c = s["case"]
    if c["op"] == "bf16":
        r = torch.arange(n, device=DEV)
        if c["page"]:
            at = (s["table"][b].long()[r // c["page"]], r % c["page"])
            return s["k"][at].double(), s["v"][at].double()
        o = int(s["offsets"][b])
        return s["k"][o:o + n].double(), s["v"][o:o + n].double()
    r = torch.arange(n, device=DEV)[:, None, None]
    g = torch.arange(c["Hkv"], device=DEV)[None, :, None]
    d = torch.arange(D, device=DEV)[None, None, :]
    rec = s["pages"][s["table"][b].long()[r // c["page"]], g, r % c["page"] // 16]      # [n, Hkv, 1, 2176]
    rec = rec.reshape(n, c["Hkv"], RECORD)
    x = r % 16
    kb = 64 * x + 16 * (d % 16 // 4) + 4 * (d // 32) + 2 * (d % 2) + d // 16 % 2
    vb = 1024 + 512 * (x // 8) + 64 * (d // 16) + 16 * (x % 8 // 2) + 8 * (x % 2) + d % 16 // 2
    t = torch.tensor(_SCALES + [0.0] * (256 - len(_SCALES)), dtype=torch.float64, device=DEV)
    full = (n, c["Hkv"], D)
    out = []
    for byte, nib, sc in ((kb, d % 4 // 2, 2048 + 4 * x + d // 32), (vb, d % 2, 2112 + 16 * (d // 32) + x)):
        code = (torch.gather(rec, 2, byte.expand(full)).long() >> (4 * nib)) & 15
        out.append((code - 8).double() * t[torch.gather(rec, 2, sc.expand(full)).long()])
    return out[0], out[1]


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "write":
        return dict(k=_exact_quant(s["k"].double()), v=_exact_quant(s["v"].double()))
    if c["op"] == "evict":
        return None          # rows chosen and copied: nothing is computed
    outs, krow, vrow = [], [], []
    weights = s["w"].double() if "w" in s else None
    for b, n0 in enumerate(s["n"]):
        n = n0 + (1 if c["append"] else 0)
        k, v = _exact_rows(s, b, n)
        if c["append"]:
            kh = _exact_hat(s["k_new"][b], s["wk"], n0, c["pairing"]).to(torch.bfloat16).double()
            vh = s["v_new"][b].double()
            if c["op"] == "kv4":
                kh, vh = _exact_quant(kh), _exact_quant(vh)
            k[n0], v[n0] = kh, vh
            krow.append(kh)
            vrow.append(vh)
        q = _exact_hat(s["q"][b], s["wq"], n0, c["pairing"])
        h = c["H"] // c["Hkv"]
        if weights is not None and c["append"]:
            weights[b, :, n0] = 0
        heads = []
        for j in range(c["H"]):
            x = (k[:, j // h] @ q[j]) / math.sqrt(128.0)
            e = torch.exp(x - x.max())
            p = e / e.sum()
            heads.append(p @ v[:, j // h])
            if weights is not None:
                weights[b, j // h, :n] += p
        outs.append(torch.stack(heads))
    res = dict(out=torch.stack(outs))
    if weights is not None:
        res["weights"] = weights
        if c["append"]:
            res["row_pos"] = None
    if c["append"] and c["op"] == "kv4":
        res.update(k_row=torch.stack(krow), v_row=torch.stack(vrow))
    return res
