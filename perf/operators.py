"""The rollout and clipping operators as measured cases, each with its plain form.

* ``append``: new keys and values into a paged cache of 8-bit values with one
  scale per block of 64 tokens and head, and the blocks that it wrote read back.
* ``attention``: grouped-head attention of the newest rows of each sequence
  over such a cache.
* ``clip``: the gradient norm of each adapter over its tensors, and clipping.

The plain forms are elementary torch operations in 32 bits.  With ``own`` the
cases call rl_step_gb300.kv and rl_step_gb300.grads instead.

The cache.  A page holds the keys and the values of 64 consecutive tokens of
one sequence: uint8 k, v [n_pages, n_kv, 64, hd] of e4m3 bytes and fp32 scales
[n_pages, n_kv], powers of two.  Inside a (page, head) tile byte order is
  k: token j, dim c at  j hd + ((c // 16) ^ s) 16 + c % 16, s = 4 (j % 2) at hd = 128, else 0
  v: token j, dim c at  (j // 4) 4 hd + ((c // 4) ^ (2 (j // 4 % 4))) 16 + 4 (c % 4) + j % 4
Row i of a sequence's n rows sits at position kv_len - n + i.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # the small transformer workload's heads (4 / 2 of 128), one token for each of 3 sequences: launch latency
        _attn("attn_small", 3, 4, 2, 128, 21, 299),
        # the 8B widths' heads (32 / 8 of 128) with one user and a long context: split over the cache
        _attn("attn_one_long", 1, 32, 8, 128, 130001, 130001),
        # a rollout step at the 8B widths: 256 sequences of the workload's 512 to 2048 tokens
        _attn("attn_rollout", 256, 32, 8, 128, 512, 2048),
        # four drafted tokens a sequence, checked at once
        _attn("attn_draft", 32, 32, 8, 128, 1023, 8191, rows=4),
        # one key/value head for each query head, 64 wide, fp32 queries, some slots of the batch empty
        _attn("attn_fp32", 41, 16, 16, 64, 0, 3001, dtype="fp32"),
        # the largest: long rollouts in a wide batch
        _attn("attn_wide_long", 64, 32, 8, 128, 4097, 32767),
        # one token a sequence into part-filled blocks, k and v read in place from a q|k|v buffer
        _append("append_step", 256, 8, 128, 1, 1, 2047, stride=32),
        # prompts of 512 to 2048 tokens, 65,536 tokens or less in all, behind a short prefix
        _append("append_prompts", 51, 8, 128, 512, 2048, 77, stride=32),
        # a few fp32 rows a sequence, odd sizes
        _append("append_fp32", 7, 3, 64, 1, 133, 500, dtype="fp32"),
        # the small transformer workload's largest adapter: 28 tensors, one group
        _clip("clip_small", 256, 512, 256, 2, 32, 1),
        # one rank-32 adapter of the 8B widths, 4 layers: 9.7 M values that stay in L2
        _clip("clip_one_8b", 4096, 12288, 1024, 4, 32, 1),
        # all 32 adapters of the 8B-width workload: 1,792 tensors, 310 M values
        _clip("clip_all_8b", 4096, 12288, 1024, 4, 32, 32),
    ]


def _attn(name, seqs, heads, kv_heads, hd, lo, hi, rows=1, dtype="bf16"):
    return {"name": name, "op": "attention", "seqs": seqs, "heads": heads, "kv_heads": kv_heads, "hd": hd,
            "lo": lo, "hi": hi, "rows": rows, "dtype": dtype}


def _append(name, seqs, kv_heads, hd, lo, hi, before, stride=0, dtype="bf16"):
    """stride: extra heads of 128 between rows (the queries of a q|k|v buffer)."""
    return {"name": name, "op": "append", "seqs": seqs, "kv_heads": kv_heads, "hd": hd, "lo": lo, "hi": hi,
            "before": before, "stride": stride, "dtype": dtype}


def _clip(name, d, f, kv, layers, rank, adapters, dtype="fp32"):
    return {"name": name, "op": "clip", "d": d, "f": f, "kv": kv, "layers": layers, "rank": rank,
            "adapters": adapters, "dtype": dtype}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "attention":
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
        hd = rng.choice([64, 128, 128])
        seqs = _log(rng, 1, 256)
        # the largest listed case reads about 1.2 M positions of 8 heads of 128
        hi = max(1, min(_log(rng, 16, 131072), 1000000 * 8 // (seqs * kv_heads)))
        c = _attn("", seqs, heads, kv_heads, hd, rng.randrange(0, hi + 1), hi, rng.choice([1, 1, 1, 2, 5, 9]), dtype)
    elif op == "append":
        seqs = _log(rng, 1, 256)
        lo = _log(rng, 1, 2048)
        hi = max(1, min(_log(rng, lo, 2 * lo), 60000 // seqs))
        c = _append("", seqs, rng.choice([1, 2, 3, 8]), rng.choice([64, 128]), min(lo, hi), hi, _log(rng, 1, 2047),
                    rng.choice([0, 4, 32]), dtype)
    else:
        d = 128 * _log(rng, 1, 32)
        c = _clip("", d, 128 * _log(rng, 1, 96), min(d, 128 * rng.choice([1, 2, 8])), rng.choice([1, 2, 4]),
                  4 * _log(rng, 1, 8), _log(rng, 1, 32), dtype)
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n lengths between lo and hi, both among them, in no order (the golden ratio's steps)."""
    got = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.999) % 1.0)) for i in range(n)]
    got[0] = hi
    if n > 1:
        got[-1] = lo
    return got


def _lens(case):
    """(kv_len, new rows) of each sequence."""
    n = case["seqs"]
    if case["op"] == "attention":
        lens = _spread(n, case["lo"], case["hi"])
        if case["rows"] == 1:
            return lens, [1] * n         # an empty slot still has its row
        return lens, [min(case["rows"] - (i % 2), ln) for i, ln in enumerate(lens)]
    rows = _spread(n, case["lo"], case["hi"])
    before = [(case["before"] * (i + 1) * 7919 // 64) % (case["before"] + 1) for i in range(n)]
    return [b + r for b, r in zip(before, rows)], rows


def _clip_sizes(case):
    """Sizes of one adapter's tensors: A [r x in] and B [out x r] of its seven projections, layer by layer."""
    d, f, kv, r = case["d"], case["f"], case["kv"], case["rank"]
    per = []
    for o, i in ((d, d), (kv, d), (kv, d), (d, d), (f, d), (f, d), (d, f)):
        per += [r * i, o * r]
    return per * case["layers"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        n = sum(_clip_sizes(case)) * case["adapters"]
        return {"bytes": 2.0 * es * n, "flops": 3.0 * n}
    lens, rows = _lens(case)
    hd, kvh = case["hd"], case["kv_heads"]
    if case["op"] == "append":
        # rows in, blocks written; then the blocks' values read back as fp32
        back = sum(ln - (ln - r) // PAGE * PAGE for ln, r in zip(lens, rows))
        return {"bytes": 2.0 * kvh * hd * (es + 1) * sum(rows) + 2.0 * kvh * hd * 5 * back,
                "flops": 4.0 * kvh * hd * sum(rows)}
    pairs = sum(r * ln - r * (r - 1) // 2 for ln, r in zip(lens, rows) if ln)
    pages = sum(-(-ln // PAGE) for ln in lens)
    return {"bytes": 2.0 * kvh * hd * sum(lens) + 8.0 * kvh * pages + 2.0 * es * case["heads"] * hd * sum(rows) +
            4.0 * case["heads"] * sum(rows),
            "flops": 4.0 * case["heads"] * hd * pairs}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _cache(g, kv_heads, hd, lens):
    """A pool of pages in random order, filled with bytes and scales such as append leaves there."""
    used = [-(-ln // PAGE) for ln in lens]
    total = sum(used)
    n_pages = total + 3 + total // 32
    width = max(max(used), 1)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    u = torch.tensor(used, dtype=torch.int64, device=DEV)
    col = torch.arange(width, device=DEV)
    first = torch.cumsum(u, 0) - u
    at = (first[:, None] + col[None, :]).clamp(max=n_pages - 1)
    table = torch.where(col[None, :] < u[:, None], order[at], torch.full_like(order[at], -1)).to(torch.int32)
    s = {"table": table.contiguous(), "kv_len": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    for name in ("k", "v"):
        x = torch.empty(n_pages, kv_heads, PAGE, hd, dtype=torch.uint8, device=DEV)
        for p in range(0, n_pages, 4096):     # pieces bound the memory of the random draws
            y = torch.randn(x[p:p + 4096].shape, generator=g, device=DEV, dtype=torch.float16) * 96
            x[p:p + 4096] = y.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name] = x
        s[name + "_scale"] = _pow2(torch.randint(-8, -5, (n_pages, kv_heads), generator=g, device=DEV))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "clip":
        # the tensors are views of one buffer per use, each 16-byte aligned, as a trainer lays them out
        sizes = _clip_sizes(case) * case["adapters"]
        s["flat"] = torch.randn(sum(sizes), generator=g, device=DEV, dtype=dt)
        per = sum(sizes) // case["adapters"]
        gain = torch.exp(torch.randn(case["adapters"], generator=g, device=DEV)) * 1e-3
        gain[0] = 2e-3
        s["flat"].view(case["adapters"], per).mul_(gain[:, None].to(dt))
        s["out"] = torch.zeros_like(s["flat"])
        s["grads"] = list(torch.split(s["flat"], sizes))
        s["outs"] = list(torch.split(s["out"], sizes))
        s["groups"] = [i // (len(sizes) // case["adapters"]) for i in range(len(sizes))]
        # clips the first adapter, and the larger half of the others or so
        s["max_norm"] = 1e-3 * math.sqrt(per)
        return s
    lens, rows = _lens(case)
    hd, kvh = case["hd"], case["kv_heads"]
    s |= _cache(g, kvh, hd, lens)
    s["row_off"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device=DEV)
    n, s["max_rows"], s["max_len"] = sum(rows), max(rows), max(max(lens), 1)
    if case["op"] == "attention":
        s["q"] = (torch.randn(n, case["heads"], hd, generator=g, device=DEV) * 2).to(dt)
        s["ragged"] = case["rows"] > 1
    else:
        # k and v as the projections leave them: columns of one row, the scale of a token's entries its own
        buf = torch.randn(n, case["stride"] + 2 * kvh, hd, generator=g, device=DEV)
        buf *= torch.exp(0.5 * torch.randn(n, 1, 1, generator=g, device=DEV))
        buf = buf.to(dt)
        s["k_new"] = buf[:, case["stride"]:case["stride"] + kvh]
        s["v_new"] = buf[:, case["stride"] + kvh:]
        # the blocks that the call writes: every position of a sequence from its first touched block on
        back = [ln - (ln - r) // PAGE * PAGE for ln, r in zip(lens, rows)]
        s["back_off"] = torch.tensor([sum(back[:i]) for i in range(len(back) + 1)], dtype=torch.int32, device=DEV)
        s["back"], s["max_back"] = sum(back), max(back)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "clip": _own_clip}[op](s)
    return {"attention": _plain_attention, "append": _plain_append, "clip": _plain_clip}[op](s)


def _own_cache(s):
    import rl_step_gb300.kv as kv
    if "cache" not in s:
        s["cache"] = kv.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return kv, s["cache"]


def _own_attention(s):
    kv, cache = _own_cache(s)
    if "workspace" not in s:
        s["workspace"] = kv.kv_workspace(s["q"].device)
    return kv.kv_attention(cache, s["table"], s["kv_len"], s["q"], s["max_len"],
                           row_off=s["row_off"] if s["ragged"] else None, max_rows=s["max_rows"],
                           workspace=s["workspace"])


def _own_append(s):
    kv, cache = _own_cache(s)
    kv.kv_append(cache, s["table"], s["kv_len"], s["k_new"], s["v_new"], row_off=s["row_off"], max_rows=s["max_rows"])
    return kv.kv_read(cache, s["table"], s["kv_len"], s["back"], row_off=s["back_off"], max_rows=s["max_back"])


def _own_clip(s):
    import rl_step_gb300.grads as grads
    if "set" not in s:
        s["set"] = grads.GradSet(s["grads"], s["groups"], out=s["outs"])
    norms = grads.clip_grads(s["set"], s["max_norm"])
    return norms, s["out"]


def _byte_of(hd):
    """Where (token, dim) sits inside a (page, head) tile of k and of v: [64 * hd] each."""
    j = torch.arange(PAGE, device=DEV)[:, None]
    c = torch.arange(hd, device=DEV)[None, :]
    at_k = j * hd + ((c // 16) ^ (4 * (j % 2) if hd == 128 else 0)) * 16 + c % 16
    at_v = (j // 4) * 4 * hd + ((c // 4) ^ (2 * (j // 4 % 4))) * 16 + 4 * (c % 4) + j % 4
    return at_k.reshape(-1), at_v.reshape(-1)


def _values(pages, scale, ids, at, hd):
    """fp32 values [..., n_kv, 64, hd] of the pages `ids` (any shape)."""
    b = pages.flatten(2)[ids][..., at].unflatten(-1, (PAGE, hd))
    return b.view(torch.float8_e4m3fn).float() * scale[ids][..., None, None]


def _plain_attention(s):
    c = s["case"]
    hd, kvh = c["hd"], c["kv_heads"]
    group, rows = c["heads"] // kvh, s["max_rows"]
    at_k, at_v = _byte_of(hd)
    kv_len, off = s["kv_len"].long(), s["row_off"].long()
    n_new = off[1:] - off[:-1]
    ids = s["table"].long().clamp(min=0)
    seqs, width = ids.shape
    q = s["q"].float()
    # [seqs, n_kv, rows * group, hd]; rows past a sequence's own repeat a valid one and are not written back
    r = torch.arange(rows, device=DEV)
    take = (off[:-1, None] + r[None, :]).clamp(max=q.shape[0] - 1)
    qs = q[take].view(seqs, rows, kvh, group, hd).permute(0, 2, 1, 3, 4).reshape(seqs, kvh, rows * group, hd)
    pos = torch.arange(width * PAGE, device=DEV)
    last = kv_len[:, None] - n_new[:, None] + r[None, :]                       # a row's own position
    last = torch.where(kv_len[:, None] > 0, last, torch.full_like(last, -1))
    seen = pos[None, None, :] <= last[:, :, None]                              # [seqs, rows, L]
    seen = seen[:, None, :, None, :].expand(seqs, kvh, rows, group, -1).reshape(seqs, kvh, rows * group, -1)
    k = _values(s["k"], s["k_scale"], ids, at_k, hd).transpose(1, 2).reshape(seqs, kvh, width * PAGE, hd)
    z = torch.matmul(qs, k.transpose(2, 3)) * (1.0 / math.sqrt(hd))
    del k
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    z = torch.exp(z - m)
    l = z.sum(-1, keepdim=True)
    v = _values(s["v"], s["v_scale"], ids, at_v, hd).transpose(1, 2).reshape(seqs, kvh, width * PAGE, hd)
    v = torch.where((pos[None, :] < kv_len[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(z, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).view(seqs, kvh, rows, group).permute(0, 2, 1, 3).reshape(seqs, rows, c["heads"])
    o = o.view(seqs, kvh, rows, group, hd).permute(0, 2, 1, 3, 4).reshape(seqs, rows, c["heads"], hd)
    row = torch.arange(q.shape[0], device=DEV)
    seq = torch.searchsorted(off[1:].contiguous(), row, right=True)
    i = row - off[seq]
    return o[seq, i].to(s["q"].dtype), lse[seq, i].contiguous()


def _exponent(a):
    """The smallest e >= -100 with a <= 448 * 2^e."""
    m, e = torch.frexp(a)                                   # a = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _pow2(e):
    """2^e, exactly (exp2 on the GPU is off by a bit)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_append(s):
    hd, kvh = s["case"]["hd"], s["case"]["kv_heads"]
    at = _byte_of(hd)
    kv_len, off = s["kv_len"].long(), s["row_off"].long()
    n_new = off[1:] - off[:-1]
    seqs = kv_len.shape[0]
    start = kv_len - n_new
    first = start // PAGE
    pages = (s["max_rows"] + PAGE - 2) // PAGE + 1                             # blocks a sequence can touch
    col = first[:, None] + torch.arange(pages, device=DEV)[None, :]
    live = col * PAGE < kv_len[:, None]
    ids = s["table"].long().gather(1, col.clamp(max=s["table"].shape[1] - 1))
    ids = torch.where(live, ids, torch.zeros_like(ids))
    pos = (col * PAGE)[:, :, None] + torch.arange(PAGE, device=DEV)            # [seqs, pages, 64]
    is_new = (pos >= start[:, None, None]) & (pos < kv_len[:, None, None])
    is_old = (pos < start[:, None, None])
    src = (off[:-1, None, None] + pos - start[:, None, None]).clamp(0, s["k_new"].shape[0] - 1)
    got = []
    for name, a in (("k", at[0]), ("v", at[1])):
        new = s[name + "_new"].float()[src].permute(0, 1, 3, 2, 4)             # [seqs, pages, n_kv, 64, hd]
        here = is_new[:, :, None, :, None] & torch.isfinite(new)
        need = _exponent(torch.where(here, new.abs(), torch.zeros_like(new)).amax((-2, -1)))
        scale = s[name + "_scale"]
        had = is_old.any(-1)[:, :, None]
        e_old = torch.frexp(scale[ids])[1] - 1
        e = torch.where(had, torch.maximum(need, e_old), need)
        old = s[name].flatten(2)[ids][..., a].unflatten(-1, (PAGE, hd)).view(torch.float8_e4m3fn).float()
        old = old * _pow2(torch.where(had, e_old - e, torch.zeros_like(e)).clamp(min=-60))[..., None, None]
        val = torch.where(is_new[:, :, None, :, None], new * _pow2(-e)[..., None, None], old)
        byte = val.to(torch.float8_e4m3fn).view(torch.uint8)
        flat = s[name].flatten(2)
        tile = torch.empty(seqs, pages, kvh, PAGE * hd, dtype=torch.uint8, device=DEV)
        tile[..., a] = byte.flatten(-2)
        flat[ids[live]] = tile[live]
        scale[ids[live]] = _pow2(e)[live]
        # the written blocks' values, in the order of the positions
        val = (byte.view(torch.float8_e4m3fn).float() * _pow2(e)[..., None, None]).permute(0, 1, 3, 2, 4)
        got.append(val[(pos < kv_len[:, None, None]) & live[:, :, None]])
    return tuple(got)


def _plain_clip(s):
    norms = torch.stack([x.float().square().sum() for x in s["grads"]])
    ids = torch.tensor(s["groups"], device=DEV)
    total = torch.zeros(s["case"]["adapters"], device=DEV).index_add_(0, ids, norms).sqrt()
    factor = torch.where(total > s["max_norm"], s["max_norm"] / total, torch.ones_like(total))
    for x, y, g in zip(s["grads"], s["outs"], s["groups"]):
        y.copy_(x.float() * factor[g])
    return total, s["out"]


# ----------------------------------------------------------------------------
# 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        x = s["flat"].double().view(case["adapters"], -1)
        n = torch.linalg.vector_norm(x, dim=1)
        f = torch.clamp(s["max_norm"] / n, max=1.0)
        return n, (x * f[:, None]).reshape(-1)
    return _exact_attention(s) if case["op"] == "attention" else _exact_append(s)


def _tile64(tile, scale, of_v):
    """[n_kv, 64 * hd] bytes of one page to [n_kv, 64, hd] doubles, by the layout's own axes."""
    kvh, hd = tile.shape[0], tile.shape[1] // PAGE
    if of_v:                                    # [16 quads, hd / 4 chunks, 4 dims, 4 tokens], chunks swapped by quad
        t = tile.view(kvh, 16, hd // 4, 4, 4)
        order = torch.arange(hd // 4, device=DEV)
        t = torch.stack([t[:, q, order ^ (2 * (q % 4))] for q in range(16)], 1)
        t = t.permute(0, 1, 4, 2, 3).reshape(kvh, PAGE, hd)
    else:
        t = tile.view(kvh, PAGE, hd // 16, 16)
        if hd == 128:
            t = torch.stack([t[:, :, :4], t[:, :, 4:]], 2)
            t = torch.stack([t[:, 0::2], t[:, 1::2].flip(2)], 2).reshape(kvh, PAGE, hd // 16, 16)
        t = t.reshape(kvh, PAGE, hd)
    return t.contiguous().view(torch.float8_e4m3fn).double() * scale.double()[:, None, None]


def _pages64(s, name, pages, hd):
    """[n_kv, 64 * len(pages), hd] doubles."""
    kvh = s[name].shape[1]
    t = s[name][pages].flatten(2)               # [p, n_kv, 64 hd]
    p = t.shape[0]
    x = _tile64(t.reshape(p * kvh, PAGE * hd), s[name + "_scale"][pages].reshape(-1), name == "v")
    return x.view(p, kvh, PAGE, hd).transpose(0, 1).reshape(kvh, p * PAGE, hd)


def _exact_attention(s):
    c = s["case"]
    lens, rows = _lens(c)
    group, hd = c["heads"] // c["kv_heads"], c["hd"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for i, (ln, r) in enumerate(zip(lens, rows)):
        if ln and r:
            pages = s["table"][i, :-(-ln // PAGE)].long()
            k, v = (_pages64(s, x, pages, hd)[:, :ln] for x in ("k", "v"))
            q = s["q"][at:at + r].double().view(r, c["kv_heads"], group, hd).permute(1, 0, 2, 3)
            z = torch.einsum("hrgd,hld->hrgl", q, k) / math.sqrt(hd)
            ahead = torch.arange(ln, device=DEV)[None, :] > torch.arange(ln - r, ln, device=DEV)[:, None]
            z = z.masked_fill(ahead[None, :, None, :], -math.inf)
            lse[at:at + r] = torch.logsumexp(z, -1).permute(1, 0, 2).reshape(r, -1)
            o = torch.einsum("hrgl,hld->hrgd", torch.softmax(z, -1), v)
            out[at:at + r] = o.permute(1, 0, 2, 3).reshape(r, c["heads"], hd)
        at += r
    return out, lse


def _two_to(e):
    """2^e as a double, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round64(x):
    """Doubles of magnitude <= 448 rounded to e4m3, ties to even."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1
    step = _two_to(e - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    lens, rows = _lens(c)
    got = {"k": [], "v": []}
    at = 0
    for i, (ln, r) in enumerate(zip(lens, rows)):
        start = ln - r
        p0, p1 = start // PAGE, -(-ln // PAGE)
        for name in ("k", "v"):
            x = s[name + "_new"][at:at + r].double()                      # [r, n_kv, hd]
            whole = []
            for p in range(p0, p1):
                lo, hi = max(start, p * PAGE), min(ln, p * PAGE + PAGE)
                new = x[lo - start:hi - start]
                # per head; the bit less keeps a quotient that is a power of two on its own exponent
                need = torch.ceil(torch.log2(new.abs().amax((0, 2)) / 448) - 1e-9)
                if lo > p * PAGE:
                    page = s["table"][i, p].long()
                    had = torch.round(torch.log2(s[name + "_scale"][page].double()))
                    e = torch.maximum(need, had)
                    old = _pages64(s, name, page[None], c["hd"])[:, :lo - p * PAGE].transpose(0, 1)
                    f = _two_to(e)[None, :, None]
                    whole.append(_round64(old / f) * f)
                else:
                    f = _two_to(need)[None, :, None]
                whole.append(_round64(new / f) * f)
            got[name] += whole
        at += r
    return torch.cat(got["k"]), torch.cat(got["v"])
