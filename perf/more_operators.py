"""What a policy says of its tokens, pages for its rollouts and orthogonal updates, as measured cases.

* ``logprobs``: log-probabilities of given tokens out of logits, with the
  entropy, the log-sum-exp and the largest alternatives of each row.
* ``gradient``: the gradient of those results in the logits.
* ``pages``: sequences of a paged key/value cache cut back to kept lengths and
  grown by new tokens: their page tables, and the position, sequence and slot
  of every new row.
* ``orthogonal``: the updates of LoRA factors made orthogonal by Newton-Schulz
  products.

The plain forms are elementary torch operations in 32 bits.  With ``own`` the
cases call rl_step_gb300.logits, rl_step_gb300.kv and rl_step_gb300.grads.

Definitions.  With z = scale * x for a row x of logits:
    lse = log sum exp(z),  logprob of y = z_y - lse,  entropy = -sum p log p,  p = exp(z - lse)
    dx_j = scale * (sum of d_logprob at y, of d_top_k at the k-th alternative, + p_j (d_lse - d_logprob - sum d_top)
                    - d_entropy p_j (log p_j + entropy))
Alternatives are in falling order, of equal ones the lowest id first.
Pages hold 64 tokens.  Cutting back gives the pages behind the kept ones to the free list so that growing by
as much takes the same ones again: growing serves the sequences in order, pages in order, from the list's end.
Newton-Schulz: x <- m / (|m| + 1e-7); five times, with a = x x^T over the shorter side,
    x <- 3.4445 x + (-4.7750 a + 2.0315 a a) x.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one user's next token over the 8B model's vocabulary, five alternatives
        _rows("logprobs_one", "logprobs", 1, 151936, 5),
        # a rollout step: 256 sequences' fp32 logits at temperature 0.7, twenty alternatives
        _rows("logprobs_step", "logprobs", 256, 151936, 20, "fp32", scale=1 / 0.7),
        # prompts scored with twenty alternatives a token
        _rows("logprobs_prompts", "logprobs", 8192, 151936, 20),
        # a batch of the small transformer workload's vocabulary, no alternatives
        _rows("logprobs_small", "logprobs", 1024, 1000, 0, "fp32"),
        # an entropy bonus beside the policy gradient, over a vocabulary whose row is no multiple of 16 bytes
        _rows("gradient_odd", "gradient", 1021, 32003, 0),
        # the same for 8,192 tokens, distilling twenty alternatives as well
        _rows("gradient_tokens", "gradient", 8192, 151936, 20),
        # 256 sequences that lose up to three refused drafted tokens and get four new rows
        _pages("pages_draft", 256, 512, 2048, 0, 3, 4, 4),
        # prompts of 512 to 2,048 tokens, 65,536 or so in all, in slots that held finished sequences
        _pages("pages_prompts", 51, 0, 0, 512, 2048, 512, 2048),
        # one small transformer adapter: 28 matrices
        _mats("orthogonal_small", 256, 512, 256, 2, 32, 1),
        # one rank-32 adapter of the 8B widths, 4 layers, bf16 updates
        _mats("orthogonal_one_8b", 4096, 12288, 1024, 4, 32, 1, "bf16"),
        # all 32 adapters of the 8B-width workload
        _mats("orthogonal_all_8b", 4096, 12288, 1024, 4, 32, 32),
    ]


def _rows(name, op, rows, vocab, top, dtype="bf16", scale=1.0):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "top": top, "dtype": dtype, "scale": scale}


def _pages(name, seqs, lo, hi, cut_lo, cut_hi, new_lo, new_hi):
    """Kept lengths in lo .. hi; cut_lo .. cut_hi tokens behind them go, new_lo .. new_hi come."""
    return {"name": name, "op": "pages", "seqs": seqs, "lo": lo, "hi": hi, "cut_lo": cut_lo, "cut_hi": cut_hi,
            "new_lo": new_lo, "new_hi": new_hi}


def _mats(name, d, f, kv, layers, rank, adapters, dtype="fp32"):
    return {"name": name, "op": "orthogonal", "d": d, "f": f, "kv": kv, "layers": layers, "rank": rank,
            "adapters": adapters, "dtype": dtype}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "gradient", "gradient", "pages", "orthogonal"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("logprobs", "gradient"):
        vocab = _log(rng, 100, 200000)
        # the largest listed case has 1.2 G logits of 2 bytes
        rows = min(_log(rng, 1, 30000), 600_000_000 // vocab)
        c = _rows("", op, rows, vocab, rng.choice([0, 0, 1, 5, 20, 32]), dtype, rng.choice([1.0, 1.0, 0.5, 1.6]))
    elif op == "pages":
        seqs = _log(rng, 1, 4096)
        hi = min(_log(rng, 1, 32768), 2_000_000 // seqs)
        cut, new = min(_log(rng, 1, 2048), 60000 // seqs), min(_log(rng, 1, 2048), 60000 // seqs)
        c = _pages("", seqs, rng.randrange(0, hi + 1), hi, rng.randrange(0, cut + 1), cut, rng.randrange(0, new + 1), new)
    else:
        d = 64 * _log(rng, 2, 64)
        c = _mats("", d, 64 * _log(rng, 2, 192), min(d, 64 * _log(rng, 1, 16)), rng.choice([1, 2, 4]),
                  4 * _log(rng, 1, 16), _log(rng, 1, 8), dtype)
    del c["name"]
    return c


def _spread(n, lo, hi, turn=0.0):
    """n numbers between lo and hi in no order (the golden ratio's steps), hi among them."""
    got = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.999 + turn) % 1.0)) for i in range(n)]
    got[n // 2] = hi
    return got


def _lens(case):
    """Kept, old and new lengths of each sequence."""
    n = case["seqs"]
    kept = _spread(n, case["lo"], case["hi"])
    cut, new = _spread(n, case["cut_lo"], case["cut_hi"], 0.31), _spread(n, case["new_lo"], case["new_hi"], 0.57)
    return kept, [a + b for a, b in zip(kept, cut)], [a + b for a, b in zip(kept, new)]


def _pages_of(n):
    return -(-n // PAGE)


def _kinds(case):
    """Shapes of one layer's factors: A [r x in] and B [out x r] of its seven projections."""
    d, f, kv, r = case["d"], case["f"], case["kv"], case["rank"]
    shapes = []
    for o, i in ((d, d), (kv, d), (kv, d), (d, d), (f, d), (f, d), (d, f)):
        shapes += [(r, i), (o, r)]
    return shapes


def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "orthogonal":
        n = case["layers"] * case["adapters"]
        # a product over the long side is 2 r^2 n: the first x x^T (half of it, being symmetric) and the last
        # polynomial times x can not be done without; what is between has r x r forms
        return {"bytes": sum(2.0 * es * a * b for a, b in _kinds(case)) * n,
                "flops": sum(3.0 * min(s) * min(s) * max(s) for s in _kinds(case)) * n}
    if case["op"] == "pages":
        kept, old, new = _lens(case)
        moved = sum(_pages_of(o) - _pages_of(k) + _pages_of(n) - _pages_of(k) for k, o, n in zip(kept, old, new))
        rows = sum(n - k for k, n in zip(kept, new))
        # a page moves from a table to the list or back, with its owner; 16 bytes come out for a row
        return {"bytes": 24.0 * case["seqs"] + 12.0 * moved + 16.0 * rows, "flops": 1.0 * (moved + rows)}
    n, t = 1.0 * case["rows"] * case["vocab"], case["rows"] * (16.0 + 12.0 * case["top"])
    if case["op"] == "logprobs":
        return {"bytes": es * n + t, "flops": 5.0 * n}
    return {"bytes": 2.0 * es * n + t, "flops": 7.0 * n}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "pages":
        return _prepare_pages(case, g, s)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "orthogonal":
        # one buffer for each factor of a layer, [layers * adapters, rows, columns]; the rank's directions differ in
        # size and share a part, as a gradient's do
        n = case["layers"] * case["adapters"]
        s["mats"], s["outs"] = [], []
        for a, b in _kinds(case):
            x = torch.randn(n, a, b, generator=g, device=DEV)
            gain = torch.exp(0.5 * torch.randn(n, min(a, b), generator=g, device=DEV))
            common = torch.randn(n, max(a, b), generator=g, device=DEV)
            if a <= b:
                x = (x + common[:, None, :]) * gain[:, :, None]
            else:
                x = (x + common[:, :, None]) * gain[:, None, :]
            s["mats"].append((x * 1e-4).to(dt))
            s["outs"].append(torch.empty_like(s["mats"][-1]))
        return s
    n, v = case["rows"], case["vocab"]
    x = torch.empty(n, v, dtype=dt, device=DEV)
    for i in range(0, n, 1024):           # pieces bound the memory of the random draws
        y = torch.randn(min(1024, n - i), v, generator=g, device=DEV) * 2.5
        # how sure the policy is differs from row to row; some tokens are not allowed
        y *= torch.exp(0.4 * torch.randn(y.shape[0], 1, generator=g, device=DEV))
        x[i:i + 1024] = y.to(dt)
    x[::7, v // 3:v // 3 + v // 50] = -math.inf
    s["x"] = x
    # targets: any token, the likeliest one in every third row, an allowed one where some are not
    s["targets"] = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    s["targets"][::3] = x[::3].float().argmax(1).to(torch.int32)
    s["targets"][::7] %= v // 3
    if case["op"] == "gradient":
        c, y = case["scale"], s["targets"].long()
        s["lse"], s["entropy"] = (torch.empty(n, device=DEV) for _ in range(2))
        for i in range(0, n, 1024):
            z = x[i:i + 1024].double() * c
            lse = torch.logsumexp(z, 1)
            s["lse"][i:i + 1024] = lse.float()
            z = z - lse[:, None]
            s["entropy"][i:i + 1024] = -(torch.exp(z) * z.clamp(min=-1e30)).sum(1).float()
        s["d_logprob"] = torch.randn(n, generator=g, device=DEV)
        s["d_entropy"] = torch.randn(n, generator=g, device=DEV) * 0.01
        masked = torch.arange(n, device=DEV) % 5 == 4      # prompt tokens without a loss
        s["d_logprob"][masked] = 0
        s["d_entropy"][masked] = 0
        if case["top"]:
            k = min(case["top"], v)
            start = torch.randint(0, v, (n, 1), generator=g, device=DEV)
            s["top_ids"] = ((start + torch.arange(k, device=DEV) * (v // k)) % v).to(torch.int32)
            s["top_ids"][::2, 0] = y[::2].to(torch.int32)
            # an id once in a row
            s["top_ids"][::2, 1:] = torch.where(s["top_ids"][::2, 1:] == s["top_ids"][::2, :1],
                                                torch.full_like(s["top_ids"][::2, 1:], -1), s["top_ids"][::2, 1:])
            s["d_top"] = torch.randn(n, k, generator=g, device=DEV) * 0.1
            s["d_top"][masked] = 0
        s["out"] = torch.empty_like(x)
    return s


def _prepare_pages(case, g, s):
    kept, old, new = _lens(case)
    used = [_pages_of(o) for o in old]
    need = sum(max(u, _pages_of(w)) for u, w in zip(used, new))
    n_pages = need + 16 + need // 8
    width = max(max(_pages_of(w), u) for u, w in zip(used, new)) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    u = torch.tensor(used, device=DEV)
    col = torch.arange(width, device=DEV)
    at = (torch.cumsum(u, 0) - u)[:, None] + col[None, :]
    mine = col[None, :] < u[:, None]
    s["table"] = torch.where(mine, order[at.clamp(max=n_pages - 1)], torch.full_like(order[:1], -1)).contiguous()
    s["kv_len"] = torch.tensor(old, dtype=torch.int32, device=DEV)
    s["keep"] = torch.tensor(kept, dtype=torch.int32, device=DEV)
    s["n_new"] = torch.tensor([w - k for w, k in zip(new, kept)], dtype=torch.int32, device=DEV)
    s["n_rows"] = sum(new) - sum(kept) + 5             # five rows more than there are, as in a padded batch
    # the pool: the pages that no sequence owns, their number, and each page's owner
    total = sum(used)
    s["free"] = torch.cat([order[total:], order[:total]]).contiguous()
    s["n_free"] = torch.tensor([n_pages - total], dtype=torch.int32, device=DEV)
    s["owner"] = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    seq = torch.arange(len(used), device=DEV)[:, None].expand(-1, width)
    s["owner"][s["table"][mine].long()] = seq[mine].to(torch.int32)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"logprobs": _own_logprobs, "gradient": _own_gradient, "pages": _own_pages,
                "orthogonal": _own_orthogonal}[op](s)
    return {"logprobs": _plain_logprobs, "gradient": _plain_gradient, "pages": _plain_pages,
            "orthogonal": _plain_orthogonal}[op](s)


def _own_logprobs(s):
    import rl_step_gb300.logits as lg
    r = lg.token_logprobs(s["x"], s["targets"], top=s["case"]["top"], scale=s["case"]["scale"])
    if not s["case"]["top"]:
        return r.logprobs, r.entropy, r.lse
    return r.logprobs, r.entropy, r.lse, r.top_ids, r.top_logprobs


def _own_gradient(s):
    import rl_step_gb300.logits as lg
    return lg.token_logprobs_backward(s["x"], s["lse"], s["entropy"], s["targets"], s["d_logprob"],
                                      d_entropy=s["d_entropy"], top_ids=s.get("top_ids"), d_top=s.get("d_top"),
                                      scale=s["case"]["scale"], out=s["out"])


def _own_pages(s):
    import rl_step_gb300.kv as kv
    if "pool" not in s:
        s["pool"] = kv.PagePool(s["free"], s["n_free"], s["owner"])
    kv.kv_release(s["pool"], s["table"], s["kv_len"], s["keep"])
    r = kv.kv_reserve(s["pool"], s["table"], s["kv_len"], s["n_new"], s["n_rows"])
    return s["table"], s["kv_len"], r.row_off, r.positions, r.seqs, r.slots, s["n_free"], s["owner"]


def _own_orthogonal(s):
    import rl_step_gb300.grads as grads
    if "set" not in s:
        s["set"] = grads.MatrixSet([m for x in s["mats"] for m in x], out=[m for x in s["outs"] for m in x])
    grads.orthogonalize(s["set"], STEPS, COEFFS, EPS)
    return s["outs"]


def _plain_logprobs(s):
    c, v = s["case"], s["case"]["vocab"]
    z = s["x"].float() * c["scale"]
    m = z.amax(1, keepdim=True)
    z = z - m
    e = torch.exp(z)
    total = e.sum(1)
    # a token that is not allowed adds nothing
    entropy = torch.log(total) - (e * z.clamp_(min=-1e30)).sum(1) / total
    del e
    y = s["targets"].long()[:, None]
    log_total = torch.log(total)
    lp = s["x"].gather(1, y).float() * c["scale"] - m - log_total[:, None]
    lse = m[:, 0] + log_total
    if not c["top"]:
        return lp[:, 0], entropy, lse
    # whole numbers in the order of the values, of equal ones the lowest id largest
    bits = s["x"].float().view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    key = (key << 32) + (v - torch.arange(v, device=DEV))
    best = torch.topk(key, min(c["top"], v), 1).values
    ids = v - (best & 0xffffffff)
    top = s["x"].gather(1, ids).float() * c["scale"] - m - log_total[:, None]
    ids = torch.where(torch.isinf(top), torch.full_like(ids, -1), ids).to(torch.int32)
    if c["top"] > v:
        more = c["top"] - v
        ids = torch.cat([ids, torch.full_like(ids[:, :1], -1).expand(-1, more)], 1)
        top = torch.cat([top, torch.full_like(top[:, :1], -math.inf).expand(-1, more)], 1)
    return lp[:, 0], entropy, lse, ids, top


def _plain_gradient(s):
    c = s["case"]
    logp = s["x"].float() * c["scale"] - s["lse"][:, None]
    p = torch.exp(logp)
    into = s["d_logprob"] + (s["d_top"] * (s["top_ids"] >= 0)).sum(1) if c["top"] else s["d_logprob"]
    d = -p * (into[:, None] + s["d_entropy"][:, None] * (logp.clamp_(min=-1e30) + s["entropy"][:, None]))
    d.scatter_add_(1, s["targets"].long()[:, None], s["d_logprob"][:, None])
    if c["top"]:
        ok = s["top_ids"] >= 0
        d.scatter_add_(1, s["top_ids"].long().clamp(min=0), s["d_top"] * ok)
    s["out"].copy_(d * c["scale"])
    return s["out"]


def _plain_pages(s):
    table, kv_len, keep, n_new = s["table"], s["kv_len"].long(), s["keep"].long(), s["n_new"].long()
    seqs, width = table.shape
    col = torch.arange(width, device=DEV)[None, :]
    seq = torch.arange(seqs, device=DEV)[:, None]
    top = s["n_free"].long()
    # cut back
    keep = torch.minimum(keep, kv_len)
    gone = (col >= (keep[:, None] + PAGE - 1) // PAGE) & (col < (kv_len[:, None] + PAGE - 1) // PAGE)
    at = gone.flatten().cumsum(0).view(seqs, width)
    count = at[-1:, -1]
    pages = table[gone].long()
    s["free"][top + count - at[gone]] = pages.to(torch.int32)
    s["owner"][pages] = -1
    table[gone] = -1
    top = top + count
    # grow
    after = keep + n_new
    fresh = (col >= (keep[:, None] + PAGE - 1) // PAGE) & (col < (after[:, None] + PAGE - 1) // PAGE)
    at = fresh.flatten().cumsum(0).view(seqs, width)
    pages = s["free"][top - at[fresh]]
    table[fresh] = pages
    s["owner"][pages.long()] = seq.expand(-1, width)[fresh].to(torch.int32)
    s["n_free"].copy_(top - at[-1:, -1])
    s["kv_len"].copy_(after)
    row_off = torch.cat([torch.zeros_like(n_new[:1]), n_new.cumsum(0)])
    row = torch.arange(s["n_rows"], device=DEV)
    of = torch.searchsorted(row_off[1:].contiguous(), row, right=True)
    live = of < seqs
    of = of.clamp(max=seqs - 1)
    pos = keep[of] + row - row_off[of]
    slot = table[of, (pos // PAGE).clamp(max=width - 1)].long() * PAGE + pos % PAGE
    none = torch.full_like(row, -1)
    return (table, s["kv_len"], row_off.to(torch.int32), torch.where(live, pos, none).to(torch.int32),
            torch.where(live, of, none).to(torch.int32), torch.where(live, slot, none), s["n_free"], s["owner"])


def _plain_orthogonal(s):
    return [out.copy_(_newton_schulz(m.float())) for m, out in zip(s["mats"], s["outs"])]


def _newton_schulz(m):
    """m [n, rows, columns], the shorter side taken for the products."""
    tall = m.shape[1] > m.shape[2]
    x = m.transpose(1, 2) if tall else m
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        a = torch.matmul(x, x.transpose(1, 2))
        x = COEFFS[0] * x + torch.matmul(COEFFS[1] * a + COEFFS[2] * torch.matmul(a, a), x)
    return x.transpose(1, 2) if tall else x


# ----------------------------------------------------------------------------
# 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return None                       # whole numbers alone
    if case["op"] == "orthogonal":
        return [torch.cat([_orthogonal64(m[i:i + 16]) for i in range(0, m.shape[0], 16)]) for m in s["mats"]]
    got = [_rows64(s, i, min(i + 512, case["rows"])) for i in range(0, case["rows"], 512)]
    if case["op"] == "gradient":
        return torch.cat(got)
    full = [torch.cat(x) for x in zip(*got)]
    if case["top"]:
        full.insert(3, None)
    return tuple(full)


def _rows64(s, a, b):
    c, x = s["case"], s["x"][a:b].double()
    y = s["targets"][a:b].long()
    rows = torch.arange(b - a, device=DEV)
    z = x * c["scale"]
    if c["op"] == "logprobs":
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        plogp = torch.special.xlogy(torch.exp(logp), torch.exp(logp))
        # p log p of the large terms from log p itself
        plogp = torch.where(logp > -700, torch.exp(logp) * logp.clamp(min=-1e300), plogp)
        got = [logp[rows, y], -plogp.sum(1), lse]
        if c["top"]:
            top = torch.sort(logp, 1, descending=True).values[:, :c["top"]]
            if top.shape[1] < c["top"]:
                top = torch.nn.functional.pad(top, (0, c["top"] - top.shape[1]), value=-math.inf)
            got.append(top)
        return got
    # the results' derivatives one by one: of a log-probability onehot - p, of the entropy -p (log p + H)
    logp = z - s["lse"][a:b].double()[:, None]
    p = torch.exp(logp)
    d = -s["d_logprob"][a:b].double()[:, None] * p
    d[rows, y] += s["d_logprob"][a:b].double()
    h = s["entropy"][a:b].double()[:, None]
    d -= s["d_entropy"][a:b].double()[:, None] * torch.where(p > 0, p * (logp + h), torch.zeros_like(p))
    for k in range(s["top_ids"].shape[1] if c["top"] else 0):
        ids, w = s["top_ids"][a:b, k].long(), s["d_top"][a:b, k].double()
        w = torch.where(ids >= 0, w, torch.zeros_like(w))
        d -= w[:, None] * p
        d[rows, ids.clamp(min=0)] += w
    return d * c["scale"]


def _orthogonal64(m):
    """The polynomial on the singular values: u p(s) v^T, from the eigenvectors of the shorter side's products."""
    x = m.double()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
    w, u = torch.linalg.eigh(x @ x.transpose(1, 2))
    gain = torch.ones_like(w)
    for _ in range(STEPS):
        t = w * gain * gain
        gain = gain * (COEFFS[0] + COEFFS[1] * t + COEFFS[2] * t * t)
    x = (u * gain[:, None, :]) @ (u.transpose(1, 2) @ x)
    return x.transpose(1, 2) if tall else x
