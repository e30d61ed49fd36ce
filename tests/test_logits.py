"""Token log-probabilities, entropy, alternatives and their gradient
(include/mlora_logits.h) against NumPy doubles.

Tolerances, with u = 2^-24.  A thread adds 8 terms of a group in a row, then its
groups (V / 16 over the team's threads), then 8 joins of three roundings each; a
term 2^a has 2 ulp of the exponential and the rounding of a, whose magnitude
times the term is below 2^-a a <= 0.54, so 4 u; the team has at least 32 threads up to
8,192 logits, 64 up to 24,576, 128 beyond.  With
    e = (8 + V / (16 threads) + 24 + 8) u
the sum of the terms is off by e of itself.  c = scale log2 e is rounded twice, the
maximum's product is exact in the sums (the terms are taken from it rounded), and
each result is rounded at most three times:
    lse: e + 4 u |lse| + 2 u max |z|,   logprob: e + 6 u (|lp| + 1)
(a logprob is a distance from the maximum, whose own rounding cancels).
The entropy log2 s - t / s: t has e of sum |term a|, and 1 + 2 |t / s| <= 1 + 2 log2 V
    entropy: e (1 + 2 log2 V)
The gradient: a = x c - lse log2 e has u (3 |lse| log2 e + 2 |z| log2 e), so
    p is off by 2^-22 + that of itself, the products by 4 u, and the sum of terms
    |p (G + d_e (log p + H))| + |own| carries these; one rounding to the type.
"""
import ctypes
import math

import numpy as np
import pytest

U = 2.0 ** -24


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    import rl_step_gb300.logits as lg
    return lg, lg._lib()


# ----------------------------------------------------------------------------
# on the CPU
# ----------------------------------------------------------------------------
P = 1 << 20                                      # never dereferenced: every call below is refused on the host


def _logits(lg, **kw):
    f = dict(logits=P, targets=P, status=None, stride=1000, n_rows=4, vocab=1000, dtype=0, scale=1.0, top=5)
    f.update(kw)
    return lg._Logits(*[f[k[0]] for k in lg._Logits._fields_])


BAD = [("logits", None), ("logits", P + 1), ("stride", 999), ("stride", -1), ("stride", 1 << 62), ("n_rows", -1),
       ("n_rows", 1 << 31), ("vocab", 0), ("vocab", (1 << 22) + 1), ("dtype", 2), ("dtype", -1), ("scale", 0.0),
       ("scale", -1.0), ("scale", math.nan), ("scale", math.inf), ("scale", 2.0 ** 21), ("top", -1), ("top", 33)]


@pytest.mark.parametrize("field,value", BAD)
def test_refusals_without_a_gpu(field, value):
    lg, lib = _lib()
    x = _logits(lg, **{field: value})
    out = lg._TokenStats(P, P, P, P, P)
    g = lg._TokenGrads(P, P, P, P, P, P, P)
    assert lib.mlora_token_logprobs(ctypes.byref(x), ctypes.byref(out), None) == -1 and lib.mlora_last_error()
    assert lib.mlora_token_logprobs_backward(ctypes.byref(x), ctypes.byref(g), 1 << 40, 1000, None) == -1


def test_refusals_of_results_and_gradients():
    lg, lib = _lib()
    x = _logits(lg)
    assert lib.mlora_token_logprobs(None, ctypes.byref(lg._TokenStats()), None) == -1
    assert lib.mlora_token_logprobs(ctypes.byref(x), None, None) == -1
    assert lib.mlora_token_logprobs(ctypes.byref(_logits(lg, targets=None)), ctypes.byref(lg._TokenStats(P)), None) == -1
    # nothing to do, or nothing wanted
    assert lib.mlora_token_logprobs(ctypes.byref(x), ctypes.byref(lg._TokenStats()), None) == 0
    assert lib.mlora_token_logprobs(ctypes.byref(_logits(lg, n_rows=0, logits=None)), ctypes.byref(lg._TokenStats(P)), None) == 0

    def rc(out=1 << 40, ld=1000, xx=x, **kw):
        f = dict(lse=P, entropy=P, top_ids=P, d_logprobs=P, d_entropy=P, d_lse=P, d_top=P)
        f.update(kw)
        g = lg._TokenGrads(*[f[k[0]] for k in lg._TokenGrads._fields_])
        return lib.mlora_token_logprobs_backward(ctypes.byref(xx), ctypes.byref(g), out, ld, None)

    assert lib.mlora_token_logprobs_backward(ctypes.byref(x), None, 1 << 40, 1000, None) == -1
    for kw in (dict(out=None), dict(out=(1 << 40) + 1), dict(ld=999), dict(ld=1 << 62), dict(lse=None),
               dict(entropy=None), dict(top_ids=None), dict(xx=_logits(lg, targets=None)),
               # an output over a part of the logits: one element on, another distance, the last row's end
               dict(out=P + 2), dict(out=P, ld=1008), dict(out=P - 2), dict(out=P + 3 * 2000 + 1998),
               # rows between rows that reach into them
               dict(xx=_logits(lg, stride=2100), out=P + 2000, ld=2200),
               dict(xx=_logits(lg, stride=1900), out=P + 2000, ld=1900)):
        assert rc(**kw) == -1, kw
    assert rc(xx=_logits(lg, n_rows=0)) == 0


def test_header_and_binding_agree(tmp_path):
    import os
    import re
    import shutil
    import subprocess
    lg, _ = _lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = [("mlora_logits", lg._Logits), ("mlora_token_stats", lg._TokenStats), ("mlora_token_grads", lg._TokenGrads)]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mlora_logits.h"', "int main(void) {"]
    for name, cls in structs:
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f[0]}));' for f in cls._fields_]
    lines.append('printf("%d %d\\n", MLORA_LOGITS_MAX_TOP, MLORA_LOGITS_MAX_VOCAB); return 0; }')
    (tmp_path / "a.c").write_text("\n".join(lines))
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"),
                    "-o", str(tmp_path / "a")], check=True, capture_output=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in structs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want + [32, 1 << 22]
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "mlora_logits.h")).read(), flags=re.S)
    for name, (_, args) in lg._SIGNATURES.items():
        m = re.search(r"\b%s\s*\(([^)]*)\)" % name, src)
        assert m and len(m.group(1).split(",")) == len(args), name


# ----------------------------------------------------------------------------
# the model
# ----------------------------------------------------------------------------
def _model_row(x, scale, top):
    """lse, entropy, ids, their logprobs and log p of one row of doubles"""
    if np.isnan(x).any() or np.isposinf(x).any():
        nan = np.full(len(x), np.nan)
        return math.nan, math.nan, np.full(top, -1), np.full(top, np.nan), nan
    if np.isneginf(x).all():
        return -math.inf, 0.0, np.full(top, -1), np.full(top, -np.inf), np.full(len(x), -np.inf)
    m = x.max()
    with np.errstate(over="ignore", invalid="ignore"):
        d = (x - m) * scale
    s = math.fsum(np.exp(d))
    lp = d - math.log(s)
    p = np.exp(lp)
    h = -math.fsum((p * np.where(p > 0, lp, 0)).tolist())
    order = np.argsort(-x, kind="stable")[:top]
    order = order[x[order] > -np.inf]
    ids, tops = np.full(top, -1), np.full(top, -np.inf)
    ids[:len(order)], tops[:len(order)] = order, lp[order]
    return m * scale + math.log(s), h, ids, tops, lp


def _e(v):
    return (8 + -(-v // 16) / (32 if v <= 8192 else 64 if v <= 24576 else 128) + 32) * U


def _near(got, want, tol, what):
    got = float(got)
    if math.isnan(want) or math.isinf(want):
        assert got == want or (math.isnan(got) and math.isnan(want)), (what, got, want)
    else:
        assert abs(got - want) <= tol, (what, got, want, tol)


def _check(x, y, scale, top, r):
    xs, (n, v) = x.double().cpu().numpy(), x.shape
    lp, h, lse = (t.double().cpu().numpy() if t is not None else None for t in r[:3])
    ids, tops = (r.top_ids.cpu().numpy(), r.top_logprobs.double().cpu().numpy()) if top else (None, None)
    y = None if y is None else y.cpu().numpy()
    e = _e(v)
    for i in range(n):
        w_lse, w_h, w_ids, w_tops, w_lp = _model_row(xs[i], scale, top)
        fin = np.abs(xs[i][np.isfinite(xs[i])] * scale)
        _near(lse[i], w_lse, e + 4 * U * abs(w_lse) + 2 * U * (fin.max() if len(fin) else 0), ("lse", i))
        _near(h[i], w_h, e * (1 + 2 * math.log2(max(v, 2))), ("entropy", i))
        if y is not None:
            want = w_lp[y[i]] if 0 <= y[i] < v else math.nan
            _near(lp[i], want, e + 6 * U * (abs(want) + 1), ("logprob", i))
        if top:
            assert (ids[i] == w_ids).all(), (i, ids[i], w_ids)
            for a, b in zip(tops[i], w_tops):
                _near(a, b, e + 6 * U * (abs(b) + 1), ("top", i))


def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib()
    return torch


def _case(torch, n, v, dtype, seed=0, spread=2.5, offset=0, gap=0):
    """logits [n, v] whose rows begin `offset` elements into a buffer, `gap` apart"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = (torch.randn(n * (v + gap) + offset + 64, generator=g, device="cuda") * spread).to(dt)
    x = buf[offset:offset + n * (v + gap)].view(n, v + gap)[:, :v]
    y = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    return buf, x, y


# ----------------------------------------------------------------------------
# on the GPU
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [1, 2, 15, 16, 17, 33, 64, 511, 1000, 4095, 4096])
def test_small_vocabularies(v, dtype):
    """a warp a row: ragged ends, rows at odd addresses, fewer ids than alternatives"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    for n, top, offset, gap, scale in ((1, 0, 0, 0, 1.0), (9, 5, 1, 0, 0.7), (17, 32, 7, 3, 1.6), (8, 1, 0, 16, 1.0)):
        buf, x, y = _case(torch, n, v, dtype, seed=v + n, offset=offset, gap=gap)
        before = buf.clone()
        _check(x, y, scale, top, lg.token_logprobs(x, y, top=top, scale=scale))
        assert torch.equal(buf, before)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,n", [(4097, 3), (8191, 5), (8192, 2500), (8193, 1300), (24576, 1300), (24577, 700), (32003, 2),
                                 (32003, 700), (151936, 1), (151936, 3), (151936, 170), (151936, 700), (200003, 2)])
def test_large_vocabularies(v, n, dtype):
    """teams of one to eight warps, or a cluster of blocks, a row: by its length and the number of rows"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, n, v, dtype, seed=v, offset=5, gap=2)
    x[0, v // 2:] = -math.inf                       # nothing in the last shares
    y[0] = v - 1                                    # a target that is not allowed
    r = lg.token_logprobs(x, y, top=20, scale=0.9)
    rows = list(range(min(n, 3))) + [n - 1]
    _check(x[rows], y[rows], 0.9, 20, lg.TokenStats(*[t[rows] for t in r]))
    again = lg.token_logprobs(x, y, top=20, scale=0.9)
    assert all(torch.equal(a, b) for a, b in zip(r, again))           # bit for bit
    few = lg.token_logprobs(x, y, top=3, scale=0.9)
    assert torch.equal(few.top_ids, r.top_ids[:, :3]) and torch.equal(few.lse, r.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [40, 1000, 20000, 151936])
def test_rows_of_special_values(v, dtype):
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 16, v, dtype, seed=5, offset=1)
    low = torch.finfo(x.dtype).min
    x[0] = 0                                                       # all equal: the first ids
    x[1] = -math.inf                                               # no distribution
    x[2] = -math.inf
    x[2, v - 1] = 3                                                # one token
    x[3] = low                                                     # a mask of the type's lowest value, all of it
    x[4] = low
    x[4, v // 2] = 1.0
    x[5, v // 3] = math.nan
    x[6, v - 2] = math.inf
    x[7] = -math.inf
    x[7, 3] = low                                                  # its only token
    x[8] = torch.arange(v, device="cuda").to(x.dtype)              # rising: equal pieces where the type ends
    x[9] = -torch.arange(v, device="cuda").to(x.dtype)
    x[10] = 3e38
    x[11] = torch.where(torch.arange(v, device="cuda") % 2 == 0, 0.0, -0.0).to(x.dtype)
    x[12] = -1e32
    x[12, 5] = -2e32
    x[13] = 1e7
    x[13, v // 2:] += 8e4
    x[14, :] = 50.0
    x[14, 7] = 50.5
    x[15, : v // 2] = -math.inf
    y[1], y[2], y[5], y[7], y[15] = 0, 0, 1, 4, 0
    top = 20
    _check(x, y, 1.0, top, lg.token_logprobs(x, y, top=top))
    # a bad row changes none beside it
    good = lg.token_logprobs(x, y, top=top)
    x[5] = 1.0
    assert torch.equal(lg.token_logprobs(x, y, top=top).lse[8:10], good.lse[8:10])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,n,offset", [(40, 64, 1), (1000, 64, 0), (20000, 64, 5), (32003, 500, 3), (151936, 3, 0),
                                        (151936, 3, 7), (151936, 320, 0)])
def test_tokens_that_are_not_allowed_cost_nothing(v, n, offset, dtype):
    """masks over a row's first ids, its two ends, all but a few tokens: with -infinity, the type's lowest value or any
    large negative number the row is taken as with -1e5, whose terms are 0 in fp32 as well, and all results have the same
    bits (a second pass over the row, which other values need, rounds its sums elsewhere)"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, n, v, dtype, seed=v, offset=offset)
    _, a, _ = _case(torch, n, v, dtype, offset=offset)             # lies as x does
    first, ends, most = (torch.zeros(v, dtype=torch.bool, device="cuda") for _ in range(3))
    first[:max(v // 3, 33)] = True
    ends[0] = ends[v - 1] = True
    most[:v - 7] = most[v - 1] = True
    y[:] = v - 2                                                   # allowed by all three
    rows = list(range(0, n, 50))
    for mask in (first, ends, most):
        a.copy_(x).masked_fill_(mask, -1e5)
        want = lg.token_logprobs(a, y, top=5, scale=0.9)
        for low in (-1e9, -1e10, -1e20, -1.2e30, torch.finfo(x.dtype).min, -math.inf):
            a.masked_fill_(mask, low)
            r = lg.token_logprobs(a, y, top=5, scale=0.9)
            for name, p, q in zip(r._fields, r, want):
                assert torch.equal(p, q), (name, low, (p != q).sum().item())
        _check(a[rows], y[rows], 0.9, 5, lg.TokenStats(*[t[rows] for t in r]))


@pytest.mark.gpu
@pytest.mark.parametrize("v", [4096, 151936])
def test_alternatives_that_few_threads_hold(v):
    """the largest groups all in one thread's stride, in more than the list holds, and in runs"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 700 if v > 4096 else 6, v, "fp32", seed=9)
    x[1, 0::16 * 32] += 100
    x[2, 5::16 * 256] += 100
    x[3, 100:700] += 50
    x[4, ::2] += 100
    x[5] = (torch.arange(v, device="cuda") // 16 % 256).float() + (torch.arange(v, device="cuda") % 7) * 0.1
    r = lg.token_logprobs(x, y, top=32)
    _check(x[:6], y[:6], 1.0, 32, lg.TokenStats(*[t[:6] for t in r]))


@pytest.mark.gpu
def test_a_sure_row_has_a_small_entropy():
    """a row whose entropy is far below fp32's steps at the size of its log-sum-exp"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    x = torch.zeros(3, 5000, device="cuda")
    x[:, 77] = torch.tensor([25.0, 40.0, 80.0], device="cuda")
    h = lg.token_logprobs(x).entropy.double().cpu().numpy()
    for i in range(3):
        want = _model_row(x[i].double().cpu().numpy(), 1.0, 0)[1]
        # s is rounded near 1, the sum of the small terms is off by e of itself
        assert abs(h[i] - want) <= 4 * U + _e(5000) * want, (h[i], want)


@pytest.mark.gpu
def test_targets_that_are_none_or_bad():
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 6, 1000, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y[1] = -1
    r = lg.token_logprobs(x, y, status=status)
    assert status.item() == 0 and torch.isnan(r.logprobs[1]) and torch.isfinite(r.logprobs[[0, 2, 3, 4, 5]]).all()
    for bad in (1000, -2, 2 ** 31 - 1):
        y[2] = bad
        status.zero_()
        r = lg.token_logprobs(x, y, top=2, status=status)
        assert status.item() == 1 and torch.isnan(r.logprobs[2]) and torch.isfinite(r.lse).all()
        d = lg.token_logprobs_backward(x, r.lse, targets=y, d_logprobs=torch.ones(6, device="cuda"), status=status.zero_())
        assert status.item() == 1 and (d[1:3] == 0).all() and (d[3] != 0).any()
    none = lg.token_logprobs(x, top=2)
    assert none.logprobs is None and torch.equal(none.lse, r.lse)
    empty = lg.token_logprobs(x[:0], y[:0], top=3)
    assert empty.lse.shape == (0,) and empty.top_ids.shape == (0, 3)


def _gradient(x, scale, y, lse, h, dl, de, dz, ids, dt):
    """the definition in doubles, and the magnitude of what is added"""
    n, v = x.shape
    z = x * scale
    out, size = np.zeros_like(x), np.zeros_like(x)
    for i in range(n):
        own = np.zeros(v)
        g = [(int(y[i]), dl[i])] if dl is not None and y[i] >= 0 else []
        g += [(int(a), b) for a, b in zip(ids[i], dt[i]) if a >= 0] if dt is not None else []
        total = sum(b for _, b in g)
        for a, b in g:
            own[a] += b
        e, w = (de[i] if de is not None else 0.0), (dz[i] if dz is not None else 0.0)
        if (e == 0 and w == 0 and all(b == 0 for _, b in g)) or lse[i] == -np.inf:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            logp = z[i] - lse[i]
            p = np.exp(logp)
            lp = np.where(p > 0, logp, 0)
            out[i] = scale * (own + p * (w - total) - e * p * (lp + h[i]))
            size[i] = scale * (np.abs(own) + p * (abs(w) + sum(abs(b) for _, b in g) + abs(e) * (np.abs(lp) + abs(h[i]))))
    return out, size


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,n,top,offset,gap", [(1, 3, 1, 0, 0), (17, 9, 3, 0, 0), (1000, 8, 5, 1, 0), (8192, 3, 0, 0, 0),
                                                (16385, 3, 20, 3, 5), (32003, 4, 32, 0, 0), (151936, 2, 20, 0, 0)])
@pytest.mark.parametrize("how", ["new", "in place", "other alignment"])
def test_gradient_is_the_definitions(v, n, top, offset, gap, dtype, how):
    torch = _torch()
    import rl_step_gb300.logits as lg
    buf, x, y = _case(torch, n, v, dtype, seed=v, offset=offset, gap=gap)
    g = torch.Generator(device="cuda").manual_seed(v + 1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    scale = 0.8
    if v > 20:
        x[1, 3:9] = -math.inf
    y[0] = -1
    r = lg.token_logprobs(x, y, scale=scale)
    dl, de, dz = rand(n), rand(n) * 0.1, rand(n) * 0.1
    dt = ids = None
    if top:
        ids = torch.randint(-1, v, (n, top), generator=g, device="cuda", dtype=torch.int32)
        ids[:, 0] = y                                   # an alternative that is the target
        if top > 2:
            ids[:, 2] = ids[:, 1]                       # and one that occurs twice
        dt = rand(n, top) * 0.3
    if n > 2:                                           # a row that gets nothing
        dl[2] = de[2] = dz[2] = 0
        if top:
            dt[2] = 0
    xs = x.double().cpu().numpy()
    if how == "new":
        out = torch.full_like(x, 9)
    elif how == "in place":
        out = x
    else:
        out = torch.full((n * (v + gap + 1) + 3,), 9, dtype=x.dtype, device="cuda")[3:].view(n, -1)[:, :v]
    rest = buf.clone()
    got = lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, de, dz, ids, dt, scale=scale, out=out)
    assert got is out
    num = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, size = _gradient(xs, scale, num(y), num(r.lse), num(r.entropy), num(dl), num(de), num(dz), num(ids), num(dt))
    z = np.abs(xs * scale)
    z = np.where(np.isfinite(z), z, 0)
    rel = 2.0 ** -22 + U * (5 * np.abs(num(r.lse))[:, None] + 3 * z + 6 + top)
    tol = size * rel + (np.abs(want) * (2.0 ** -8 if dtype == "bf16" else U)) + 1e-38
    d = np.abs(out.double().cpu().numpy() - want)
    assert (d <= tol).all(), (d / tol).max()
    if n > 2:
        assert (out[2] == 0).all()
    if how == "in place" and gap:
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[offset:offset + n * (v + gap)].view(n, v + gap)[:, :v] = False
        assert torch.equal(buf[keep], rest[keep])       # nothing between the rows


@pytest.mark.gpu
def test_gradient_against_differences():
    """central differences of every result of the forward's model, in doubles"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 3, 40, "fp32", seed=2)
    scale, top = 0.7, 4
    r = lg.token_logprobs(x, y, top=top, scale=scale)
    g = torch.Generator(device="cuda").manual_seed(3)
    dl, de, dz = (torch.randn(3, generator=g, device="cuda") for _ in range(3))
    dt = torch.randn(3, top, generator=g, device="cuda")
    got = lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, de, dz, r.top_ids, dt, scale=scale).double().cpu().numpy()
    xs, ids = x.double().cpu().numpy(), r.top_ids.cpu().numpy()
    w = [t.double().cpu().numpy() for t in (dl, de, dz, dt)]

    def loss(i, row):
        lse, h, _, _, lp = _model_row(row, scale, top)
        return w[0][i] * lp[int(y[i])] + w[1][i] * h + w[2][i] * lse + (w[3][i] * lp[ids[i]]).sum()

    for i in range(3):
        for j in range(40):
            a, b = xs[i].copy(), xs[i].copy()
            a[j] += 1e-5
            b[j] -= 1e-5
            diff = (loss(i, a) - loss(i, b)) / 2e-5
            assert abs(diff - got[i, j]) <= 1e-5 * (1 + abs(diff)), (i, j)


@pytest.mark.gpu
def test_gradient_of_rows_without_numbers():
    """NaN logits: zeros where nothing comes in, NaN else; no distribution: zeros"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 4, 1000, "fp32")
    x[0, 5] = math.nan
    x[1, 6] = math.nan
    x[2] = -math.inf
    r = lg.token_logprobs(x, y)
    d = lg.token_logprobs_backward(x, r.lse, r.entropy, y, torch.tensor([0., 1, 1, 1], device="cuda"),
                                   torch.tensor([0., 0, 1, 1], device="cuda"))
    assert (d[0] == 0).all() and torch.isnan(d[1]).all() and (d[2] == 0).all() and torch.isfinite(d[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [100, 9000])
def test_gradient_beside_the_logits(v, dtype):
    """rows of one buffer that hold logits and their gradient side by side; many rows of short ones"""
    torch = _torch()
    import rl_step_gb300 as m
    import rl_step_gb300.logits as lg
    n = 1500 if v < 1000 else 20
    g = torch.Generator(device="cuda").manual_seed(v)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.randn(n, 2 * v + 6, generator=g, device="cuda").to(dt)
    x, d = buf[:, :v], buf[:, v + 3:2 * v + 3]
    rest = buf.clone()
    y = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.randn(n, generator=g, device="cuda")
    r = lg.token_logprobs(x, y, top=2)
    lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, dl, top_ids=r.top_ids, d_top=r.top_logprobs, out=d)
    want = lg.token_logprobs_backward(x.contiguous(), r.lse, r.entropy, y, dl, dl, top_ids=r.top_ids, d_top=r.top_logprobs)
    assert torch.equal(d, want)
    assert torch.equal(x, rest[:, :v]) and torch.equal(buf[:, v:v + 3], rest[:, v:v + 3])
    assert torch.equal(buf[:, 2 * v + 3:], rest[:, 2 * v + 3:])
    rows = list(range(0, n, 137)) + [n - 1]
    _check(x[rows], y[rows], 1.0, 2, lg.TokenStats(*[t[rows] for t in r]))
    with pytest.raises(m.MLoRAError):                       # one row for all
        lg.token_logprobs(x[:1].expand(4, v), y[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_between_the_logits_at_another_distance(dtype):
    """rows that overlap no row of the logits although they lie between them, and one row in place with any distance"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    n, v = 5, 1000
    g = torch.Generator(device="cuda").manual_seed(4)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.randn(6 * n * v, generator=g, device="cuda").to(dt)
    x = torch.as_strided(buf, (n, v), (5000, 1))                     # [0, 1000), [5000, 6000), .. [20000, 21000)
    d = torch.as_strided(buf, (n, v), (4300, 1), 1300)               # [1300, 2300), [5600 ..: one reaches into a row
    y = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.randn(n, generator=g, device="cuda")
    rest = buf.clone()
    r = lg.token_logprobs(x, y)
    import rl_step_gb300 as m
    with pytest.raises(m.MLoRAError):
        lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, dl, out=d)
    assert torch.equal(buf, rest)
    d = torch.as_strided(buf, (n, v), (5500, 1), 1700)               # 1700, 7200, 12700, 18200 and 23700 on
    want = lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, dl)
    lg.token_logprobs_backward(x, r.lse, r.entropy, y, dl, dl, out=d)
    assert torch.equal(d, want)
    d.copy_(torch.as_strided(rest, (n, v), (5500, 1), 1700))
    assert torch.equal(buf, rest)
    # one row: its distance to the next says nothing
    es = x.element_size()
    c = lg._Logits(x.data_ptr(), y.data_ptr(), None, 5000, 1, v, lg._dtype(dt), 1.0, 0)
    q = lg._TokenGrads(r.lse.data_ptr(), r.entropy.data_ptr(), None, dl.data_ptr(), dl.data_ptr(), None, None)
    stream = torch.cuda.current_stream().cuda_stream
    assert lg._lib().mlora_token_logprobs_backward(ctypes.byref(c), ctypes.byref(q), x.data_ptr() + es, v, stream) == -1
    assert lg._lib().mlora_token_logprobs_backward(ctypes.byref(c), ctypes.byref(q), x.data_ptr(), v, stream) == 0
    assert torch.equal(x[0], want[0]) and torch.equal(buf[1000:], rest[1000:])


@pytest.mark.gpu
def test_rows_beyond_two_gigabytes():
    """offsets beyond 31 bits: the last rows of 2.4 G logits"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    n, v = 17000, 140000
    x = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 15339, 15340, n - 1]
    for i in rows:
        x[i] = (torch.randn(v, generator=g, device="cuda") * 2).bfloat16()
    y = torch.full((n,), v - 1, dtype=torch.int32, device="cuda")
    r = lg.token_logprobs(x, y, top=4)
    _check(x[rows], y[rows], 1.0, 4, lg.TokenStats(*[t[rows] for t in r]))
    assert (r.top_ids[1] == torch.arange(4, device="cuda")).all()
    xs = x[n - 1].double().cpu().numpy()[None]
    lg.token_logprobs_backward(x, r.lse, targets=y, d_logprobs=torch.ones(n, device="cuda"), out=x)
    want, _ = _gradient(xs, 1.0, [v - 1], r.lse[n - 1:].double().cpu().numpy(), [0], [1.0], None, None, None, None)
    d = np.abs(x[n - 1].double().cpu().numpy() - want[0])
    assert (d <= 2.0 ** -8 * np.abs(want[0]) + 1e-4 * np.abs(want[0]) + 1e-38).all()


@pytest.mark.gpu
def test_captured_on_another_stream_and_two_at_once():
    torch = _torch()
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 40, 20000, "bf16", seed=4)
    dl = torch.randn(40, device="cuda")
    graphs, outs, xs = [], [], []
    side = torch.cuda.Stream()
    for k in range(2):
        xk, yk = x.clone(), y.clone()
        dk = torch.empty_like(xk)
        side.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            r = lg.token_logprobs(xk, yk, top=5)
            lg.token_logprobs_backward(xk, r.lse, r.entropy, yk, dl, d_entropy=dl, out=dk)
        graphs.append(gr)
        outs.append((r, dk))
        xs.append((xk, yk))
    for step in range(2):
        for k, (xk, yk) in enumerate(xs):
            xk.copy_(torch.roll(x, step + 3 * k, 1))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for (xk, yk), (r, dk) in zip(xs, outs):
            want = lg.token_logprobs(xk, yk, top=5)
            assert all(torch.equal(a, b) for a, b in zip(r, want))
            assert torch.equal(dk, lg.token_logprobs_backward(xk, want.lse, want.entropy, yk, dl, d_entropy=dl))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r = lg.token_logprobs(x, y, top=5, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(r.lse, lg.token_logprobs(x, y, top=5).lse)


@pytest.mark.gpu
def test_python_refusals():
    torch = _torch()
    import rl_step_gb300 as m
    import rl_step_gb300.logits as lg
    _, x, y = _case(torch, 4, 100, "fp32")
    lse = torch.zeros(4, device="cuda")
    for bad in (lambda: lg.token_logprobs(x[0], y), lambda: lg.token_logprobs(x.half(), y), lambda: lg.token_logprobs(x.cpu()),
                lambda: lg.token_logprobs(x.t()), lambda: lg.token_logprobs(x, y.long()), lambda: lg.token_logprobs(x, y[:3]),
                lambda: lg.token_logprobs(x, y.cpu()),
                lambda: lg.token_logprobs_backward(x, lse[:3], targets=y, d_logprobs=lse),
                lambda: lg.token_logprobs_backward(x, lse, targets=y, d_logprobs=lse.double()),
                lambda: lg.token_logprobs_backward(x, lse, targets=y, d_logprobs=lse, out=x.bfloat16()),
                lambda: lg.token_logprobs_backward(x, lse, d_top=torch.zeros(4, 2, device="cuda")),
                lambda: lg.token_logprobs_backward(x, lse, d_top=torch.zeros(4, 2, device="cuda"), top_ids=y)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lg.token_logprobs(x, y, top=33), lambda: lg.token_logprobs(x, y, scale=-1.0),
                lambda: lg.token_logprobs(x[:, :0]),
                lambda: lg.token_logprobs_backward(x, None, targets=y, d_logprobs=lse),
                lambda: lg.token_logprobs_backward(x, lse, d_logprobs=lse),
                lambda: lg.token_logprobs_backward(x, lse, d_entropy=lse),
                lambda: lg.token_logprobs_backward(x[:3], lse[:3], targets=y[:3], d_logprobs=lse[:3], out=x[1:])):
        with pytest.raises(m.MLoRAError):
            bad()


# ----------------------------------------------------------------------------
# the transformer model's rows
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("lm,max_tokens", [("recompute", 640), ("keep_logits", 640), ("recompute", 64)])
def test_stats_of_the_transformers_rows(lm, max_tokens):
    """against the oracle's logits, and against mlora_tf_forward; the handle's next step is not changed by them"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    import rl_step_gb300.transformer as t
    from test_rollout import Setup
    s = Setup(max_tokens=max_tokens, qk_std=0.05)
    t.tf_set_lm_backward(s.h, lm)
    rng = np.random.default_rng(3)
    lens = [200, 77, 130, 1, 150] if max_tokens > 100 else [30, 9]
    ads = np.repeat(np.arange(len(lens)) % 3, lens)
    pos = np.concatenate([np.arange(k) for k in lens])
    n = len(pos)
    toks, tgts = rng.integers(0, s.cfg.vocab, n), rng.integers(0, s.cfg.vocab, n)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(toks), i32(tgts), i32(pos), i32(ads))
    lp = t.tf_forward(s.h, *args)
    dl = torch.randn(n, device="cuda")

    def step():
        out, _ = t.tf_forward_backward_custom(s.h, *args, dl)
        g = t.tf_read_adapter(s.h, 0, 0, "q", "A", "grad").clone()
        t.tf_optim_step(s.h, lr=0.0)
        return out.clone(), g

    first = step()
    r = lg.tf_forward_stats(s.h, *args, top=7)
    # the same fp32 logits, their sums in another order: both within e of the definition's, twice
    assert (lp - r.logprobs).abs().max().item() <= 2 * _e(s.cfg.vocab) + 12 * U * (1 + lp.abs().max().item()) + 2.0 ** -20
    again = step()
    assert torch.equal(first[0], again[0])
    assert torch.allclose(first[1], again[1], rtol=1e-4, atol=1e-6 * first[1].abs().max().item())   # atomics' order
    # the distribution: entropy, alternatives and target agree with one another over scales
    for scale in (1.0, 0.5):
        w = lg.tf_forward_stats(s.h, *args, top=32, scale=scale)
        assert (w.top_ids >= 0).all() and (w.top_logprobs[:, :-1] >= w.top_logprobs[:, 1:]).all()
        assert torch.equal(w.top_ids[:, :7], r.top_ids)
        assert (w.entropy > 0).all() and (w.entropy <= math.log(s.cfg.vocab) * 1.0001).all()
        hit = w.top_ids == args[1][:, None]
        rows = hit.any(1)
        assert torch.equal(w.top_logprobs[hit], w.logprobs[rows])
    none = lg.tf_forward_stats(s.h, args[0], None, *args[2:], top=7)
    assert none.logprobs is None and torch.equal(none.entropy, r.entropy) and torch.equal(none.top_ids, r.top_ids)
    # a bad token is flagged and gets nothing
    bad = args[0].clone()
    bad[3] = s.cfg.vocab
    b = lg.tf_forward_stats(s.h, bad, *args[1:], top=7)
    assert t.tf_check_status(s.h) == -2
    assert torch.isnan(b.logprobs[3]) and torch.isnan(b.entropy[3]) and (b.top_ids[3] == -1).all()


@pytest.mark.gpu
def test_stats_of_the_transformer_match_the_oracle():
    torch = _torch()
    import rl_step_gb300.logits as lg
    from test_rollout import Setup
    s = Setup(max_tokens=256, qk_std=0.05)
    rng = np.random.default_rng(8)
    lens = [90, 33]
    ads, pos = np.repeat([0, 2], lens), np.concatenate([np.arange(k) for k in lens])
    toks = rng.integers(0, s.cfg.vocab, 123)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    r = lg.tf_forward_stats(s.h, i32(toks), i32(toks), i32(pos), i32(ads), top=3)
    # every id's logprob of each row from the oracle: a column of targets at a time
    cols = rng.choice(s.cfg.vocab, 5, replace=False)
    for cidx in cols:
        want = s.o.forward(toks, np.full(123, cidx), pos, ads)
        got = lg.tf_forward_stats(s.h, i32(toks), i32(np.full(123, cidx)), i32(pos), i32(ads)).logprobs
        assert np.abs(got.cpu().numpy() - want).max() <= 2e-2          # the model's own bound
    best = r.top_ids[:, 0].cpu().numpy()
    want = s.o.forward(toks, best, pos, ads)
    assert np.abs(r.top_logprobs[:, 0].cpu().numpy() - want).max() <= 2e-2


@pytest.mark.gpu
@pytest.mark.parametrize("fails", [1, 2])
def test_a_step_after_statistics_that_failed(fails):
    """a launch of the statistics fails (by the library's hook, on the host): the error is returned, and the logits that are
    in the backward's buffer by then are none of the next step's"""
    torch = _torch()
    import rl_step_gb300 as m
    import rl_step_gb300.logits as lg
    import rl_step_gb300.transformer as t
    from test_rollout import Setup
    hook = lg._lib().mlk_test_fail_stats_at
    hook.restype, hook.argtypes = None, [ctypes.c_int64]
    s = Setup(max_tokens=640, qk_std=0.05, vocab=990)    # 992 .. 1023: columns that the backward reads and does not write
    rng = np.random.default_rng(5)
    n = 600                                              # five tiles of rows, two at a time
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(rng.integers(0, s.cfg.vocab, n)), i32(rng.integers(0, s.cfg.vocab, n)), i32(np.arange(n)), i32(np.zeros(n)))
    dl = torch.randn(n, device="cuda")

    def step():
        out, _ = t.tf_forward_backward_custom(s.h, *args, dl)
        g = t.tf_read_adapter(s.h, 0, 0, "q", "A", "grad").clone()
        t.tf_optim_step(s.h, lr=0.0)
        return out.clone(), g

    first = step()
    hook(fails)
    with pytest.raises(m.MLoRAError):
        lg.tf_forward_stats(s.h, *args, top=3)
    again = step()
    assert torch.equal(first[0], again[0]) and torch.isfinite(again[1]).all()
    assert torch.allclose(first[1], again[1], rtol=1e-4, atol=1e-6 * first[1].abs().max().item())   # atomics' order
    assert torch.isfinite(lg.tf_forward_stats(s.h, *args, top=3).entropy).all()                     # the hook is off again


@pytest.mark.gpu
def test_statistics_captured_replayed_and_on_another_stream():
    """the batch is read at replay; the same bits as calls outside a graph"""
    torch = _torch()
    import rl_step_gb300.logits as lg
    from test_rollout import Setup
    s = Setup(max_tokens=640, qk_std=0.05)
    rng = np.random.default_rng(6)
    n = 500
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pos, ads = i32(np.r_[np.arange(350), np.arange(150)]), i32(np.r_[np.zeros(350), np.ones(150)])
    batches = [(i32(rng.integers(0, s.cfg.vocab, n)), i32(rng.integers(0, s.cfg.vocab, n)), pos, ads) for _ in range(2)]
    want = [lg.tf_forward_stats(s.h, *b, top=6, scale=0.7) for b in batches]
    held = tuple(t.clone() for t in batches[0])
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        r = lg.tf_forward_stats(s.h, *held, top=6, scale=0.7)
    for k in (0, 1, 0):
        for d, t in zip(held, batches[k]):
            d.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want[k]))
    side.wait_stream(torch.cuda.current_stream())
    r = lg.tf_forward_stats(s.h, *batches[1], top=6, scale=0.7, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, want[1]))
    empty = lg.tf_forward_stats(s.h, *[t[:0] for t in batches[0]], top=6)
    assert empty.lse.shape == (0,) and empty.top_ids.shape == (0, 6)
