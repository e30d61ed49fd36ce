"""Rollouts of the transformer model over its 8-bit caches, and the iteration
they are part of: prompts, drafted and single tokens, next tokens, a policy
step on them, a clipped update, and rollouts with the updated adapters.

The reference is the CPU model in doubles with one change: attention reads the
keys and values that the caches hold (read back exactly).  So the tolerance is
that of the model's bf16 activations alone, 2e-2 on logprobs, as for its forward.
What the caches hold is tested apart: against the model's own rotated keys and
values, whose distance is at most 2^-4 of each value by the rounding to e4m3
(a page's small values: 2^-10 of its scale, below 2^-10 of its largest value),
plus the activations' storage, 2.5e-2 as for gradients.
"""
import ctypes
import math

import numpy as np
import pytest

import oracle
import workloads.transformer as wt
from _gpu_util import dev, rel_fro
from oracle import transformer_oracle as to

LP_TOL = 2e-2
PAGE = 64


def test_rollout_refuses_without_a_handle():
    import __graft_entry__
    __graft_entry__.build()
    import rl_step_gb300.kv as kv
    lib = kv._lib()
    b, c = kv._TfBatch(), kv._TfContext()
    p = ctypes.c_void_p(4096)
    assert lib.mlora_tf_forward_cached(None, ctypes.byref(b), ctypes.byref(c), p, None) == -1
    assert lib.mlora_tf_sample_cached(None, ctypes.byref(b), ctypes.byref(c), p, p, p, None) == -1
    assert b"NULL" in lib.mlora_last_error()


def test_context_struct_and_binding_agree(tmp_path):
    import os
    import shutil
    import subprocess
    import rl_step_gb300.kv as kv
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    fields = [f[0] for f in kv._TfContext._fields_]
    body = "".join(f'printf("%zu ", offsetof(mlora_tf_context, {f}));' for f in fields)
    (tmp_path / "a.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mlora_kv.h"\nint main(void) {'
                                  + body + 'printf("%zu", sizeof(mlora_tf_context)); return 0; }')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", include, str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True, capture_output=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(kv._TfContext, f).offset for f in fields] + [ctypes.sizeof(kv._TfContext)]


def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch


def _handle(cfg, base, ad, max_tokens):
    import rl_step_gb300.transformer as t
    dbase = {"E": dev(base["E"]), "Wout": dev(base["Wout"]), "final_norm": dev(base["final_norm"]),
             "attn_norm": [dev(g) for g in base["attn_norm"]], "mlp_norm": [dev(g) for g in base["mlp_norm"]],
             "W": {p: [dev(w) for w in base["W"][p]] for p in t.PROJ}}
    A = {p: [[dev(x) for x in row] for row in ad["A"][p]] for p in t.PROJ}
    B = {p: [[dev(x) for x in row] for row in ad["B"][p]] for p in t.PROJ}
    return t.tf_create(cfg.vocab, cfg.d_model, cfg.n_heads, cfg.n_kv_heads, cfg.d_ffn, cfg.n_layers, cfg.ranks,
                       cfg.alphas, max_tokens, dbase, A, B, rope_theta=cfg.rope_theta, rms_eps=cfg.rms_eps)


class Setup:
    def __init__(self, max_tokens=1024, **overrides):
        self.cfg = wt.get_tf_config("tf_small", **overrides)
        self.base, self.ad = wt.make_tf_base_weights(self.cfg), wt.make_tf_adapters(self.cfg)
        self.h = _handle(self.cfg, self.base, self.ad, max_tokens)
        c = self.cfg
        self.o = oracle.TransformerOracle(self.base, self.ad, c.ranks, c.alphas, c.n_heads, c.n_kv_heads, c.head_dim,
                                          c.rope_theta, c.rms_eps)

    def caches(self, n_pages):
        import rl_step_gb300.kv as kv
        return [kv.KvCache.empty(n_pages, self.cfg.n_kv_heads, self.cfg.head_dim) for _ in range(self.cfg.n_layers)]


@pytest.fixture(scope="module")
def small():
    _torch()
    return Setup(qk_std=0.05)


def _tables(torch, lengths, seed=3):
    """page table [n, width] of shuffled page ids, and the number of pages"""
    need = [-(-n // PAGE) for n in lengths]
    ids = np.random.default_rng(seed).permutation(sum(need) + 3)
    table = np.full((len(lengths), max(need)), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = ids[at:at + k]
        at += k
    return torch.from_numpy(table).cuda(), len(ids)


def _int(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _reference(o, toks, ids, kc, vc):
    """logprob rows' hidden states of flattened sequences with keys and values given"""
    pos = np.concatenate([np.arange(len(t)) for t in toks])
    flat = np.concatenate(toks)
    ad = np.concatenate([np.full(len(t), a) for t, a in zip(toks, ids)])
    ends = np.cumsum([len(t) for t in toks])
    seqs = [np.arange(e - len(t), e) for t, e in zip(toks, ends)]
    groups = {int(a): np.nonzero(ad == a)[0] for a in np.unique(ad)}
    x = to._widen(o._E[flat])
    ks, vs = [], []
    for l in range(o.L):
        y, _ = to.rmsnorm(x, o.g_attn[l], o.eps)
        q = to.rope(o._proj("q", l, y, groups, None), pos, o.nh, o.hd, o.theta)
        ks.append(to.rope(o._proj("k", l, y, groups, None), pos, o.nkv, o.hd, o.theta))
        vs.append(o._proj("v", l, y, groups, None))
        att, _ = to.attention(q, kc[l], vc[l], seqs, o.nh, o.nkv, o.hd)
        x = x + o._proj("o", l, att, groups, None)
        y, _ = to.rmsnorm(x, o.g_mlp[l], o.eps)
        g, u = o._proj("gate", l, y, groups, None), o._proj("up", l, y, groups, None)
        x = x + o._proj("down", l, oracle.silu(g) * u, groups, None)
    return to.rmsnorm(x, o.g_final, o.eps)[0], ks, vs


def _read_back(torch, s, caches, table, lengths):
    import rl_step_gb300.kv as kv
    off = np.concatenate([[0], np.cumsum(lengths)])
    n = int(off[-1])
    out = [[], []]
    for c in caches:
        k, v = kv.kv_read(c, table, _int(torch, lengths), n, row_off=_int(torch, off), max_rows=max(lengths))
        for dst, x in zip(out, (k, v)):
            dst.append(x.double().cpu().numpy().reshape(n, -1))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("cut", [False, True])
def test_rollout_logprobs_match_the_model_on_cached_keys(small, cut):
    """ragged prompts in two parts, three drafted tokens, then single tokens across a page's end"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = small
    rng = np.random.default_rng(5)
    total = [170, 1 + 3 + 9, 64 + 3 + 9, 130, 64 + 40, 30]
    ids = [0, 2, 1, 0, 2, 1]
    toks = [rng.integers(0, s.cfg.vocab, n + 1).astype(np.int32) for n in total]
    table, n_pages = _tables(torch, total)
    caches = s.caches(n_pages)
    ws = kv.kv_workspace(nbytes=kv.WORKSPACE_BYTES if cut else 0)
    done = [0] * len(total)
    got = [np.full(n, np.nan) for n in total]

    def step(counts):
        rows = [toks[i][done[i]:done[i] + n] for i, n in enumerate(counts)]
        tgt = [toks[i][done[i] + 1:done[i] + n + 1] for i, n in enumerate(counts)]
        ad = np.concatenate([np.full(n, a) for n, a in zip(counts, ids)])
        off = np.concatenate([[0], np.cumsum(counts)])
        now = [d + n for d, n in zip(done, counts)]
        single = set(counts) == {1}
        lp = kv.tf_forward_cached(s.h, caches, _int(torch, np.concatenate(rows)), _int(torch, np.concatenate(tgt)),
                                  _int(torch, ad), table, _int(torch, now), max(now),
                                  row_off=None if single else _int(torch, off), max_rows=max(counts), workspace=ws)
        lp = lp.cpu().numpy()
        for i, n in enumerate(counts):
            got[i][done[i]:done[i] + n] = lp[off[i]:off[i + 1]]
            done[i] += n

    prompt = [n - 12 for n in total]
    step([n // 2 for n in prompt])                      # a sequence of one token has no row here
    step([n - n // 2 for n in prompt])
    step([3] * len(total))
    for _ in range(9):
        step([1] * len(total))
    assert done == total
    assert t.tf_check_status(s.h) == 0 and all(kv.kv_check_status(c) == 0 for c in caches)
    kc, vc = _read_back(torch, s, caches, table, total)
    xf, ks, vs = _reference(s.o, [x[:-1] for x in toks], ids, kc, vc)
    ref = s.o.logprobs_from_hidden(xf, np.concatenate([x[1:] for x in toks]))[0]
    err = np.abs(np.concatenate(got) - ref)
    print(f"\nlogprob max|err| {err.max():.2e}, rms {np.sqrt((err ** 2).mean()):.2e}")
    assert err.max() <= LP_TOL
    for have, want in ((kc, ks), (vc, vs)):
        for l in range(s.o.L):
            assert rel_fro(have[l], want[l]) <= 2.0 ** -4 + 2.0 ** -10 * 8 + 2.5e-2


@pytest.mark.gpu
def test_padded_rows_and_bad_rows(small):
    """empty slots, rows behind the last sequence, a bad adapter, token, length and page"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = small
    rng = np.random.default_rng(6)
    n = 7
    table, n_pages = _tables(torch, [100] * n)
    caches = s.caches(n_pages)
    ws = kv.kv_workspace(nbytes=0)                     # rows do not depend on the batch
    prompt = rng.integers(0, s.cfg.vocab, 70 * n).astype(np.int32)
    ad = np.repeat(np.arange(n) % 3, 70)
    off = np.arange(n + 1) * 70
    kv.tf_forward_cached(s.h, caches, _int(torch, prompt), None, _int(torch, ad), table, _int(torch, [70] * n), 70,
                         row_off=_int(torch, off), max_rows=70, workspace=ws)
    tok, tgt, ad1 = rng.integers(0, s.cfg.vocab, n), rng.integers(0, s.cfg.vocab, n), np.arange(n) % 3

    def decode(tok, tgt, ad1, lens, tab, max_len=71):
        lp = kv.tf_forward_cached(s.h, caches, _int(torch, tok), _int(torch, tgt), _int(torch, ad1), tab,
                                  _int(torch, lens), max_len, workspace=ws)
        return lp.cpu().numpy(), t.tf_check_status(s.h), [kv.kv_check_status(c) for c in caches]

    full, rc, crc = decode(tok, tgt, ad1, [71] * n, table)
    assert np.isfinite(full).all() and rc == 0 and crc == [0] * s.cfg.n_layers
    lens = [71] * n
    lens[2] = 0                                        # an empty slot: NaN, no error
    lp, rc, crc = decode(tok, tgt, ad1, lens, table)
    assert np.isnan(lp[2]) and rc == 0 and crc == [0] * s.cfg.n_layers
    keep = np.arange(n) != 2
    assert np.array_equal(lp[keep], full[keep])
    # three rows behind the last sequence
    lp = kv.tf_forward_cached(s.h, caches, _int(torch, tok), _int(torch, tgt), _int(torch, ad1), table[:4],
                              _int(torch, [71] * 4), 71, workspace=ws).cpu().numpy()
    assert np.array_equal(lp[:4], full[:4]) and np.isnan(lp[4:]).all() and t.tf_check_status(s.h) == 0
    for what in ("adapter", "token", "target", "length", "max_len", "page"):
        tk, tg, aa, ll, tab = tok.copy(), tgt.copy(), ad1.copy(), [71] * n, table.clone()
        bad = 3
        if what == "adapter":
            aa[bad] = 3
        elif what == "token":
            tk[bad] = s.cfg.vocab
        elif what == "target":
            tg[bad] = -1
        elif what == "length":
            ll[bad] = -5
        elif what == "max_len":
            ll[bad] = 72
        else:
            tab[bad, 1] = n_pages
        before = [[x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)] for c in caches]
        lp, rc, crc = decode(tk, tg, aa, ll, tab)
        assert np.isnan(lp[bad]), what
        keep = np.arange(n) != bad
        assert np.array_equal(lp[keep], full[keep]), what
        assert rc == (0 if what == "page" else -2), what
        if what in ("length", "max_len", "page"):
            assert crc == [-2] * s.cfg.n_layers
        else:
            assert crc == [0] * s.cfg.n_layers
        for c, old in zip(caches, before):             # the bad row's page is put back
            for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old):
                x.copy_(y)
        assert np.array_equal(decode(tok, tgt, ad1, [71] * n, table)[0], full)
    nothing = kv.tf_forward_cached(s.h, caches, _int(torch, tok), _int(torch, tgt), _int(torch, ad1), table[:0],
                                   _int(torch, []), 71, workspace=ws, row_off=_int(torch, [0]), max_rows=0)
    assert torch.isnan(nothing).all() and t.tf_check_status(s.h) == 0


@pytest.mark.gpu
def test_refusals_of_a_context(small):
    torch = _torch()
    import rl_step_gb300.kv as kv
    s = small
    table, n_pages = _tables(torch, [10, 10])
    caches = s.caches(n_pages)
    z = _int(torch, [1, 2])
    args = (s.h, caches, z, z, z, table, _int(torch, [1, 1]))
    for kw in (dict(max_len=0), dict(max_len=1025), dict(max_len=1, max_rows=2)):
        with pytest.raises(Exception):
            kv.tf_forward_cached(*args, **kw)
    with pytest.raises(ValueError):
        kv.tf_forward_cached(s.h, caches[:1], *args[2:], max_len=1)
    for bad in (kv.KvCache.empty(n_pages, 2, 64), kv.KvCache.empty(n_pages, 4, 128)):
        with pytest.raises(Exception):
            kv.tf_forward_cached(s.h, [caches[0], bad], *args[2:], max_len=1)
    with pytest.raises(ValueError):
        kv.tf_sample_cached(s.h, caches, z, z, torch.zeros(3, device="cuda"), table, z, 1)


@pytest.mark.gpu
def test_next_tokens_invert_the_distribution(small):
    """one prompt in 200 slots, their whole distribution from the rows' logprobs, 200 uniforms.

    Tolerance on the distribution function: a tile's and a column's fp32 running sums add at most
    4 + 256 terms, 300 u; the logits of the picked tile are formed again, both sides with fp32 sums of d
    products: 2 d u |x| |w| on a logit, the same relative change of its probability."""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = small
    n, T = 200, 5
    rng = np.random.default_rng(8)
    prompt = rng.integers(0, s.cfg.vocab, T).astype(np.int32)
    table = _int(torch, np.arange(n)[:, None])
    caches = s.caches(n)
    ws = kv.kv_workspace(nbytes=0)
    off = _int(torch, np.arange(n + 1) * T)
    ad = _int(torch, np.full(n * T, 1))
    toks = _int(torch, np.tile(prompt, n))
    lens = _int(torch, [T] * n)
    u = torch.linspace(0, 1, n, device="cuda")[:-1]
    u = torch.cat([u, torch.tensor([0.9999999], device="cuda")])
    kv.tf_forward_cached(s.h, caches, toks, None, ad, table, lens, T, row_off=off, max_rows=T, workspace=ws)
    dist = []
    one, last = _int(torch, np.full(n, 1)), _int(torch, np.full(n, prompt[-1]))
    nxt, lp = kv.tf_sample_cached(s.h, caches, last, one, u, table, lens, T, workspace=ws)
    for v0 in range(0, s.cfg.vocab, n):                # the last row again, with every id as its target
        tgt = _int(torch, np.minimum(np.arange(v0, v0 + n), s.cfg.vocab - 1))
        dist.append(kv.tf_forward_cached(s.h, caches, last, tgt, one, table, lens, T, workspace=ws))
    logp = torch.cat(dist)[:s.cfg.vocab].double().cpu().numpy()
    assert t.tf_check_status(s.h) == 0
    cdf = np.cumsum(np.exp(logp))
    eps = 2.0 ** -24
    wmax = np.sqrt((s.o.Wout ** 2).sum(1).max())
    xnorm = np.sqrt(s.cfg.d_model) * np.abs(s.o.g_final).max()
    dz = 2 * s.cfg.d_model * eps * wmax * xnorm
    tol = 300 * eps + 2 * dz + 1e-5                    # 1e-5: __expf and the fp32 logprobs, a few 2^-20
    nxt, lp, u = nxt.cpu().numpy(), lp.cpu().numpy().astype(np.float64), u.double().cpu().numpy()
    assert (nxt >= 0).all() and (np.diff(nxt) >= 0).all()
    assert (cdf[nxt] + tol > u).all()
    assert (np.where(nxt > 0, cdf[nxt - 1], 0.0) - tol <= u).all()
    assert (np.abs(lp - logp[nxt]) <= dz + 8 * eps * np.abs(logp[nxt]) + 1e-5).all()
    # slots without a row, bad uniforms
    lens2 = lens.clone()
    lens2[3] = 0
    u2 = torch.full((n,), 0.5, device="cuda")
    a, la = kv.tf_sample_cached(s.h, caches, last, one, u2, table, lens2, T, workspace=ws)
    assert t.tf_check_status(s.h) == 0
    assert int(a[3]) == -1 and bool(torch.isnan(la[3])) and int((a >= 0).sum()) == n - 1
    u2[7] = 1.0
    u2[9] = float("nan")
    b, lb = kv.tf_sample_cached(s.h, caches, last, one, u2, table, lens2, T, workspace=ws)
    assert t.tf_check_status(s.h) == -2
    assert sorted(np.nonzero(b.cpu().numpy() < 0)[0].tolist()) == [3, 7, 9]
    none, _ = kv.tf_sample_cached(s.h, caches, last[:0], one[:0], u2[:0], table[:0], lens[:0], T, workspace=ws)
    assert none.numel() == 0
    c, lc = kv.tf_sample_cached(s.h, caches, last[:0], one[:0], u2, table, lens2, T, workspace=ws,
                                row_off=_int(torch, [0] * (n + 1)), max_rows=1)
    assert (c == -1).all() and torch.isnan(lc).all()


@pytest.mark.gpu
def test_an_iteration_of_rollout_policy_step_and_clipped_update():
    """prompts, 70 sampled tokens a sequence (eager, and the same as a replayed graph), PPO on them with
    the sampled logprobs, an update clipped per adapter, and a rollout that sees the new weights"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = Setup(qk_std=0.05)
    rng = np.random.default_rng(9)
    ids = np.array([0, 1, 2, 1, 0])
    plen = np.array([3, 64, 17, 100, 1])
    n, G = len(ids), 70
    full = plen + G
    table, n_pages = _tables(torch, full.tolist())
    prompts = [rng.integers(0, s.cfg.vocab, k).astype(np.int32) for k in plen]
    off = np.concatenate([[0], np.cumsum(plen)])
    uni = torch.rand(G, n, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    ad1 = _int(torch, ids)
    max_len = int(full.max())

    def rollout(graph):
        caches = s.caches(n_pages)
        ws = kv.kv_workspace()
        toks, lps = torch.zeros(G, n, dtype=torch.int32, device="cuda"), torch.zeros(G, n, device="cuda")
        tok, lp = kv.tf_sample_cached(s.h, caches, _int(torch, np.concatenate(prompts)),
                                      _int(torch, np.repeat(ids, plen)), uni[0].contiguous(), table, _int(torch, plen),
                                      max_len, row_off=_int(torch, off), max_rows=int(plen.max()), workspace=ws)
        toks[0], lps[0] = tok, lp
        cur, lens, u = tok.clone(), _int(torch, plen + 1), uni[1].clone()

        def decode():
            kv.tf_sample_cached(s.h, caches, cur, ad1, u, table, lens, max_len, workspace=ws, next_out=tok,
                                logprob_out=lp)
        g = None
        for i in range(1, G):
            u.copy_(uni[i])
            if graph and i == 2:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    decode()
            if g is None:
                decode()
            else:
                g.replay()
            toks[i], lps[i] = tok, lp
            cur.copy_(tok)
            lens += 1
        assert t.tf_check_status(s.h) == 0 and all(kv.kv_check_status(c) == 0 for c in caches)
        return toks.cpu().numpy(), lps.cpu().numpy()

    toks, lps = rollout(False)
    toks_g, lps_g = rollout(True)
    assert np.array_equal(toks, toks_g) and np.array_equal(lps, lps_g)      # bit for bit
    assert (toks >= 0).all() and np.isfinite(lps).all()
    # PPO on the sampled tokens: the prompt's rows get no advantage
    seqs = [np.concatenate([p, toks[:, i]]) for i, p in enumerate(prompts)]
    tokens = np.concatenate([x[:-1] for x in seqs])
    targets = np.concatenate([x[1:] for x in seqs])
    positions = np.concatenate([np.arange(len(x) - 1) for x in seqs])
    ads = np.concatenate([np.full(len(x) - 1, a) for x, a in zip(seqs, ids)])
    sampled = np.concatenate([np.concatenate([np.zeros(k - 1), lps[:, i]]) for i, k in enumerate(plen)])
    adv = np.concatenate([np.concatenate([np.zeros(k - 1), np.full(G, 1.0 + i)]) for i, k in enumerate(plen)])
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")
    lp, _ = t.tf_forward_backward(s.h, _int(torch, tokens), _int(torch, targets), _int(torch, positions),
                                  _int(torch, ads), "ppo", advantages=f32(adv), sampler_logprobs=f32(sampled),
                                  clip_eps=0.2)
    assert t.tf_check_status(s.h) == 0 and torch.isfinite(lp).all()
    read = lambda a, kind: {(l, p, f): t.tf_read_adapter(s.h, a, l, p, f, kind).double().cpu().numpy()
                            for l in range(s.cfg.n_layers) for p in t.PROJ for f in "AB"}
    grads = [read(a, "grad") for a in range(3)]
    weights = [read(a, "weight") for a in range(3)]
    norms = [math.sqrt(sum(float((x * x).sum()) for x in g.values())) for g in grads]
    assert min(norms) > 0
    max_norm = sorted(norms)[1] * 0.9                   # two adapters are clipped, one is not
    skipped, got = t.tf_optim_step_clipped(s.h, max_norm, lr=1e-3)
    eps = 2.0 ** -24
    assert t.tf_check_status(s.h) == 0 and skipped.sum().item() == 0
    for a in range(3):
        assert abs(float(got[a]) - norms[a]) <= 35 * eps * norms[a]
        f = min(1.0, max_norm / norms[a])
        m, w = read(a, "m"), read(a, "weight")
        b1, b2 = float(np.float32(0.9)), float(np.float32(0.999))
        for key, x in grads[a].items():
            g = f * x
            # the factor 36 u, its product u, 1 - b1 and the product with it 2 u
            assert (np.abs(m[key] - (1 - b1) * g) <= 40 * eps * np.abs((1 - b1) * g) + 1e-40).all()
            want = oracle.adam_update(weights[a][key], g, 0.0, 0.0, 1, 1e-3, b1, b2, 1e-8, 0.0)[0]
            # the update, at most lr: the moments' 40 u and 78 u / 2, a few u of its own arithmetic; the weight's rounding
            assert (np.abs(w[key] - want) <= 1e-3 * 128 * eps + 1.01 * eps * np.abs(want)).all()
    after, lps2 = rollout(False)
    assert np.isfinite(lps2).all() and not np.array_equal(lps2, lps)        # the new weights


@pytest.mark.gpu
def test_two_streams_and_one_handle_each():
    """rollouts of two handles on two streams at once give what each gives alone"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    hs = [Setup(qk_std=0.05), Setup(qk_std=0.05, seed=2002)]
    rng = np.random.default_rng(11)
    data = []
    for s in hs:
        table, n_pages = _tables(torch, [90, 33, 128])
        toks = _int(torch, rng.integers(0, s.cfg.vocab, 251))
        data.append((s, table, n_pages, toks, _int(torch, [0, 90, 123, 251]), _int(torch, np.repeat([0, 1, 2], [90, 33, 128])),
                     _int(torch, [90, 33, 128]), kv.kv_workspace()))

    def run(d, caches, lp, stream=None):
        s, table, n_pages, toks, off, ad, lens, ws = d
        kv.tf_forward_cached(s.h, caches, toks, toks, ad, table, lens, 128, row_off=off, max_rows=128, workspace=ws,
                             logprobs_out=lp, stream=stream)

    caches = [d[0].caches(d[2]) for d in data]
    lps = [torch.empty(251, device="cuda") for _ in data]
    for d, c, lp in zip(data, caches, lps):
        run(d, c, lp)
    alone = [lp.clone() for lp in lps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for d, c, lp, st in zip(data, caches, lps, streams):
            run(d, c, lp, st)
    torch.cuda.synchronize()
    for a, b in zip(alone, lps):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("length", [-5, 72, 10 ** 6])
def test_a_sequence_out_of_range_leaves_its_pages(small, length):
    """a length below zero, beyond the call's max_len (but within the table) and beyond the table: nothing of the
    sequence is appended, in any layer, by rows whose keys would make every page's scale grow"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = small
    rng = np.random.default_rng(13)
    table, n_pages = _tables(torch, [100] * 3)
    caches = s.caches(n_pages)
    ws = kv.kv_workspace()
    prompt = _int(torch, rng.integers(0, s.cfg.vocab, 210))
    kv.tf_forward_cached(s.h, caches, prompt, None, _int(torch, np.repeat([0, 1, 2], 70)), table, _int(torch, [70] * 3),
                         70, row_off=_int(torch, [0, 70, 140, 210]), max_rows=70, workspace=ws)
    for c in caches:                                   # stored scales below any that the next row needs
        c.k_scale.mul_(2.0 ** -20)
        c.v_scale.mul_(2.0 ** -20)
    before = [[x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)] for c in caches]
    own = table[1, :2].long()
    tok, ad = _int(torch, [5, 6, 7]), _int(torch, [0, 1, 2])
    for call in ("forward", "sample"):
        if call == "forward":
            lp = kv.tf_forward_cached(s.h, caches, tok, tok, ad, table, _int(torch, [71, length, 71]), 71, workspace=ws)
        else:
            nxt, lp = kv.tf_sample_cached(s.h, caches, tok, ad, torch.full((3,), 0.5, device="cuda"), table,
                                          _int(torch, [71, length, 71]), 71, workspace=ws)
            assert nxt[1] == -1 and (nxt[[0, 2]] >= 0).all()
        assert torch.isnan(lp[1]) and torch.isfinite(lp[[0, 2]]).all()
        assert t.tf_check_status(s.h) == -2 and [kv.kv_check_status(c) for c in caches] == [-2] * s.cfg.n_layers
        for c, old in zip(caches, before):
            for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old):
                assert torch.equal(x[own], y[own])


@pytest.mark.gpu
def test_layers_that_share_pages_are_refused(small):
    """one pool for two layers would hold the last one's keys and values alone"""
    torch = _torch()
    import rl_step_gb300 as m
    import rl_step_gb300.kv as kv
    s = small
    z, lens, table = _int(torch, [1, 2]), _int(torch, [1, 1]), _int(torch, [[0], [1]])
    a, b = s.caches(4)[:2]
    whole = kv.KvCache.empty(6, s.cfg.n_kv_heads, s.cfg.head_dim)
    part = lambda i, j: kv.KvCache(whole.k[i:j], whole.v[i:j], whole.k_scale[i:j], whole.v_scale[i:j])
    for pair in ([a, a], [a, kv.KvCache(b.k, a.v, b.k_scale, b.v_scale)], [part(0, 4), part(2, 6)],
                 [a, kv.KvCache(b.k, b.v, a.k_scale, b.v_scale)], [a, kv.KvCache(a.v, b.v, b.k_scale, b.v_scale)]):
        with pytest.raises(m.MLoRAError):
            kv.tf_forward_cached(s.h, pair, z, z, z, table, lens, 1)
    lp = kv.tf_forward_cached(s.h, [part(0, 3), part(3, 6)], z, z, z, table, lens, 1)      # side by side
    assert torch.isfinite(lp).all()


@pytest.mark.gpu
def test_joined_attention_counts_as_a_launch(small):
    """where long sequences may be cut, each layer launches one kernel more"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.transformer as t
    s = small
    table = _int(torch, [np.arange(16)])
    caches = s.caches(16)
    z = _int(torch, [1])
    n = []
    for nbytes in (0, kv.WORKSPACE_BYTES):
        ws = kv.kv_workspace(nbytes=nbytes)
        at = t._lib().mlora_tf_kernel_launches(s.h.ptr)
        kv.tf_forward_cached(s.h, caches, z, z, z, table, _int(torch, [1]), 1024, workspace=ws)
        n.append(t._lib().mlora_tf_kernel_launches(s.h.ptr) - at)
    assert n[1] == n[0] + s.cfg.n_layers
