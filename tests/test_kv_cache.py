"""The 8-bit key/value cache (include/mlora_kv.h) against tests/_kv_model.py.

append and read move values between formats by rules without rounding choices,
so their bytes, scales and values have to be equal.

Tolerances of the attention, per element, with u = 2^-24 (fp32's half step),
A = sum_i p_i |v_i| and S = max_i |scale| sum_d |q_d k_d| of the row (doubles):
  scores: q and the bytes enter exactly (bf16) or as two fp16 parts (fp32,
    relative 2^-22); hd products are added in fp32, then scaled: at most
    d = (hd + 8) u S + 2^-22 S, and 2^-23 |s - m| log2(e) from the exponent's
    own rounding, |s - m| <= 2 S: together D = (hd + 16) u S + 2^-22 S
  each p_i then has a relative error of 2 D (itself and the sum), exp2 adds
    2^-22, the fp16 rounding of p 2^-11 (bf16) or 2^-22 (fp32), and the sums
    over n positions at most n u each
  below 2^-14 fp16's rounding is absolute, 2^-25: p_i is held as p'_i = 2^12
    2^(s_i log2(e) - m + ev_i - unit) with ev_i the exponent of its page's value
    scale, unit at most the largest of them, and m reached by some position, so
    that the result's divisor sum_i p'_i 2^(unit - ev_i) is at least 2^12.  n errors
    of 2^-25 on bytes of at most 448 < 2^9, in units of 2^unit, make at most
    n 2^-25 2^9 2^(unit - 12) = n 2^-28 2^unit <= F = n 2^-28 max_page 2^ev
  out: (4 D + P + 2 n u + 2^-20) A + F + half a step of the type, with P = 2^-11 or 2^-22
  lse: 2 D + n u + 2^-22 + 2 u |lse|
(the products' order inside a matrix instruction may truncate instead of
round: that is a full step, 2 u, which the factor 2 on D covers).
"""
import ctypes
import math

import numpy as np
import pytest

import _kv_model as M

EPS = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


# ----------------------------------------------------------------------------
# on the CPU: layout and refusals
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("hd", [64, 128])
def test_page_layout_is_a_permutation(hd):
    for m in M.maps(hd):
        assert sorted(m.reshape(-1)) == list(range(64 * hd))


@pytest.mark.parametrize("hd", [64, 128])
def test_fragment_reads_touch_distinct_banks(hd):
    """The 16-byte reads of eight consecutive lanes (token g of a key tile, or
    token quad t of a value tile) fall on 32 different 4-byte banks."""
    for j in range(2):
        for a in range(hd // 64):
            for ph in range(4):
                lanes = range(8 * ph, 8 * ph + 8)
                k = [M.byte_k(4 * ((ln // 4) >> 1) + 2 * j + ((ln // 4) & 1), (ln % 4 + 4 * a) * 16, hd)
                     for ln in lanes]
                assert sorted((x // 16) % 8 for x in k) == list(range(8))
    for m in range(hd // 32):
        for ph in range(4):
            v = [M.byte_v(4 * (ln % 4), 32 * m + 4 * (ln // 4), hd) for ln in range(8 * ph, 8 * ph + 8)]
            assert sorted((x // 16) % 8 for x in v) == list(range(8))


def test_model_rounds_like_torch():
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.linspace(-448, 448, 20001), np.logspace(-6, 2.6, 5000)]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(M.e4m3_byte(x), want)


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    import rl_step_gb300.kv as kv
    return kv, kv._lib()


def _valid():
    kv, lib = _lib()
    p = 4096                                           # never dereferenced: every call below is refused on the host
    c = kv._KvCache(p, p, p, p, None, 4, 2, 128)
    q = kv._KvSeqs(p, p, None, 3, 3, 2, 1)
    a = kv._KvAttn(p, p, p, p, 512, 512, 65536, 128, 0, 4, 0.1)
    return kv, lib, c, q, a


_BAD = [("c", "n_pages", 0), ("c", "n_kv_heads", 0), ("c", "n_kv_heads", 1025), ("c", "head_dim", 96),
        ("c", "k", None), ("c", "v_scale", None), ("c", "v", 4104), ("q", "n_seqs", -1), ("q", "n_rows", -1),
        ("q", "n_rows", 2), ("q", "n_rows", 1 << 31), ("q", "max_pages", 0), ("q", "max_rows", -1),
        ("q", "max_rows", 2), ("q", "page_table", None), ("q", "kv_len", None)]


@pytest.mark.parametrize("where,field,value", _BAD + [
    ("a", "n_heads", 3), ("a", "n_heads", 0), ("a", "scale", math.inf), ("a", "scale", math.nan), ("a", "max_len", -1),
    ("a", "q", None), ("a", "out", None), ("a", "q", 4104), ("a", "q_stride", 511), ("a", "q_stride", 516),
    ("a", "out_stride", 256), ("a", "workspace", 4104), ("a", "workspace_bytes", -1),
    ("a", "dtype", 2)])
def test_attention_refuses(where, field, value):
    kv, lib, c, q, a = _valid()
    setattr({"c": c, "q": q, "a": a}[where], field, value)
    assert lib.mlora_kv_attention(ctypes.byref(c), ctypes.byref(q), ctypes.byref(a), None) == -1
    assert lib.mlora_last_error()


@pytest.mark.parametrize("out,out_stride", [(4096, 1024), (4096 + 16, 512), (4096 + 1024, 512), (4096 - 512, 512),
                                            (4096 + 512, 1024), (4096 + 2048, 512), (4096 + 512, 768), (4096 - 2048, 1024)])
def test_attention_refuses_an_output_that_overlaps_other_queries(out, out_stride):
    """three rows of 512 elements (1 KB) at 4096 on: an output is the queries themselves, or apart from them"""
    kv, lib, c, q, a = _valid()
    a.out, a.out_stride = out, out_stride
    assert lib.mlora_kv_attention(ctypes.byref(c), ctypes.byref(q), ctypes.byref(a), None) == -1
    assert b"overlap" in lib.mlora_last_error()


@pytest.mark.parametrize("q_stride,out_stride,out", [(1 << 62, 1 << 62, 4096), (1 << 62, 512, 4096 + 1024), (512, 1 << 60, 0),
                                                     (1 << 62, 1 << 62, 4096 + 16)])
@pytest.mark.parametrize("n", [1, 3])
def test_attention_refuses_rows_beyond_memory(q_stride, out_stride, out, n):
    """distances whose products with the rows or the element size leave 64 bits"""
    kv, lib, c, q, a = _valid()
    q.n_seqs = q.n_rows = n
    a.q_stride, a.out_stride = q_stride, out_stride
    a.out = out or a.out
    assert lib.mlora_kv_attention(ctypes.byref(c), ctypes.byref(q), ctypes.byref(a), None) == -1
    assert b"apart" in lib.mlora_last_error()


@pytest.mark.parametrize("where,field,value", _BAD)
def test_append_and_read_refuse(where, field, value):
    kv, lib, c, q, _ = _valid()
    setattr({"c": c, "q": q}[where], field, value)
    p = ctypes.c_void_p(4096)
    assert lib.mlora_kv_append(ctypes.byref(c), ctypes.byref(q), 0, p, 256, p, 256, None) == -1
    assert lib.mlora_kv_read(ctypes.byref(c), ctypes.byref(q), 0, p, p, None) == -1


def test_append_refuses_rows():
    kv, lib, c, q, _ = _valid()
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    for args in ((0, None, 256, p, 256), (0, p, 256, None, 256), (0, p, 255, p, 256), (0, p, 256, p, 260),
                 (0, odd, 256, p, 256), (2, p, 256, p, 256), (1, p, 258, p, 256)):
        assert lib.mlora_kv_append(ctypes.byref(c), ctypes.byref(q), *args, None) == -1
    assert lib.mlora_kv_read(ctypes.byref(c), ctypes.byref(q), 0, odd, p, None) == -1
    q.row_off, q.max_rows, q.n_seqs, q.n_rows = 4096, 1 << 30, 1 << 20, (1 << 31) - 1     # more blocks than a grid holds
    assert lib.mlora_kv_append(ctypes.byref(c), ctypes.byref(q), 0, p, 256, p, 256, None) == -1
    assert lib.mlora_kv_read(ctypes.byref(c), ctypes.byref(q), 0, p, p, None) == -1


def test_nothing_to_do_is_no_error():
    kv, lib, c, q, a = _valid()
    q.n_seqs = 0
    assert lib.mlora_kv_attention(ctypes.byref(c), ctypes.byref(q), ctypes.byref(a), None) == 0
    q.n_seqs, q.row_off, q.max_rows = 3, 4096, 0
    assert lib.mlora_kv_append(ctypes.byref(c), ctypes.byref(q), 0, None, 256, None, 256, None) == 0


def test_kv_header_and_binding_agree(tmp_path):
    import os
    import re
    import shutil
    import subprocess
    kv, _ = _lib()
    import rl_step_gb300.grads as gr
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = [("mlora_kv_cache", kv._KvCache), ("mlora_kv_seqs", kv._KvSeqs), ("mlora_kv_attn", kv._KvAttn),
               ("mlora_grad_set", gr._GradSet)]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mlora_kv.h"', "int main(void) {"]
    for name, cls in structs:
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f[0]}));' for f in cls._fields_]
    lines.append('printf("%d %d\\n", MLORA_KV_PAGE, MLORA_KV_WORKSPACE_BYTES); return 0; }')
    (tmp_path / "a.c").write_text("\n".join(lines))
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"),
                    "-o", str(tmp_path / "a")], check=True, capture_output=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in structs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want + [kv.PAGE, kv.WORKSPACE_BYTES]
    src = re.sub(r"/\*.*?\*/", "", "".join(open(os.path.join(root, "include", h)).read()
                                          for h in ("mlora_kv.h", "mlora.h")), flags=re.S)
    for name, (_, args) in {**kv._SIGNATURES, **gr._SIGNATURES}.items():
        m = re.search(r"\b%s\s*\(([^)]*)\)" % name, src)
        assert m and len(m.group(1).split(",")) == len(args), name


# ----------------------------------------------------------------------------
# on the GPU
# ----------------------------------------------------------------------------
def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib()
    return torch


class Setup:
    """A cache on the GPU beside its model; sequences own pages in a shuffled order."""

    def __init__(self, caps, n_kv, hd, seed=0, extra=3):
        self.torch = torch = _torch()
        import rl_step_gb300.kv as kv
        self.kv, self.hd, self.n_kv = kv, hd, n_kv
        self.rng = np.random.default_rng(seed)
        used = [-(-c // 64) for c in caps]
        total = sum(used) + extra
        order = self.rng.permutation(total).astype(np.int32)
        width = max(max(used), 1)
        self.table = np.full((len(caps), width), -1, np.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.model = M.Cache(total, n_kv, hd)
        for x in "kv":                                   # stale bytes, NaN among them
            self.model.b[x][:] = self.rng.integers(0, 256, self.model.b[x].shape)
            self.model.e[x][:] = 30
        self.cache = kv.KvCache(*[torch.from_numpy(self.model.pages(x)).cuda() for x in "kv"],
                                *[torch.full((total, n_kv), 2.0 ** 30, device="cuda") for _ in range(2)])
        self.len = [0] * len(caps)
        self.dtable = torch.from_numpy(self.table).cuda()

    def i32(self, x):
        return self.torch.tensor(list(x), dtype=self.torch.int32, device="cuda")

    def off(self, rows):
        return self.i32(np.concatenate([[0], np.cumsum(rows)]))

    def rows(self, n, dtype, spread=1.0):
        x = self.rng.standard_normal((n, 2 * self.n_kv, self.hd)) * np.exp(spread * self.rng.standard_normal((n, 1, 1)))
        t = self.torch.from_numpy(x.astype(np.float32)).cuda()
        return t.bfloat16() if dtype == "bf16" else t

    def append(self, rows, dtype="bf16", x=None, use_off=True):
        """rows[s] new tokens of each sequence, on both sides."""
        n = sum(rows)
        x = self.rows(n, dtype) if x is None else x
        k, v = x[:, :self.n_kv], x[:, self.n_kv:]         # strided views
        self.len = [a + b for a, b in zip(self.len, rows)]
        self.kv.kv_append(self.cache, self.dtable, self.i32(self.len), k, v,
                          row_off=self.off(rows) if use_off else None, max_rows=max(rows) if use_off else 1)
        kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
        at = 0
        for s, r in enumerate(rows):
            if r:
                self.model.append(self.table[s], self.len[s] - r, {"k": kn[at:at + r], "v": vn[at:at + r]})
            at += r

    def check_state(self):
        """bytes of every position a sequence holds, and the scales of its pages"""
        for x, pages, scale in (("k", self.cache.k, self.cache.k_scale), ("v", self.cache.v, self.cache.v_scale)):
            got, sc = pages.cpu().numpy(), scale.cpu().numpy()
            want = self.model.pages(x)
            m = M.maps(self.hd)[0 if x == "k" else 1]
            for s, n in enumerate(self.len):
                for p in range(-(-n // 64)):
                    live = m[:min(n - 64 * p, 64)].reshape(-1)
                    g = got[self.table[s, p]].reshape(self.n_kv, -1)[:, live]
                    w = want[self.table[s, p]].reshape(self.n_kv, -1)[:, live]
                    nan = ((g & 0x7f) == 0x7f) & ((w & 0x7f) == 0x7f)        # a NaN's sign says nothing
                    assert np.array_equal(np.where(nan, 0, g), np.where(nan, 0, w)), (x, s, p)
                    assert np.array_equal(sc[self.table[s, p]],
                                          2.0 ** self.model.e[x][self.table[s, p]].astype(np.float64)), (x, s, p)
        assert self.kv.kv_check_status(self.cache) == 0


def _attend(st, rows, heads, dtype="bf16", q=None, scale=None, use_off=True, slack=0, **kw):
    """kv_attention of each sequence's newest rows[s], checked against the model."""
    torch = st.torch
    n = sum(rows)
    if q is None:
        q = torch.from_numpy(st.rng.standard_normal((n, heads, st.hd)).astype(np.float32) * 2).cuda()
        q = q.bfloat16() if dtype == "bf16" else q
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, max(max(st.len), 1) + slack, scale=scale,
                                  row_off=st.off(rows) if use_off else None, max_rows=max(rows) if use_off else 1, **kw)
    assert st.kv.kv_check_status(st.cache) == 0
    _compare(st, rows, q, out, lse, dtype, scale)
    return q, out, lse


def _compare(st, rows, q, out, lse, dtype, scale=None):
    sc = 1 / math.sqrt(st.hd) if scale is None else scale
    qn, on, ln = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    u = 2.0 ** -24
    at = 0
    for s, r in enumerate(rows):
        if not r:
            continue
        n = st.len[s]
        k, v = (st.model.values(x, st.table[s], n) for x in "kv")
        o, l, mass, big = M.attention(qn[at:at + r], k, v, max(n - r, -r), sc)
        D = ((st.hd + 16) * u + 2.0 ** -22) * big
        P = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
        kv = np.arange(q.shape[1]) // (q.shape[1] // st.n_kv)
        top = 2.0 ** st.model.e["v"][st.table[s, :-(-n // 64)]].astype(np.float64).max(0, initial=-200.0)
        tol = (4 * D + P + 2 * n * u + 2.0 ** -20)[..., None] * mass + EPS[dtype] * np.abs(o) + \
            (n * 2.0 ** -28 * top)[kv][:, None] + 1e-40
        bad = np.abs(on[at:at + r] - o) > tol
        assert not bad.any(), (s, float((np.abs(on[at:at + r] - o) / tol).max()))
        fin = np.isfinite(l)
        assert np.array_equal(fin, np.isfinite(ln[at:at + r]))
        assert np.array_equal(ln[at:at + r][~fin], l[~fin])
        d = np.abs(ln[at:at + r][fin] - l[fin])
        assert (d <= 2 * D[fin] + n * u + 2.0 ** -22 + 2 * u * np.abs(l[fin])).all(), (s, float(d.max()))
        at += r


@pytest.mark.gpu
@pytest.mark.parametrize("hd,n_kv,dtype", [(128, 2, "bf16"), (64, 3, "bf16"), (128, 1, "fp32"), (64, 5, "fp32")])
def test_append_in_pieces_equals_the_model(hd, n_kv, dtype):
    st = Setup([300, 1, 64, 129, 200, 70], n_kv, hd, seed=hd + n_kv)
    for rows in ([1, 1, 1, 1, 1, 1], [0, 0, 3, 63, 5, 0], [62, 0, 60, 1, 130, 1], [1, 0, 0, 64, 1, 65], [200, 0, 0, 0, 2, 3]):
        st.append(rows, dtype)
        st.check_state()


@pytest.mark.gpu
def test_append_one_token_each_without_row_off():
    st = Setup([90] * 5, 2, 128, seed=3)
    for _ in range(70):
        st.append([1] * 5, use_off=False)
    st.check_state()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_extreme_values(dtype):
    """zeros, infinities, NaN, the largest and the smallest magnitudes, and scales that jump"""
    st = Setup([130], 1, 64, seed=9)
    x = st.rows(130, dtype).float()
    x[3] = 0
    x[5, :, 7], x[6, :, 8], x[9, :, 1] = math.inf, -math.inf, math.nan
    x[20:30] *= 1e30
    x[30] = 3.3e38
    x[31] = 1e-44
    x[64:] *= 1e-38                                       # the second page: below the smallest scale
    x = x.bfloat16() if dtype == "bf16" else x
    for a, b in ((0, 1), (1, 4), (4, 5), (5, 6), (6, 25), (25, 30), (30, 31), (31, 66), (66, 130)):
        st.append([b - a], dtype, x[a:b])
        st.check_state()
    st2 = Setup([70], 1, 64, seed=9)
    st2.append([3], dtype, x[:3] * 0)                      # a page of zeros, then ordinary values
    st2.append([60], dtype, x[64:124])
    st2.check_state()


@pytest.mark.gpu
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "fp32"), (128, "fp32"), (64, "bf16")])
def test_read_returns_the_stored_values(hd, dtype):
    torch = _torch()
    st = Setup([150, 64, 1, 77], 3, hd, seed=5)
    st.append([150, 64, 1, 77])
    for rows in ([150, 64, 1, 77], [1, 1, 1, 1], [65, 0, 1, 14]):
        k, v = st.kv.kv_read(st.cache, st.dtable, st.i32(st.len), sum(rows), row_off=st.off(rows), max_rows=max(rows),
                             dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
        for x, got in (("k", k), ("v", v)):
            want = np.concatenate([st.model.values(x, st.table[s], st.len[s])[st.len[s] - r:] for s, r in enumerate(rows)])
            assert np.array_equal(got.double().cpu().numpy(), want)
    assert st.kv.kv_check_status(st.cache) == 0


_SHAPES = [  # heads, kv heads, hd
    (4, 2, 128), (8, 1, 64), (3, 3, 128), (24, 2, 64), (40, 2, 128), (7, 1, 128), (64, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,n_kv,hd", _SHAPES)
def test_attention_single_rows(heads, n_kv, hd, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]
    st = Setup(lens, n_kv, hd, seed=heads)
    st.append(lens)
    _attend(st, [1] * len(lens), heads, dtype, use_off=False)
    _attend(st, [1] * len(lens), heads, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,n_kv,hd", _SHAPES)
def test_attention_several_rows(heads, n_kv, hd, dtype):
    """drafted tokens and short prompts: ragged rows, rows that see only themselves"""
    lens = [1, 5, 33, 64, 66, 130, 257]
    st = Setup(lens, n_kv, hd, seed=heads + 1)
    st.append(lens)
    _attend(st, [1, 5, 2, 0, 3, 9, 4], heads, dtype)
    _attend(st, [1, 5, 33, 20, 66, 70, 40], heads, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("n_seqs,length", [(1, 20000), (2, 9001), (3, 4097)])
def test_attention_split_over_a_long_cache(n_seqs, length):
    """few long sequences: the work is cut along the positions and joined; a small
    workspace gives fewer parts and the same values"""
    torch = _torch()
    lens = [length - 117 * i for i in range(n_seqs)]
    st = Setup(lens, 2, 128, seed=n_seqs)
    st.append(lens)
    ws = st.kv.kv_workspace()
    q, out, lse = _attend(st, [1] * n_seqs, 8, workspace=ws)
    _, o2, l2 = _attend(st, [1] * n_seqs, 8, q=q, workspace=ws)
    assert torch.equal(out, o2) and torch.equal(lse, l2)               # bit for bit
    for nbytes in (0, 16, 40000, 300000, 4000000):
        _attend(st, [1] * n_seqs, 8, q=q, workspace=st.kv.kv_workspace(nbytes=nbytes))
    _attend(st, [3] * n_seqs, 8)
    _attend(st, [1] * n_seqs, 8, q=q, slack=100000)                    # a loose bound of the lengths


@pytest.mark.gpu
def test_attention_concentrated_and_wide_scores():
    """scores of +-200, one position with all the weight, values of very different scales"""
    st = Setup([700, 700, 65], 1, 128, seed=2)
    x = st.rows(1465, "bf16", spread=0.1).float()
    x[100:164, 1] *= 1e-12                                 # tiny values on one page ..
    x[700 + 64:700 + 128, 1] *= 1e9                        # .. large ones on another
    st.append([700, 700, 65], x=x.bfloat16())
    torch = st.torch
    k = st.model.values("k", st.table[0], 700)
    q = torch.from_numpy(np.stack([k[120, 0] * 3, k[5, 0] * 2])[None].repeat(3, 0).astype(np.float32)).cuda().bfloat16()
    _attend(st, [1, 1, 1], 2, q=q)
    _attend(st, [1, 1, 1], 2, q=q * 0)
    _attend(st, [1, 1, 1], 2, q=q, scale=-0.3)
    _attend(st, [1, 1, 1], 2, q=q * 1e-20)
    _attend(st, [1, 1, 1], 2, "fp32", q=q.float() * 1e20, scale=1e-21)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_nan_and_infinity(dtype):
    """NaN in a cached key or value, and infinities in a query, reach exactly the
    rows and dims of the formula; stale NaN behind the end reach nothing"""
    torch = _torch()
    st = Setup([100, 100, 100], 1, 64, seed=4)
    x = st.rows(300, "bf16").float()
    x[10, 0, 3] = math.nan                                 # sequence 0: a key
    x[150, 1, 5] = math.inf                                # sequence 1: a value (stored as NaN)
    st.append([100, 100, 100], x=x.bfloat16())
    q = torch.ones(3, 2, 64, device="cuda")
    q[2, 1, 9] = math.inf
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q if dtype == "fp32" else q.bfloat16(), 100)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    nan = torch.isnan(out[1])
    assert nan[:, 5].all() and int(nan.sum()) == 2 and torch.isfinite(lse[1]).all()
    assert torch.isfinite(out[2, 0]).all() and torch.isnan(out[2, 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [9, 70])
def test_nan_of_a_later_row_does_not_reach_the_rows_before_it(n, dtype):
    """a key and a value that are NaN at the same call's later rows: masked for the earlier ones"""
    torch = _torch()
    st = Setup([30 + n, 30 + n], 1, 128, seed=n)
    x = st.rows(60 + 2 * n, "bf16").float()
    x[30 + n - 3, 1, [0, 77]] = math.nan                   # sequence 0: values of its third newest row
    x[60 + 2 * n - 2, 0, 5] = math.nan                     # sequence 1: a key of its second newest row
    st.append([30 + n, 30 + n], x=x.bfloat16())
    q = torch.randn(2 * n, 3, 128, device="cuda")
    q = q if dtype == "fp32" else q.bfloat16()
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, 30 + n, row_off=st.off([n, n]), max_rows=n)
    a = torch.isnan(out[:n])
    assert not a[:n - 3].any() and a[n - 3:][:, :, [0, 77]].all() and int(a.sum()) == 3 * 3 * 2
    assert torch.isfinite(lse[:n]).all()
    assert torch.isfinite(out[n:-2]).all() and torch.isnan(out[-2:]).all() and torch.isnan(lse[-2:]).all()


@pytest.mark.gpu
def test_empty_slots_and_rows_behind_the_end():
    torch = _torch()
    st = Setup([64, 0, 10, 0], 2, 128, seed=6)
    st.append([64, 0, 10, 0])
    q = torch.randn(6, 4, 128, device="cuda").bfloat16()
    out = torch.full((6, 4, 128), 7.0, device="cuda").bfloat16()
    lse = torch.full((6, 4), 7.0, device="cuda")
    st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, 64, out=out, lse=lse)
    assert (out[4:] == 7).all() and (lse[4:] == 7).all()
    for s in (1, 3):
        assert (out[s] == 0).all() and (lse[s] == -math.inf).all()
    _compare(st, [1, 0, 1, 0], q[[0, 2]], out[[0, 2]], lse[[0, 2]], "bf16")
    before = st.cache.k.clone(), st.cache.v.clone()
    x = st.rows(4, "bf16")
    st.kv.kv_append(st.cache, st.dtable, st.i32([0, 0, 0, 0]), x[:, :2], x[:, 2:])
    assert torch.equal(before[0], st.cache.k) and torch.equal(before[1], st.cache.v)
    k, v = st.kv.kv_read(st.cache, st.dtable, st.i32([0] * 4), 4)
    assert st.kv.kv_check_status(st.cache) == 0


@pytest.mark.gpu
def test_bad_sequences_are_flagged_and_leave_the_others_alone():
    """every range error that only the device sees: NaN rows or skipped writes, status, and the
    neighbours as if it were not there"""
    torch = _torch()
    for bad in ("len<0", "len>cap", "len>max", "page", "rows>max", "off<0", "off>n", "rows>len"):
        st = Setup([128, 100, 128], 2, 128, seed=7)
        st.append([128, 100, 128])
        good = _attend(st, [2, 3, 2], 4)
        q = good[0]
        lens, off, table, max_rows, max_len = list(st.len), [0, 2, 5, 7], st.table.copy(), 3, 128
        if bad == "len<0":
            lens[1] = -5
        elif bad == "len>cap":
            lens[1], max_len = 129, 1 << 40
        elif bad == "len>max":
            lens[1], max_len = 128, 127
            lens[0] = lens[2] = 127
        elif bad == "page":
            table[1, 0] = st.cache.n_pages
            table[1, 1] = -1
        elif bad == "rows>max":
            max_rows = 2
        elif bad == "off<0":
            off = [0, 2, -3, 7]
        elif bad == "off>n":
            off = [0, 2, 9, 7]
        elif bad == "rows>len":
            lens[1] = 2
        kw = dict(row_off=st.i32(off), max_rows=max_rows)
        tab = torch.from_numpy(table).cuda()
        before = st.cache.k.clone(), st.cache.v.clone(), st.cache.k_scale.clone(), st.cache.v_scale.clone()
        out, lse = st.kv.kv_attention(st.cache, tab, st.i32(lens), q, max_len, **kw)
        assert st.kv.kv_check_status(st.cache) == -2 and st.kv.kv_check_status(st.cache) == 0, bad
        if bad in ("len<0", "len>cap", "len>max", "page", "rows>max", "rows>len"):
            assert torch.isnan(out[2:5]).all() and torch.isnan(lse[2:5]).all(), bad
        if bad not in ("len>max", "off<0", "off>n"):
            for i in (slice(0, 2), slice(5, 7)):
                assert torch.equal(out[i], good[1][i]) and torch.equal(lse[i], good[2][i]), bad
        # nothing of a bad sequence is written
        st.kv.kv_append(st.cache, tab, st.i32(lens), *[torch.zeros(7, 2, 128, device="cuda")] * 2, **kw)
        if bad in ("len<0", "len>cap", "page", "rows>max", "rows>len"):
            assert st.kv.kv_check_status(st.cache) == -2, bad
            own = torch.from_numpy(st.table[1]).cuda().long()
            for a, b in zip(before, (st.cache.k, st.cache.v, st.cache.k_scale, st.cache.v_scale)):
                assert torch.equal(a[own], b[own]), bad
        st.kv.kv_read(st.cache, tab, st.i32(lens), 7, **kw)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_shared_prefix_pages():
    """two sequences over the same first pages, each with a tail of its own"""
    st = Setup([128, 20, 30], 2, 128, seed=8)
    st.append([128, 0, 0])
    x = st.rows(50, "bf16")
    st.append([0, 20, 30], x=x)
    table = np.concatenate([np.repeat(st.table[:1, :2], 2, 0), st.table[1:, :1]], 1)
    q = st.torch.randn(2, 4, 128, device="cuda").bfloat16()
    out, lse = st.kv.kv_attention(st.cache, st.torch.from_numpy(table).cuda(), st.i32([148, 158]), q, 158)
    st.table, st.len = table, [148, 158]
    _compare(st, [1, 1], q, out, lse, "bf16")


@pytest.mark.gpu
def test_rows_of_strided_buffers_and_outputs():
    """q, k, v as column blocks of one buffer, out as a column block of another"""
    torch = _torch()
    st = Setup([70, 70], 2, 64, seed=10)
    buf = torch.randn(140, 4 + 2 + 2 + 1, 64, device="cuda").bfloat16()
    st.append([70, 70], x=buf[:, 4:8])
    st.check_state()
    big = torch.zeros(2, 6, 64, device="cuda").bfloat16()
    q = buf[69::70, :4]
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, 70, out=big[:, 1:5])
    _compare(st, [1, 1], q, out, lse, "bf16")
    assert (big[:, 0] == 0).all() and (big[:, 5] == 0).all()


@pytest.mark.gpu
def test_captured_steps_replay_on_new_data_and_another_stream():
    """append and attention in one graph: the lengths, tables and rows are read at replay"""
    torch = _torch()
    st = Setup([200, 200, 200], 2, 128, seed=11)
    st.append([100, 63, 1])
    k, v = torch.zeros(3, 2, 128, device="cuda").bfloat16(), torch.zeros(3, 2, 128, device="cuda").bfloat16()
    q, lens = torch.zeros(3, 8, 128, device="cuda").bfloat16(), st.i32(st.len)
    out, lse, ws = torch.zeros_like(q), torch.zeros(3, 8, device="cuda"), st.kv.kv_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            st.kv.kv_append(st.cache, st.dtable, lens, k, v)
            st.kv.kv_attention(st.cache, st.dtable, lens, q, 200, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        x = st.rows(3, "bf16")
        k.copy_(x[:, :2])
        v.copy_(x[:, 2:])
        q.normal_()
        lens += 1
        st.len = [n + 1 for n in st.len]
        g.replay()
        torch.cuda.synchronize()
        for s in range(3):
            st.model.append(st.table[s], st.len[s] - 1, {"k": x[s:s + 1, :2].float().cpu().numpy(),
                                                         "v": x[s:s + 1, 2:].float().cpu().numpy()})
        st.check_state()
        _compare(st, [1, 1, 1], q, out, lse, "bf16")


@pytest.mark.gpu
def test_two_calls_at_once_with_a_workspace_each():
    torch = _torch()
    st = Setup([6000, 5000], 2, 128, seed=12)
    st.append([6000, 5000])
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    want = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, 6000)
    lens = st.i32(st.len)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [st.kv.kv_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, w in zip(streams, ws):
            got.append(st.kv.kv_attention(st.cache, st.dtable, lens, q, 6000, workspace=w, stream=s))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.gpu
def test_a_row_does_not_depend_on_its_batch():
    """without a workspace no sequence is cut: bit for bit the same row in every batch"""
    torch = _torch()
    lens = [900, 3, 450, 64, 2000]
    st = Setup(lens, 2, 128, seed=13)
    st.append(lens)
    q = torch.randn(5, 8, 128, device="cuda").bfloat16()
    ws = st.kv.kv_workspace(nbytes=0)
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(lens), q, 2000, workspace=ws)
    other = [n if s == 2 else 1 for s, n in enumerate(lens)]
    o2, l2 = st.kv.kv_attention(st.cache, st.dtable, st.i32(other), q, 2000, workspace=ws)
    assert torch.equal(out[2], o2[2]) and torch.equal(lse[2], l2[2])
    o3, l3 = st.kv.kv_attention(st.cache, st.dtable[2:3].contiguous(), st.i32([450]), q[2:3], 450, workspace=ws)
    assert torch.equal(out[2:3], o3) and torch.equal(lse[2:3], l3)


@pytest.mark.gpu
def test_python_refusals():
    torch = _torch()
    st = Setup([64], 2, 128)
    kv, c, tab, lens = st.kv, st.cache, st.dtable, st.i32([3])
    x = torch.zeros(1, 2, 128, device="cuda")
    for f in (lambda: kv.kv_append(c, tab, lens, x.half(), x.half()), lambda: kv.kv_append(c, tab.long(), lens, x, x),
              lambda: kv.kv_append(c, tab, lens, x, x.bfloat16()), lambda: kv.kv_append(c, tab, lens[:0], x, x),
              lambda: kv.kv_append(c, tab, lens, x.cpu(), x), lambda: kv.kv_append(c, tab, lens.cpu(), x, x),
              lambda: kv.kv_attention(c, tab, lens, x[:, :, ::2], 64), lambda: kv.kv_attention(c, tab, lens, x[0], 64),
              lambda: kv.kv_attention(c, tab, lens, x, 64, lse=torch.zeros(1, 3, device="cuda")),
              lambda: kv.kv_attention(c, tab, lens, x, 64, out=x.bfloat16()),
              lambda: kv.KvCache(c.k, c.v[:1], c.k_scale, c.v_scale),
              lambda: kv.KvCache(c.k.cpu(), c.v.cpu(), c.k_scale.cpu(), c.v_scale.cpu())):
        with pytest.raises(ValueError):
            f()
    import rl_step_gb300 as m
    with pytest.raises(m.MLoRAError):
        kv.kv_attention(c, tab, lens, torch.zeros(1, 3, 128, device="cuda"), 64)       # 3 heads over 2
    with pytest.raises(m.MLoRAError):
        kv.kv_attention(c, tab, lens, x, 64, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")[4:])
    with pytest.raises(m.MLoRAError):
        kv.kv_append(c, tab, lens, x, x, max_rows=2)                                   # row_off is missing


@pytest.mark.gpu
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "bf16"), (128, "fp32"), (64, "fp32")])
@pytest.mark.parametrize("most", [1, 2, 5, 6, 13, 14, 29, 30, 64, 65, 130])
def test_append_any_rows_at_any_offset(hd, dtype, most):
    """every size class of a call, new rows at every place of a group of four and of a page, scales that
    grow and that do not, units with infinities and NaN, and with nothing finite"""
    before = [0, 1, 2, 3, 5, 31, 62, 63, 64, 65, 127]
    rows = [max(1, min(most, r)) for r in (most, most, 1, 2, most, 3, most, 4, most, most - 1, most)]
    caps = [b + 2 * r for b, r in zip(before, rows)]
    st = Setup(caps, 2, hd, seed=most)
    st.append(before, dtype)
    for gain, bad in ((1e-3, False), (300.0, True)):
        n = sum(rows)
        x = st.rows(n, "fp32") * gain
        if bad:
            x[::3, 0, 5] = math.inf
            x[1::4, 3, hd - 1] = math.nan
            x[rows[0]:rows[0] + rows[1]] = -math.inf       # a whole sequence's rows
        st.append(rows, dtype, x=x.bfloat16() if dtype == "bf16" else x)
        st.check_state()
    n = sum(st.len)
    k, v = st.kv.kv_read(st.cache, st.dtable, st.i32(st.len), n, row_off=st.off(st.len), max_rows=max(st.len))
    at = 0
    for s, ln in enumerate(st.len):
        for name, got in (("k", k), ("v", v)):
            want = st.model.values(name, st.table[s], ln)
            g = got[at:at + ln].double().cpu().numpy()
            assert np.array_equal(np.isnan(g), np.isnan(want)) and np.array_equal(g[~np.isnan(g)], want[~np.isnan(want)])
        at += ln


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_wide_groups_and_odd_bounds(dtype):
    """a hundred query heads on one key head, a bound of the lengths beyond 2^62, scale 0, the output over the queries"""
    torch = _torch()
    lens = [1, 63, 200, 641]
    st = Setup(lens, 1, 64, seed=12)
    st.append(lens)
    ws = st.kv.kv_workspace()
    q, out, lse = _attend(st, [1, 3, 2, 5], 100, dtype, workspace=ws)
    _attend(st, [1, 3, 2, 5], 100, dtype, q=q, workspace=ws, slack=2 ** 62)
    _attend(st, [1, 3, 2, 5], 100, dtype, q=q, workspace=ws, scale=0.0)
    same = q.clone()
    o2, l2 = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), same, 641, row_off=st.off([1, 3, 2, 5]), max_rows=5,
                                out=same, workspace=ws)
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.gpu
def test_outputs_on_another_stream_do_not_meet_the_current_ones_writes():
    """memory that the current stream has still to write when it is handed out again: results asked for on
    another stream must not lie there"""
    torch = _torch()
    st = Setup([3500, 1300], 2, 64, seed=21)
    st.append([3500, 1300])
    q = torch.randn(4800, 8, 64, device="cuda")
    lens, off = st.i32(st.len), st.off([3500, 1300])
    ws = st.kv.kv_workspace()
    args = (st.cache, st.dtable, lens)
    want = st.kv.kv_attention(*args, q, 3500, row_off=off, max_rows=3500, workspace=ws)
    wk, wv = st.kv.kv_read(*args, 4800, row_off=off, max_rows=3500)
    big = torch.zeros(1 << 28, device="cuda")
    s = torch.cuda.Stream()

    def meet(nbytes, call):
        """call(), while blocks of nbytes each wait to be filled with 255 by the current stream"""
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes]
        torch.cuda.synchronize()
        for _ in range(100):                               # some 30 ms of work before the fills
            big.mul_(1.0)
        for x in old:
            x.fill_(255)
        del old, x
        got = call()
        s.synchronize()
        torch.cuda.synchronize()
        return got
    out, lse = meet([q.numel() * 4], lambda: st.kv.kv_attention(*args, q, 3500, row_off=off, max_rows=3500, workspace=ws,
                                                                stream=s))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    k, v = meet([wk.numel() * 4] * 2, lambda: st.kv.kv_read(*args, 4800, row_off=off, max_rows=3500, stream=s))
    assert torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.gpu
def test_pages_beyond_four_gigabytes():
    """page ids whose bytes lie behind 2^32: the same results as from a small pool"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    n_pages, n_kv, hd = 70000, 8, 128                      # 4.6 GB each of keys and values
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    high = [69999, 65536, 65535, 32768, 69000, 1, 68001]
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(410, 2 * n_kv, hd, generator=g, device="cuda").bfloat16()
    q = torch.randn(5, 16, hd, generator=g, device="cuda").bfloat16()
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    got = []
    for pool, ids in ((n_pages, high), (7, list(range(7)))):
        c = kv.KvCache.empty(pool, n_kv, hd)
        table = i32([ids[:4] , ids[4:] + [-1]])
        kv.kv_append(c, table, i32([250, 160]), x[:, :n_kv], x[:, n_kv:], row_off=i32([0, 250, 410]), max_rows=250)
        out, lse = kv.kv_attention(c, table, i32([250, 160]), q, 250, row_off=i32([0, 2, 5]), max_rows=3)
        k, v = kv.kv_read(c, table, i32([250, 160]), 410, row_off=i32([0, 250, 410]), max_rows=250)
        assert kv.kv_check_status(c) == 0
        got.append((out, lse, k, v))
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dtype", [(8, "bf16"), (24, "bf16"), (16, "fp32")])
def test_attention_many_units(heads, dtype):
    """100 sequences of 8 key/value heads: short, long (cut) and empty ones, whole batch and without a workspace"""
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(0, 90, 92)] + [0, 1, 63, 64, 65, 600, 601, 777]
    st = Setup(lens, 8, 128, seed=33)
    st.append(lens)
    live = [1 if n else 0 for n in lens]
    q, out, lse = _attend(st, live, heads, dtype, workspace=st.kv.kv_workspace())
    _, o2, l2 = _attend(st, live, heads, dtype, q=q, workspace=st.kv.kv_workspace())
    assert st.torch.equal(out, o2) and st.torch.equal(lse, l2)
    _attend(st, live, heads, dtype, q=q, workspace=st.kv.kv_workspace(nbytes=0))
    _attend(st, live, heads, dtype, q=q, slack=5000)


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
def test_small_parts_of_fp32_queries_count(hd):
    """queries of 2^-16 of their row's largest, whose key dim is zero: q is held to 2^-22 of itself and 2^-36 of
    the power of two above the largest, 2 here"""
    st = Setup([130, 40], 2, hd, seed=47)
    x = st.rows(170, "fp32", spread=0.0)
    x[:, :2, 0] = 0                                        # the large dim's keys
    x[:, :2] *= 2.0 ** 16
    st.append([130, 40], "fp32", x)
    torch = st.torch
    q = torch.from_numpy(st.rng.standard_normal((2, 4, hd)).astype(np.float32)).cuda() * 2.0 ** -16
    q[:, :, 0] = 1.5
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, 130)
    u, qn = 2.0 ** -24, q.double().cpu().numpy()
    for s in range(2):
        k, v = (st.model.values(x, st.table[s], st.len[s]) for x in "kv")
        o, l, mass, big = M.attention(qn[s:s + 1], k, v, st.len[s] - 1, 1 / math.sqrt(hd))
        most = np.abs(k).sum(2).max(0)[np.arange(4) // 2][None] * 2.0 ** -36 * 2 / math.sqrt(hd)
        D = ((hd + 16) * u + 2.0 ** -22) * big + most
        assert (np.abs(lse[s].double().cpu().numpy() - l) <= 2 * D + st.len[s] * u + 2.0 ** -22 + 2 * u * np.abs(l)).all()
        assert (np.abs(out[s].double().cpu().numpy() - o) <= (4 * D + 2 * st.len[s] * u + 2.0 ** -20)[..., None] * mass + 2 * u * np.abs(o)).all()


@pytest.mark.gpu
def test_small_probabilities_of_fp32_rows_count():
    """weights down to 2^-22 of the largest, each alone in its dim of the values: held to 2^-22 of themselves.

    q and k are small integers and 7/16, so the products are exact; the score in units of log2 is rounded three
    times (scale log2 e, its product, the difference): 3 u 23, times ln 2 in p; exp2 2^-22, the sum of 23 terms
    and the division 25 u."""
    n, hd = 23, 64
    st = Setup([n], 1, hd, seed=48)
    torch = st.torch
    x = torch.zeros(n, 2, hd, device="cuda")
    j = torch.arange(n, device="cuda").float()
    x[:, 0, 0] = -torch.clamp(j, max=16)
    x[:, 0, 1] = -torch.clamp(j - 16, min=0)
    x[1:, 0, 2] = -0.4375
    x[torch.arange(n), 1, torch.arange(n)] = 1.125
    st.append([n], "fp32", x)
    q = torch.zeros(1, 1, hd, device="cuda")
    q[0, 0, :3] = 1.0
    sc = float(np.float32(math.log(2)))
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32([n]), q, n, scale=sc)
    k, v = (st.model.values(x, st.table[0], n) for x in "kv")
    o, l, _, _ = M.attention(q.double().cpu().numpy(), k, v, n - 1, sc)
    got, want = out.double().cpu().numpy()[0, 0, :n], o[0, 0, :n]
    u = 2.0 ** -24
    assert (np.abs(got / want - 1) <= 3 * u * 23 * math.log(2) + 2 * 2.0 ** -22 + 2.0 ** -22 + 25 * u).all()


# ----------------------------------------------------------------------------
# Pages of very different value scales.  In the attention each dimension of a
# result stands for itself: with p relative to its row's largest,
#   |out_d - o_d| <= (4 D + P + 2 n u + 2^-20) A_d + half a step of the type + C sum_i |v_id|
# where C = 2^-33 (bf16) or 2^-44 (fp32) is the absolute rounding of a p: fp16's
# half step 2^-25 (and 2^-11 of it on fp32, whose low part is held 2^11 times as
# large) at p' >= 2^(12 - 3) p, and on bf16 once more, before the factor 2^-3 .. 1.  Pages below 2^-64 of the largest scale of the row's
# pages may count as zero in out, never in lse.
# ----------------------------------------------------------------------------
def _scaled_pages(pages, n_kv, hd, seed, outlier=False):
    """a Setup whose sequence s has the pages pages[s], of values times 2^e each (None: zero); outlier: dim 5
    alone is that large, and the others ordinary where that leaves them bits"""
    st = Setup([64 * len(p) - 3 for p in pages], n_kv, hd, seed=seed)
    lens = [64 * len(p) - 3 for p in pages]
    x = st.rows(sum(lens), "fp32", spread=0.0)
    at = 0
    for p, n in zip(pages, lens):
        for i, e in enumerate(p):
            rows = x[at + 64 * i:min(at + 64 * i + 64, at + n), n_kv:]
            if outlier:
                rows[..., 5] *= 2.0 ** e
            else:
                rows *= 0.0 if e is None else 2.0 ** e
        at += n
    st.append(lens, "fp32", x)
    st.check_state()
    return st


def _compare_dims(st, rows, q, out, lse, dtype, scale=None):
    sc = 1 / math.sqrt(st.hd) if scale is None else scale
    qn, on, ln = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    u = 2.0 ** -24
    P, C = (2.0 ** -11, 2.0 ** -33) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -44)
    at = 0
    for s, r in enumerate(rows):
        n = st.len[s]
        k, v = (st.model.values(x, st.table[s], n) for x in "kv")
        e = np.repeat(st.model.e["v"][st.table[s, :-(-n // 64)]], 64, 0)[:n]             # [n, n_kv]
        gone = e < e.max(0) - 64
        o, l, mass, big = M.attention(qn[at:at + r], k, v, n - r, sc)
        lost = M.attention(qn[at:at + r], k, v * gone[:, :, None], n - r, sc)[2]
        kv = np.arange(q.shape[1]) // (q.shape[1] // st.n_kv)
        D = ((st.hd + 16) * u + 2.0 ** -22) * big
        tol = (4 * D + P + 2 * n * u + 2.0 ** -20)[..., None] * mass + EPS[dtype] * np.abs(o) + \
            C * np.abs(v).sum(0)[kv] + lost + 1e-40
        err = np.abs(on[at:at + r] - o)
        assert (err <= tol).all(), (s, float((err / tol).max()))
        d = np.abs(ln[at:at + r] - l)
        assert (d <= 2 * D + n * u + 2.0 ** -22 + 2 * u * np.abs(l)).all(), (s, float(d.max()))
        at += r


def _scale_cases(kind, rng):
    """pages, heads, n_kv, hd, rows of a sequence: one of each form of the kernel"""
    gap = lambda n: [int(x) for x in rng.choice([0, 4, 5, 20, 38, 60], n)]
    if kind == "single rows":
        return [gap(3), [0, 60], [60, 0], [38, 0, 0], [4, 0, 5, 0, 9, 0]], 4, 2, 128, 1
    if kind == "heads of 64":
        return [gap(4), [0, 45], [45, 0]], 3, 3, 64, 1
    if kind == "cut":
        return [gap(70), gap(41)], 4, 2, 128, 1
    if kind == "16 pairs":
        return [gap(3), gap(12)], 12, 2, 128, 3
    if kind == "64 pairs":
        return [gap(3), gap(11)], 16, 1, 64, 9
    return [gap(3) for _ in range(76)], 8, 8, 128, 1       # many units


_KINDS = ["single rows", "heads of 64", "cut", "16 pairs", "64 pairs", "many units"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", _KINDS)
def test_a_large_value_in_one_dim_leaves_the_others(kind, dtype):
    """a page whose scale is 2^4 to 2^60 times its neighbours' for one dim's sake: the other dims are the neighbours'"""
    pages, heads, n_kv, hd, r = _scale_cases(kind, np.random.default_rng(41))
    st = _scaled_pages(pages, n_kv, hd, 43, outlier=True)
    torch = st.torch
    rows = [r] * len(pages)
    for gain in (0.0, 1.0):
        q = torch.from_numpy(st.rng.standard_normal((sum(rows), heads, hd)).astype(np.float32)).cuda() * gain
        q = q.bfloat16() if dtype == "bf16" else q
        out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, max(st.len), row_off=st.off(rows), max_rows=r)
        _compare_dims(st, rows, q, out, lse, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", _KINDS)
def test_every_page_counts_whatever_its_scale(kind, dtype):
    """zeros beside values of up to 2^110 in every order: each position has its share of the sum"""
    pages, heads, n_kv, hd, r = _scale_cases(kind, np.random.default_rng(42))
    rng = np.random.default_rng(44)
    pages = [[[None, -100, -30, 0, 45, 110][int(rng.integers(6))] for _ in p] for p in pages]
    pages[0], pages[1] = ([None, 60, None] if len(pages[0]) < 9 else pages[0]), ([110, None] if len(pages[1]) < 9 else pages[1])
    st = _scaled_pages(pages, n_kv, hd, 45)
    torch = st.torch
    rows = [r] * len(pages)
    for gain in (0.0, 1.0):
        q = torch.from_numpy(st.rng.standard_normal((sum(rows), heads, hd)).astype(np.float32)).cuda() * gain
        q = q.bfloat16() if dtype == "bf16" else q
        for nbytes in (st.kv.WORKSPACE_BYTES, 0):
            out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32(st.len), q, max(st.len), row_off=st.off(rows),
                                          max_rows=r, workspace=st.kv.kv_workspace(nbytes=nbytes))
            _compare_dims(st, rows, q, out, lse, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,rows,nbytes", [(1, 1, None), (1, 1, 0), (12, 1, None), (24, 3, None)])
def test_the_sum_over_many_positions_of_zero_values(heads, rows, nbytes, dtype):
    """70,000 equal scores over values that are all zero: lse = log n.  Every term is the same power of two, so
    the sums are exact; the logarithm and its scaling are a few u."""
    n, hd = 70000, 64
    st = Setup([n], 1, hd, seed=46)
    x = st.rows(n, "bf16")
    x[:, 1] = 0
    st.append([n], x=x)
    torch = st.torch
    q = torch.zeros(rows, heads, hd, device="cuda", dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
    ws = st.kv.kv_workspace() if nbytes is None else st.kv.kv_workspace(nbytes=nbytes)
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32([n]), q, n, row_off=st.off([rows]), max_rows=rows, workspace=ws)
    want = np.log(np.arange(n - rows + 1, n + 1))[:, None]
    assert (np.abs(lse.double().cpu().numpy() - want) <= 8 * 2.0 ** -24 * want + 2.0 ** -22).all()
    assert (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scales_that_make_up_for_tiny_or_huge_factors(dtype):
    """ordinary scores from queries, keys and a scale whose exponents are far from zero, and queries of zero"""
    torch = _torch()
    for kgain, qgain, sc in ((2.0 ** -70, 2.0 ** -60, 2.0 ** 126), (2.0 ** -60, 2.0 ** -68, float(np.float32(3.0e38))),
                             (2.0 ** 100, 2.0 ** 10, 2.0 ** -113), (2.0 ** 60, 2.0 ** 66, 2.0 ** -129),
                             (2.0 ** -60, 2.0 ** 100, 2.0 ** -43), (2.0 ** 110, 0.0, 2.0 ** 30)):
        st = Setup([100, 65, 1], 2, 64, seed=49)
        x = st.rows(166, "fp32", spread=0.1)
        x[:, :2] *= kgain
        st.append([100, 65, 1], "fp32", x)
        q = torch.from_numpy(st.rng.standard_normal((3, 4, 64)).astype(np.float32)).cuda() * qgain
        _attend(st, [1, 1, 1], 4, dtype, q=q.bfloat16() if dtype == "bf16" else q, scale=sc)


@pytest.mark.gpu
def test_the_status_is_read_and_cleared_on_the_stream():
    """kv_check_status(cache, stream): read and cleared in that stream's order, so that no later call's bit there is lost"""
    torch = _torch()
    st = Setup([64], 1, 64, seed=50)
    s = torch.cuda.Stream()

    class Word:
        def __init__(self, value):
            self.value, self.where = value, []

        def item(self):
            self.where.append(torch.cuda.current_stream())
            return self.value

        def zero_(self):
            self.where.append(torch.cuda.current_stream())
    st.cache.status = Word(1)
    assert st.kv.kv_check_status(st.cache, stream=s) == -2
    assert st.cache.status.where == [s, s]
    st.cache.status = Word(3)
    assert st.kv.kv_check_status(st.cache) == -5 and set(st.cache.status.where) == {torch.cuda.current_stream()}


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 70])
def test_outputs_beside_the_queries_are_taken(n):
    """columns and rows of one buffer that do not touch the queries', in every order"""
    torch = _torch()
    st = Setup([70], 2, 64, seed=51)
    st.append([70])
    buf = torch.randn(4 * n, 9, 64, device="cuda").bfloat16()
    off, lens = st.off([n]), st.i32([70])
    want = None
    x = torch.randn(n, 4, 64, device="cuda").bfloat16()
    for q, out in ((buf[:n, :4], buf[:n, 4:8]), (buf[:n, 5:], buf[:n, 1:5]), (buf[:n, :4], buf[n:2 * n, 2:6]),
                   (buf[::2][:n, :4], buf[1::2][:n, :4]), (buf[::2][:n, :4], buf[:n, 4:8]), (buf[:n, 4:8], buf[::4][:n, :4]),
                   (buf[3 * n:, :4], buf[::3][:n, 4:8]), (buf[:n, :4], buf[:n, :4])):
        q.copy_(x)
        o, lse = st.kv.kv_attention(st.cache, st.dtable, lens, q, 70, row_off=off, max_rows=n, out=out)
        if want is None:
            want = o.clone(), lse
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_a_nan_among_zero_values_reaches_the_rows_that_see_it(rows, dtype):
    """values that count as zero beside their neighbours', one of them NaN: its dim is NaN, the others are the formula's"""
    st = Setup([256, 256], 1, 128, seed=52)
    x = st.rows(512, "fp32", spread=0.0)
    x[64:128, 1] = 0                                       # sequence 0: its second page, which every row sees whole
    x[70, 1, 5] = math.nan
    x[256 + 192:, 1] = 0                                   # sequence 1: its last page, which holds the newest rows
    x[256 + 216, 1, 9] = math.inf
    x[256:256 + 192, 1] *= 2.0 ** 40
    st.append([256, 256], "fp32", x)
    torch = st.torch
    q = torch.from_numpy(st.rng.standard_normal((2 * rows, 4, 128)).astype(np.float32)).cuda()
    q = q.bfloat16() if dtype == "bf16" else q
    out, lse = st.kv.kv_attention(st.cache, st.dtable, st.i32([256, 256]), q, 256, row_off=st.off([rows, rows]), max_rows=rows)
    assert torch.isfinite(lse).all()
    nan = torch.isnan(out)
    sees = torch.zeros_like(nan)
    sees[:rows, :, 5] = True
    sees[[rows + i for i in range(rows) if 256 - rows + i >= 216], :, 9] = True
    assert torch.equal(nan, sees)
    for y in "kv":
        st.model.b[y] = np.where((st.model.b[y] & 0x7f) == 0x7f, 0, st.model.b[y])
    _compare_dims(st, [rows, rows], q, torch.where(nan, torch.zeros_like(out), out) + _model_dims(st, rows, q, sees), lse, dtype)


def _model_dims(st, rows, q, where):
    """the model's results at `where`, 0 elsewhere"""
    torch = st.torch
    got = np.zeros(tuple(q.shape))
    for s in range(len(st.len)):
        k, v = (st.model.values(x, st.table[s], st.len[s]) for x in "kv")
        got[s * rows:(s + 1) * rows] = M.attention(q[s * rows:(s + 1) * rows].double().cpu().numpy(), k, v, st.len[s] - rows,
                                                   1 / math.sqrt(st.hd))[0]
    return torch.where(where, torch.from_numpy(got).cuda(), torch.zeros(q.shape, device="cuda", dtype=torch.float64)).to(q.dtype)
