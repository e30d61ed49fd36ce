"""Page tables made on the GPU (mlora_kv_reserve, mlora_kv_release) against a plain
Python model: whole numbers, so everything has to be equal."""
import ctypes

import numpy as np
import pytest

PAGE = 64


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    import rl_step_gb300.kv as kv
    return kv, kv._lib()


# ----------------------------------------------------------------------------
# on the CPU
# ----------------------------------------------------------------------------
P = 4096                                         # never dereferenced


def _args(kv, **kw):
    f = dict(free_pages=P, n_free=P, owner=P, status=None, n_pages=4, page_table=P, kv_len=P, n_new=P, row_off=P,
             positions=P, seqs=P, slots=P, n_rows=8, n_seqs=3, max_pages=2)
    f.update(kw)
    return (kv._KvPool(*[f[k[0]] for k in kv._KvPool._fields_]), kv._KvGrowth(*[f[k[0]] for k in kv._KvGrowth._fields_]))


@pytest.mark.parametrize("field,value", [("free_pages", None), ("n_free", None), ("owner", None), ("n_pages", 0),
                                         ("page_table", None), ("kv_len", None), ("n_new", None), ("row_off", None),
                                         ("n_rows", -1), ("n_rows", 1 << 31), ("n_seqs", -1), ("n_seqs", 2 ** 31 - 1),
                                         ("max_pages", 0)])
def test_refusals_without_a_gpu(field, value):
    kv, lib = _lib()
    p, g = _args(kv, **{field: value})
    assert lib.mlora_kv_reserve(ctypes.byref(p), ctypes.byref(g), None) == -1 and lib.mlora_last_error()
    if field in ("n_new", "row_off", "n_rows"):
        return
    assert lib.mlora_kv_release(ctypes.byref(p), g.page_table, g.kv_len, P, g.n_seqs, g.max_pages, None) == -1


def test_null_and_nothing_to_do():
    kv, lib = _lib()
    p, g = _args(kv)
    assert lib.mlora_kv_reserve(None, ctypes.byref(g), None) == -1 and lib.mlora_kv_reserve(ctypes.byref(p), None, None) == -1
    assert lib.mlora_kv_release(None, P, P, P, 3, 2, None) == -1
    assert lib.mlora_kv_release(ctypes.byref(p), None, None, None, 0, 2, None) == 0


def test_header_and_binding_agree(tmp_path):
    import os
    import re
    import shutil
    import subprocess
    kv, _ = _lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = [("mlora_kv_pool", kv._KvPool), ("mlora_kv_growth", kv._KvGrowth)]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mlora_kv.h"', "int main(void) {"]
    for name, cls in structs:
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f[0]}));' for f in cls._fields_]
    lines.append('return 0; }')
    (tmp_path / "a.c").write_text("\n".join(lines))
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"),
                    "-o", str(tmp_path / "a")], check=True, capture_output=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in structs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "mlora_kv.h")).read(), flags=re.S)
    for name in ("mlora_kv_reserve", "mlora_kv_release"):
        m = re.search(r"\b%s\s*\(([^)]*)\)" % name, src)
        assert m and len(m.group(1).split(",")) == len(kv._SIGNATURES[name][1]), name


# ----------------------------------------------------------------------------
# the model
# ----------------------------------------------------------------------------
class Model:
    def __init__(self, n_pages, n_seqs, width, seed=0):
        self.n_pages, self.width = n_pages, width
        self.free = list(np.random.default_rng(seed).permutation(n_pages))
        self.owner = [-1] * n_pages
        self.table = np.full((n_seqs, width), -1, np.int64)
        self.len = [0] * n_seqs

    def reserve(self, new, n_rows):
        """(row_off, positions, seqs, slots, status)"""
        bad = pages = rows = 0
        avail = len(self.free)
        off, pos, seqs, slots = [], [], [], []
        for s, add in enumerate(new):
            off.append(len(pos))
            n = self.len[s]
            if n < 0 or add < 0 or n + add > self.width * PAGE:
                bad |= 1
                continue
            need = -(-(n + add) // PAGE) - -(-n // PAGE)
            pages, rows = pages + need, rows + add
            if add and rows > n_rows:
                bad |= 1
                continue
            if need and pages > avail:
                bad |= 4
                continue
            for k in range(need):
                page = self.free.pop()
                self.owner[page] = s
                self.table[s, -(-n // PAGE) + k] = page
            for p in range(n, n + add):
                pos.append(p)
                seqs.append(s)
                slots.append(int(self.table[s, p // PAGE]) * PAGE + p % PAGE)
            self.len[s] = n + add
        off.append(len(pos))
        fill = [-1] * (n_rows - len(pos))
        return off, pos + fill, seqs + fill, slots + fill, bad

    def release(self, keep):
        bad = 0
        for s in reversed(range(len(self.len))):
            n = self.len[s]
            if n < 0 or n > self.width * PAGE or keep[s] < 0:
                bad |= 1
                continue
            if keep[s] >= n:
                continue
            for k in reversed(range(-(-keep[s] // PAGE), -(-n // PAGE))):
                page = self.table[s, k]
                self.table[s, k] = -1
                if page < 0 or page >= self.n_pages:
                    bad |= 1
                elif self.owner[page] == s:
                    self.owner[page] = -1
                    self.free.append(page)
            self.len[s] = keep[s]
        return bad


def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib()
    return torch


class Both:
    """The model and the device's state side by side."""

    def __init__(self, n_pages, n_seqs, width, seed=0):
        self.torch = _torch()
        import rl_step_gb300.kv as kv
        self.kv, self.m = kv, Model(n_pages, n_seqs, width, seed)
        self.pool = kv.PagePool(self.i32(self.m.free), self.i32([n_pages]), self.i32(self.m.owner))
        self.push()

    def i32(self, a):
        return self.torch.tensor(np.asarray(a), dtype=self.torch.int32, device="cuda")

    def push(self):
        self.table, self.len = self.i32(self.m.table), self.i32(self.m.len)

    def check(self):
        n = self.pool.n_free.item()
        assert n == len(self.m.free)
        assert self.pool.free[:n].tolist() == [int(x) for x in self.m.free]
        assert self.pool.owner.tolist() == self.m.owner
        assert (self.table.cpu().numpy() == self.m.table).all() and self.len.tolist() == self.m.len

    def reserve(self, new, n_rows=None):
        n_rows = int(np.clip(new, 0, None).sum()) + 3 if n_rows is None else n_rows
        r = self.kv.kv_reserve(self.pool, self.table, self.len, self.i32(new), n_rows)
        off, pos, seqs, slots, bad = self.m.reserve(list(map(int, new)), n_rows)
        self.check()
        assert r.row_off.tolist() == off and r.positions.tolist() == pos and r.seqs.tolist() == seqs
        assert r.slots.tolist() == slots and r.slots.dtype == self.torch.int64
        assert self.kv.kv_pool_check_status(self.pool) == (-2 if bad & 1 else -4 if bad & 4 else 0)
        assert self.pool.status.item() == 0
        return bad

    def release(self, keep=None):
        self.kv.kv_release(self.pool, self.table, self.len, None if keep is None else self.i32(keep))
        bad = self.m.release([0] * len(self.m.len) if keep is None else list(map(int, keep)))
        self.check()
        assert self.kv.kv_pool_check_status(self.pool) == (-2 if bad else 0)
        return bad


# ----------------------------------------------------------------------------
# on the GPU
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("n_seqs,width,most", [(1, 1, 64), (1, 40, 2500), (3, 5, 100), (255, 6, 70), (256, 4, 9),
                                               (257, 8, 200), (1024, 3, 40), (1025, 4, 3), (2500, 9, 100), (40, 130, 8000)])
def test_growing_and_cutting_back(n_seqs, width, most):
    """random growths and cuts: empty sequences, whole and part-filled pages, one block's rounds and rows apart"""
    rng = np.random.default_rng(n_seqs)
    b = Both(n_seqs * width + 5, n_seqs, width, seed=n_seqs)
    for step in range(5):
        room = width * PAGE - np.array(b.m.len)
        new = np.minimum(rng.integers(0, most + 1, n_seqs), room)
        if step == 1:
            new[:] = np.minimum(1, room)             # one token each
        if step == 2 and n_seqs > 1:
            new[rng.integers(0, n_seqs, n_seqs // 2)] = 0
        assert b.reserve(new) == 0
        keep = np.array(b.m.len) - rng.integers(0, most + 1, n_seqs)
        if step == 3:
            keep[::2] = np.array(b.m.len)[::2] + 7   # nothing to cut
        assert b.release(np.maximum(keep, 0)) == 0
    assert b.release() == 0
    assert len(b.m.free) == b.m.n_pages


@pytest.mark.gpu
def test_a_release_undoes_a_growth():
    b = Both(200, 20, 10, seed=2)
    rng = np.random.default_rng(1)
    b.reserve(rng.integers(0, 300, 20))
    free, table, lens = list(b.m.free), b.m.table.copy(), list(b.m.len)
    new = rng.integers(0, 200, 20)
    b.reserve(new)
    grown = b.m.table.copy()
    b.release(lens)
    assert b.m.free == free and (b.m.table == table).all()
    b.reserve(new)
    assert (b.m.table == grown).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n_seqs", [5, 1500])
def test_too_few_pages_and_rows(n_seqs):
    """what does not fit is left as it is, and what needs nothing is served all the same"""
    rng = np.random.default_rng(4)
    width = 4
    b = Both(n_seqs, n_seqs, width, seed=4)
    new = rng.integers(0, 120, n_seqs)
    new[-2:] = [130, 0]
    assert b.reserve(new) == 4
    assert b.reserve(np.minimum(63 - (np.array(b.m.len) + 63) % 64, 5)) in (0, 4)      # rests of pages
    b.release()
    assert b.reserve(np.full(n_seqs, 10), n_rows=10 * n_seqs - 1) == 1                 # a row too few
    assert b.m.len[-1] == 0 and b.m.len[0] == 10
    assert b.reserve(np.zeros(n_seqs, int), n_rows=0) == 0
    assert b.reserve(np.full(n_seqs, 1), n_rows=0) == 1


@pytest.mark.gpu
def test_numbers_out_of_range():
    b = Both(40, 6, 3, seed=5)
    assert b.reserve([10, -1, 193, 192, 0, 2 ** 31 - 1], n_rows=400) == 1
    assert b.m.len == [10, 0, 0, 192, 0, 0]
    b.m.len[1], b.m.len[4] = -5, 193                 # lengths that no call left there
    b.push()
    assert b.reserve([1, 1, 1, 0, 1, 1]) == 1
    assert b.release([0, 0, 0, 64, 0, -1]) == 1
    b.m.len[1], b.m.len[4] = 0, 0
    b.push()
    b.reserve([64, 64, 64, 0, 64, 64])
    b.m.table[0, 0], b.m.table[2, 0] = 40, -7        # page ids out of range
    b.push()
    assert b.release() == 1


@pytest.mark.gpu
def test_a_pool_whose_number_is_out_of_range_is_left():
    torch = _torch()
    b = Both(8, 2, 3)
    for n in (-1, 9, 2 ** 31 - 1):
        b.pool.n_free.fill_(n)
        r = b.kv.kv_reserve(b.pool, b.table, b.len, b.i32([5, 0]), 5)
        assert b.kv.kv_pool_check_status(b.pool) == -2 and b.len.tolist() == [0, 0] and r.row_off.tolist() == [0, 0, 0]
        b.kv.kv_release(b.pool, b.table, b.len)
        assert b.kv.kv_pool_check_status(b.pool) == -2 and b.pool.n_free.item() == n
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_shared_pages_stay_with_their_owner():
    """a prefix in two rows goes back once, when its owner lets it go; a page listed twice by its own row too"""
    b = Both(20, 3, 4, seed=6)
    b.reserve([130, 0, 0])
    b.m.table[1, :2] = b.m.table[0, :2]
    b.m.len[1] = 128
    b.push()
    b.reserve([0, 100, 0])
    assert b.release([130, 0, 0]) == 0
    assert len(b.m.free) == 20 - 3
    b.m.table[2, 0] = b.m.table[0, 2]                # and of another's last page
    b.m.len[2] = 5
    b.push()
    assert b.release() == 0
    assert sorted(b.m.free) == list(range(20))
    b.reserve([192, 0, 0])
    b.m.table[0, 2] = b.m.table[0, 0]
    twice = b.m.table[0].copy()
    b.push()
    b.kv.kv_release(b.pool, b.table, b.len)
    n = b.pool.n_free.item()
    ids = b.pool.free[:n].tolist()
    assert n == 19 and len(set(ids)) == 19 and b.pool.owner[int(twice[0])].item() == -1


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4, 1500])
def test_no_growth_inside_a_page_of_another_sequence(n):
    """a row cut to a length inside a shared page, a prefix that ends inside one, and a page that its owner has given back:
    no slot in them, the sequence is left as it is and those behind it are served"""
    torch = _torch()
    b = Both(20, n, 4, seed=8)
    rest = [0] * (n - 4)
    b.reserve([130, 0, 0, 40] + rest)
    b.m.table[1, :2], b.m.len[1] = b.m.table[0, :2], 128
    b.m.table[2, :3], b.m.len[2] = b.m.table[0, :3], 130
    b.push()
    assert b.release([130, 100, 130, 40] + rest) == 0
    table, free = b.m.table.copy(), list(b.m.free)

    def grow(new, lens, off, slots, status=-2):
        r = b.kv.kv_reserve(b.pool, b.table, b.len, b.i32(new + rest), 64)
        assert b.kv.kv_pool_check_status(b.pool) == status
        assert b.len.tolist() == lens + rest and (b.table.cpu().numpy() == table).all()
        assert r.row_off.tolist() == off + [off[-1]] * len(rest)
        assert r.slots.tolist() == slots + [-1] * (64 - len(slots)) and b.pool.n_free.item() == len(free)

    def at(s, pos):
        return int(table[s, pos // PAGE]) * PAGE + pos % PAGE

    grow([0, 5, 3, 0], [130, 100, 130, 40], [0, 0, 0, 0, 0], [])
    grow([1, 5, 3, 2], [131, 100, 130, 42], [0, 1, 1, 1, 3], [at(0, 130), at(3, 40), at(3, 41)])
    grow([0, 0, 0, 1], [131, 100, 130, 43], [0, 0, 0, 0, 1], [at(3, 42)], status=0)
    # 30 tokens would need a page as well: it is not taken
    grow([0, 30, 0, 1], [131, 100, 130, 44], [0, 0, 0, 0, 1], [at(3, 43)])
    # the same without rows asked for
    new, row_off = b.i32([0, 5, 3, 1] + rest), b.i32([0] * (n + 1))
    q = b.kv._KvGrowth(b.table.data_ptr(), b.len.data_ptr(), new.data_ptr(), row_off.data_ptr(), None, None, None, 64, n, 4)
    torch.cuda.synchronize()
    assert b.kv._lib().mlora_kv_reserve(b.pool._ref, ctypes.byref(q), None) == 0
    assert b.kv.kv_pool_check_status(b.pool) == -2 and b.len.tolist() == [131, 100, 130, 45] + rest
    # an entry that is no page
    bad = b.table.clone()
    for entry in (-1, 20, 2 ** 31 - 1, -2 ** 31):
        bad[3, 0] = entry
        r = b.kv.kv_reserve(b.pool, bad, b.len, b.i32([0, 0, 0, 1] + rest), 1)
        assert b.kv.kv_pool_check_status(b.pool) == -2 and b.len.tolist() == [131, 100, 130, 45] + rest
        assert r.slots.tolist() == [-1]
    # the owner gives its pages back: nobody's now, and soon another's
    b.m.len[:4] = [131, 100, 130, 45]
    assert b.release([0, 100, 130, 45] + rest) == 0
    table, free = b.m.table.copy(), list(b.m.free)
    grow([0, 5, 3, 0], [0, 100, 130, 45], [0, 0, 0, 0, 0], [])
    # cut back to whole pages both grow in pages of their own
    assert b.release([0, 64, 128, 45] + rest) == 0
    assert b.reserve([0, 5, 70, 1] + rest) == 0
    assert b.m.owner[b.m.table[1, 1]] == 1 and b.m.owner[b.m.table[2, 2]] == b.m.owner[b.m.table[2, 3]] == 2


@pytest.mark.gpu
def test_captured_growth_replays_and_other_stream():
    """a decode step's cut and growth as a graph: lengths and lists are read at replay"""
    torch = _torch()
    b = Both(600, 70, 8, seed=7)
    rng = np.random.default_rng(3)
    b.reserve(rng.integers(1, 300, 70))
    keep, new = b.len.clone(), torch.zeros_like(b.len)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        b.kv.kv_release(b.pool, b.table, b.len, keep)
        r = b.kv.kv_reserve(b.pool, b.table, b.len, new, 300)
    torch.cuda.synchronize()
    for _ in range(4):
        k, a = [max(0, n - int(rng.integers(0, 70))) for n in b.m.len], rng.integers(0, 4, 70)
        keep.copy_(b.i32(k))
        new.copy_(b.i32(a))
        g.replay()
        b.m.release(k)
        off, pos, seqs, slots, bad = b.m.reserve(list(map(int, a)), 300)
        b.check()
        assert bad == 0 and r.row_off.tolist() == off and r.positions.tolist() == pos and r.slots.tolist() == slots
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a = b.i32(np.ones(70))
    r = b.kv.kv_reserve(b.pool, b.table, b.len, a, 70, stream=st)
    torch.cuda.synchronize()
    assert b.m.reserve([1] * 70, 70)[3] == r.slots.tolist()
    b.check()


@pytest.mark.gpu
def test_slots_beyond_four_gigabytes():
    """page ids whose slots leave 32 bits"""
    torch = _torch()
    n_pages = 1 << 26
    import rl_step_gb300.kv as kv
    pool = kv.PagePool.empty(n_pages)
    pool.n_free.fill_(n_pages)
    pool.free[-3:] = torch.tensor([n_pages - 3, n_pages - 2, n_pages - 1], dtype=torch.int32, device="cuda")
    table, lens = torch.full((1, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    r = kv.kv_reserve(pool, table, lens, lens + 130, 130)
    assert r.slots[0].item() == (n_pages - 1) * 64 and r.slots[129].item() == (n_pages - 3) * 64 + 1
    assert kv.kv_pool_check_status(pool) == 0


@pytest.mark.gpu
def test_python_refusals():
    torch = _torch()
    import rl_step_gb300.kv as kv
    pool = kv.PagePool.empty(8)
    t, n = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: kv.kv_reserve(pool, t[0], n, n, 1), lambda: kv.kv_reserve(pool, t, n[:1], n, 1),
                lambda: kv.kv_reserve(pool, t, n, n.long(), 1), lambda: kv.kv_reserve(pool, t.cpu(), n, n, 1),
                lambda: kv.kv_reserve(pool, t[:, :2], n, n, 1), lambda: kv.kv_release(pool, t, n, n[:1]),
                lambda: kv.kv_release(pool, t.long(), n), lambda: kv.PagePool(n, n, n),
                lambda: kv.PagePool(n.cpu(), n[:1].cpu(), n.cpu()), lambda: kv.PagePool(n, n[:1], n.long())):
        with pytest.raises(ValueError):
            bad()
    import rl_step_gb300 as m
    with pytest.raises(m.MLoRAError):
        kv.kv_reserve(pool, t, n, n, -1)
    r = kv.kv_reserve(pool, t[:0], n[:0], n[:0], 2)
    assert r.row_off.tolist() == [0] and r.slots.tolist() == [-1, -1]


@pytest.mark.gpu
def test_a_rollout_over_tables_made_on_the_gpu():
    """prompts, sampled tokens, refused drafted tokens and finished sequences: what the model gives is bit for bit what
    tables made on the host give, and the tokens are scored with their entropies and alternatives"""
    torch = _torch()
    import rl_step_gb300.kv as kv
    import rl_step_gb300.logits as lg
    from test_rollout import Setup
    s = Setup(max_tokens=600, qk_std=0.05)
    rng = np.random.default_rng(2)
    lens, ads = [70, 9, 130], [0, 2, 1]
    n_pages, width = 16, 4
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    caches = s.caches(n_pages)
    pool = kv.PagePool.empty(n_pages)
    table, kv_len = torch.full((3, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    prompt = rng.integers(0, s.cfg.vocab, sum(lens))
    ad = i32(ads)
    r = kv.kv_reserve(pool, table, kv_len, i32(lens), 220)      # eleven rows more than there are
    ids = torch.where(r.seqs >= 0, ad[r.seqs.clamp(min=0).long()], torch.zeros_like(r.seqs))
    toks = torch.zeros(220, dtype=torch.int32, device="cuda")
    toks[:sum(lens)] = i32(prompt)
    u = torch.full((3,), 0.37, device="cuda")
    got = [kv.tf_sample_cached(s.h, caches, toks, ids, u, table, kv_len, 256, row_off=r.row_off, max_rows=130)]
    for step in range(4):
        kv.kv_reserve(pool, table, kv_len, i32([1, 1, 1]), 3)
        got.append(kv.tf_sample_cached(s.h, caches, got[-1][0], ad, u, table, kv_len, 256))
    # three drafted tokens each, of which one, none and three are kept
    before = kv_len.clone()
    draft = i32(rng.integers(0, s.cfg.vocab, 9))
    r = kv.kv_reserve(pool, table, kv_len, i32([3, 3, 3]), 9)
    lp = kv.tf_forward_cached(s.h, caches, draft, draft, ad[r.seqs.long()], table, kv_len, 256, row_off=r.row_off, max_rows=3)
    kv.kv_release(pool, table, kv_len, before + i32([1, 0, 3]))
    kv.kv_reserve(pool, table, kv_len, i32([1, 1, 1]), 3)
    got.append(kv.tf_sample_cached(s.h, caches, got[-1][0], ad, u, table, kv_len, 256))
    assert kv.kv_pool_check_status(pool) == 0

    # the same with tables from the host
    c2 = s.caches(n_pages)
    t2 = i32(np.arange(12).reshape(3, 4))
    n2 = i32(lens)
    want = [kv.tf_sample_cached(s.h, c2, i32(prompt), i32(np.repeat(ads, lens)), u, t2, n2, 256,
                                row_off=i32([0, 70, 79, 209]), max_rows=130)]
    for step in range(4):
        n2 = n2 + 1
        want.append(kv.tf_sample_cached(s.h, c2, want[-1][0], ad, u, t2, n2, 256))
    lp2 = kv.tf_forward_cached(s.h, c2, draft, draft, ad.repeat_interleave(3), t2, n2 + 3, 256, row_off=i32([0, 3, 6, 9]), max_rows=3)
    n2 = n2 + i32([1, 0, 3]) + 1
    want.append(kv.tf_sample_cached(s.h, c2, want[-1][0], ad, u, t2, n2, 256))
    assert torch.equal(kv_len, n2) and torch.equal(lp, lp2)
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)

    # what was sampled, scored by the training forward: its logprobs (to the rounding of sums of 1,000 terms in another
    # order, 2 (8 + 2 + 32) 2^-24 and six roundings of each), entropies and alternatives
    import rl_step_gb300.transformer as t
    seq = np.concatenate([np.r_[prompt[a:a + k], [int(g[0][i]) for g in got[:5]]] for i, (a, k) in enumerate(zip([0, 70, 79], lens))])
    pos = np.concatenate([np.arange(k + 5) for k in lens])
    batch = i32(seq), i32(np.r_[seq[1:], 0]), i32(pos), i32(np.repeat(ads, [k + 5 for k in lens]))
    st = lg.tf_forward_stats(s.h, *batch, top=4)
    lp = t.tf_forward(s.h, *batch)
    assert ((st.logprobs - lp).abs() <= 2.0 ** -24 * (84 + 12 * (1 + lp.abs())) + 2.0 ** -20).all()
    assert (st.entropy > 0).all() and (st.top_ids >= 0).all() and (st.top_logprobs[:, 0] >= st.logprobs).all()

    # sequences that have ended give their pages to new ones
    kv.kv_release(pool, table, kv_len, torch.where(i32([1, 0, 0]) > 0, kv_len, torch.zeros_like(kv_len)))
    kv.kv_reserve(pool, table, kv_len, i32([0, 200, 190]), 390)
    assert kv.kv_pool_check_status(pool) == 0
    kv.kv_release(pool, table, kv_len)
    assert pool.n_free.item() == n_pages and sorted(pool.free.tolist()) == list(range(n_pages))
