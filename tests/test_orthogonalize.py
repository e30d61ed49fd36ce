"""Updates made orthogonal (mlora_orthogonalize) against the definition in doubles.

Tolerance.  A product's terms are off by at most 2^-20 of themselves (three
products of fp16 parts of 11 bits; the fourth is left out), so with |X|_F = 1 the first A is
off by E, |E|_F <= 2^-20.  A step's polynomial Q = a + b A + c A^2 is then off by
(|b| + 2 |c| |A|) E <= 10 E, x Q(x^2) has a slope of at most 3.9 where singular values
fall (0 .. 1.2), and A's own error grows by a^2 = 11.9 a step inside a phase of at most
three steps (A is formed anew between phases): 10 (3.9^2 + 11.9 3.9 + 141) = 2,000 for a
phase of three, 10 (3.9 + 11.9) 3.9^3 = 9,400 for the two steps before it, of which
3.9^3 holds for directions that are still small, whose part of E is small too (E is
relative to rows).  A bound that counts every term at its worst is 2^-20 x 1e4; errors
of random sign in 32 or more columns add up to less than a tenth of it: 2^-10 of the
result's norm is the tolerance for any matrix.  Singular values that do not differ much
have no such growth (Q is at most 5 in size, three such factors): 2^-20 x 5^3 / 8 = 2^-16
for those.  bf16 results: 2^-8 of each value besides.
"""
import ctypes
import math

import numpy as np
import pytest

COEFFS = (3.4445, -4.7750, 2.0315)


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    import rl_step_gb300.grads as gr
    return gr, gr._lib()


# ----------------------------------------------------------------------------
# on the CPU
# ----------------------------------------------------------------------------
def _set(gr, src=(4096, 8192), dst=None, rows=(4, 100), cols=(64, 8), dtype=1):
    n = len(src)
    keep = ((ctypes.c_void_p * n)(*src), None if dst is None else (ctypes.c_void_p * n)(*dst),
            (ctypes.c_int64 * n)(*rows), (ctypes.c_int64 * n)(*cols))
    m = gr._MatrixSet(*keep, n, dtype)
    m._keep = keep
    return m


def test_refusals_without_a_gpu():
    gr, lib = _lib()

    def rc(m, a=1.0, b=1.0, c=1.0, eps=1e-7, steps=5):
        p = gr._NewtonSchulz(a, b, c, eps, steps)
        return lib.mlora_orthogonalize(ctypes.byref(m) if m is not None else None, ctypes.byref(p), None)

    good = _set(gr, rows=(0, 5), cols=(3, 0))
    assert rc(good) == 0                                        # nothing to do
    assert rc(None) == -1 and lib.mlora_orthogonalize(ctypes.byref(good), None, None) == -1
    for kw in (dict(a=math.nan), dict(b=math.inf), dict(c=-math.inf), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(steps=0), dict(steps=13)):
        assert rc(good, **kw) == -1 and lib.mlora_last_error(), kw
    for kw in (dict(dtype=2), dict(rows=(65, 100), cols=(65, 8)), dict(rows=(-1, 100)), dict(cols=(64, -8)),
               dict(cols=(1 << 31, 8)), dict(src=(None, 8192)), dict(src=(4098, 8192)), dict(dtype=0, src=(4097, 8192)),
               dict(dst=(4096, None)), dict(dst=(4096, 8194))):
        assert rc(_set(gr, **kw)) == -1 and lib.mlora_last_error(), kw


def test_header_and_binding_agree(tmp_path):
    import os
    import re
    import shutil
    import subprocess
    gr, _ = _lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = [("mlora_matrix_set", gr._MatrixSet), ("mlora_newton_schulz", gr._NewtonSchulz)]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mlora.h"', "int main(void) {"]
    for name, cls in structs:
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f[0]}));' for f in cls._fields_]
    lines.append('printf("%d\\n", MLORA_ORTHO_MAX_STEPS); return 0; }')
    (tmp_path / "a.c").write_text("\n".join(lines))
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"),
                    "-o", str(tmp_path / "a")], check=True, capture_output=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.split()]
    want = []
    for _, cls in structs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want + [12]
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "mlora.h")).read(), flags=re.S)
    m = re.search(r"\bmlora_orthogonalize\s*\(([^)]*)\)", src)
    assert m and len(m.group(1).split(",")) == len(gr._SIGNATURES["mlora_orthogonalize"][1])


def _model(m, steps=5, co=COEFFS, eps=1e-7):
    """The definition, in doubles, as it stands."""
    x = np.asarray(m, dtype=np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.linalg.norm(x) + eps)
    for _ in range(steps):
        a = x @ x.T
        x = co[0] * x + (co[1] * a + co[2] * (a @ a)) @ x
    return x.T if tall else x


def test_the_model_brings_singular_values_near_one():
    rng = np.random.default_rng(0)
    s = np.linalg.svd(_model(rng.standard_normal((16, 200))), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3


# ----------------------------------------------------------------------------
# on the GPU
# ----------------------------------------------------------------------------
def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib()
    return torch


def _check(m, out, tol, **kw):
    want = _model(m.double().cpu().numpy(), **kw)
    got = out.double().cpu().numpy()
    err = np.linalg.norm(got - want)
    more = 2.0 ** -8 if out.element_size() == 2 else 2.0 ** -24
    assert err <= (tol + more) * np.linalg.norm(want) + 1e-30, (m.shape, err / np.linalg.norm(want))


SHAPES = [(1, 1), (1, 7), (9, 1), (3, 3), (4, 4096), (4096, 4), (8, 33), (33, 8), (16, 16), (16, 1000), (1000, 16),
          (17, 31), (31, 17), (32, 4096), (12288, 32), (32, 1023), (1023, 32), (20, 777), (777, 20), (64, 64), (64, 2048),
          (2048, 64), (50, 999), (999, 50), (63, 5), (36, 5120), (5120, 36), (64, 25600), (25600, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("how", ["new", "in place", "odd addresses"])
def test_shapes(dtype, how):
    """ranks around the tiles', odd sizes, long sides around a block's part, one set of all"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    off = 1 if how == "odd addresses" else 0
    total = sum(a * b + 24 for a, b in SHAPES)
    buf = (torch.randn(total, generator=g, device="cuda") * 1e-3).to(dt)
    res = torch.full_like(buf, 7)
    mats, outs, at = [], [], 0
    for a, b in SHAPES:
        mats.append(buf[at + off:at + off + a * b].view(a, b))
        outs.append(res[at + off:at + off + a * b].view(a, b))
        at += -(-(a * b + 8) // 8) * 8
    before = [m.clone() for m in mats]
    if how == "in place":
        ms = gr.MatrixSet(mats)
        got = gr.orthogonalize(ms)
        assert got[0] is mats[0]
    else:
        rest = buf.clone()
        ms = gr.MatrixSet(mats, out=outs)
        got = gr.orthogonalize(ms)
        assert torch.equal(buf, rest)
        for o in outs:
            first = o.clone()
            o.fill_(7)
            assert not torch.equal(first, o)
        assert (res == 7).all()                             # nothing between the outputs
        got = gr.orthogonalize(ms)
    for m, o in zip(before, got):
        _check(m, o, 2.0 ** -10)
    if how == "new":
        again = [o.clone() for o in got]
        gr.orthogonalize(ms)
        assert all(torch.equal(a, b) for a, b in zip(again, got))         # bit for bit
        one = gr.orthogonalize(gr.MatrixSet([mats[13]]))[0]               # alone
        assert torch.equal(one, again[13])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(32, 4096), (4096, 32), (64, 3000), (3000, 64), (8, 500), (12, 2000)])
def test_like_singular_values_are_held_closely(shape):
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(3)
    m = torch.randn(*shape, generator=g, device="cuda")
    _check(m, gr.orthogonalize(gr.MatrixSet([m], out=[torch.empty_like(m)]))[0], 2.0 ** -16)


@pytest.mark.gpu
@pytest.mark.parametrize("low", [1e-1, 1e-2, 1e-3, 1e-4, 0.0])
def test_spread_singular_values(low):
    """a spectrum down to `low` of its largest value, and one of lower rank: as near as the same formula in fp32 products
    is, times four"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    rng = np.random.default_rng(5)
    for r, n in ((32, 1500), (64, 700), (8, 3000)):
        u, v = np.linalg.qr(rng.standard_normal((r, r)))[0], np.linalg.qr(rng.standard_normal((n, r)))[0]
        s = np.geomspace(1, low, r) if low else np.r_[np.ones(r // 2), np.zeros(r - r // 2)]
        for m in ((u * s) @ v.T, ((u * s) @ v.T).T.copy()):
            m = torch.from_numpy(m * 37.0).float().cuda()
            out = gr.orthogonalize(gr.MatrixSet([m], out=[torch.empty_like(m)]))[0]
            want = _model(m.double().cpu().numpy())
            x = m if m.shape[0] < m.shape[1] else m.t()
            x = x / (x.norm() + 1e-7)
            for _ in range(5):
                a = x @ x.t()
                x = COEFFS[0] * x + (COEFFS[1] * a + COEFFS[2] * (a @ a)) @ x
            plain = (x if m.shape[0] < m.shape[1] else x.t()).double().cpu().numpy()
            err, ref = np.linalg.norm(out.double().cpu().numpy() - want), np.linalg.norm(plain - want)
            assert err <= 2.0 ** -10 * np.linalg.norm(want)
            assert err <= 4 * ref + 2.0 ** -18 * np.linalg.norm(want), (m.shape, err, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", list(range(1, 13)))
def test_steps_and_coefficients(steps):
    """every division into phases; coefficients that converge (1.5, -0.5, 0)"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(steps)
    for shape in ((32, 600), (600, 13)):
        m = torch.randn(*shape, generator=g, device="cuda")
        for co in (COEFFS, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)):
            out = gr.orthogonalize(gr.MatrixSet([m], out=[torch.empty_like(m)]), steps, co)[0]
            _check(m, out, 2.0 ** -10, steps=steps, co=co)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_extreme_magnitudes_and_eps(dtype):
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(7)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    base = [torch.randn(16, 300, generator=g, device="cuda"), torch.randn(300, 40, generator=g, device="cuda")]
    for scale, eps in ((1e-30, 1e-30), (1e-38, 1e-38), (1e37, 1e-7), (1e18, 1.0), (1e-12, 1e-7), (1e-7, 1e-7), (1.0, 50.0)):
        mats = [(b * scale).to(dt) for b in base]
        outs = gr.orthogonalize(gr.MatrixSet(mats, out=[torch.empty_like(m) for m in mats]), eps=eps)
        e = float(np.float32(eps))
        for m, o in zip(mats, outs):
            _check(m, o, 2.0 ** -10, eps=e)
    # one large value beside small ones, rows of very different size
    m = base[0].clone()
    m[3, 5] = 1e20
    m[7] *= 1e-6
    m = m.to(dt)
    _check(m, gr.orthogonalize(gr.MatrixSet([m], out=[torch.empty_like(m)]))[0], 2.0 ** -10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_zeros_and_values_that_are_no_numbers(dtype):
    """zeros stay zero; NaN and infinities fill their matrix and no other"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(7)
    good = torch.randn(32, 500, generator=g, device="cuda").to(dt)
    alone = gr.orthogonalize(gr.MatrixSet([good.clone()]))[0]
    zero, nan, inf = torch.zeros_like(good), good.clone(), good.t().contiguous()
    nan[31, 499], inf[0, 0] = math.nan, -math.inf
    for eps in (1e-7, 1e-38):
        mats = [zero.clone(), good.clone(), nan.clone(), inf.clone(), torch.zeros(1, 1, dtype=dt, device="cuda")]
        gr.orthogonalize(gr.MatrixSet(mats), eps=eps)
        assert (mats[0] == 0).all() and (mats[4] == 0).all()
        assert torch.isnan(mats[2]).all() and torch.isnan(mats[3]).all()
        if eps == 1e-7:
            assert torch.equal(mats[1], alone)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_parts_of_very_different_size(dtype):
    """zeros, tiny and huge values in the first columns (a warp's first tile says how it scales), outliers behind them"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(11)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    mats = []
    for first in (0.0, 1e-9, 1e6, 1e-25):
        for shape in ((32, 900), (900, 32), (12, 300), (300, 60)):
            m = torch.randn(*shape, generator=g, device="cuda")
            wide = m if shape[0] < shape[1] else m.t()
            wide[:, :256] *= first
            mats.append(m.to(dt))
    m = torch.randn(16, 5000, generator=g, device="cuda")
    m[3, 4999] = 1e5
    m[5, 40] = -3e4
    mats += [m.to(dt), (m.t() * 1e-3).to(dt).contiguous()]
    outs = gr.orthogonalize(gr.MatrixSet(mats, out=[torch.empty_like(m) for m in mats]))
    for m, o in zip(mats, outs):
        _check(m, o, 2.0 ** -10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("co,steps", [((5.0, 5.0, 5.0), 5), ((5.0, 5.0, 5.0), 6), ((5.0, 5.0, 5.0), 9), ((5.0, 5.0, 5.0), 12),
                                      ((1e10, 0.0, 0.0), 12), ((1.0, -1e20, 0.0), 3), ((1.0, 1.0, 1e30), 2)])
def test_an_iteration_that_diverges_gives_nan(co, steps, dtype):
    """x grows to a few times 5 |x|^5 a step from |x| near 1: beyond fp32's range after five.  (1, -1e20, 0): 1e20, 1e80;
    (1, 1, 1e30): its second A is beyond 1e60.  No number that an optimizer would take, whatever the shape"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(steps)
    for shape in ((32, 600), (600, 13), (64, 900), (8, 8), (4096, 16), (32, 12288)):
        m = torch.randn(*shape, generator=g, device="cuda").to(dt)
        out, zero = (gr.orthogonalize(gr.MatrixSet([x], out=[torch.empty_like(x)]), steps, co)[0] for x in (m, torch.zeros_like(m)))
        assert torch.isnan(out).all(), (shape, torch.isfinite(out).sum().item())
        assert (zero == 0).all()
        m_in_place = m.clone()
        gr.orthogonalize(gr.MatrixSet([m_in_place]), steps, co)
        assert torch.isnan(m_in_place).all()


@pytest.mark.gpu
def test_elements_far_below_the_others():
    """one step of x <- x is M / |M|, element by element.  The norm is off by 2^-20 (its squares' factors), P and M by 2^-22
    each, the product of their low parts 2^-22, the result 2^-24: 2^-19 with room for P's and the norm's own roundings; an
    element whose low part is below fp16's normal range by 2^-25 of what |M|, in 2^14 .. 2^15, is scaled to: 2^-39"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(6)
    for shape in ((32, 2048), (2048, 32), (12, 300), (300, 60)):
        m = torch.randn(*shape, generator=g, device="cuda")
        m *= 10.0 ** torch.randint(-9, 1, shape, generator=g, device="cuda")
        out = gr.orthogonalize(gr.MatrixSet([m], out=[torch.empty_like(m)]), 1, (1.0, 0.0, 0.0))[0].double()
        want = m.double() / (m.double().norm() + float(np.float32(1e-7)))
        assert ((out - want).abs() <= 2.0 ** -19 * want.abs() + 2.0 ** -39).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_one_matrix_alone_and_among_many(dtype):
    """the number and lengths of a set's matrices say over how many blocks one is spread, and so the order of its sums: the
    results differ by what each is off at most, 2^-20 + 2^-24 / s, and by two roundings to bf16 of values that far apart
    (each half a step of 2^-7 at most); a set as it is repeats bit for bit"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(21)
    mats = [m for m in torch.randn(400, 32, 4096, generator=g, device="cuda").to(dt)]
    outs = [torch.empty_like(m) for m in mats]
    ms = gr.MatrixSet(mats, out=outs)
    gr.orthogonalize(ms)
    first = [o.clone() for o in outs]
    gr.orthogonalize(ms)
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    for i in (0, 7, 399):
        alone = gr.orthogonalize(gr.MatrixSet([mats[i]], out=[torch.empty_like(mats[i])]))[0]
        for o in (alone, outs[i]):
            _check(mats[i], o, 2.0 ** -16)
        s = torch.linalg.svdvals(mats[i].double())
        bound = 2 * (2.0 ** -20 + 2.0 ** -24 * (s.norm() / s[-1]).item())
        a, b = alone.double(), outs[i].double()
        apart = (a - b).abs()
        if dtype == "bf16":
            # neighbours at most, where the values before the rounding lie on two sides of a middle
            assert (apart <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + bound * b.norm()).all()
        else:
            assert (apart.norm() <= (bound + 2.0 ** -24) * b.norm()).item(), (apart.norm() / b.norm()).item()


@pytest.mark.gpu
def test_more_matrices_than_a_launch_holds():
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1500, 8, 40, generator=g, device="cuda")
    y = torch.randn(100, 70, 32, generator=g, device="cuda")
    mats = [m for m in x] + [m for m in y]
    outs = [torch.empty_like(m) for m in mats]
    gr.orthogonalize(gr.MatrixSet(mats, out=outs))
    for i in list(range(0, 1600, 97)) + [1299, 1300, 1301, 1499, 1500, 1599]:
        _check(mats[i], outs[i], 2.0 ** -10)


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream():
    torch = _torch()
    import rl_step_gb300.grads as gr
    g = torch.Generator(device="cuda").manual_seed(2)
    mats = [torch.randn(32, 900, generator=g, device="cuda"), torch.randn(512, 16, generator=g, device="cuda")]
    outs = [torch.empty_like(m) for m in mats]
    ms = gr.MatrixSet(mats, out=outs)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        gr.orthogonalize(ms)
    torch.cuda.synchronize()
    for _ in range(2):
        for m in mats:
            m.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for m, o in zip(mats, outs):
            _check(m, o, 2.0 ** -10)
    want = [o.clone() for o in outs]
    st = [torch.cuda.Stream() for _ in range(2)]
    sets = [gr.MatrixSet(mats, out=[torch.empty_like(m) for m in mats]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, k in zip(st, sets):
            gr.orthogonalize(k, stream=s)
    torch.cuda.synchronize()
    for k in sets:
        assert all(torch.equal(a, b) for a, b in zip(k.out, want))


@pytest.mark.gpu
def test_python_refusals():
    torch = _torch()
    import rl_step_gb300 as m
    import rl_step_gb300.grads as gr
    x = torch.randn(8, 100, device="cuda")
    for bad in (lambda: gr.MatrixSet([]), lambda: gr.MatrixSet([x.cpu()]), lambda: gr.MatrixSet([x.t()]),
                lambda: gr.MatrixSet([x[0]]), lambda: gr.MatrixSet([x.half()]), lambda: gr.MatrixSet([x, x]),
                lambda: gr.MatrixSet([x, x.bfloat16()]), lambda: gr.MatrixSet([x], out=[x[:4]]),
                lambda: gr.MatrixSet([x[:4]], out=[x[2:6]])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gr.orthogonalize(gr.MatrixSet([torch.zeros(65, 70, device="cuda")])),
                lambda: gr.orthogonalize(gr.MatrixSet([x]), steps=0), lambda: gr.orthogonalize(gr.MatrixSet([x]), eps=0.0),
                lambda: gr.orthogonalize(gr.MatrixSet([x]), coefficients=(1.0, math.inf, 0.0))):
        with pytest.raises(m.MLoRAError):
            bad()


@pytest.mark.gpu
def test_an_update_of_the_transformers_factors():
    """gradients of the transformer's adapters, clipped and made orthogonal, as a user's optimizer takes them"""
    torch = _torch()
    import rl_step_gb300.grads as gr
    import rl_step_gb300.transformer as t
    from test_rollout import Setup
    s = Setup(max_tokens=256, qk_std=0.05)
    rng = np.random.default_rng(4)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    n = 150
    toks = rng.integers(0, s.cfg.vocab, n + 1)
    t.tf_forward_backward(s.h, i32(toks[:-1]), i32(toks[1:]), i32(np.arange(n)), i32(np.zeros(n)), "cross_entropy",
                          weights=torch.ones(n, device="cuda"))
    grads = [t.tf_read_adapter(s.h, 0, l, p, f, "grad") for l in range(s.cfg.n_layers) for p in t.PROJ for f in "AB"]
    before = [g.clone() for g in grads]
    norms = gr.clip_grads(gr.GradSet(grads), 1e-3)
    gr.orthogonalize(gr.MatrixSet(grads))
    assert torch.isfinite(norms).all()
    f = min(1.0, 1e-3 / norms.item())
    for b, g in zip(before, grads):
        assert g.norm() > 0
        # clipping first changes eps's part alone; gradients of few tokens have small singular values
        want = _model(b.double().cpu().numpy() * f)
        assert np.linalg.norm(g.double().cpu().numpy() - want) <= 2.0 ** -6 * np.linalg.norm(want)
