"""Group norm with an activation on node rows and 8-bit checkpoints: refusals and definitions on the CPU,
kernels against float64 on the GPU (element by element, within bounds derived from the formulas)."""
import ctypes

import numpy as np
import pytest

import workloads
from tests._norm_side import keep64, norm64, norm_bounds

torch = pytest.importorskip("torch")
etp = pytest.importorskip("equivariant_mlip_tensor_edge_b200")

DEV = "cuda:0"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def _np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ CPU: definitions and refusals

@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("lmax,c,groups", [(0, 6, 2), (2, 4, 1)])
def test_gradient_formula_against_differences(lmax, c, groups, act):
    """The float64 backward of the test side against central differences of its forward: the
    truncation error of step 1e-5 is of order 1e-10, the rounding error of order 1e-11."""
    rng = np.random.default_rng(3)
    ptr = [0, 3, 3, 8]
    x = rng.standard_normal((9, (lmax + 1) ** 2 * c))
    w, b, g = 1 + 0.3 * rng.standard_normal((lmax + 1, c)), rng.standard_normal(c), rng.standard_normal(x.shape)

    def loss(x, w, b):
        return float((norm64(x, w, b, lmax, groups, ptr, 1e-3, act)[0] * g).sum())
    stats = norm64(x, w, b, lmax, groups, ptr, 1e-3, act)[1]
    grads = norm64(x, w, b, lmax, groups, ptr, 1e-3, act, grad=g, stats=stats)
    for i, got in enumerate(grads):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in got.shape)
            args = [[x, w, b], [x, w, b]]
            for sign, a in zip((1, -1), args):
                a[i] = a[i].copy()
                a[i][at] += sign * 1e-5
            diff = (loss(*args[0]) - loss(*args[1])) / 2e-5
            assert abs(diff - got[at]) <= 1e-7 * (1 + abs(diff)), (i, at)


def test_norm_commutes_with_rotations():
    """A rotation mixes the components of a rank; the norm and its gate commute with it."""
    rng = np.random.default_rng(5)
    q = np.linalg.qr(rng.standard_normal((3, 3)))[0]
    x = rng.standard_normal((7, 4, 8))
    w, b = rng.standard_normal((2, 8)), rng.standard_normal(8)

    def turn(v):
        v = v.reshape(7, 4, 8).copy()
        v[:, 1:] = np.einsum("ij,njc->nic", q, v[:, 1:])
        return v.reshape(7, 32)
    a = norm64(turn(x), w, b, 1, 2, [0, 7], 1e-5, "silu")[0]
    assert np.abs(a - turn(norm64(x.reshape(7, 32), w, b, 1, 2, [0, 7], 1e-5, "silu")[0])).max() < 1e-12


def test_library_refuses_bad_norm_arguments_before_device_work():
    lib, fake, odd = etp.load_library(), ctypes.c_void_p(4096), ctypes.c_void_p(4100)
    nb = lib.etp_group_norm_workspace_bytes(2, 64, 8, 1, 0)
    assert nb > 0 and lib.etp_group_norm_workspace_bytes(2, 64, 8, 1, 1) > nb

    def fwd(lmax=2, c=64, g=8, n=10, s=1, ptr=None, dtype=0, x=fake, eps=1e-5, act=1, out=fake, stats=fake, fmt=0,
            q=None, scale=None, ws=fake, nb=1 << 30):
        out = ctypes.c_void_p(1 << 20) if out is fake else out
        return lib.etp_group_norm(lmax, c, g, n, s, ptr, dtype, x, None, None, eps, act, 0, out, stats, fmt, q, scale,
                                  ws, nb, None)
    for bad in (dict(lmax=4), dict(lmax=-1), dict(g=7), dict(g=0), dict(c=1028, g=1), dict(c=260, g=65),
                dict(c=257, g=1), dict(c=514, g=1), dict(c=512, g=256), dict(lmax=3, c=260, g=1)):
        assert fwd(**bad) == 3, bad
        assert lib.etp_group_norm_workspace_bytes(bad.get("lmax", 2), bad.get("c", 64), bad.get("g", 8), 1, 0) == 0, bad
    for bad in (dict(n=-1), dict(s=-1, ptr=fake), dict(s=2), dict(dtype=3), dict(act=2), dict(fmt=3), dict(x=None),
                dict(out=None), dict(stats=None), dict(x=odd), dict(out=odd), dict(eps=-1.0), dict(eps=float("nan")),
                dict(fmt=1), dict(fmt=1, q=ctypes.c_void_p(4097), scale=fake), dict(ws=None), dict(nb=nb - 1),
                dict(ws=ctypes.c_void_p(4096 + 16))):
        assert fwd(**bad) == 1, bad
        assert lib.etp_last_error().decode().startswith("etp_group_norm")

    def bwd(n=10, s=1, ptr=None, x=fake, fmt=0, q=None, scale=None, stats=fake, go=fake, gx=ctypes.c_void_p(1 << 20),
            gw=fake, gb=fake, nb=1 << 30):
        return lib.etp_group_norm_backward(2, 64, 8, n, s, ptr, 0, x, fmt, q, scale, stats, None, None, 1, go, 0, gx,
                                           gw, gb, fake, nb, None)
    other = ctypes.c_void_p(1 << 20)
    assert fwd(out=ctypes.c_void_p(4096 + 16 * 64)) == 1 and "overlap" in lib.etp_last_error().decode()
    assert bwd(gx=other, go=other) == 1 and "overlap" in lib.etp_last_error().decode()
    assert bwd(gx=other, x=ctypes.c_void_p((1 << 20) - 64)) == 1
    for bad in (dict(gx=None, gw=None, gb=None), dict(x=None), dict(fmt=1), dict(go=None), dict(go=odd), dict(gx=odd),
                dict(stats=None), dict(nb=nb)):
        assert bwd(**bad) == 1, bad


def test_library_refuses_bad_checkpoint_arguments_before_device_work():
    lib, fake = etp.load_library(), ctypes.c_void_p(4096)
    for call in (lib.etp_checkpoint_store, lib.etp_checkpoint_restore):
        assert call(0, 0, 4, 4, fake, fake, fake, None) == 1
        assert call(1, 5, 4, 4, fake, fake, fake, None) == 1
        assert call(1, 0, -1, 4, fake, fake, fake, None) == 1
        assert call(1, 0, 4, 4, None, fake, fake, None) == 1
        assert call(1, 0, 1 << 40, 4, fake, fake, fake, None) == 3
        assert call(1, 0, 0, 4, None, None, None, None) == 0
        assert call(2, 1, 4, 0, None, None, None, None) == 0
    assert lib.etp_checkpoint_store(1, 0, 4, 4, ctypes.c_void_p(4098), fake, fake, None) == 1


def test_binding_refuses_bad_arguments():
    x = torch.zeros(4, 18)
    with pytest.raises(ValueError):
        etp.group_norm(x, None, None, 2, 1)       # no CPU fallback
    with pytest.raises(ValueError):
        etp.checkpoint8(x)
    with pytest.raises(ValueError):
        etp.group_norm_function("int4")
    with pytest.raises(ValueError):
        etp.edge_conv_function("fp8")


# ------------------------------------------------------------------ GPU: checkpoints

def _awkward(rows, cols, dtype, seed):
    """Values of many sizes with zeros, ties, a NaN, infinities, subnormal and largest values among them."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1)))).to(TYPES[dtype])
    fin = torch.finfo(TYPES[dtype])
    if rows >= 8:
        x[0] = 0
        x[1, ::2] = -0.0
        x[2, cols // 2] = float("nan")
        x[3, 0] = -float("inf")
        x[4] = fin.max
        x[5] = -fin.smallest_normal / 4
        x[6] = torch.arange(cols).to(x.dtype) % 9 - 4.5
        x[7] = fin.smallest_normal * 3
        x[7, 0] = fin.max
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (9, 31), (13, 32), (8, 33), (40, 576), (11, 100), (300, 2048), (700, 3),
                                       (40, 5), (9, 17), (9, 20011)])
def test_checkpoint_is_exact(rows, cols, dtype, fmt):
    x = _awkward(rows, cols, dtype, rows + cols)
    ck = etp.checkpoint8(x.to(DEV), fmt)
    val, code, byte = keep64(_np(x), fmt)
    assert ck.format == fmt and ck.nbytes == rows * cols + rows * -(-cols // 32)
    assert np.array_equal(ck.scale.cpu().numpy(), byte)
    assert np.array_equal(_np(ck.q.float()), code)
    for to in TYPES.values():
        most = torch.finfo(to).max
        want = torch.from_numpy(np.clip(val, -most, most)).to(to)   # held to the type's range, NaN kept
        got = ck.restore(dtype=to)
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
        assert torch.equal(got.isnan().cpu(), want.isnan())
    assert ck.restore().dtype == TYPES[dtype]


@pytest.mark.gpu
def test_checkpoint_views_shapes_and_out():
    x = torch.randn(6, 5, 70, device=DEV)
    part = x[:, 1:4, 3:]                     # neither contiguous nor aligned
    ck = etp.checkpoint8(part)
    assert ck.q.shape == (6, 3, 67) and ck.scale.shape == (6, 3, 3)
    want, _, _ = keep64(_np(part).reshape(18, 67), "int8")
    out = torch.empty(6, 3, 67, device=DEV)
    assert ck.restore(out=out) is out
    assert np.array_equal(_np(out).reshape(18, 67), want)
    flat = torch.randn(1 + 4 * 64, device=DEV)[1:].view(4, 64)    # whole blocks, 4-byte aligned only
    assert np.array_equal(_np(etp.checkpoint8(flat).restore()), keep64(_np(flat), "int8")[0])
    assert etp.checkpoint8(torch.empty(0, 64, device=DEV)).restore().shape == (0, 64)
    with pytest.raises(ValueError):
        ck.restore(out=torch.empty(6, 3, 66, device=DEV))
    with pytest.raises(ValueError):
        etp.Checkpoint8(ck.q, ck.scale[..., :2], torch.float32).restore()
    with pytest.raises(ValueError):
        etp.checkpoint8(x.double())
    with pytest.raises(ValueError):
        etp.checkpoint8(x, "none")


# ------------------------------------------------------------------ GPU: group norm

def _starts(kind, n, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return [0, n]
    if kind == "pad":            # rows before the first and behind the last structure
        return [min(1, n), (n + 1) // 2, (n + 1) // 2, max(n - 2, (n + 1) // 2)]
    if kind == "rows":           # a structure for every row
        return list(range(n + 1))
    cuts = np.sort(rng.integers(0, n + 1, max(1, n // 9)))
    return [0] + cuts.tolist() + [n]


def _norm_inputs(n, lmax, c, dtype, seed, offset=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, (lmax + 1) ** 2 * c)) * np.exp(rng.standard_normal((n, 1)))
    x[:, :c] += offset
    x = torch.from_numpy(x).to(TYPES[dtype])
    w = (1 + 0.3 * rng.standard_normal((lmax + 1, c))).astype(np.float32)
    b = (0.3 * rng.standard_normal(c)).astype(np.float32)
    g = torch.from_numpy(rng.standard_normal(x.shape)).to(TYPES[dtype])
    return x, w, b, g


def _within(got, want, bound, what, most=np.inf):
    # a value that reaches past the type's largest finite one (`most`, and half a step) is infinite there
    past = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= most * (1 + 2.0 ** -12))
    got = np.where(past, want, got)
    off = np.abs(got - want) - bound
    assert np.isfinite(got).all() and off.max() <= 0, (what, float(np.abs(got - want).max()), float(off.max()))


SHAPES = [(1, 0, 1, 1, "one"), (1, 2, 64, 8, "one"), (21, 2, 64, 8, "one"), (700, 1, 32, 4, "ragged"),
          (333, 3, 128, 16, "ragged"), (150, 2, 36, 3, "pad"), (90, 1, 50, 5, "rows"), (257, 0, 252, 7, "ragged"),
          (40, 3, 255, 5, "pad"), (64, 0, 1024, 64, "ragged"), (5000, 0, 8, 2, "ragged"), (3001, 2, 20, 5, "one"),
          (2500, 1, 96, 3, "ragged"), (77, 1, 64, 64, "rows"), (9, 1, 1024, 64, "ragged"), (31, 3, 256, 1, "pad"),
          (11, 2, 454, 1, "one"), (12, 0, 512, 2, "rows")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,lmax,c,groups,kind", SHAPES)
def test_norm_forward(n, lmax, c, groups, kind, dtype):
    x, w, b, _ = _norm_inputs(n, lmax, c, dtype, n + c)
    ptr = _starts(kind, n)
    act = "none" if n % 5 == 0 else "silu"
    out, stats, ck = etp.group_norm(x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV), lmax, groups,
                                    None if kind == "one" else torch.tensor(ptr, dtype=torch.int32, device=DEV),
                                    activation=act)
    want, st = norm64(_np(x), w, b, lmax, groups, ptr, 1e-5, act)
    assert ck is None
    u = 2.0 ** -24
    # the mean is a float64 sum rounded once; the deviation as norm_bounds says
    _within(_np(stats)[:, 0], st[:, 0], 2 * u * np.abs(st[:, 0]) + 1e-12, "mean")
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * u * st[:, 1:], "deviation")
    info = torch.finfo(TYPES[dtype])
    _within(_np(out), want, norm_bounds(_np(x), w, b, lmax, groups, ptr, act, st, info.eps if dtype != "float32" else 0,
                                        tiny=info.smallest_normal), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,lmax,c,groups,kind", SHAPES)
def test_norm_backward(n, lmax, c, groups, kind, dtype, keep):
    x, w, b, g = _norm_inputs(n, lmax, c, dtype, n + c)
    ptr = _starts(kind, n)
    act = "none" if n % 5 == 0 else "silu"
    xd, wd, bd = x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    node_ptr = None if kind == "one" else torch.tensor(ptr, dtype=torch.int32, device=DEV)
    out, stats, ck = etp.group_norm(xd, wd, bd, lmax, groups, node_ptr, activation=act, checkpoint=keep)
    if keep:      # the same checkpoint as the call of its own makes, whichever kernel wrote it
        alone = etp.checkpoint8(xd, keep)
        assert torch.equal(alone.scale, ck.scale) and torch.equal(alone.q.view(torch.int8), ck.q.view(torch.int8))
    got = etp.group_norm_backward(ck if keep else xd, stats, wd, bd, g.to(DEV), lmax, groups, node_ptr, act)
    xin = keep64(_np(x), keep)[0] if keep else _np(x)
    st = _np(stats)
    want = norm64(xin, w, b, lmax, groups, ptr, 1e-5, act, grad=_np(g), stats=st)
    info = torch.finfo(TYPES[dtype])
    bounds = norm_bounds(xin, w, b, lmax, groups, ptr, act, st, info.eps if dtype != "float32" else 0, grad=_np(g),
                         tiny=info.smallest_normal)
    for a, e, t, what in zip(got, want, bounds, ("grad_x", "grad_weight", "grad_bias")):
        _within(_np(a), e, t + 1e-30, what, info.max if dtype == "float16" and what == "grad_x" else np.inf)
    again = etp.group_norm_backward(ck if keep else xd, stats, wd, bd, g.to(DEV), lmax, groups, node_ptr, act)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("tail", ["ragged", "long"])
def test_norm_of_more_rows_than_a_block_holds(tail):
    """100 rows of 4 KB for each of 148 blocks, small structures among them, or one over the second half."""
    n, lmax, c, groups = 14800, 3, 64, 8
    x, w, b, g = _norm_inputs(n, lmax, c, "float32", 21)
    ptr = _starts("ragged", n)
    if tail == "long":
        ptr = [p for p in ptr if p < n // 2] + [n]
    node_ptr = torch.tensor(ptr, dtype=torch.int32, device=DEV)
    xd, wd, bd = x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    out, stats, ck = etp.group_norm(xd, wd, bd, lmax, groups, node_ptr, checkpoint="int8")
    want, st = norm64(_np(x), w, b, lmax, groups, ptr, 1e-5, "silu")
    tiny = torch.finfo(torch.float32).smallest_normal
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    _within(_np(out), want, norm_bounds(_np(x), w, b, lmax, groups, ptr, "silu", st, 0, tiny=tiny), "out")
    alone = etp.checkpoint8(xd)
    assert torch.equal(alone.scale, ck.scale) and torch.equal(alone.q, ck.q)
    got = etp.group_norm_backward(ck, stats, wd, bd, g.to(DEV), lmax, groups, node_ptr)
    kept, st = _np(ck.restore()), _np(stats)
    want = norm64(kept, w, b, lmax, groups, ptr, 1e-5, "silu", grad=_np(g), stats=st)
    bounds = norm_bounds(kept, w, b, lmax, groups, ptr, "silu", st, 0, grad=_np(g), tiny=tiny)
    for a, e, t, what in zip(got, want, bounds, ("grad_x", "grad_weight", "grad_bias")):
        _within(_np(a), e, t + 1e-30, what)


@pytest.mark.gpu
def test_norm_of_values_far_from_zero():
    """Scalars around 1000 with spread 1: the sums of squares cancel 6 digits, which 64-bit sums keep."""
    x, w, b, _ = _norm_inputs(400, 1, 32, "float32", 4, offset=1000.0)
    ptr = _starts("ragged", 400)
    out, stats, _ = etp.group_norm(x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV), 1, 4,
                                   torch.tensor(ptr, dtype=torch.int32, device=DEV))
    want, st = norm64(_np(x), w, b, 1, 4, ptr, 1e-5, "silu")
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    _within(_np(out), want, norm_bounds(_np(x), w, b, 1, 4, ptr, "silu", st, 0), "out")


@pytest.mark.gpu
def test_norm_without_affine_and_partial_gradients():
    x, _, _, g = _norm_inputs(50, 2, 16, "float32", 8)
    xd, gd = x.to(DEV), g.to(DEV)
    out, stats, _ = etp.group_norm(xd, None, None, 2, 4)
    want, st = norm64(_np(x), None, None, 2, 4, [0, 50], 1e-5, "silu")
    _within(_np(out), want, norm_bounds(_np(x), None, None, 2, 4, [0, 50], "silu", st, 0), "out")
    gx, gw, gb = etp.group_norm_backward(xd, stats, None, None, gd, 2, 4)
    only_x = etp.group_norm_backward(xd, stats, None, None, gd, 2, 4, want_grad_affine=False)
    only_w = etp.group_norm_backward(xd, stats, None, None, gd, 2, 4, want_grad_x=False)
    assert torch.equal(only_x[0], gx) and only_x[1] is None and only_x[2] is None
    assert only_w[0] is None and torch.equal(only_w[1], gw) and torch.equal(only_w[2], gb)
    assert etp.group_norm_backward(xd, stats, None, None, gd, 2, 4, want_grad_x=False, want_grad_affine=False) == (None,) * 3


@pytest.mark.gpu
@pytest.mark.parametrize("c", [32, 20])
def test_rows_of_no_structure(c):
    """Rows outside the structures: left alone in a given tensor, zero in a new one, never read by the
    sums, and part of the checkpoint."""
    n, lmax = 200, 1
    x, w, b, g = _norm_inputs(n, lmax, c, "float32", 6)
    ptr = [3, 90, 90, 150]
    outside = [0, 1, 2] + list(range(150, n))
    x[outside] = float("nan")
    g[outside] = float("nan")
    xd, gd, wd, bd = x.to(DEV), g.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    node_ptr = torch.tensor(ptr, dtype=torch.int32, device=DEV)
    new, stats, ck = etp.group_norm(xd, wd, bd, lmax, 2, node_ptr, checkpoint="int8")
    given = torch.full_like(xd, 5.0)
    assert etp.group_norm(xd, wd, bd, lmax, 2, node_ptr, out=given)[0] is given
    assert (new[outside] == 0).all() and (given[outside] == 5).all() and torch.equal(new[3:150], given[3:150])
    assert torch.isfinite(new).all() and torch.isfinite(stats).all() and (stats[1] == 0).all()
    assert ck.restore()[outside].isnan().all() and ck.restore()[3:150].isfinite().all()
    gx, gw, gb = etp.group_norm_backward(ck, stats, wd, bd, gd, lmax, 2, node_ptr)
    held = torch.full_like(xd, 5.0)
    etp.group_norm_backward(ck, stats, wd, bd, gd, lmax, 2, node_ptr, grad_x=held)
    assert (gx[outside] == 0).all() and (held[outside] == 5).all() and torch.equal(gx[3:150], held[3:150])
    assert torch.isfinite(gx).all() and torch.isfinite(gw).all() and torch.isfinite(gb).all()


@pytest.mark.gpu
def test_no_rows_and_no_structures():
    w, b = torch.ones(2, 8, device=DEV), torch.zeros(8, device=DEV)
    none = torch.empty(0, 32, device=DEV)
    out, stats, _ = etp.group_norm(none, w, b, 1, 2, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 32) and stats.shape == (3, 3, 2) and (stats == 0).all()
    gx, gw, gb = etp.group_norm_backward(none, stats, w, b, none, 1, 2, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert gx.shape == (0, 32) and (gw == 0).all() and (gb == 0).all()
    x = torch.randn(5, 32, device=DEV)
    empty = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, stats, _ = etp.group_norm(x, w, b, 1, 2, empty)
    assert (out == 0).all() and stats.shape == (0, 3, 2)
    gx, gw, gb = etp.group_norm_backward(x, stats, w, b, x, 1, 2, empty)
    assert (gx == 0).all() and (gw == 0).all() and (gb == 0).all()


@pytest.mark.gpu
def test_not_a_number_stays_in_its_structure():
    x, w, b, _ = _norm_inputs(60, 1, 16, "float32", 2)
    x[25, 3] = float("nan")
    x[45, 20] = float("inf")
    out, stats, _ = etp.group_norm(x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV), 1, 4,
                                   torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV))
    assert out[:20].isfinite().all()
    assert stats[1, :2, 0].isnan().all() and stats[1, :, 1:].isfinite().all()
    assert stats[2, 2, 1] == 0      # 1 / sqrt(inf)


@pytest.mark.gpu
def test_bad_node_ptr(monkeypatch):
    x = torch.randn(40, 32, device=DEV)
    bad = torch.tensor([0, 30, 20, 40], dtype=torch.int32, device=DEV)
    monkeypatch.setenv("ETP_VALIDATE", "1")
    with pytest.raises(etp.EtpError) as e:
        etp.group_norm(x, None, None, 1, 2, bad)
    assert e.value.status == 4
    with pytest.raises(etp.EtpError):
        etp.group_norm(x, None, None, 1, 2, torch.tensor([0, 41], dtype=torch.int32, device=DEV))
    etp.group_norm(x, None, None, 1, 2, torch.tensor([0, 30, 30, 40], dtype=torch.int32, device=DEV))


@pytest.mark.gpu
def test_binding_checks_shapes_and_types():
    x = torch.randn(6, 32, device=DEV)
    stats = torch.zeros(1, 3, 2, device=DEV)
    for bad in (lambda: etp.group_norm(x, None, None, 2, 2), lambda: etp.group_norm(x[0], None, None, 1, 2),
                lambda: etp.group_norm(x, torch.ones(8, device=DEV), None, 1, 2),
                lambda: etp.group_norm(x, None, torch.ones(9, device=DEV), 1, 2),
                lambda: etp.group_norm(x, None, None, 1, 2, activation="relu"),
                lambda: etp.group_norm(x.double(), None, None, 1, 2),
                lambda: etp.group_norm(x, None, None, 1, 2, out=torch.empty(6, 31, device=DEV)),
                lambda: etp.group_norm(x, None, torch.ones(8), 1, 2),
                lambda: etp.group_norm(x, None, None, 1, 2, workspace=torch.empty(1 << 22, dtype=torch.uint8)),
                lambda: etp.group_norm_backward(x, stats, None, None, x.half(), 1, 2),
                lambda: etp.group_norm_backward(x, stats[:, :2], None, None, x, 1, 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: etp.group_norm(x, None, None, 1, 3), lambda: etp.group_norm(x, None, None, 1, 2, out=x),
                lambda: etp.group_norm_backward(x, stats, None, None, x.clone(), 1, 2, grad_x=x)):
        with pytest.raises(etp.EtpError):
            bad()


@pytest.mark.gpu
def test_views_other_streams_and_workspace():
    """Rows of a larger tensor (unaligned, not contiguous), another stream, a kept workspace."""
    x, w, b, g = _norm_inputs(300, 1, 24, "float32", 9)
    wd, bd = torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    xd, gd = x.to(DEV), g.to(DEV)
    want = etp.group_norm(xd, wd, bd, 1, 3)
    wide = torch.zeros(301, 97, device=DEV)
    wide[1:, 1:] = xd
    assert torch.equal(etp.group_norm(wide[1:, 1:], wd, bd, 1, 3)[0], want[0])
    flat = torch.empty(1 + xd.numel(), device=DEV)[1:].view_as(xd).copy_(xd)
    assert torch.equal(etp.group_norm(flat, wd, bd, 1, 3)[0], want[0])
    back = etp.group_norm_backward(xd, want[1], wd, bd, gd, 1, 3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 3:      # calls at once, each with its own workspace
        with torch.cuda.stream(s):
            y, st, _ = etp.group_norm(xd, wd, bd, 1, 3)
            got.append((y, st) + etp.group_norm_backward(xd, st, wd, bd, gd, 1, 3))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want[:2] + back))
    ws = torch.empty(etp.group_norm_workspace_bytes(1, 24, 3, 1, backward=True), dtype=torch.uint8, device=DEV).fill_(255)
    assert torch.equal(etp.group_norm(xd, wd, bd, 1, 3, workspace=ws)[0], want[0])
    assert torch.equal(etp.group_norm_backward(xd, want[1], wd, bd, gd, 1, 3, workspace=ws)[0], back[0])


@pytest.mark.gpu
def test_captured_and_replayed():
    x, w, b, g = _norm_inputs(500, 2, 32, "float32", 12)
    ptr = torch.tensor(_starts("ragged", 500), dtype=torch.int32, device=DEV)
    wd, bd, gd = torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV), g.to(DEV)
    xd = torch.zeros_like(x, device=DEV)

    def step():
        y, st, ck = etp.group_norm(xd, wd, bd, 2, 4, ptr, checkpoint="e4m3")
        return (y, st, ck.restore()) + etp.group_norm_backward(ck, st, wd, bd, gd, 2, 4, ptr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(2):
        xd.copy_(x.roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step())), k


@pytest.mark.gpu
def test_more_than_2_31_values():
    """8.4 M rows of 256 bfloat16: offsets past 32 bits, in the rows of the last structure."""
    n, c = (1 << 23) + 5, 256
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.empty(n, c, dtype=torch.bfloat16, device=DEV)
    x.normal_()
    ptr = [0, n - 70, n]
    out, stats, ck = etp.group_norm(x, None, None, 0, 8, torch.tensor(ptr, dtype=torch.int32, device=DEV), checkpoint="int8")
    last = _np(x[-70:])
    want, st = norm64(last, None, None, 0, 8, [0, 70], 1e-5, "silu")
    bound = norm_bounds(last, None, None, 0, 8, [0, 70], "silu", st, torch.finfo(torch.bfloat16).eps)
    _within(_np(out[-70:]), want, bound, "out")
    kept = keep64(last, "int8")[0]
    assert np.array_equal(_np(ck.restore(dtype=torch.float32)[-70:]), kept)
    del out
    gx, gw, gb = etp.group_norm_backward(ck, stats, None, None, x, 0, 8, torch.tensor(ptr, dtype=torch.int32, device=DEV))
    want = norm64(kept, None, None, 0, 8, [0, 70], 1e-5, "silu", grad=last, stats=_np(stats[1:]))
    bound = norm_bounds(kept, None, None, 0, 8, [0, 70], "silu", _np(stats[1:]), torch.finfo(torch.bfloat16).eps, grad=last)
    _within(_np(gx[-70:]), want[0], bound[0], "grad_x")


# ------------------------------------------------------------------ GPU: used together

def _tiny():
    wl = workloads.make("tiny")
    conv = etp.EdgeConv(wl.irreps, wl.lmax, wl.irreps, wl.n_basis, float(wl.r_cut))
    g = etp.neighbors(torch.from_numpy(wl.pos).to(DEV), float(wl.r_cut), cell=wl.cell, pbc=wl.pbc)
    return wl, conv, g


@pytest.mark.gpu
@pytest.mark.parametrize("keep", ["int8", "e4m3"])
def test_conv_gradients_from_a_checkpoint(keep):
    """backward, backward_weights and the autograd path at a Checkpoint8 equal those at the values it holds."""
    wl, conv, g = _tiny()
    x = torch.from_numpy(wl.features()).to(DEV)
    W = torch.from_numpy(wl.weights(conv.n_paths)).to(DEV)
    go = torch.from_numpy(wl.cotangent()).to(DEV)
    ck = etp.checkpoint8(x, keep)
    held = ck.restore()
    want = conv.backward(g, held, W, go) + (conv.backward_weights(g, held, go),)
    got = conv.backward(g, ck, W, go) + (conv.backward_weights(g, ck, go),)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    xr, vr, Wr = x.clone().requires_grad_(), g.edge_vec.clone().requires_grad_(), W.clone().requires_grad_()
    out = etp.edge_conv_function(keep).apply(conv, g, xr, vr, Wr)
    assert torch.equal(out, conv.forward(g, x, W))
    out.backward(go)
    assert all(torch.equal(p.grad, q) for p, q in zip((xr, vr, Wr), want))


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8", "e4m3"])
def test_training_block(keep):
    """Two convolutions with a norm between them: every gradient of the autograd path equals the chain of
    the library's calls made by hand; without a checkpoint the loss changes along a direction as its
    gradient says."""
    wl, conv, g = _tiny()
    c, groups = wl.channels, 2
    norm, edge = etp.group_norm_function(keep), etp.edge_conv_function(keep)
    ptr = torch.tensor([0, 12, 12, wl.n_nodes], dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(1)
    leaves = [torch.from_numpy(wl.features()), g.edge_vec.cpu(), torch.from_numpy(wl.weights(conv.n_paths)),
              1 + 0.2 * torch.randn(wl.lmax + 1, c, generator=gen), 0.2 * torch.randn(c, generator=gen),
              torch.from_numpy(wl.weights(conv.n_paths)).flip(0).contiguous()]
    go = torch.from_numpy(wl.cotangent()).to(DEV)

    def run(x, v, W1, w, b, W2):
        y = edge.apply(conv, g, x, v, W1)
        return edge.apply(conv, g, norm.apply(y, w, b, wl.lmax, groups, ptr), v, W2)
    leaves = [t.to(DEV).requires_grad_() for t in leaves]
    run(*leaves).backward(go)
    x, v, W1, w, b, W2 = [t.detach() for t in leaves]
    y = conv.forward(g, x, W1)
    z, stats, kept = etp.group_norm(y, w, b, wl.lmax, groups, ptr, checkpoint=keep)
    hold = (lambda t: etp.checkpoint8(t, keep)) if keep else (lambda t: t)
    gz, gv2 = conv.backward(g, hold(z), W2, go)
    gy, gw, gb = etp.group_norm_backward(kept if keep else y, stats, w, b, gz, wl.lmax, groups, ptr)
    gx, gv1 = conv.backward(g, hold(x), W1, gy)
    want = [gx, gv1 + gv2, conv.backward_weights(g, hold(x), gy), gw, gb, conv.backward_weights(g, hold(z), go)]
    for p, q in zip(leaves, want):
        assert torch.equal(p.grad, q)
    if keep is None:
        for t, grad in list(zip(leaves, want))[2:5]:    # a central difference along a random direction
            d = torch.randn(t.shape, generator=gen).to(DEV)
            d /= d.norm()
            h = 2e-2
            at = [[p.detach() + (s * h * d if p is t else 0) for p in leaves] for s in (1, -1)]
            up, down = (float((run(*a).detach().double() * go.double()).sum()) for a in at)
            slope = float((grad.double() * d.double()).sum())
            scale = float(grad.double().norm())
            # truncation: h^2 / 6 of the third derivative, whose size is of the gradient's order; rounding:
            # 2^-24 of each of the sum's terms over h
            size = float((run(*leaves).detach().double() * go.double()).abs().sum())
            assert abs((up - down) / (2 * h) - slope) <= 10 * h * h * scale + 40 * 2.0 ** -24 * size / h


@pytest.mark.gpu
def test_half_precision_rows_through_autograd():
    x, w, b, g = _norm_inputs(30, 1, 16, "bfloat16", 3)
    xr = x.to(DEV).requires_grad_()
    wr, br = torch.from_numpy(w).to(DEV).requires_grad_(), torch.from_numpy(b).to(DEV).requires_grad_()
    etp.group_norm_function("int8").apply(xr, wr, br, 1, 4).backward(g.to(DEV))
    y, st, ck = etp.group_norm(x.to(DEV), wr.detach(), br.detach(), 1, 4, checkpoint="int8")
    want = etp.group_norm_backward(ck, st, wr.detach(), br.detach(), g.to(DEV), 1, 4)
    assert xr.grad.dtype == torch.bfloat16
    assert all(torch.equal(p.grad, q) for p, q in zip((xr, wr, br), want))


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8"])
def test_broadcast_cotangent_and_partial_leaves(keep):
    """sum() hands down an expanded cotangent; leaves that need no gradient get none."""
    x, w, b, _ = _norm_inputs(40, 1, 24, "float32", 14)
    xd, wd, bd = x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    fn = etp.group_norm_function(keep)
    y, st, ck = etp.group_norm(xd, wd, bd, 1, 3, checkpoint=keep)
    want = etp.group_norm_backward(ck if keep else xd, st, wd, bd, torch.ones_like(y), 1, 3)
    for needs in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
        leaves = [t.clone().requires_grad_(n) for t, n in zip((xd, wd, bd), needs)]
        fn.apply(*leaves, 1, 3).sum().backward()
        for leaf, grad, n in zip(leaves, want, needs):
            assert torch.equal(leaf.grad, grad) if n else leaf.grad is None
