"""Group norm and 8-bit checkpoints where sizes, ranges and arguments end: the launch plan replayed on the
CPU, refusals, and kernels against float64 on the GPU."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

from tests._norm_side import keep64, norm64, norm_bounds
from tests.test_norm_checkpoint import DEV, TYPES, _norm_inputs, _np, _starts, _within, etp, torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


# ------------------------------------------------------------------ bytes of a tile

@pytest.mark.skipif(shutil.which(NVCC) is None, reason="no nvcc")
def test_plan_brings_every_byte_of_every_tile(tmp_path):
    """The launch plan over many shapes and row counts, on the host: each tile's bytes are copied, in bulk or
    by hand, within the array and the slot."""
    exe = tmp_path / "norm_plan"
    csrc = os.path.join(ROOT, "equivariant_mlip_tensor_edge_b200", "csrc")
    subprocess.run([NVCC, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I" + os.path.join(ROOT, "include"),
                    "-I" + csrc, os.path.join(ROOT, "tests", "c", "norm_plan.cu"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith(" 0 wrong"), run.stdout + run.stderr


def test_all_threads_meet_at_the_same_barriers():
    """A grid or block barrier has to be one statement for all threads of a block: none stands in a branch that
    the copying warp or the computing ones take alone."""
    with open(os.path.join(ROOT, "equivariant_mlip_tensor_edge_b200", "csrc", "etp_norm_sweep.h")) as f:
        body = f.read().split("k_norm(const")[1].split("// ---------------------------------------------------------------- launch")[0]
    assert body.count("this_grid().sync()") == 1
    depth = 0
    for line in body.splitlines():
        if "__syncthreads()" in line:
            assert depth == 1, line        # of the kernel's own block
        depth += line.count("{") - line.count("}")
    assert depth == 0


def _check_forward(x, w, b, lmax, groups, ptr, act, out, stats, dtype):
    want, st = norm64(_np(x), w, b, lmax, groups, ptr, 1e-5, act)
    info = torch.finfo(TYPES[dtype])
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    _within(_np(out), want, norm_bounds(_np(x), w, b, lmax, groups, ptr, act, st, info.eps if dtype != "float32" else 0,
                                        tiny=info.smallest_normal), "out")


def _check_backward(xin, w, b, g, lmax, groups, ptr, act, stats, got, dtype):
    st, info = _np(stats), torch.finfo(TYPES[dtype])
    want = norm64(xin, w, b, lmax, groups, ptr, 1e-5, act, grad=_np(g), stats=st)
    bounds = norm_bounds(xin, w, b, lmax, groups, ptr, act, st, info.eps if dtype != "float32" else 0, grad=_np(g),
                         tiny=info.smallest_normal)
    for a, e, t, what in zip(got, want, bounds, ("grad_x", "grad_weight", "grad_bias")):
        _within(_np(a), e, t + 1e-30, what, info.max if dtype == "float16" and what == "grad_x" else float("inf"))


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,lmax,c,groups", [(871, 2, 32, 4), (931, 1, 32, 4), (198, 0, 64, 8), (514, 0, 1, 1), (519, 0, 1, 1)])
def test_short_rows_at_the_end_of_the_array(n, lmax, c, groups, dtype, keep):
    """Fewer than 16 bytes of an array behind a tile that is not the last: rows (or rows of scales) of
    under 16 bytes, a block's border a row or a few before the end."""
    x, w, b, g = _norm_inputs(n, lmax, c, dtype, n)
    ptr = _starts("ragged", n)
    xd, wd, bd = x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    node_ptr = torch.tensor(ptr, dtype=torch.int32, device=DEV)
    out, stats, ck = etp.group_norm(xd, wd, bd, lmax, groups, node_ptr, checkpoint=keep)
    _check_forward(x, w, b, lmax, groups, ptr, "silu", out, stats, dtype)
    got = etp.group_norm_backward(ck if keep else xd, stats, wd, bd, g.to(DEV), lmax, groups, node_ptr)
    _check_backward(keep64(_np(x), keep)[0] if keep else _np(x), w, b, g, lmax, groups, ptr, "silu", stats, got, dtype)


# ------------------------------------------------------------------ no rows

def test_backward_without_rows_may_have_no_gradient_to_write():
    """An empty grad_x has no address: asking for it alone is a valid call."""
    lib, fake = etp.load_library(), ctypes.c_void_p(4096)

    def bwd(n):
        return lib.etp_group_norm_backward(1, 8, 2, n, 1, None, 0, None, 0, None, None, fake, None, None, 1, None, 0, None,
                                           None, None, fake, 1 << 30, None)
    assert bwd(0) == 0
    assert bwd(1) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8"])
def test_gradients_of_no_rows(keep):
    none = torch.empty(0, 32, device=DEV)
    w, b = torch.ones(2, 8, device=DEV), torch.zeros(8, device=DEV)
    ptr = torch.zeros(3, dtype=torch.int32, device=DEV)
    out, stats, ck = etp.group_norm(none, w, b, 1, 2, ptr, checkpoint=keep)
    gx, gw, gb = etp.group_norm_backward(ck if keep else none, stats, w, b, none, 1, 2, ptr, want_grad_affine=False)
    assert gx.shape == (0, 32) and gw is None and gb is None
    for affine in ((None, None), (w, b)):      # absent, and frozen
        x = torch.empty(0, 32, device=DEV, requires_grad=True)
        etp.group_norm_function(keep).apply(x, *affine, 1, 2, ptr).sum().backward()
        assert x.grad.shape == (0, 32)


# ------------------------------------------------------------------ sizes past a C int

@pytest.mark.parametrize("cols", [1 << 32, (1 << 32) + 64, 1 << 31])
def test_binding_refuses_sizes_past_a_c_int(monkeypatch, cols):
    """Sizes of 2^31 and more are refused, not cut to their lower 32 bits (tensors without memory here)."""
    monkeypatch.setattr(etp, "_one_device", lambda *tensors: 0)
    monkeypatch.setattr(etp, "_call", lambda index, where, *args: pytest.fail(f"{where} was called"))
    meta = dict(device="meta")
    x = torch.empty(cols, dtype=torch.bfloat16, **meta)
    ck = etp.Checkpoint8(torch.empty(cols, dtype=torch.int8, **meta), torch.empty(-(-cols // 32), dtype=torch.uint8, **meta),
                         torch.bfloat16)
    tall, wide = x.view(cols, 1), x.view(1, cols)
    many = torch.empty(cols + 1, dtype=torch.int32, **meta)
    few = torch.empty(4, 1, dtype=torch.bfloat16, **meta)
    stats = torch.empty(1, 2, 1, **meta)
    for call in (lambda: etp.checkpoint8(x), lambda: etp.checkpoint8(wide), ck.restore,
                 lambda: etp.group_norm(tall, None, None, 0, 1), lambda: etp.group_norm(wide, None, None, 0, 1),
                 lambda: etp.group_norm(few, None, None, 0, cols + 1), lambda: etp.group_norm(few, None, None, 0, 1, many),
                 lambda: etp.group_norm_backward(tall, stats, None, None, tall, 0, 1),
                 lambda: etp.group_norm_backward(wide, stats, None, None, wide, 0, 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [(1 << 31) - 1, (1 << 31) - 4])
def test_checkpoint_of_the_longest_rows(cols):
    """One row of nearly 2^31 values has the codes of the same values in rows of 32 (whose tail is checked apart)."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.empty(cols, dtype=torch.bfloat16, device=DEV).normal_()
    ck = etp.checkpoint8(x)
    whole = cols // 32 * 32
    rows = etp.checkpoint8(x[:whole].view(-1, 32))
    assert torch.equal(ck.q[:whole].view(-1, 32), rows.q) and torch.equal(ck.scale[:-1], rows.scale[:, 0])
    held, codes, byte = keep64(_np(x[whole:])[None], "int8")
    assert (_np(ck.q[whole:]) == codes).all() and int(ck.scale[-1]) == byte[0, 0]
    back = ck.restore()
    assert torch.equal(back[:whole].view(-1, 32), rows.restore())
    assert (_np(back[whole:]) == _np(torch.from_numpy(held).to(torch.bfloat16))).all()


# ------------------------------------------------------------------ precision

@pytest.mark.gpu
@pytest.mark.parametrize("offset,step", [(1e4, 2.0 ** -8), (1e5, 2.0 ** -6), (1e6, 2.0 ** -4)])
def test_deviation_of_values_far_from_zero(offset, step):
    """Scalars of spread 1 far from zero, in multiples of `step` of under 2^24 steps, at most 32 to a sum: the
    sums of x and x^2 are exact in 64 bits, so nothing but what is made of them can spoil the deviation."""
    rng = np.random.default_rng(11)
    n, c, groups = 200, 32, 8
    x = np.round((offset + rng.standard_normal((n, 4 * c))) / step) * step
    x[:, c:] -= offset
    assert np.abs(x).max() / step < 1 << 24 and (x.astype(np.float32) == x).all()
    ptr = [0, 1] + list(range(8, n, 8)) + [n]     # structures of up to 8 rows, of 4 channels a group
    out, stats, _ = etp.group_norm(torch.from_numpy(x).float().to(DEV), None, None, 1, groups,
                                   torch.tensor(ptr, dtype=torch.int32, device=DEV))
    want, st = norm64(x, None, None, 1, groups, ptr, 1e-5, "silu")
    _within(_np(stats)[:, 0], st[:, 0], 2.0 ** -24 * np.abs(st[:, 0]), "mean")
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    _within(_np(out), want, norm_bounds(x, None, None, 1, groups, ptr, "silu", st, 0), "out")


@pytest.mark.gpu
def test_deviation_of_a_long_structure():
    """100048 equal rows of 1024 channels: 676 to a thread, whose squares of l > 0 a 32-bit sum would round
    the same way each time (56 x 2^-24 in the end). Within the bound of the short ones: a row's squares in
    32 bits, the rest in 64."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    n, c, groups = 148 * 676, 1024, 64
    row = torch.full((1, 4 * c), 0.9, device=DEV)
    row[:, :c:2] = -0.9
    out, stats, _ = etp.group_norm(row.expand(n, -1), None, None, 1, groups)
    want, st = norm64(_np(row), None, None, 1, groups, [0, 1], 1e-5, "silu")
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    bound = norm_bounds(_np(row), None, None, 1, groups, [0, 1], "silu", st, 0)
    for r in (0, n // 2, n - 1):
        _within(_np(out[r:r + 1]), want, bound, "out")


# ------------------------------------------------------------------ waits that give up

def test_status_word_gates_the_norm_until_it_is_read():
    """A kernel that gives up a bounded wait stores its code in the status word of the norm's calls, and every
    later one returns ETP_ERR_CUDA before any CUDA work. Here the test writes the word itself."""
    lib, fake, other = etp.load_library(), ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)
    word = lib.etp_group_norm_status_word()
    assert word and word[0] == 0

    def fwd(x=fake):
        return lib.etp_group_norm(1, 8, 2, 4, 1, None, 0, x, None, None, 1e-5, 1, 0, other, fake, 0, None, None, fake, 1 << 30, None)

    def bwd():
        return lib.etp_group_norm_backward(1, 8, 2, 4, 1, None, 0, fake, 0, None, None, fake, None, None, 1, fake, 0, other,
                                           None, None, fake, 1 << 30, None)
    code = ctypes.c_int(-1)
    try:
        word[0] = 2
        assert fwd() == 5 and "code 2" in lib.etp_last_error().decode()
        assert bwd() == 5 and "code 2" in lib.etp_last_error().decode()
        assert fwd(x=None) == 1          # arguments are checked first
        assert lib.etp_group_norm_status(None, ctypes.byref(code)) == 5 and code.value == 2 and word[0] == 0
        assert lib.etp_group_norm_status(None, ctypes.byref(code)) == 0 and code.value == 0
        word[0] = 3
        with pytest.raises(etp.EtpError) as e:
            etp.group_norm_check_status()
        assert e.value.status == 5 and "code 3" in str(e.value)
        etp.group_norm_check_status()
    finally:
        word[0] = 0


@pytest.mark.gpu
def test_status_word_on_the_device(monkeypatch):
    """Calls leave the word alone; a code in it stops the binding's calls until it is read."""
    x = torch.randn(40, 32, device=DEV)
    word = etp.load_library().etp_group_norm_status_word()
    want = etp.group_norm(x, None, None, 1, 2)[0]
    etp.group_norm_check_status(torch.device(DEV))
    try:
        word[0] = 1
        for call in (lambda: etp.group_norm(x, None, None, 1, 2),
                     lambda: etp.group_norm_backward(x, torch.zeros(1, 3, 2, device=DEV), None, None, x, 1, 2)):
            with pytest.raises(etp.EtpError) as e:
                call()
            assert e.value.status == 5
        with pytest.raises(etp.EtpError):
            etp.group_norm_check_status(torch.device(DEV))
    finally:
        word[0] = 0
    monkeypatch.setenv("ETP_VALIDATE", "1")
    assert torch.equal(etp.group_norm(x, None, None, 1, 2)[0], want)


@pytest.mark.gpu
def test_first_call_of_a_process_may_be_captured():
    """The word is made by the first call, also one that a stream captures."""
    program = (
        "import torch, equivariant_mlip_tensor_edge_b200 as etp\n"
        "x = torch.randn(40, 32, device='cuda')\n"
        "torch.cuda.synchronize()\n"
        "graph = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(graph):\n"
        "    y = etp.group_norm(x, None, None, 1, 2)[0]\n"
        "graph.replay()\n"
        "torch.cuda.synchronize()\n"
        "etp.group_norm_check_status(x.device)\n"
        "assert torch.equal(y, etp.group_norm(x, None, None, 1, 2)[0])\n"
        "print('captured')\n")
    run = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


# ------------------------------------------------------------------ buffers that a program uses again

@pytest.mark.gpu
def test_node_ptr_changed_before_the_backward_is_refused():
    """A batch's node_ptr overwritten for the next one would give wrong gradients: autograd says so, as it
    does for x and the weights."""
    x = torch.randn(20, 32, device=DEV, requires_grad=True)
    w = torch.ones(2, 8, device=DEV, requires_grad=True)
    for change in (0, 1):
        ptr = torch.tensor([0, 12, 20], dtype=torch.int32, device=DEV)
        y = etp.group_norm_function().apply(x, w, None, 1, 2, ptr)
        if change:
            ptr.copy_(torch.tensor([0, 4, 20], dtype=torch.int32))
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.sum().backward()
        else:
            y.sum().backward()


def test_workspace_with_strides_is_refused(monkeypatch):
    """An expanded or strided workspace has fewer bytes behind its address than elements."""
    monkeypatch.setattr(etp, "_one_device", lambda *tensors: 0)
    monkeypatch.setattr(etp, "_call", lambda index, where, *args: pytest.fail(f"{where} was called"))
    x, stats = torch.zeros(4, 32), torch.zeros(1, 3, 2)
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 22), torch.empty(1 << 22, 2, dtype=torch.uint8)[:, 0]):
        for call in (lambda: etp.group_norm(x, None, None, 1, 2, workspace=ws),
                     lambda: etp.group_norm_backward(x, stats, None, None, x, 1, 2, workspace=ws)):
            with pytest.raises(ValueError, match="contiguous"):
                call()


@pytest.mark.gpu
def test_bad_node_ptr_of_no_rows(monkeypatch):
    none, w = torch.empty(0, 32, device=DEV), torch.ones(2, 8, device=DEV)
    monkeypatch.setenv("ETP_VALIDATE", "1")
    bad, good = (torch.tensor(p, dtype=torch.int32, device=DEV) for p in ([0, 5], [0, 0]))
    stats = etp.group_norm(none, w, None, 1, 2, good)[1]
    etp.group_norm_backward(none, stats, w, None, none, 1, 2, good)
    for call in (lambda: etp.group_norm(none, w, None, 1, 2, bad),
                 lambda: etp.group_norm_backward(none, stats, w, None, none, 1, 2, bad)):
        with pytest.raises(etp.EtpError) as e:
            call()
        assert e.value.status == 4


# ------------------------------------------------------------------ range

@pytest.mark.gpu
@pytest.mark.parametrize("keep", [None, "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("power,eps", [(57, 1e-5), (57, 0.0), (-57, 0.0)])
def test_values_of_the_stated_range(power, eps, dtype, keep):
    """Values around 2^57, up to 2^60, and deviations around 2^-57 without eps."""
    n, lmax, c, groups = 300, 2, 32, 4
    x, w, b, g = _norm_inputs(n, lmax, c, dtype, 31)
    x = (x.clamp(-8, 8).float() * 2.0 ** power).to(x.dtype)
    ptr = _starts("ragged", n)
    xd, wd, bd = x.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(b).to(DEV)
    node_ptr = torch.tensor(ptr, dtype=torch.int32, device=DEV)
    out, stats, ck = etp.group_norm(xd, wd, bd, lmax, groups, node_ptr, eps=eps, checkpoint=keep)
    want, st = norm64(_np(x), w, b, lmax, groups, ptr, eps, "silu")
    info = torch.finfo(TYPES[dtype])
    half = info.eps if dtype != "float32" else 0
    _within(_np(stats)[:, 1:], st[:, 1:], 16 * 2.0 ** -24 * st[:, 1:], "deviation")
    _within(_np(out), want, norm_bounds(_np(x), w, b, lmax, groups, ptr, "silu", st, half, tiny=info.smallest_normal), "out")
    got = etp.group_norm_backward(ck if keep else xd, stats, wd, bd, g.to(DEV), lmax, groups, node_ptr)
    _check_backward(keep64(_np(x), keep)[0] if keep else _np(x), w, b, g, lmax, groups, ptr, "silu", stats, got, dtype)


# ------------------------------------------------------------------ first calls at once

def test_first_calls_of_two_threads():
    """A thread's first call may come between any two lines of another's."""
    for line in range(1, 9):
        spec = importlib.util.spec_from_file_location("etp_again", etp.__file__)
        again = importlib.util.module_from_spec(spec)
        sys.modules["etp_again"] = again
        seen = [0]

        def other(frame, event, arg):
            if frame.f_code.co_name != "_dtype_code":
                return None
            if event == "line":
                seen[0] += 1
                if seen[0] == line:
                    sys.settrace(None)
                    assert again._dtype_code(torch.bfloat16) == 1
            return other
        try:
            spec.loader.exec_module(again)
            sys.settrace(other)
            assert again._dtype_code(torch.float32) == 0
        finally:
            sys.settrace(None)
            del sys.modules["etp_again"]
