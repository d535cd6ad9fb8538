"""Refusals and launch plans of the 8-bit linear layer's operators, without a
GPU: the C planner with made-up addresses, and the binding's own checks."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import software_pipelining_amd as tp
from software_pipelining_amd import tilepipe
from tests import linear8_forms as forms

OK, INVALID, MISALIGNED, OVERLAP = 0, 1, 2, 4
BF16, FP16, FP32, E4M3, E5M2 = range(5)
A, B, C, D, E, F, G = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(7))


def lib():
    return tilepipe._load()


def norm(x=A, xs=256, r=B, rs=256, w=C, rows=7, cols=256, dtype=BF16, eps=1e-6, sum_=D, ss=256, out=E,
         os_=256, out_type=E4M3, scale=F, rstd=G):
    plan = tilepipe._CPlan()
    st = lib().tp_plan_rms_norm(x, xs, r, rs, w, rows, cols, dtype, eps, sum_, ss, out, os_, out_type,
                                scale, rstd, ctypes.byref(plan))
    return st, plan


@pytest.mark.parametrize("change, status", [
    ({}, OK),
    ({"rows": 0}, OK),
    ({"cols": 0, "xs": 1, "rs": 1, "ss": 1, "os_": 1}, OK),
    ({"rstd": 0}, OK),
    ({"out_type": BF16, "scale": 0}, OK),
    ({"r": 0, "sum_": 0}, OK),
    ({"xs": 255}, INVALID),
    ({"os_": 255}, INVALID),
    ({"rows": -1}, INVALID),
    ({"cols": (1 << 24) + 1, "xs": 1 << 25, "rs": 1 << 25, "ss": 1 << 25, "os_": 1 << 25}, INVALID),
    ({"dtype": E4M3}, INVALID),
    ({"dtype": 7}, INVALID),
    ({"out_type": FP16}, INVALID),
    ({"eps": -1.0}, INVALID),
    ({"eps": float("nan")}, INVALID),
    ({"x": 0}, INVALID),
    ({"w": 0}, INVALID),
    ({"out": 0}, INVALID),
    ({"r": 0}, INVALID),
    ({"sum_": 0}, INVALID),
    ({"scale": 0}, INVALID),
    ({"out_type": BF16}, INVALID),
    ({"x": A + 1}, MISALIGNED),
    ({"w": C + 1}, MISALIGNED),
    ({"scale": F + 2}, MISALIGNED),
    ({"rstd": G + 1}, MISALIGNED),
    ({"out": E + 1}, OK),                                  # 8-bit rows have no alignment
    ({"sum_": A}, OK),                                     # in place of x
    ({"sum_": B}, OK),                                     # in place of the residual
    ({"sum_": A + 2}, OVERLAP),
    ({"sum_": A, "ss": 257}, OVERLAP),
    ({"out": D + 16}, OVERLAP),
    ({"out": A}, OVERLAP),                                 # another type than x
    ({"scale": C + 4}, OVERLAP),
    ({"rstd": F}, OVERLAP),
    ({"out": A, "out_type": BF16, "scale": 0}, OK),
])
def test_norm_refusals(change, status):
    assert norm(**change)[0] == status


def test_norm_plans_cover_every_width():
    for dtype in (BF16, FP16, FP32):
        for cols in (1, 7, 64, 512, 513, 2048, 8192, 12288, 16384, 20000, 1 << 20):
            for rows in (1, 300, 100000):
                st, plan = norm(rows=rows, cols=cols, xs=cols, rs=cols, ss=cols, os_=cols, dtype=dtype,
                                w=A + (1 << 45), x=A, r=A + (1 << 46), sum_=A + (1 << 47),
                                out=A + (1 << 48), scale=A + (1 << 49), rstd=A + (1 << 50))
                assert st == OK
                assert 64 <= plan.threads <= 1024 and plan.threads % 64 == 0
                assert 0 < plan.grid <= rows and plan.lds_bytes <= 160 * 1024


def backward(dy=A, dys=256, x=B, xs=256, w=C, rstd=C + 65536, ds=D, dss=256, rows=9, cols=256, dtype=FP16,
             dx=E, dxs=256, dw=F, ws=G, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = max(0, lib().tp_rms_norm_backward_workspace_bytes(rows, cols, dtype))
    plan = tilepipe._CPlan()
    return lib().tp_plan_rms_norm_backward(dy, dys, x, xs, w, rstd, ds, dss, rows, cols, dtype, dx, dxs, dw,
                                           ws, ws_bytes, ctypes.byref(plan))


@pytest.mark.parametrize("change, status", [
    ({}, OK),
    ({"ds": 0}, OK),
    ({"rows": 0}, OK),
    ({"dx": A}, OK),
    ({"dx": D}, OK),
    ({"dx": B + 2}, OVERLAP),
    ({"dw": B}, OVERLAP),
    ({"ws": A}, OVERLAP),
    ({"ws": F + 16}, OVERLAP),
    ({"dw": C}, OVERLAP),
    ({"dw": 0}, INVALID),
    ({"rstd": 0}, INVALID),
    ({"ws": 0}, INVALID),
    ({"ws_bytes": 16}, INVALID),
    ({"dxs": 255}, INVALID),
    ({"dtype": E5M2}, INVALID),
    ({"dw": F + 2}, MISALIGNED),
    ({"dy": A + 1}, MISALIGNED),
    ({"cols": 40000, "dys": 40000, "xs": 40000, "dss": 40000, "dxs": 40000, "dx": A}, OVERLAP),  # read twice
    ({"cols": 40000, "dys": 40000, "xs": 40000, "dss": 40000, "dxs": 40000, "dx": E}, OK),
])
def test_backward_refusals(change, status):
    assert backward(**change) == status


def quantize(x=A, xs=300, rows=200, cols=300, dtype=BF16, square=0, out_type=E5M2, q=B, qs=304, scale=C, qt=D,
             qts=208, scale_t=E):
    plan = tilepipe._CPlan()
    return lib().tp_plan_block_quantize(x, xs, rows, cols, dtype, square, out_type, q, qs, scale, qt, qts,
                                        scale_t, ctypes.byref(plan))


@pytest.mark.parametrize("change, status", [
    ({}, OK),
    ({"q": 0, "scale": 0}, OK),
    ({"qt": 0, "scale_t": 0}, OK),
    ({"rows": 0}, OK),
    ({"q": 0, "scale": 0, "qt": 0, "scale_t": 0}, INVALID),
    ({"scale": 0}, INVALID),
    ({"scale_t": 0}, INVALID),
    ({"x": 0}, INVALID),
    ({"square": 2}, INVALID),
    ({"out_type": BF16}, INVALID),
    ({"dtype": E4M3}, INVALID),
    ({"qs": 299}, INVALID),
    ({"qts": 199}, INVALID),
    ({"xs": 1 << 22}, INVALID),            # rows over 2^22 bytes apart
    ({"x": A + 1}, MISALIGNED),
    ({"scale": C + 1}, MISALIGNED),
    ({"q": A}, OVERLAP),
    ({"qt": B + 8}, OVERLAP),
    ({"scale": D}, OVERLAP),
])
def test_quantize_refusals(change, status):
    assert quantize(**change) == status


def matmul(a=A, a_s=272, at=E4M3, sa=B, b=C, bs=272, bt=E4M3, sb=D, square=1, m=100, n=200, k=272, out=E, os_=200,
           ot=BF16, ws=F, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = max(0, lib().tp_block_matmul_workspace_bytes(m, n, k, ot))
    plan = tilepipe._CPlan()
    return lib().tp_plan_block_matmul(a, a_s, at, sa, b, bs, bt, sb, square, m, n, k, out, os_, ot, ws, ws_bytes,
                                      ctypes.byref(plan))


@pytest.mark.parametrize("change, status", [
    ({}, OK),
    ({"square": 0}, OK),
    ({"at": E5M2, "bt": E5M2, "ot": FP32}, OK),
    ({"m": 0}, OK),
    ({"k": 0, "a": 0, "b": 0, "sa": 0, "sb": 0}, OK),
    ({"a": A + 1, "b": C + 3}, OK),        # 8-bit rows have no alignment
    ({"at": BF16}, INVALID),
    ({"ot": E4M3}, INVALID),
    ({"square": -1}, INVALID),
    ({"a_s": 271}, INVALID),
    ({"os_": 199}, INVALID),
    ({"a": 0}, INVALID),
    ({"sb": 0}, INVALID),
    ({"out": 0}, INVALID),
    ({"k": (1 << 22) + 1, "a_s": 1 << 23, "bs": 1 << 23}, INVALID),
    ({"bs": (1 << 22) + 1}, INVALID),
    ({"m": 1, "n": 5_000_000, "k": 64, "os_": 5_000_000, "ot": FP32, "out": E + (1 << 40)}, OK),       # one long row
    ({"m": 3, "n": 5_000_000, "k": 64, "os_": 5_000_000, "ot": FP32, "out": E + (1 << 40)}, OK),
    ({"m": 100, "os_": 5_000_000, "out": E + (1 << 40)}, OK),
    ({"m": 64, "os_": 1 << 22, "ot": FP32, "out": E + (1 << 40)}, OK),                             # 2^30 bytes of a tile
    ({"m": 65, "os_": 1 << 22, "ot": FP32, "out": E + (1 << 40)}, INVALID),
    ({"m": 300, "os_": 1 << 20, "ot": FP32, "out": E + (1 << 40)}, OK),
    ({"m": 300, "os_": (1 << 20) + 1, "ot": FP32, "out": E + (1 << 40)}, INVALID),
    ({"sa": B + 2}, MISALIGNED),
    ({"out": E + 1}, MISALIGNED),
    ({"out": A}, OVERLAP),
    ({"out": D}, OVERLAP),
    ({"m": 100, "n": 64, "k": 16384, "a_s": 16384, "bs": 16384, "os_": 64}, OK),      # a split sum
    ({"m": 100, "n": 64, "k": 16384, "a_s": 16384, "bs": 16384, "os_": 64, "ws": 0}, INVALID),
    ({"m": 100, "n": 64, "k": 16384, "a_s": 16384, "bs": 16384, "os_": 64, "ws_bytes": 8}, INVALID),
    ({"m": 100, "n": 64, "k": 16384, "a_s": 16384, "bs": 16384, "os_": 64, "ws": E}, OVERLAP),
])
def test_matmul_refusals(change, status):
    assert matmul(**change) == status


def test_matmul_tile_shapes():
    """The products that the GPU tests take for each shape of tile have it."""
    for (m, n, k), narrow, wide in forms.TILE_SHAPES:
        for ot in (BF16, FP16, FP32):
            plan = tilepipe._CPlan()
            need = lib().tp_block_matmul_workspace_bytes(m, n, k, ot)
            st = lib().tp_plan_block_matmul(1 << 44, k, E4M3, 1 << 45, 1 << 46, k, E4M3, 1 << 47, 0, m, n, k,
                                            1 << 48, n, ot, 1 << 49, need, ctypes.byref(plan))
            assert st == OK and (plan.threads // 64, plan.tile_units) == (narrow if ot == BF16 else wide)


def matmul_plan(m, n, k, ot, square=0):
    plan = tilepipe._CPlan()
    need = lib().tp_block_matmul_workspace_bytes(m, n, k, ot)
    st = lib().tp_plan_block_matmul(1 << 44, k, E4M3, 1 << 45, 1 << 46, k, E4M3, 1 << 47, square, m, n, k, 1 << 48, n, ot,
                                    1 << 49, need, ctypes.byref(plan))
    assert st == OK
    return plan, max(1, need // (m * n * 4))


def test_matmul_plans_say_what_is_launched():
    """Stages, LDS and workgroups of each shape: the stages' blocks of 128 bytes,
    two sets of 16 bytes of scales a row, and 1 KiB; rounded up to the 8 XCDs."""
    side = {64: (64, 3), 128: (128, 2), 256: (256, 2)}
    for (m, n, k), _, _ in forms.TILE_SHAPES:
        for ot in (BF16, FP16, FP32):
            plan, splits = matmul_plan(m, n, k, ot)
            wide, stages = (256, 3) if plan.threads == 512 and plan.tile_units == 128 else side[plan.tile_units]
            assert plan.stages == stages
            assert plan.lds_bytes == (plan.tile_units + wide) * (stages * 128 + 32) + 1024 <= 160 * 1024
            assert plan.num_tiles == -(-m // plan.tile_units) * -(-n // wide)
            assert plan.grid == -(-plan.num_tiles * splits // 8) * 8
    for (m, n, k), slots in forms.FEW_ROWS:
        for ot in (BF16, FP16, FP32):
            plan, splits = matmul_plan(m, n, k, ot)
            assert (plan.threads, plan.stages, plan.tile_units) == (512, slots, -(-m // 16) * 16)
            assert plan.lds_bytes == 8 * (plan.tile_units + 16) * (slots * 128 + 32) <= 160 * 1024
            assert plan.grid == plan.num_tiles * splits == -(-n // 16) * splits
    plan = tilepipe._CPlan()
    assert lib().tp_plan_block_quantize(A, 300, 200, 300, BF16, 0, E5M2, B, 304, C, D, 208, E, ctypes.byref(plan)) == OK
    assert 128 * 128 < plan.lds_bytes <= 40 * 1024 and (plan.threads, plan.grid) == (256, 6)


def test_workspace_sizes():
    ws = lib().tp_block_matmul_workspace_bytes
    assert ws(1, 1, 1, BF16) == 0 and ws(0, 5, 5, BF16) == 0
    assert ws(-1, 1, 1, BF16) == -1 and ws(1, 1, 1, E4M3) == -1
    # whole products of each split, and the count of splits within the sum's blocks
    for m, n, k in ((100, 64, 16384), (2000, 1544, 10007), (70, 70, 600), (17, 16, 40000)):
        for ot in (BF16, FP32):
            need = ws(m, n, k, ot)
            assert need % (m * n * 4) == 0
            splits = need // (m * n * 4)
            assert splits == 0 or 2 <= splits <= -(-k // 128)
    gs = lib().tp_rms_norm_backward_workspace_bytes
    assert gs(0, 5, BF16) == 0 and gs(5, 0, BF16) == 0 and gs(5, 5, E5M2) == -1
    assert gs(1000, 512, FP32) % (512 * 4) == 0
    # the join's 32-bit offsets reach all of it
    for cols in (1 << 22, (1 << 23) + 8, (1 << 24) - 1, 1 << 24):
        for dtype in (BF16, FP32):
            assert cols * 4 <= gs(10000, cols, dtype) < 1 << 31


def test_build_without_torch_keeps_the_library(monkeypatch, tmp_path, capsys):
    """The direct binding needs torch's headers; the library does not."""
    from software_pipelining_amd import build
    old = tmp_path / "_linear8.so"
    old.write_bytes(b"of an older build")
    monkeypatch.setattr(build, "BINDING", str(old))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libtilepipe.so"))
    monkeypatch.setattr(build, "_compile", lambda unit, save_temps: str(unit))
    ran = []
    monkeypatch.setattr(build, "_run", lambda cmd: ran.append(cmd) or open(cmd[cmd.index("-o") + 1], "wb").close())
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setitem(sys.modules, "torch.utils", None)
    assert build.build(jobs=2, verbose=False) == str(tmp_path / "libtilepipe.so")
    assert os.path.exists(build.LIB) and len(ran) == 1
    assert not old.exists() and "without the direct binding" in capsys.readouterr().err


def test_star_import_without_torch():
    """The planning calls need no torch, and a star import of them neither."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from software_pipelining_amd import *\n"
            "assert plan_row_shift(0x1000, 0x2000, 4).threads and 'rms_norm' not in globals()\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(tp.__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)
    scope = {}
    exec("from software_pipelining_amd import *", scope)
    assert scope["rms_norm"] is tp.rms_norm and scope["RmsNorm"] is tp.RmsNorm


def test_binding_refusals_without_a_gpu():
    x = torch.zeros(4, 8)
    w = torch.zeros(8)
    with pytest.raises(TypeError, match="torch.Tensor"):
        tp.rms_norm([1.0], w)
    with pytest.raises(TypeError, match="dtype"):
        tp.rms_norm(x.double(), w)
    with pytest.raises(ValueError, match="GPU tensor"):
        tp.rms_norm(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        tp.rms_norm_backward(x, x, w, torch.zeros(4))
    with pytest.raises(ValueError, match="GPU tensor"):
        tp.block_quantize(x)
    with pytest.raises(TypeError, match="dtype"):
        tp.block_matmul(x, w, x, w)
    with pytest.raises(AttributeError):
        tp.no_such_operator
