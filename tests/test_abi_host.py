"""Host-side tests of the C ABI: the library loads, exports every entry point
the header declares, sizes its workspace as documented and rejects bad
arguments before queuing any work.  No call here reaches the GPU: every call
with device pointers carries one argument the host checks refuse."""
from __future__ import annotations

import os
import re

import pytest

import flash_mixed_chunk_gb300 as fm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "flash_mca.h")


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(flash_mca_\w+)\s*\(", text)))


def test_header_declares_the_documented_entry_points():
    names = declared_functions()
    for must in ("flash_mca_forward", "flash_mca_workspace_bytes", "flash_mca_status_string",
                 "flash_mca_forward_host", "flash_mca_host_arena_bytes"):
        assert must in names


def test_library_exports_every_declared_symbol():
    names = declared_functions()
    for name in names:
        assert hasattr(fm.lib, name), f"{name} declared in the header but not exported"
    assert sorted(fm.EXPORTED_SYMBOLS) == names, "binding and header disagree"


def test_library_is_in_tree_and_not_the_oracle():
    assert os.path.dirname(fm.library_path) == os.path.join(ROOT, "flash_mixed_chunk_gb300")
    # the product binding never imports the oracle
    src = open(os.path.join(ROOT, "flash_mixed_chunk_gb300", "__init__.py")).read()
    assert "oracle" not in src.replace("no CPU fallback", "")


def test_status_strings():
    for code in range(8):
        sname = fm.flash_mca_status_string(code)
        assert sname.startswith("FMCA_")
    assert "unknown" in fm.flash_mca_status_string(99)
    assert fm.flash_mca_version() == "0.1.0"


def walk_segments(B, n, e, C):
    """Segments of the chunk axis the tensor-core path's chunk walkers use:
    about 144 (sequence, 256 e columns, segment) units, every segment
    non-empty (the last slice of e may be narrower)."""
    G = n // C
    slices = B * (-(-e // 256))
    S = max(1, min(G, 144 // slices)) if slices else 1
    L = -(-G // S)
    return -(-G // L)


@pytest.mark.parametrize("B,n,s,e,C,causal", [(2, 8192, 128, 1536, 256, 1),
                                              (4, 4096, 128, 1536, 256, 0),
                                              (1, 256, 32, 64, 64, 1),
                                              (3, 96, 48, 80, 32, 0)])
def test_workspace_bytes_formula(B, n, s, e, C, causal):
    """Enough for either path: fp32 states and prefix (SIMT) or, on the tensor
    cores, the bf16 local sums of each chunk's segment (causal), the segment
    totals/carries, the work counters and the bf16 rows T0, T1, T2; no
    per-chunk states and no [B*n][C] buffer of relu^2 weights."""
    a = lambda x: (x + 255) // 256 * 256
    G = n // C
    Gp = G if causal else 1
    simt = a(4 * B * G * s * e) + a(4 * B * Gp * s * e)
    tc = (a(2 * B * G * s * e) * causal + a(2 * B * walk_segments(B, n, e, C) * s * e) + 256
          + a(3 * 2 * B * n * s))  # + the bf16 rows T0, T1, T2
    for dt in (fm.FMCA_F32, fm.FMCA_BF16):
        assert fm.flash_mca_workspace_bytes(B, n, s, e, C, causal, dt) == max(simt, tc)


def test_workspace_bytes_zero_for_rejected_shapes():
    assert fm.flash_mca_workspace_bytes(1, 100, 32, 64, 30, 1, fm.FMCA_F32) == 0   # C !| n
    assert fm.flash_mca_workspace_bytes(1, 64, 32, 64, 128, 1, fm.FMCA_F32) == 0   # C > n
    assert fm.flash_mca_workspace_bytes(0, 64, 32, 64, 64, 1, fm.FMCA_F32) == 0
    assert fm.flash_mca_workspace_bytes(1, 64, 512, 64, 64, 1, fm.FMCA_F32) == 0   # s > 256
    assert fm.flash_mca_workspace_bytes(1, 64, 32, 64, 64, 1, 7) == 0              # bad dtype


def test_auto_path_choice():
    bf, f32 = fm.FMCA_BF16, fm.FMCA_F32
    assert fm.flash_mca_auto_path(2, 8192, 128, 1536, 256, 1, bf) == fm.FMCA_PATH_TCGEN05
    assert fm.flash_mca_auto_path(1, 32768, 128, 2048, 256, 1, bf) == fm.FMCA_PATH_TCGEN05
    assert fm.flash_mca_auto_path(1, 256, 128, 256, 128, 0, bf) == fm.FMCA_PATH_TCGEN05
    assert fm.flash_mca_auto_path(2, 8192, 128, 1536, 256, 1, f32) == fm.FMCA_PATH_SIMT
    assert fm.flash_mca_auto_path(1, 256, 32, 64, 64, 1, f32) == fm.FMCA_PATH_SIMT
    assert fm.flash_mca_auto_path(1, 512, 64, 256, 256, 1, bf) == fm.FMCA_PATH_SIMT   # s != 128
    assert fm.flash_mca_auto_path(1, 512, 128, 200, 256, 1, bf) == fm.FMCA_PATH_SIMT  # e % 64
    # e a multiple of 64 but not of 256: the forward pass's own forms take it
    assert fm.flash_mca_auto_path(1, 512, 128, 640, 256, 1, bf) == fm.FMCA_PATH_TCGEN05
    assert fm.flash_mca_auto_path(1, 512, 128, 320, 256, 1, bf) == fm.FMCA_PATH_TCGEN05
    assert fm.flash_mca_auto_path(1, 512, 128, 256, 64, 1, bf) == fm.FMCA_PATH_SIMT   # C = 64
    assert fm.flash_mca_auto_path(1, 500, 128, 256, 64, 1, bf) == -1


def test_launch_counts():
    bf = fm.FMCA_BF16
    # chunks of 256: the segment walkers (local sums, totals, T rows), then
    # the row-pair kernel, which forms the segment carries (or, bidirectional,
    # the total) itself
    assert fm.flash_mca_launch_count(2, 8192, 128, 1536, 256, 1, bf) == 2
    assert fm.flash_mca_launch_count(4, 4096, 128, 1536, 256, 0, bf) == 2
    # chunks of 128, bidirectional: walkers, the total, the fused chunk kernel
    assert fm.flash_mca_launch_count(4, 4096, 128, 1536, 128, 0, bf) == 3
    # one segment per sequence (B * e / 256 >= 144 units): no carries
    assert fm.flash_mca_launch_count(16, 1024, 128, 2560, 256, 1, bf) == 2
    # without a global term: the T0 / T1 rows and the fused chunk kernel
    assert fm.flash_mca_launch_count(8, 1024, 128, 1536, 1024, 1, bf,
                                     lin_norm=fm.FMCA_LIN_NORM_NONE) == 2
    assert fm.flash_mca_launch_count(8, 1024, 128, 1536, 1024, 1, bf, fm.FMCA_PATH_SIMT,
                                     lin_norm=fm.FMCA_LIN_NORM_NONE) == 3
    assert fm.flash_mca_launch_count(2, 8192, 128, 1536, 256, 1, bf,
                                     lin_norm=fm.FMCA_LIN_NORM_POSITION) == 2
    assert fm.flash_mca_launch_count(2, 8192, 128, 1536, 256, 1, bf, fm.FMCA_PATH_SIMT) == 3
    assert fm.flash_mca_launch_count(1, 512, 64, 256, 256, 1, bf, fm.FMCA_PATH_TCGEN05) == 0
    # e % 256 != 0: every form but the stored-weights one (no global term,
    # chunks over 256 tokens), which goes to the CUDA cores
    assert fm.flash_mca_launch_count(2, 2048, 128, 640, 256, 1, bf) == 2
    assert fm.flash_mca_launch_count(2, 2048, 128, 640, 512, 1, bf, fm.FMCA_PATH_TCGEN05,
                                     lin_norm=fm.FMCA_LIN_NORM_NONE) == 0
    assert fm.flash_mca_launch_count(2, 2048, 128, 640, 512, 1, bf,
                                     lin_norm=fm.FMCA_LIN_NORM_NONE) == 3
    assert fm.flash_mca_launch_count(2, 2048, 128, 768, 512, 1, bf,
                                     lin_norm=fm.FMCA_LIN_NORM_NONE) == 2
    assert fm.flash_mca_launch_count(1, 500, 128, 256, 64, 1, bf) == 0


# A fake device address: aligned, never dereferenced (each call below fails a
# host check first).
P = 0x7F0000000000
BIG = 1 << 40


def fwd(**kw):
    args = dict(Z=P, V=P + 0x10000000, U=P + 0x20000000, g=P + 0x30000000, b=P + 0x30001000,
                O=P + 0x40000000, B=1, n=256, s=32, e=64, C=64, causal=1, dt=fm.FMCA_F32,
                ws=P + 0x50000000, wsb=BIG, path=fm.FMCA_PATH_AUTO)
    args.update(kw)
    return fm.lib.flash_mca_forward_path(args["Z"], args["V"], args["U"], args["g"], args["b"],
                                         args["O"], args["B"], args["n"], args["s"], args["e"],
                                         args["C"], args["causal"], args["dt"], args["ws"],
                                         args["wsb"], args["path"], None)


def test_validation_codes():
    assert fwd(C=60) == fm.FMCA_ERR_SHAPE
    assert fwd(C=512) == fm.FMCA_ERR_SHAPE
    assert fwd(B=0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(e=-1) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(dt=5) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(path=9) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(Z=0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(O=0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(g=0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(s=300) == fm.FMCA_ERR_UNSUPPORTED
    assert fwd(V=P + 0x10000008) == fm.FMCA_ERR_ALIGN
    assert fwd(O=P + 0x40000004) == fm.FMCA_ERR_ALIGN
    assert fwd(ws=0) == fm.FMCA_ERR_WORKSPACE
    assert fwd(ws=P + 0x50000010) == fm.FMCA_ERR_ALIGN
    assert fwd(wsb=100) == fm.FMCA_ERR_WORKSPACE
    # O overlapping an input or the workspace
    assert fwd(O=P + 0x10000000) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(O=P + 0x50000000) == fm.FMCA_ERR_INVALID_ARG
    # explicit tensor-core path on a shape it does not cover: no fallback
    assert fwd(path=fm.FMCA_PATH_TCGEN05) == fm.FMCA_ERR_UNSUPPORTED
    assert fwd(dt=fm.FMCA_BF16, s=64, e=256, n=512, C=256,
               path=fm.FMCA_PATH_TCGEN05) == fm.FMCA_ERR_UNSUPPORTED


def test_host_entry_validation():
    f = fm.lib.flash_mca_forward_host
    good = dict(B=1, n=256, s=32, e=64, C=64, causal=1, dt=fm.FMCA_F32)
    need = fm.flash_mca_host_arena_bytes(1, 256, 32, 64, 64, 1, fm.FMCA_F32)
    assert need > fm.flash_mca_workspace_bytes(1, 256, 32, 64, 64, 1, fm.FMCA_F32)
    h = P  # host pointers are never touched either
    assert f(h, h, h, h, h, h, 1, 256, 32, 64, 60, 1, fm.FMCA_F32, P, need, None) == fm.FMCA_ERR_SHAPE
    assert f(0, h, h, h, h, h, 1, 256, 32, 64, 64, 1, fm.FMCA_F32, P, need, None) == fm.FMCA_ERR_INVALID_ARG
    assert f(h, h, h, h, h, h, 1, 256, 32, 64, 64, 1, fm.FMCA_F32, 0, need, None) == fm.FMCA_ERR_WORKSPACE
    assert f(h, h, h, h, h, h, 1, 256, 32, 64, 64, 1, fm.FMCA_F32, P, need - 1, None) == fm.FMCA_ERR_WORKSPACE
    assert f(h, h, h, h, h, h, 1, 256, 32, 64, 64, 1, fm.FMCA_F32, P + 16, need, None) == fm.FMCA_ERR_ALIGN


def test_selftest_rejects_bad_limits():
    assert fm.lib.flash_mca_selftest_timeout(0, None) == fm.FMCA_ERR_INVALID_ARG
    assert fm.lib.flash_mca_selftest_timeout(20_000_000, None) == fm.FMCA_ERR_INVALID_ARG


def test_python_binding_rejects_bad_tensors():
    import torch
    Z = torch.zeros(1, 256, 32)
    V = torch.zeros(1, 256, 64)
    with pytest.raises(ValueError):
        fm.flash_mca_forward(Z, V, V, torch.zeros(4, 32), torch.zeros(4, 32), V, 64, True, Z)
    with pytest.raises(ValueError):
        fm.forward(Z[0], V, V, torch.zeros(4, 32), torch.zeros(4, 32), 64, True)


def fwd_ex(opts, **kw):
    args = dict(Z=P, V=P + 0x10000000, U=P + 0x20000000, g=P + 0x30000000, b=P + 0x30001000,
                O=P + 0x40000000, B=1, n=256, s=32, e=64, C=64, causal=1, dt=fm.FMCA_F32,
                ws=P + 0x50000000, wsb=BIG, path=fm.FMCA_PATH_AUTO)
    args.update(kw)
    return fm.lib.flash_mca_forward_ex(args["Z"], args["V"], args["U"], args["g"], args["b"],
                                       args["O"], args["B"], args["n"], args["s"], args["e"],
                                       args["C"], args["causal"], args["dt"], args["ws"],
                                       args["wsb"], args["path"], opts, None)


def test_default_options():
    import ctypes
    o = fm.FmcaOptions()
    assert fm.lib.flash_mca_default_options(256, ctypes.byref(o)) == fm.FMCA_OK
    assert o.quad_scale == 1.0 / 65536.0 and o.lin_norm == fm.FMCA_LIN_NORM_N
    assert fm.lib.flash_mca_default_options(0, ctypes.byref(o)) == fm.FMCA_ERR_INVALID_ARG
    assert fm.lib.flash_mca_default_options(64, None) == fm.FMCA_ERR_INVALID_ARG


def test_options_validation_codes():
    import ctypes
    for q, ln in ((-1.0, 0), (float("nan"), 0), (float("inf"), 0), (0.5, 4), (0.5, -1)):
        o = fm.FmcaOptions(q, ln)
        assert fwd_ex(ctypes.byref(o)) == fm.FMCA_ERR_INVALID_ARG, (q, ln)
    # valid options still go through the other host checks first
    o = fm.FmcaOptions(0.25, fm.FMCA_LIN_NORM_POSITION)
    assert fwd_ex(ctypes.byref(o), C=60) == fm.FMCA_ERR_SHAPE
    assert fwd_ex(ctypes.byref(o), ws=0) == fm.FMCA_ERR_WORKSPACE
    assert fwd_ex(None, V=P + 0x10000008) == fm.FMCA_ERR_ALIGN


def test_decode_state_bytes_and_validation():
    import ctypes
    nb = fm.flash_mca_decode_state_bytes(2, 32, 64, 16, fm.FMCA_F32)
    a = lambda x: (x + 255) // 256 * 256
    assert nb == a(4 * 2 * 32 * 64) + a(4 * 2 * 16 * 32) + a(4 * 2 * 16 * 64)
    # bf16: the fp32 sum, its bf16 copy, and the bf16 chunk cache
    assert fm.flash_mca_decode_state_bytes(2, 32, 64, 16, fm.FMCA_BF16) == \
        a(4 * 2 * 32 * 64) + a(2 * 2 * 32 * 64) + a(2 * 2 * 16 * 32) + a(2 * 2 * 16 * 64)
    for bad in ((0, 32, 64, 16), (2, 300, 64, 16), (2, 32, 64, 2048), (2, 32, 0, 16)):
        assert fm.flash_mca_decode_state_bytes(*bad, fm.FMCA_F32) == 0
    step = fm.lib.flash_mca_decode_step
    base = dict(z=P, v=P + 0x1000, u=P + 0x2000, g=P + 0x3000, b=P + 0x4000, o=P + 0x5000,
                B=2, s=32, e=64, C=16, t=5, n=64, dt=fm.FMCA_F32, opts=None,
                st=P + 0x100000, stb=nb)

    def call(**kw):
        d = dict(base)
        d.update(kw)
        return step(d["z"], d["v"], d["u"], d["g"], d["b"], d["o"], d["B"], d["s"], d["e"], d["C"],
                    d["t"], d["n"], d["dt"], d["opts"], d["st"], d["stb"], None)
    assert call(t=-1) == fm.FMCA_ERR_INVALID_ARG
    assert call(n=5) == fm.FMCA_ERR_INVALID_ARG          # n_norm must exceed t
    assert call(C=4096) == fm.FMCA_ERR_INVALID_ARG
    assert call(z=0) == fm.FMCA_ERR_INVALID_ARG
    assert call(v=P + 0x1004) == fm.FMCA_ERR_ALIGN
    assert call(stb=nb - 1) == fm.FMCA_ERR_WORKSPACE
    assert call(st=0) == fm.FMCA_ERR_WORKSPACE
    assert call(st=P + 0x100010) == fm.FMCA_ERR_ALIGN
    assert call(o=P + 0x1000) == fm.FMCA_ERR_INVALID_ARG    # o overlaps v
    o = fm.FmcaOptions(0.1, 7)
    assert call(opts=ctypes.byref(o)) == fm.FMCA_ERR_INVALID_ARG
    # the per-position and tokens-summed divisors do not need n_norm
    o = fm.FmcaOptions(0.1, fm.FMCA_LIN_NORM_SUMMED)
    assert call(opts=ctypes.byref(o), n=0, stb=0) == fm.FMCA_ERR_WORKSPACE
    reset = fm.lib.flash_mca_decode_reset
    assert reset(P + 0x100000, nb - 1, 2, 32, 64, 16, fm.FMCA_F32, None) == fm.FMCA_ERR_WORKSPACE
    assert reset(P + 0x100010, nb, 2, 32, 64, 16, fm.FMCA_F32, None) == fm.FMCA_ERR_ALIGN
    assert reset(P + 0x100000, nb, 0, 32, 64, 16, fm.FMCA_F32, None) == fm.FMCA_ERR_INVALID_ARG


def test_backward_workspace_and_validation():
    nb = fm.flash_mca_backward_workspace_bytes(2, 64, 16, 32, 16, 1, fm.FMCA_F32)
    a = lambda x: (x + 255) // 256 * 256
    G, rows = 4, 128
    want = (a(4 * 2 * G * 16 * 32) * 3 + a(4 * rows * 32) + 2 * a(4 * 2 * G * 16 * 16) +
            a(4 * 4 * rows * 16) + a(4 * 8 * 16 * 2))
    assert nb == want
    assert fm.flash_mca_backward_workspace_bytes(2, 64, 16, 32, 60, 1, fm.FMCA_F32) == 0
    f = fm.lib.flash_mca_backward
    base = dict(Z=P, V=P + 0x10000, U=P + 0x20000, g=P + 0x30000, b=P + 0x31000, dO=P + 0x40000,
                dZ=P + 0x50000, dV=P + 0x60000, dU=P + 0x70000, dg=P + 0x80000, db=P + 0x81000,
                B=2, n=64, s=16, e=32, C=16, causal=1, dt=fm.FMCA_F32, opts=None,
                ws=P + 0x100000, wsb=nb)

    def call(**kw):
        d = dict(base)
        d.update(kw)
        return f(d["Z"], d["V"], d["U"], d["g"], d["b"], d["dO"], d["dZ"], d["dV"], d["dU"],
                 d["dg"], d["db"], d["B"], d["n"], d["s"], d["e"], d["C"], d["causal"], d["dt"],
                 d["opts"], d["ws"], d["wsb"], None)
    assert call(C=60) == fm.FMCA_ERR_SHAPE
    assert call(dO=0) == fm.FMCA_ERR_INVALID_ARG
    assert call(dg=0) == fm.FMCA_ERR_INVALID_ARG
    assert call(dV=P + 0x60004) == fm.FMCA_ERR_ALIGN
    assert call(ws=0) == fm.FMCA_ERR_WORKSPACE
    assert call(wsb=nb - 1) == fm.FMCA_ERR_WORKSPACE
    assert call(ws=P + 0x100010) == fm.FMCA_ERR_ALIGN
    assert call(dZ=P + 0x10000) == fm.FMCA_ERR_INVALID_ARG   # dZ overlaps V
    assert call(dU=P + 0x60000) == fm.FMCA_ERR_INVALID_ARG   # dU overlaps dV
    import ctypes
    o = fm.FmcaOptions(0.1, 9)
    assert call(opts=ctypes.byref(o)) == fm.FMCA_ERR_INVALID_ARG


def test_gau_projection_validation():
    f = fm.lib.flash_mca_gau_project
    X, W, U, V, Z = P, P + 0x100000, P + 0x200000, P + 0x300000, P + 0x400000
    assert f(0, W, U, V, Z, 128, 64, 64, 64, None) == fm.FMCA_ERR_INVALID_ARG
    assert f(X, W, U, V, Z, 0, 64, 64, 64, None) == fm.FMCA_ERR_INVALID_ARG
    assert f(X, W, U, V, Z, 128, 60, 64, 64, None) == fm.FMCA_ERR_UNSUPPORTED   # d % 8
    assert f(X, W, U, V, Z, 128, 64, 96, 64, None) == fm.FMCA_ERR_UNSUPPORTED   # e % 64
    assert f(X, W, U, V, Z, 128, 64, 64, 32, None) == fm.FMCA_ERR_UNSUPPORTED   # s % 64
    assert f(X + 8, W, U, V, Z, 128, 64, 64, 64, None) == fm.FMCA_ERR_ALIGN
    assert f(X, W, X, V, Z, 128, 64, 64, 64, None) == fm.FMCA_ERR_INVALID_ARG   # U overlaps X
    assert f(X, W, U, U, Z, 128, 64, 64, 64, None) == fm.FMCA_ERR_INVALID_ARG   # V overlaps U
    g = fm.lib.flash_mca_gau_output
    assert g(X, W, U, 128, 64, 96, None) == fm.FMCA_ERR_UNSUPPORTED             # d % 64
    assert g(X, W, X, 128, 64, 64, None) == fm.FMCA_ERR_INVALID_ARG             # Out overlaps Y
    assert g(X, W, U + 4, 128, 64, 64, None) == fm.FMCA_ERR_ALIGN


def test_backward_saved_validation():
    # the saved mode exists for the tensor-core shapes only: fp32, or bf16 with
    # s != 128, is refused before any pointer is looked at
    f = fm.lib.flash_mca_backward_saved

    def call(B, n, s, e, C, dt):
        return f(P, P, P, P, P, P, P, P, P, P, P, B, n, s, e, C, 1, dt, None, P, 1 << 30, None)
    assert call(2, 64, 16, 32, 16, fm.FMCA_F32) == fm.FMCA_ERR_UNSUPPORTED
    assert call(1, 512, 64, 256, 256, fm.FMCA_BF16) == fm.FMCA_ERR_UNSUPPORTED
    assert call(1, 512, 128, 200, 256, fm.FMCA_BF16) == fm.FMCA_ERR_UNSUPPORTED
    assert call(2, 64, 16, 32, 60, fm.FMCA_F32) == fm.FMCA_ERR_SHAPE   # C does not divide n


def test_backward_launch_count():
    bf, f32 = fm.FMCA_BF16, fm.FMCA_F32
    cnt = fm.flash_mca_backward_launch_count
    # tensor cores: forward kernels (chunk walkers, segment carries, scaled
    # prefix, relu^2 weights, output kernel: 5; 3 when the forward pass's local
    # sums and carries are kept; 2 without a global term), 2 elementwise, 3
    # product launches, the reverse scan (global term only), 2 for dZ /
    # dgamma / dbeta
    assert cnt(2, 1024, 128, 512, 256, True, bf) == 13
    assert cnt(2, 1024, 128, 512, 256, True, bf, saved=True) == 11
    assert cnt(2, 1024, 128, 512, 256, True, bf, lin_norm=fm.FMCA_LIN_NORM_NONE) == 9
    # CUDA cores
    assert cnt(2, 1024, 128, 512, 256, True, f32) == 12
    assert cnt(2, 1024, 128, 512, 256, True, f32, lin_norm=fm.FMCA_LIN_NORM_NONE) == 7
    assert cnt(2, 1024, 128, 512, 256, True, f32, saved=True) == 0
    assert cnt(2, 1024, 128, 512, 60, True, bf) == 0        # C does not divide n


def test_forward_seq_rejects_before_queueing():
    """flash_mca_forward_seq checks its arguments on the host before anything is
    queued: bidirectional attention and the no-global-term variant are not
    covered, the piece must start on a chunk boundary, state pointers must be
    16-byte aligned and state_out must not overlap the other buffers.  The
    pointers here are never dereferenced."""
    import ctypes
    B, n, s, e, C = 1, 512, 128, 256, 256
    P = 0x7F0000000000
    z, v, u, g, b, o = P, P + (1 << 24), P + (2 << 24), P + (3 << 24), P + (3 << 24) + 4096, P + (4 << 24)
    ws = P + (8 << 24)
    nb = fm.flash_mca_workspace_bytes(B, n, s, e, C, 1, fm.FMCA_BF16)
    opts = fm.flash_mca_default_options(C)
    state = P + (16 << 24)

    def call(causal, offset, lin_norm=fm.FMCA_LIN_NORM_N, s_in=state, s_out=state, dt=fm.FMCA_BF16):
        opts.lin_norm = lin_norm
        seq = fm.FmcaSeq(s_in, s_out, offset, 0)
        return fm.lib.flash_mca_forward_seq(z, v, u, g, b, o, B, n, s, e, C, causal, dt, ws, nb,
                                            ctypes.byref(opts), ctypes.byref(seq), None)
    assert call(0, 0) == fm.FMCA_ERR_UNSUPPORTED                      # bidirectional
    assert call(1, 0, lin_norm=fm.FMCA_LIN_NORM_NONE) == fm.FMCA_ERR_UNSUPPORTED
    assert call(1, 0, dt=fm.FMCA_F32) != fm.FMCA_OK                   # not the tensor-core path
    assert call(1, 128) == fm.FMCA_ERR_INVALID_ARG                    # off a chunk boundary
    assert call(1, -256) == fm.FMCA_ERR_INVALID_ARG
    assert call(1, 0, s_in=state + 4) == fm.FMCA_ERR_ALIGN
    assert call(1, 0, s_out=o) == fm.FMCA_ERR_INVALID_ARG             # state_out overlaps O


def test_layer_norm_rejects_before_queueing():
    """flash_mca_layer_norm and its backward pass: argument checks on the host.
    The pointers here are never dereferenced."""
    P = 0x7F0000000000
    x, r, w, b, h, y, mn, rs = [P + (k << 24) for k in range(8)]
    bf = fm.FMCA_BF16

    def fwd(x=x, r=r, w=w, b=b, h=h, y=y, mn=mn, rs=rs, M=0, d=64, eps=1e-5, dt=bf):
        return fm.lib.flash_mca_layer_norm(x, r, w, b, h, y, mn, rs, M, d, eps, dt, None)
    assert fwd() == fm.FMCA_ERR_INVALID_ARG                      # no rows
    assert fwd(M=4, d=0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(M=4, d=8193) == fm.FMCA_ERR_UNSUPPORTED
    assert fwd(M=4, dt=2) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(M=4, eps=-1.0) == fm.FMCA_ERR_INVALID_ARG
    assert fwd(M=4, eps=float("nan")) == fm.FMCA_ERR_INVALID_ARG
    for k in ("x", "w", "b", "y", "h"):                          # h: needed with a residual
        assert fwd(M=4, **{k: None}) == fm.FMCA_ERR_INVALID_ARG
    for k, v in (("x", x), ("r", r), ("w", w), ("b", b), ("h", h), ("y", y)):
        assert fwd(M=4, **{k: v + 8}) == fm.FMCA_ERR_ALIGN
    assert fwd(M=4, mn=mn + 2) == fm.FMCA_ERR_ALIGN and fwd(M=4, rs=rs + 1) == fm.FMCA_ERR_ALIGN
    for k, v in (("y", x), ("y", r), ("y", h), ("h", x + 128), ("h", r - 128), ("h", w), ("mn", rs),
                 ("rs", y)):
        assert fwd(M=4, **{k: v}) == fm.FMCA_ERR_INVALID_ARG     # overlaps

    nb = fm.flash_mca_layer_norm_backward_workspace_bytes
    # one partial row of dw and db a block: at least 8 rows a block up to d =
    # 256, 2 up to 1024, one beyond; 304 blocks at most (456 up to d = 256 and
    # from 1025 to 2048)
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    assert nb(1, 768) == up(8 * 768) and nb(17, 768) == up(9 * 8 * 768)
    assert nb(17, 256) == up(3 * 8 * 256)
    assert nb(100000, 768) == up(304 * 8 * 768) and nb(5, 1025) == up(5 * 8 * 1025)
    assert nb(100000, 256) == up(456 * 8 * 256) and nb(100000, 2048) == up(456 * 8 * 2048)
    assert nb(100000, 257) == up(304 * 8 * 257) and nb(100000, 2049) == up(304 * 8 * 2049)
    assert nb(0, 768) == 0 and nb(4, 0) == 0 and nb(4, 8193) == 0

    dy, hh, dh, dx, dw, db, ws = [P + (k << 24) for k in range(8, 15)]

    def bwd(dy=dy, hh=hh, w=w, mn=mn, rs=rs, dh=dh, dx=dx, dw=dw, db=db, M=4, d=64, dt=bf, ws=ws,
            size=1 << 20):
        return fm.lib.flash_mca_layer_norm_backward(dy, hh, w, mn, rs, dh, dx, dw, db, M, d, dt, ws,
                                                    size, None)
    assert bwd(M=0) == fm.FMCA_ERR_INVALID_ARG and bwd(d=9000) == fm.FMCA_ERR_UNSUPPORTED
    assert bwd(dt=7) == fm.FMCA_ERR_INVALID_ARG
    for k in ("dy", "hh", "w", "mn", "rs", "dx", "dw", "db"):
        assert bwd(**{k: None}) == fm.FMCA_ERR_INVALID_ARG
    assert bwd(ws=None) == fm.FMCA_ERR_WORKSPACE and bwd(size=100) == fm.FMCA_ERR_WORKSPACE
    assert bwd(ws=ws + 16) == fm.FMCA_ERR_ALIGN and bwd(dh=dh + 4) == fm.FMCA_ERR_ALIGN
    for k, v in (("dx", dy), ("dx", dh), ("dw", db), ("db", ws), ("dx", ws), ("dw", w), ("ws", hh)):
        assert bwd(**{k: v}) == fm.FMCA_ERR_INVALID_ARG


def test_training_wrappers_refuse_host_tensors():
    import torch
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        fm.layer_norm(x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        fm.layer_norm_backward(x, x, w, torch.zeros(2), torch.zeros(2))


def test_projection_gradients_reject_before_queueing():
    """Argument checks of the projections' gradients; no pointer is
    dereferenced."""
    P = 0x7F0000000000
    a = [P + (k << 28) for k in range(8)]
    big = 1 << 40
    nb = fm.flash_mca_gau_project_backward_workspace_bytes
    slots = 2 * 152 * 128 * 256 * 4  # two fp32 tiles a CTA
    # dpre in boxes of 64 x 64, tokens and columns rounded up to 256
    assert nb(1000, 768, 1536, 128) == 1024 * 3328 * 2 + slots
    assert nb(1, 64, 64, 64) == 256 * 256 * 2 + slots
    assert nb(0, 64, 64, 64) == 0 and nb(4, 60, 64, 64) == 0 and nb(4, 64, 32, 64) == 0
    assert nb(4, 64, 64, 96) == 0 and nb(1 << 21, 768, 1536, 128) == 0

    def proj(X=a[0], Wt=a[1], dU=a[2], dV=a[3], dZ=a[4], dX=a[5], dWt=a[6], M=100, d=64, e=64, s=64,
             ws=a[7], size=big):
        return fm.lib.flash_mca_gau_project_backward(X, Wt, dU, dV, dZ, dX, dWt, M, d, e, s, ws,
                                                     size, None)
    for k in ("X", "Wt", "dU", "dV", "dZ", "dX", "dWt"):
        assert proj(**{k: None}) == fm.FMCA_ERR_INVALID_ARG
        assert proj(**{k: a[0] + (99 << 28) + 2}) == fm.FMCA_ERR_ALIGN
    assert proj(M=0) == fm.FMCA_ERR_INVALID_ARG and proj(d=12) == fm.FMCA_ERR_UNSUPPORTED
    assert proj(e=100) == fm.FMCA_ERR_UNSUPPORTED and proj(s=8) == fm.FMCA_ERR_UNSUPPORTED
    assert proj(ws=None) == fm.FMCA_ERR_WORKSPACE and proj(size=1000) == fm.FMCA_ERR_WORKSPACE
    assert proj(ws=a[7] + 128) == fm.FMCA_ERR_ALIGN
    small = nb(100, 64, 64, 64)
    for k, v in (("dX", a[0]), ("dWt", a[1]), ("dX", a[2]), ("dWt", a[5]), ("ws", a[4]), ("dX", a[7])):
        assert proj(**{k: v, "size": small}) == fm.FMCA_ERR_INVALID_ARG

    ob = fm.flash_mca_gau_output_backward_workspace_bytes
    assert ob(100, 64, 64) == slots and ob(0, 64, 64) == 0 and ob(4, 60, 64) == 0
    assert ob(4, 64, 32) == 0

    def outp(Y=a[0], Wo=a[1], dO=a[2], dY=a[3], dW=a[4], M=100, e=64, d=64, ws=a[5], size=slots):
        return fm.lib.flash_mca_gau_output_backward(Y, Wo, dO, dY, dW, M, e, d, ws, size, None)
    for k in ("Y", "Wo", "dO", "dY", "dW"):
        assert outp(**{k: None}) == fm.FMCA_ERR_INVALID_ARG
        assert outp(**{k: a[0] + (99 << 28) + 8}) == fm.FMCA_ERR_ALIGN
    assert outp(M=-1) == fm.FMCA_ERR_INVALID_ARG and outp(e=4) == fm.FMCA_ERR_UNSUPPORTED
    assert outp(d=8) == fm.FMCA_ERR_UNSUPPORTED and outp(size=slots - 1) == fm.FMCA_ERR_WORKSPACE
    for k, v in (("dY", a[0]), ("dW", a[2]), ("dY", a[4]), ("ws", a[1])):
        assert outp(**{k: v}) == fm.FMCA_ERR_INVALID_ARG


def test_vocab_loss_rejects_before_queueing():
    P = 0x7F0000000000
    a = [P + (k << 28) for k in range(10)]
    fb, bb = fm.flash_mca_vocab_loss_workspace_bytes, fm.flash_mca_vocab_loss_backward_workspace_bytes
    for f in (fb, bb):
        assert f(0, 10, 64) == 0 and f(4, 0, 64) == 0 and f(4, 10, 0) == 0 and f(4, 10, 12) == 0
        assert f(1 << 22, 10, 512) == 0 and f(4, 1 << 22, 512) == 0
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    # index, target and logit of a row, X, two fp32 pairs a row and 256 columns (128
    # while the tiles of 128 x 128 are 152 at most)
    assert fb(100, 1000, 64) == 256 + 3 * up(400) + up(100 * 128) + up(100 * 8 * 2 * 8)
    assert fb(100, 19456, 64) == 256 + 3 * up(400) + up(100 * 128) + up(100 * 8 * 2 * 152)
    assert fb(100, 19457, 64) == 256 + 3 * up(400) + up(100 * 128) + up(100 * 8 * 2 * 77)
    # the logits never lie in the workspace: a piece of 256 MiB at most
    assert bb(16384, 250000, 64) < (256 << 20) + (64 << 20)
    assert fb(16384, 250000, 64) < 16384 * 250000 * 2 / 16
    nf, nb = fb(100, 1000, 64), bb(100, 1000, 64)

    def fwd(X=a[0], W=a[1], t=a[2], loss=a[3], lse=a[4], M=100, V=1000, d=64, ws=a[5], size=nf):
        return fm.lib.flash_mca_vocab_loss(X, W, t, loss, lse, M, V, d, ws, size, None)

    def bwd(X=a[0], W=a[1], t=a[2], lse=a[3], g=a[4], dX=a[5], dW=a[6], M=100, V=1000, d=64, ws=a[7],
            size=nb):
        return fm.lib.flash_mca_vocab_loss_backward(X, W, t, lse, g, dX, dW, M, V, d, ws, size, None)
    for f, names in ((fwd, ("X", "W", "t", "loss", "lse")),
                     (bwd, ("X", "W", "t", "lse", "g", "dX", "dW"))):
        for k in names:
            assert f(**{k: None}) == fm.FMCA_ERR_INVALID_ARG
            off = 4 if k == "t" else 2 if k in ("loss", "lse", "g") else 8
            assert f(**{k: P + (99 << 28) + off}) == fm.FMCA_ERR_ALIGN
        assert f(M=0) == fm.FMCA_ERR_INVALID_ARG and f(V=-5) == fm.FMCA_ERR_INVALID_ARG
        assert f(d=60) == fm.FMCA_ERR_UNSUPPORTED and f(M=1 << 26) == fm.FMCA_ERR_UNSUPPORTED
        assert f(ws=None) == fm.FMCA_ERR_WORKSPACE and f(size=255) == fm.FMCA_ERR_WORKSPACE
        assert f(ws=a[9] + 16) == fm.FMCA_ERR_ALIGN
    for k, v in (("loss", a[4]), ("lse", a[2]), ("loss", a[0]), ("ws", a[1]), ("lse", a[5])):
        assert fwd(**{k: v}) == fm.FMCA_ERR_INVALID_ARG
    for k, v in (("dX", a[0]), ("dW", a[1]), ("dW", a[5]), ("dX", a[4]), ("ws", a[3]), ("dX", a[7])):
        assert bwd(**{k: v}) == fm.FMCA_ERR_INVALID_ARG


def test_tensor_core_training_wrappers_refuse_host_tensors():
    import torch
    X, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    t, r = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for call in (lambda: fm.vocab_loss(X, W, t), lambda: fm.vocab_loss_backward(X, W, t, r, r),
                 lambda: fm.gau_project_backward(X, W, X, X, X),
                 lambda: fm.gau_output_backward(X, W, X)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_vocab_loss_refuses_depths_beyond_its_products():
    """A product's depth is one tile's k steps: up to 2^24 they stay well within a
    second (the waits' limit) and their number within 32 bits, which ceil(d / 64)
    left at d = 2^31 - 8."""
    for f in (fm.flash_mca_vocab_loss_workspace_bytes,
              fm.flash_mca_vocab_loss_backward_workspace_bytes):
        assert f(1, 1, 1 << 24) > 0 and f(100, 127, 1 << 24) > 0
        for d in ((1 << 24) + 8, 1 << 28, 2 ** 31 - 64, 2 ** 31 - 8):
            assert f(1, 1, d) == 0
    P = 0x7F0000000000
    a = [P + (k << 36) for k in range(8)]
    for d in ((1 << 24) + 8, 2 ** 31 - 8):
        assert fm.lib.flash_mca_vocab_loss(*a[:5], 1, 1, d, a[5], 0, None) == \
            fm.FMCA_ERR_UNSUPPORTED
        assert fm.lib.flash_mca_vocab_loss_backward(*a[:7], 1, 1, d, a[7], 0, None) == \
            fm.FMCA_ERR_UNSUPPORTED


def test_training_sizes_beyond_32_bits_are_refused():
    """The C ABI takes sizes as int: 2^32 + 4 rows are not 4 rows."""
    import torch
    big = (1 << 32) + 4
    assert fm.flash_mca_layer_norm_backward_workspace_bytes(4, 8) > 0
    assert fm.flash_mca_layer_norm_backward_workspace_bytes(big, 8) == 0
    assert fm.flash_mca_layer_norm_backward_workspace_bytes(4, (1 << 32) + 8) == 0
    assert fm.flash_mca_gau_project_backward_workspace_bytes(big, 64, 64, 64) == 0
    assert fm.flash_mca_gau_project_backward_workspace_bytes(4, 64, 64, (1 << 32) + 64) == 0
    assert fm.flash_mca_gau_output_backward_workspace_bytes(big, 64, 64) == 0
    assert fm.flash_mca_vocab_loss_workspace_bytes(big, 10, 64) == 0
    assert fm.flash_mca_vocab_loss_backward_workspace_bytes(4, (1 << 33) + 10, 64) == 0
    # the calls themselves, on tensors without memory
    bf, f32 = torch.bfloat16, torch.float32
    t = lambda *shape, dtype=bf: torch.empty(*shape, dtype=dtype, device="meta")  # noqa: E731
    dev = t(1).get_device()
    v = t(8, dtype=f32)
    rows = t(big, dtype=f32)
    x, ws = t(big, 8), t(1 << 20, dtype=torch.uint8)
    y = t(big, 64)
    for call in (
            lambda: fm._layer_norm(dev, None, x, None, v, v, None, x, None, None, 1e-5),
            lambda: fm._layer_norm_backward(dev, None, x, x, v, rows, rows, None, x, v, v, ws),
            lambda: fm._gau_project_backward(dev, None, y, t(192, 64), y, y, y, y, t(192, 64), ws),
            lambda: fm._gau_output_backward(dev, None, y, t(64, 64), y, y, t(64, 64), ws),
            lambda: fm._vocab_loss(dev, None, x, t(10, 8), t(big, dtype=torch.int64), rows, rows,
                                   ws),
            lambda: fm._vocab_loss_backward(dev, None, t(4, 8), x, t(4, dtype=torch.int64),
                                            t(4, dtype=f32), t(4, dtype=f32), t(4, 8), x, ws)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
