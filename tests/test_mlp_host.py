"""CPU checks of the MLP operators: the header's entry points are exported, arguments are
refused on the host before anything is enqueued, and the tests' own MXFP8 reference agrees with
nearest-by-enumeration and with torch's E4M3 rounding."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import mlp_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dq_mlp.h")
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x10004)
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def dqlib():
    import dual_scale_w4a4_amd as dq

    if not os.path.exists(dq.LIB_PATH):
        from dual_scale_w4a4_amd import build

        build.build()
    L = dq.lib()  # the package calls these through its compiled binding; here through ctypes
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    norm = [P, I, P, P, I64, I64, P, I, ctypes.c_double, P, I, I, F, P, P]
    L.dq_norm_quantize_act_async.argtypes = [*norm, P, P]
    L.dq_norm_quantize_act.argtypes = [*norm, P, ctypes.c_size_t, P]
    L.dq_gemm_mx_epilogue.argtypes = [P, P, I, I64, I64, P, P, P, P, I, P, I64, I, P, P]
    L.dq_gated_mx.argtypes = [P, P, I, I64, I64, P, P, P, P, P, P, I, I64, I, P, P]
    L.dq_gated_mx_quantized.argtypes = [P, P, I, I64, I64, P, P, P, P, P, P, I, I64, P, I, P, P, P]
    return dq


def test_header_and_exports(dqlib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dq_[a-z0-9_]+)\s*\(", src)))
    assert names == ["dq_gated_mx", "dq_gated_mx_quantized", "dq_gemm_mx_epilogue",
                     "dq_norm_quantize_act", "dq_norm_quantize_act_async"]
    out = subprocess.run(["nm", "-D", "--defined-only", dqlib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if " T " in l}
    assert set(names) <= exported


def test_header_compiles_as_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text(f'#define __HIP_PLATFORM_AMD__ 1\n#include "{HEADER}"\nint main(void) {{ return '
                 "DQ_FMT_MXFP8 != 4 || DQ_ACTIVATION_GELU_TANH != 4; }\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-I/opt/rocm/include", str(c)], check=True)


NORM = dict(X=FAKE, xt=1, R=FAKE, h=FAKE, tokens=4, cols=256, w=FAKE, wt=1, eps=1e-5, b=FAKE,
            fmt=4, group=32, g=0.0, codes=FAKE, scales=FAKE)


@pytest.mark.parametrize("change,want", [
    (dict(X=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG),
    (dict(R=None), ARG), (dict(h=None), ARG),        # residual in without out, and out without in
    (dict(tokens=0), ARG), (dict(cols=0), ARG), (dict(cols=250), ARG), (dict(group=8), ARG),
    (dict(cols=96, group=64), ARG), (dict(tokens=1 << 40), ARG), (dict(cols=1 << 40), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG),
    (dict(fmt=3), ARG), (dict(fmt=3, g=float("nan")), ARG), (dict(fmt=3, g=float("inf")), ARG),
    (dict(X=ODD), ARG), (dict(R=ODD), ARG), (dict(h=ODD), ARG), (dict(w=ODD), ARG),
    (dict(b=ODD), ARG), (dict(codes=ctypes.c_void_p(0x10008)), ARG),
    (dict(fmt=0, scales=ctypes.c_void_p(0x10001)), ARG),
    (dict(h=ctypes.c_void_p(0x10100)), ARG),         # overlaps X and residual
    (dict(fmt=5), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED), (dict(xt=2), UNSUPPORTED),
    (dict(wt=7), UNSUPPORTED),
])
def test_norm_arguments_are_refused(dqlib, change, want):
    a = list(dict(NORM, **change).values())
    L = dqlib.lib()
    assert L.dq_norm_quantize_act_async(*a, FAKE, None) == want
    assert L.dq_norm_quantize_act(*a, None, 0, None) == want


def test_norm_status_and_workspace_are_checked(dqlib):
    a = list(NORM.values())
    L = dqlib.lib()
    assert L.dq_norm_quantize_act_async(*a, None, None) == ARG
    assert L.dq_norm_quantize_act_async(*a, ctypes.c_void_p(0x10002), None) == ARG
    assert L.dq_norm_quantize_act(*a, FAKE, 16, None) == WORKSPACE
    assert L.dq_norm_quantize_act(*a, ctypes.c_void_p(0x10010), 256, None) == ARG


EPI = dict(xc=FAKE, xs=FAKE, fmt=2, tokens=4, K=512, wc=FAKE, ws=FAKE, a=FAKE, bias=FAKE, act=0,
           res=FAKE, out=64, yt=1, y=FAKE)
GATED = dict(xc=FAKE, xs=FAKE, fmt=2, tokens=4, K=512, gc=FAKE, gs=FAKE, ag=FAKE, uc=FAKE, us=FAKE,
             au=FAKE, act=2, inner=64, yt=1, y=FAKE)
GATEDQ = dict(xc=FAKE, xs=FAKE, fmt=2, tokens=4, K=512, gc=FAKE, gs=FAKE, ag=FAKE, uc=FAKE,
              us=FAKE, au=FAKE, act=2, inner=64, b=FAKE, qfmt=4, codes=FAKE, scales=FAKE)
SHARED = [(dict(xc=None), ARG), (dict(xs=None), ARG), (dict(tokens=0), ARG), (dict(K=0), ARG),
          (dict(K=256), ARG), (dict(K=768), ARG), (dict(K=1 << 23), ARG),
          (dict(tokens=1 << 31), ARG), (dict(xc=ODD), ARG), (dict(xs=ODD), ARG),
          (dict(fmt=0), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(fmt=5), UNSUPPORTED),
          (dict(act=5), UNSUPPORTED), (dict(act=-1), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(wc=None), ARG), (dict(ws=None), ARG), (dict(y=None), ARG), (dict(out=0), ARG),
    (dict(out=1 << 31), ARG), (dict(wc=ODD), ARG), (dict(ws=ctypes.c_void_p(0x10002)), ARG),
    (dict(a=ODD), ARG), (dict(bias=ODD), ARG), (dict(y=ctypes.c_void_p(0x10001)), ARG),
    (dict(res=ctypes.c_void_p(0x10001)), ARG),
    (dict(res=ctypes.c_void_p(0x10020)), ARG),       # overlaps Y
    (dict(yt=2), UNSUPPORTED), (dict(yt=0, fmt=4), UNSUPPORTED),  # fp32 from MXFP8
])
def test_epilogue_arguments_are_refused(dqlib, change, want):
    assert dqlib.lib().dq_gemm_mx_epilogue(*dict(EPI, **change).values(), None) == want


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(gc=None), ARG), (dict(us=None), ARG), (dict(y=None), ARG), (dict(inner=0), ARG),
    (dict(uc=ODD), ARG), (dict(us=ctypes.c_void_p(0x10002)), ARG), (dict(ag=ODD), ARG),
    (dict(au=ODD), ARG), (dict(y=ctypes.c_void_p(0x10001)), ARG), (dict(yt=2), UNSUPPORTED),
    (dict(yt=0, fmt=4), UNSUPPORTED),
])
def test_gated_arguments_are_refused(dqlib, change, want):
    assert dqlib.lib().dq_gated_mx(*dict(GATED, **change).values(), None) == want


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(gs=None), ARG), (dict(uc=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG),
    (dict(inner=0), ARG), (dict(inner=48), ARG), (dict(codes=ODD), ARG), (dict(b=ODD), ARG),
    (dict(qfmt=3), UNSUPPORTED), (dict(qfmt=0), UNSUPPORTED),
])
def test_gated_quantized_arguments_are_refused(dqlib, change, want):
    assert dqlib.lib().dq_gated_mx_quantized(*dict(GATEDQ, **change).values(), None) == want


def _apart(call, **pointers):
    """The call with every array at an address of its own (never dereferenced)."""
    names = [k for k, v in call.items() if isinstance(v, ctypes.c_void_p)]
    return {**call, **{k: ctypes.c_void_p((i + 1) << 44) for i, k in enumerate(names)}, **pointers}


def _at(call, other, offset=0):
    return ctypes.c_void_p(_apart(call)[other].value + offset)


@pytest.mark.parametrize("call,entry,out,others", [
    (NORM, "dq_norm_quantize_act_async", "codes", ["X", "R", "h", "w", "b", "scales"]),
    (NORM, "dq_norm_quantize_act_async", "scales", ["X", "R", "h", "w", "b", "codes"]),
    (NORM, "dq_norm_quantize_act_async", "h", ["w", "b"]),
    (EPI, "dq_gemm_mx_epilogue", "y", ["xc", "xs", "wc", "ws", "a", "bias"]),
    (GATED, "dq_gated_mx", "y", ["xc", "xs", "gc", "gs", "ag", "uc", "us", "au"]),
    (GATEDQ, "dq_gated_mx_quantized", "codes", ["xc", "xs", "gc", "gs", "ag", "uc", "us", "au", "b"]),
    (GATEDQ, "dq_gated_mx_quantized", "scales", ["xc", "gs", "au", "b", "codes"]),
])
def test_overlapping_outputs_are_refused(dqlib, call, entry, out, others):
    tail = [FAKE, None] if entry.endswith("async") else [None]
    for o in others:
        for offset in (0, 16):
            args = list(_apart(call, **{out: _at(call, o, offset)}).values())
            assert getattr(dqlib.lib(), entry)(*args, *tail) == ARG, (out, o, offset)


def test_in_place_residuals_overlap_exactly_or_not_at_all(dqlib):
    L = dqlib.lib()
    for other in ("X", "R"):
        args = list(_apart(NORM, h=_at(NORM, other, 16)).values())
        assert L.dq_norm_quantize_act_async(*args, FAKE, None) == ARG
    shifted = _apart(NORM, h=_at(NORM, "X"), R=_at(NORM, "X", 32))  # h is X, but cuts into R
    assert L.dq_norm_quantize_act_async(*shifted.values(), FAKE, None) == ARG
    args = list(_apart(EPI, y=_at(EPI, "res", 16)).values())
    assert L.dq_gemm_mx_epilogue(*args, None) == ARG


def test_channels_past_the_limit_are_refused(dqlib):
    L, out = dqlib.lib(), (1 << 22) + 32
    assert L.dq_gemm_mx_epilogue(*_apart(EPI, out=out).values(), None) == ARG
    assert L.dq_gated_mx(*_apart(GATED, inner=out).values(), None) == ARG
    assert L.dq_gated_mx_quantized(*_apart(GATEDQ, inner=out).values(), None) == ARG


def test_binding_refuses_without_a_gpu(dqlib):
    import torch

    t = torch.zeros(2, 64)
    u = torch.zeros(2, 256, dtype=torch.uint8)
    pk = dict(codes=u, scales=u, out=64, K=512)
    calls = dqlib._calls()
    for f in (lambda: dqlib.act_outputs(t, "mxfp8", 32), lambda: dqlib.act_outputs(3, "mxfp8", 32),
              lambda: dqlib.norm_quantize_act(t, "mxfp8", 32),
              lambda: dqlib.norm_quantize_act_async(t, "mxfp8", 32, u, u, None),
              lambda: dqlib.gemm_mx_epilogue(u, u, pk), lambda: dqlib.gemm_mx_epilogue(u, u, {}),
              lambda: dqlib.gemm_mx_epilogue(u, u, [1]),
              lambda: dqlib.gemm_mx_epilogue(u, u, dict(pk, K=500)),
              lambda: dqlib.gated_mx(u, u, pk, pk),
              lambda: dqlib.gated_mx_quantized(u, u, pk, dict(pk, out=0), "mxfp8")):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        calls.epilogue(u)  # a fixed number of positional arguments
    with pytest.raises(TypeError):
        dqlib.gemm_mx_epilogue(u, u, dict(pk, K="512"))


def test_mxfp8_is_no_format_of_the_solver(dqlib):
    L = dqlib.lib()
    init = dqlib._Init(None, None, 0.0, 0)
    assert L.dq_solve(FAKE, 1, 128, 256, 4, 32, 2, ctypes.byref(init), FAKE, FAKE, FAKE, FAKE,
                      FAKE, FAKE, None, 0, None) == UNSUPPORTED
    assert L.dq_quantize_act_async(FAKE, 1, 4, 256, 4, 32, None, 0.0, None, FAKE, FAKE, FAKE,
                                   None, 0, None) == UNSUPPORTED


def test_reference_e4m3_is_nearest_with_ties_to_even():
    vals = ref.e4m3_values()
    pos = np.sort(vals[np.isfinite(vals) & (vals >= 0)][:127])
    pos = np.unique(pos)
    mids = (pos[:-1] + pos[1:]) / 2
    v = np.concatenate([pos, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        [448.0, 500.0, 1e9, 2.0 ** -30]])
    code = ref.e4m3_codes(v)
    for x, c in zip(v, code):
        d = np.abs(np.minimum(x, 448.0) - pos)
        near = np.flatnonzero(d == d.min())
        want = near[0] if len(near) == 1 else near[near % 2 == 0][0]  # index = byte
        assert c == want, (x, c, want)
    neg = ref.e4m3_codes(-v)
    assert np.array_equal(neg & 0x7F, code) and np.all((neg == 0) == (code == 0))


def test_reference_e4m3_agrees_with_torch():
    import torch

    x = np.random.default_rng(3).standard_normal(4096) * 2.0 ** np.random.default_rng(4).integers(
        -12, 8, 4096)
    x = np.clip(x, -448, 448).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    t = np.where(t == 0x80, 0, t)
    assert np.array_equal(ref.e4m3_codes(x.astype(np.float64)), t)
