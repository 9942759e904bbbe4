"""CPU checks of include/dq_layer.h: the entry points are exported, the header is C, and what the host
checks refuse, one fault at a time, and what they accept.

Every array of a call lies at an address of its own and the call without the fault passes every
check, which shows by DQ_ERR_HIP: the calls are made in a process to which no GPU is visible, so
that an accepted one finds no device and nothing is enqueued or read."""
import ctypes
import json
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dq_layer.h")
ARG, UNSUPPORTED, WORKSPACE, ACCEPTED = 1, 2, 5, 6
NAN, INF = float("nan"), float("inf")

_CHILD = r"""
import ctypes, json, sys
L = ctypes.CDLL(sys.argv[1])
n = ctypes.c_int(0)
rc = L.hipGetDeviceCount(ctypes.byref(n))
print(json.dumps("a GPU is visible" if rc == 0 and n.value else "ready"), flush=True)
if rc == 0 and n.value:
    sys.exit(0)
P, I, I64, F, D, S = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                      ctypes.c_size_t)
norm = [P, I, I, P, D, P, P, P, F, P, I64, I64, P, I, D, P, I, P, I, I, F, P, P, P]
for name, types in dict(
        dq_block_norm_quantize_act_async=[*norm, P],
        dq_block_norm_quantize_act=[*norm, S, P],
        dq_gemm_mx_adapters=[P, P, I, I64, I64, P, P, P, P, P, P, I64, I, P, P, P, I, P, I64, I, P, P,
                             S, P],
        dq_moe_route=[P, I, I64, I64, P, I, I64, P, I, I, I, F, P, P, P, S, P],
        dq_moe_mx=[P, P, I, I64, I64, P, P, I, I64, P, P, P, P, P, P, I, I64, P, I, P, P, P, P, I64, I,
                   P, P, S, P]).items():
    getattr(L, name).argtypes = types
for line in sys.stdin:
    name, args = json.loads(line)
    print(getattr(L, name)(*[float(a) if isinstance(a, str) else a for a in args], None), flush=True)
"""


@pytest.fixture(scope="module")
def dqlib():
    import dual_scale_w4a4_amd as dq

    if not os.path.exists(dq.LIB_PATH):
        from dual_scale_w4a4_amd import build

        build.build()
    return dq


@pytest.fixture(scope="module")
def status(dqlib):
    """status(entry, call): what the entry point returns for the call's values."""
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    child = subprocess.Popen([sys.executable, "-c", _CHILD, dqlib.LIB_PATH], stdin=subprocess.PIPE,
                             stdout=subprocess.PIPE, text=True, env=env)
    hello = json.loads(child.stdout.readline())
    if hello != "ready":
        child.wait()
        pytest.skip(hello)

    def call(entry, values):
        # floats as text: JSON has no NaN
        args = [repr(v) if isinstance(v, float) else v for v in values.values()]
        child.stdin.write(json.dumps([entry, args]) + "\n")
        child.stdin.flush()
        return int(child.stdout.readline())

    yield call
    child.stdin.close()
    child.wait()


def test_header_and_exports(dqlib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dq_[a-z0-9_]+)\s*\(", src)))
    assert names == ["dq_adapter_workspace_bytes", "dq_block_norm_quantize_act",
                     "dq_block_norm_quantize_act_async", "dq_gemm_mx_adapters", "dq_moe_mx",
                     "dq_moe_route", "dq_moe_route_workspace_bytes", "dq_moe_workspace_bytes"]
    out = subprocess.run(["nm", "-D", "--defined-only", dqlib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert set(names) <= {l.split()[-1] for l in out.splitlines() if " T " in l}


def test_header_compiles_as_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text(f'#define __HIP_PLATFORM_AMD__ 1\n#include "{HEADER}"\n'
                 "int main(void) { return DQ_SCORE_SIGMOID != 1; }\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-I/opt/rocm/include", str(c)], check=True)


def _at(k):
    return (k + 1) << 44  # an address of its own


NORM = dict(X=_at(0), xt=1, post_norm=1, post=_at(1), post_eps=1e-5, gate=_at(2), tgate=_at(3),
            R=_at(4), rs=0.5, h=_at(5), tokens=4, cols=256, w=_at(6), wt=1, eps=1e-5, xo=_at(7), xot=1,
            b=_at(8), fmt=4, group=32, g=0.0, codes=_at(9), scales=_at(10), status=_at(11))
NORM_BLOCKING = {**{k: v for k, v in NORM.items() if k != "status"}, "ws": _at(11), "ws_bytes": 256}
ADAPT = dict(xc=_at(0), xs=_at(1), fmt=2, tokens=40, K=512, wc=_at(2), ws=_at(3), a=_at(4), bias=_at(5),
             X=_at(6), ids=_at(7), adapters=3, rank=16, A=_at(8), B=_at(9), scale=_at(10), act=0,
             res=_at(11), out=64, yt=1, y=_at(12), space=_at(13), bytes=1 << 20)
ROUTE = dict(X=_at(0), xt=1, tokens=4, cols=256, W=_at(1), wt=1, experts=8, bias=_at(2), score=0,
             top_k=2, renorm=1, scale=1.0, ids=_at(3), weights=_at(4), space=_at(5), bytes=256)
MOE = dict(xc=_at(0), xs=_at(1), fmt=2, tokens=4, K=512, ids=_at(2), weights=_at(3), top_k=2, experts=3,
           gc=_at(4), gs=_at(5), ag=_at(6), uc=_at(7), us=_at(8), au=_at(9), act=2, inner=1024, b=_at(10),
           mid=4, dc=_at(11), ds=_at(12), ad=_at(13), res=_at(14), out=64, yt=1, y=_at(15),
           space=_at(16), bytes=1 << 20)
CALLS = {"dq_block_norm_quantize_act_async": NORM, "dq_block_norm_quantize_act": NORM_BLOCKING,
         "dq_gemm_mx_adapters": ADAPT, "dq_moe_route": ROUTE, "dq_moe_mx": MOE}
NORMS = ["dq_block_norm_quantize_act_async", "dq_block_norm_quantize_act"]


def _off(call, name, by):
    return {name: call[name] + by}


@pytest.mark.parametrize("entry", CALLS)
def test_the_unchanged_call_passes_every_check(status, entry):
    assert status(entry, CALLS[entry]) == ACCEPTED


@pytest.mark.parametrize("change", [
    dict(R=None), dict(post=None), dict(post=None, post_norm=0), dict(gate=None), dict(tgate=None),
    dict(w=None), dict(w=None, post=None, wt=7), dict(xo=None), dict(xo=None, xot=7), dict(b=None),
    dict(xt=0), dict(wt=0), dict(xot=0), dict(tokens=1), dict(cols=32), dict(cols=16, group=16),
    dict(cols=64, group=64), dict(eps=5e-324), dict(eps=1.7e308), dict(post_eps=5e-324),
    dict(post_norm=0, post=None, post_eps=0.0), dict(post_norm=0, post=None, post_eps=NAN),
    dict(rs=0.0), dict(rs=-3e38), dict(fmt=0), dict(fmt=1), dict(fmt=2), dict(fmt=3, g=1.0),
    dict(g=-1.0), dict(fmt=0, scales=_at(10) + 2), dict(scales=_at(10) + 1),
    dict(fmt=2, codes=_at(9) + 8), dict(tgate=_at(3) + 4), dict(h=_at(0)), dict(h=_at(4)),
    dict(X=_at(4), h=_at(4)), dict(X=_at(4)), dict(tokens=2 ** 31 - 1, cols=256),
    dict(tokens=1, cols=1 << 40)])
@pytest.mark.parametrize("entry", NORMS)
def test_norm_accepts(status, entry, change):
    assert status(entry, {**CALLS[entry], **change}) == ACCEPTED


@pytest.mark.parametrize("change,want", [
    (dict(X=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(h=None), ARG),
    (dict(post_norm=2), ARG), (dict(post_norm=-1), ARG), (dict(post_norm=0), ARG), (dict(tokens=0), ARG),
    (dict(tokens=-1), ARG), (dict(cols=0), ARG), (dict(cols=-32), ARG), (dict(cols=250), ARG),
    (dict(cols=240), ARG), (dict(group=8), ARG), (dict(group=128), ARG), (dict(group=0), ARG),
    (dict(cols=96, group=64), ARG), (dict(tokens=1 << 31, cols=32), ARG),
    (dict(tokens=1, cols=(1 << 40) + 32), ARG), (dict(tokens=2, cols=(1 << 39) + 32), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG),
    (dict(post_eps=0.0), ARG), (dict(post_eps=-1.0), ARG), (dict(post_eps=NAN), ARG),
    (dict(post_eps=INF), ARG), (dict(rs=NAN), ARG), (dict(rs=INF), ARG), (dict(rs=-INF), ARG),
    (dict(fmt=3), ARG), (dict(fmt=3, g=-1.0), ARG), (dict(fmt=3, g=NAN), ARG), (dict(fmt=3, g=INF), ARG),
    *[(_off(NORM, n, 8), ARG) for n in ("X", "post", "gate", "R", "h", "w", "xo", "b", "codes")],
    (_off(NORM, "tgate", 2), ARG), ({"fmt": 2, **_off(NORM, "codes", 4)}, ARG),
    ({"fmt": 0, **_off(NORM, "scales", 1)}, ARG),
    (dict(fmt=5), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED), (dict(xt=2), UNSUPPORTED),
    (dict(xt=-1), UNSUPPORTED), (dict(wt=2), UNSUPPORTED), (dict(wt=2, post=None), UNSUPPORTED),
    (dict(wt=2, w=None), UNSUPPORTED), (dict(xot=2), UNSUPPORTED), (dict(xot=-1), UNSUPPORTED)])
@pytest.mark.parametrize("entry", NORMS)
def test_norm_refuses(status, entry, change, want):
    assert status(entry, {**CALLS[entry], **change}) == want


def test_norm_status_and_workspace(status):
    entry = NORMS[0]
    assert status(entry, {**NORM, "status": None}) == ARG
    for by, want in ((1, ARG), (2, ARG), (3, ARG), (4, ACCEPTED)):
        assert status(entry, {**NORM, **_off(NORM, "status", by)}) == want
    entry, call = NORMS[1], NORM_BLOCKING
    assert status(entry, {**call, "ws_bytes": 255}) == WORKSPACE
    for by, want in ((16, ARG), (128, ARG), (256, ACCEPTED)):
        assert status(entry, {**call, **_off(call, "ws", by)}) == want
    assert status(entry, {**call, "ws": None, "ws_bytes": 0}) == ACCEPTED


@pytest.mark.parametrize("change", [
    dict(tokens=1), dict(tokens=2 ** 31 - 1 - 256, bytes=1 << 50), dict(K=1 << 22), dict(K=1536),
    dict(out=1), dict(out=37), dict(out=1 << 22), dict(fmt=4), dict(act=4), dict(yt=0), dict(a=None),
    dict(bias=None), dict(scale=None), dict(res=None), dict(res=ADAPT["y"]), dict(adapters=1),
    dict(adapters=1 << 20), dict(rank=8), dict(rank=256), dict(rank=24), _off(ADAPT, "ws", 4),
    _off(ADAPT, "ids", 4), _off(ADAPT, "scale", 4), _off(ADAPT, "y", 2), _off(ADAPT, "res", 2),
    dict(yt=0, y=ADAPT["y"] + 4), *[_off(ADAPT, n, 16) for n in ("xc", "xs", "wc", "a", "bias", "X", "A", "B")]])
def test_adapters_accept(status, change):
    assert status("dq_gemm_mx_adapters", {**ADAPT, **change}) == ACCEPTED


@pytest.mark.parametrize("change,want", [
    *[({n: None}, ARG) for n in ("xc", "xs", "wc", "ws", "X", "ids", "A", "B", "y", "space")],
    *[(_off(ADAPT, n, 8), ARG) for n in ("xc", "xs", "wc", "a", "bias", "X", "A", "B")],
    (_off(ADAPT, "ws", 2), ARG), (_off(ADAPT, "ids", 2), ARG), (_off(ADAPT, "scale", 2), ARG),
    (_off(ADAPT, "y", 1), ARG), (_off(ADAPT, "res", 1), ARG), (dict(yt=0, y=ADAPT["y"] + 2), ARG),
    (_off(ADAPT, "space", 128), ARG), (dict(tokens=0), ARG), (dict(tokens=2 ** 31 - 256), ARG),
    (dict(K=0), ARG), (dict(K=256), ARG), (dict(K=768), ARG), (dict(K=(1 << 22) + 512), ARG),
    (dict(out=0), ARG), (dict(out=(1 << 22) + 32), ARG), (dict(adapters=0), ARG),
    (dict(adapters=-1), ARG), (dict(adapters=(1 << 20) + 1), ARG), (dict(rank=0), ARG),
    (dict(rank=12), ARG), (dict(rank=264), ARG), (dict(rank=-8), ARG), (dict(bytes=256), WORKSPACE),
    (dict(fmt=0), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(act=5), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(yt=2), UNSUPPORTED), (dict(yt=0, fmt=4), UNSUPPORTED)])
def test_adapters_refuse(status, change, want):
    assert status("dq_gemm_mx_adapters", {**ADAPT, **change}) == want


@pytest.mark.parametrize("change", [
    dict(tokens=1), dict(tokens=2 ** 31 - 1 - 256, bytes=1 << 50), dict(cols=8), dict(cols=1 << 22),
    dict(xt=0), dict(wt=0), dict(experts=2), dict(experts=1024, bytes=1 << 20), dict(bias=None),
    dict(score=1), dict(top_k=1), dict(top_k=8), dict(experts=1024, top_k=32, bytes=1 << 20),
    dict(renorm=0), dict(scale=0.0), dict(scale=-3e38), _off(ROUTE, "bias", 4), _off(ROUTE, "ids", 4),
    _off(ROUTE, "weights", 4), _off(ROUTE, "X", 16), _off(ROUTE, "W", 16)])
def test_route_accepts(status, change):
    assert status("dq_moe_route", {**ROUTE, **change}) == ACCEPTED


@pytest.mark.parametrize("change,want", [
    *[({n: None}, ARG) for n in ("X", "W", "ids", "weights", "space")],
    (_off(ROUTE, "X", 8), ARG), (_off(ROUTE, "W", 8), ARG), (_off(ROUTE, "bias", 2), ARG),
    (_off(ROUTE, "ids", 2), ARG), (_off(ROUTE, "weights", 2), ARG), (_off(ROUTE, "space", 16), ARG),
    (dict(tokens=0), ARG), (dict(tokens=2 ** 31 - 256), ARG), (dict(cols=0), ARG), (dict(cols=12), ARG),
    (dict(cols=(1 << 22) + 8), ARG), (dict(experts=0), ARG), (dict(experts=1025, bytes=1 << 30), ARG),
    (dict(top_k=0), ARG), (dict(top_k=9), ARG), (dict(experts=64, top_k=33, bytes=1 << 20), ARG),
    (dict(renorm=2), ARG), (dict(renorm=-1), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG),
    (dict(bytes=255), WORKSPACE), (dict(xt=2), UNSUPPORTED), (dict(wt=-1), UNSUPPORTED),
    (dict(score=2), UNSUPPORTED), (dict(score=-1), UNSUPPORTED)])
def test_route_refuses(status, change, want):
    assert status("dq_moe_route", {**ROUTE, **change}) == want


BIG = dict(bytes=1 << 40)


@pytest.mark.parametrize("change", [
    dict(tokens=1), {**BIG, "tokens": 2 ** 31 - 1 - 256}, {**BIG, "K": 1 << 22}, {**BIG, "inner": 1 << 22},
    {**BIG, "out": 1 << 22}, dict(K=1536), dict(inner=512), dict(out=32), {**BIG, "top_k": 32},
    dict(top_k=1), dict(top_k=3), {**BIG, "top_k": 7}, dict(experts=1), {**BIG, "experts": 1024},
    dict(fmt=4), dict(mid=2), dict(fmt=2, mid=2, yt=0), dict(act=4), dict(ag=None), dict(au=None),
    dict(ad=None), dict(b=None), dict(res=None), dict(res=MOE["y"]), _off(MOE, "ids", 4),
    _off(MOE, "weights", 4), *[_off(MOE, n, 4) for n in ("gs", "us", "ds")], dict(uc=MOE["gc"]),
    *[_off(MOE, n, 16) for n in ("xc", "xs", "gc", "uc", "dc", "ag", "au", "ad", "b", "res", "y")]])
def test_moe_accepts(status, change):
    assert status("dq_moe_mx", {**MOE, **change}) == ACCEPTED


@pytest.mark.parametrize("change,want", [
    *[({n: None}, ARG) for n in ("xc", "xs", "ids", "weights", "gc", "gs", "uc", "us", "dc", "ds", "y",
                                 "space")],
    *[(_off(MOE, n, 8), ARG) for n in ("xc", "xs", "gc", "uc", "dc", "ag", "au", "ad", "b", "res", "y")],
    *[(_off(MOE, n, 2), ARG) for n in ("gs", "us", "ds", "ids", "weights")],
    (_off(MOE, "space", 64), ARG), (dict(tokens=0), ARG), (dict(tokens=2 ** 31 - 256, **BIG), ARG),
    (dict(K=0), ARG), (dict(K=768), ARG), (dict(K=(1 << 22) + 512, **BIG), ARG), (dict(inner=256), ARG),
    (dict(inner=544), ARG), (dict(inner=(1 << 22) + 512, **BIG), ARG), (dict(out=0), ARG),
    (dict(out=48), ARG), (dict(out=(1 << 22) + 32, **BIG), ARG), (dict(top_k=0), ARG),
    (dict(top_k=33, **BIG), ARG), (dict(experts=0), ARG), (dict(experts=1025, **BIG), ARG),
    (dict(bytes=4096), WORKSPACE), (dict(fmt=0), UNSUPPORTED), (dict(fmt=5), UNSUPPORTED),
    (dict(mid=0), UNSUPPORTED), (dict(mid=3), UNSUPPORTED), (dict(act=5), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(yt=2), UNSUPPORTED), (dict(yt=0), UNSUPPORTED),
    (dict(yt=0, mid=2, fmt=4), UNSUPPORTED)])
def test_moe_refuses(status, change, want):
    assert status("dq_moe_mx", {**MOE, **change}) == want


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=1), dict(tokens=100000), dict(top_k=9, experts=1000)])
def test_workspaces_are_what_the_calls_need(dqlib, status, sizes):
    c = {**MOE, **sizes}
    n = dqlib.moe_workspace_bytes(c["tokens"], c["K"], c["inner"], c["out"], c["experts"], c["top_k"])
    assert n % 256 == 0
    for by, want in ((0, ACCEPTED), (-1, WORKSPACE)):
        assert status("dq_moe_mx", {**c, "bytes": n + by}) == want
    c = {**ADAPT, **{k: v for k, v in sizes.items() if k in ADAPT}}
    n = dqlib.adapter_workspace_bytes(c["tokens"], c["K"], c["rank"])
    for by, want in ((0, ACCEPTED), (-1, WORKSPACE)):
        assert status("dq_gemm_mx_adapters", {**c, "bytes": n + by}) == want
    c = {**ROUTE, **sizes}
    n = dqlib.moe_route_workspace_bytes(c["tokens"], c["experts"])
    for by, want in ((0, ACCEPTED), (-1, WORKSPACE)):
        assert status("dq_moe_route", {**c, "bytes": n + by}) == want


def test_workspace_bytes_refuse(dqlib):
    for f, bad in ((dqlib.moe_workspace_bytes, [(0, 512, 512, 32, 1, 1), (1, 500, 512, 32, 1, 1),
                                                (1, 512, 256, 32, 1, 1), (1, 512, 512, 33, 1, 1),
                                                (1, 512, 512, 32, 0, 1), (1, 512, 512, 32, 1, 33)]),
                   (dqlib.adapter_workspace_bytes, [(0, 512, 8), (1, 500, 8), (1, 512, 4), (1, 512, 264)]),
                   (dqlib.moe_route_workspace_bytes, [(0, 1), (1, 0), (1, 1025)])):
        for args in bad:
            with pytest.raises(dqlib.DQError):
                f(*args)
    L = dqlib.lib()
    assert L.dq_moe_workspace_bytes(1, 512, 512, 32, 1, 1, None) == ARG
    assert L.dq_adapter_workspace_bytes(1, 512, 8, None) == ARG
    assert L.dq_moe_route_workspace_bytes(1, 1, None) == ARG
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def _bytes(entry, call):
    """The bytes of every array of a call, with its sizes as above."""
    if entry in NORMS:
        x = 4 * 256 * (2 if call["xt"] else 4)
        w = 256 * (2 if call["wt"] else 4)
        return dict(X=x, R=x, h=x, post=w, w=w, gate=1024, b=1024, tgate=16,
                    xo=4 * 256 * (2 if call["xot"] else 4), codes=4 * (256 if call["fmt"] == 4 else 128),
                    scales=4 * 8 * (2 if call["fmt"] == 0 else 1),
                    **({"ws": 256} if "ws" in call else {"status": 4}))
    if entry == "dq_gemm_mx_adapters":
        y = 40 * 64 * (2 if call["yt"] else 4)
        return dict(xc=40 * (512 if call["fmt"] == 4 else 256), xs=40 * 16, wc=64 * 256, ws=64 * 16,
                    a=256, bias=256, X=40 * 1024, ids=160, A=3 * 16 * 1024, B=3 * 64 * 32, scale=12,
                    res=y, y=y, space=call["bytes"])
    if entry == "dq_moe_route":
        return dict(X=4 * 256 * (2 if call["xt"] else 4), W=8 * 256 * (2 if call["wt"] else 4), bias=32,
                    ids=32, weights=32, space=256)
    y = 4 * 64 * (2 if call["yt"] else 4)
    w, d = 3 * 1024 * 512, 3 * 64 * 1024
    return dict(xc=4 * (512 if call["fmt"] == 4 else 256), xs=64, ids=32, weights=32, gc=w // 2,
                gs=w // 32, uc=w // 2, us=w // 32, dc=d // 2, ds=d // 32, ag=12288, au=12288, b=12288,
                ad=768, res=y, y=y, space=call["bytes"])


OUTPUTS = {NORMS[0]: ["codes", "scales", "h", "xo", "status"], NORMS[1]: ["codes", "scales", "h", "xo", "ws"],
           "dq_gemm_mx_adapters": ["y", "space"], "dq_moe_route": ["ids", "weights", "space"],
           "dq_moe_mx": ["y", "space"]}


@pytest.mark.parametrize("entry,change", [(e, {}) for e in CALLS] + [
    (NORMS[0], dict(fmt=0, xot=0)), (NORMS[0], dict(fmt=2)), (NORMS[0], dict(xt=0, wt=0)),
    ("dq_gemm_mx_adapters", dict(yt=0)), ("dq_gemm_mx_adapters", dict(fmt=4)),
    ("dq_moe_route", dict(xt=0, wt=0)), ("dq_moe_mx", dict(fmt=4)), ("dq_moe_mx", dict(yt=0, mid=2))])
def test_an_output_overlaps_no_other_array(dqlib, status, entry, change):
    # either array may end where the other begins, and neither may reach a byte into the other
    call = {**CALLS[entry], **change}
    if entry == "dq_gemm_mx_adapters":
        call["bytes"] = dqlib.adapter_workspace_bytes(40, 512, 16)
    if entry == "dq_moe_mx":
        call["bytes"] = dqlib.moe_workspace_bytes(4, 512, 1024, 64, 3, 2)
    size = _bytes(entry, call)
    for out in OUTPUTS[entry]:
        for other in size:
            if other == out:
                continue
            # steps that keep the output's alignment; sizes that are no whole steps reach over
            step = 256 if out in ("ws", "space") else 16
            up = lambda n: -(-n // step) * step  # noqa: E731
            last = up(size[other]) - step
            cases = [(call[other] + up(size[other]), ACCEPTED), (call[other] + last, ARG),
                     (call[other] - up(size[out]), ACCEPTED),
                     (call[other] - up(size[out]) + step, ARG if size[out] > step else None),
                     (call[other], ARG)]
            if (out, other) in (("h", "X"), ("h", "R"), ("y", "res")):
                cases[-1] = (call[other], ACCEPTED)  # in place
            for where, want in cases:
                if want is not None:
                    assert status(entry, {**call, out: where}) == want, (out, other, where)


def test_binding_refuses_without_a_gpu(dqlib):
    import torch

    t, u = torch.zeros(2, 64), torch.zeros(2, 256, dtype=torch.uint8)
    pk = dict(codes=u, scales=u, out=64, K=512)
    ids, w = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    for f in (lambda: dqlib.block_norm_quantize_act(t, "mxfp8", 32),
              lambda: dqlib.block_norm_quantize_act_async(t, "mxfp8", 32, u, u, None),
              lambda: dqlib.gemm_mx_adapters(u, u, pk, t, ids, t, t),
              lambda: dqlib.gemm_mx_adapters(u, u, {}, t, ids, t, t),
              lambda: dqlib.moe_route(t, t, 1), lambda: dqlib.moe_route(t, 3, 1),
              lambda: dqlib.moe_mx(u, u, ids, w, pk, pk, dict(pk, K=512), 1),
              lambda: dqlib.moe_mx(u, u, ids, w, pk, pk, {}, 1)):
        with pytest.raises(ValueError):
            f()
    calls = dqlib._calls()
    for f in (calls.block_norm, calls.adapters, calls.moe, calls.route):
        with pytest.raises(TypeError):
            f(u)  # a fixed number of positional arguments
