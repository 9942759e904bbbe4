"""What the MLP operators' host checks refuse, one fault at a time, and what they accept.

Every array of a call lies at an address of its own and the call without the fault passes every
check, which shows by DQ_ERR_HIP: the calls are made in a process to which no GPU is visible, so
that an accepted one finds no device and nothing is enqueued or read."""
import json
import os
import subprocess
import sys

import pytest

ARG, UNSUPPORTED, WORKSPACE, ACCEPTED = 1, 2, 5, 6

_CHILD = r"""
import ctypes, json, sys
L = ctypes.CDLL(sys.argv[1])
n = ctypes.c_int(0)
rc = L.hipGetDeviceCount(ctypes.byref(n))
print(json.dumps("a GPU is visible" if rc == 0 and n.value else "ready"), flush=True)
if rc == 0 and n.value:
    sys.exit(0)
P, I, I64, F, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double
norm = [P, I, P, P, I64, I64, P, I, D, P, I, I, F, P, P, P]
for name, types in dict(
        dq_norm_quantize_act_async=[*norm, P],
        dq_norm_quantize_act=[*norm, ctypes.c_size_t, P],
        dq_gemm_mx_epilogue=[P, P, I, I64, I64, P, P, P, P, I, P, I64, I, P, P],
        dq_gated_mx=[P, P, I, I64, I64, P, P, P, P, P, P, I, I64, I, P, P],
        dq_gated_mx_quantized=[P, P, I, I64, I64, P, P, P, P, P, P, I, I64, P, I, P, P, P]).items():
    getattr(L, name).argtypes = types
for line in sys.stdin:
    name, args = json.loads(line)
    print(getattr(L, name)(*[float(a) if isinstance(a, str) else a for a in args], None), flush=True)
"""


@pytest.fixture(scope="module")
def status():
    """status(entry, call): what the entry point returns for the call's values."""
    import dual_scale_w4a4_amd as dq

    if not os.path.exists(dq.LIB_PATH):
        from dual_scale_w4a4_amd import build

        build.build()
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    child = subprocess.Popen([sys.executable, "-c", _CHILD, dq.LIB_PATH], stdin=subprocess.PIPE,
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


def _at(k):
    return (k + 1) << 44  # an address of its own


# The calls, of 4 tokens
NORM = dict(X=_at(0), xt=1, R=_at(1), h=_at(2), tokens=4, cols=256, w=_at(3), wt=1, eps=1e-5,
            b=_at(4), fmt=4, group=32, g=0.0, codes=_at(5), scales=_at(6), status=_at(7))
NORM_BLOCKING = {**{k: v for k, v in NORM.items() if k != "status"}, "ws": _at(7), "ws_bytes": 256}
EPI = dict(xc=_at(0), xs=_at(1), fmt=2, tokens=4, K=512, wc=_at(2), ws=_at(3), a=_at(4), bias=_at(5),
           act=0, res=_at(6), out=64, yt=1, y=_at(7))
GATED = dict(xc=_at(0), xs=_at(1), fmt=2, tokens=4, K=512, gc=_at(2), gs=_at(3), ag=_at(4), uc=_at(5),
             us=_at(6), au=_at(7), act=2, inner=64, yt=1, y=_at(8))
GATEDQ = dict(xc=_at(0), xs=_at(1), fmt=2, tokens=4, K=512, gc=_at(2), gs=_at(3), ag=_at(4),
              uc=_at(5), us=_at(6), au=_at(7), act=2, inner=64, b=_at(8), qfmt=4, codes=_at(9),
              scales=_at(10))
CALLS = {"dq_norm_quantize_act_async": NORM, "dq_norm_quantize_act": NORM_BLOCKING,
         "dq_gemm_mx_epilogue": EPI, "dq_gated_mx": GATED, "dq_gated_mx_quantized": GATEDQ}
NORMS = ["dq_norm_quantize_act_async", "dq_norm_quantize_act"]
PRODUCTS = ["dq_gemm_mx_epilogue", "dq_gated_mx", "dq_gated_mx_quantized"]
NVFP4 = dict(fmt=3, g=1.0)


def _off(call, name, by):
    return {name: call[name] + by}


@pytest.mark.parametrize("entry", CALLS)
def test_the_unchanged_call_passes_every_check(status, entry):
    assert status(entry, CALLS[entry]) == ACCEPTED


@pytest.mark.parametrize("change", [
    dict(R=None, h=None), dict(w=None), dict(b=None), dict(xt=0), dict(wt=0), dict(tokens=1),
    dict(cols=32), dict(cols=16, group=16), dict(cols=64, group=64), dict(eps=5e-324),
    dict(eps=1.7e308), dict(fmt=0), dict(fmt=1), dict(fmt=2), NVFP4, dict(fmt=3, g=1e-45),
    dict(g=-1.0), dict(fmt=0, scales=_at(6) + 2), dict(scales=_at(6) + 1),
    dict(fmt=2, codes=_at(5) + 8), dict(h=_at(0)), dict(h=_at(1)), dict(X=_at(1), h=_at(1)),
    dict(w=None, wt=7), dict(tokens=2 ** 31 - 1, cols=256), dict(tokens=1, cols=1 << 40)])
@pytest.mark.parametrize("entry", NORMS)
def test_norm_accepts(status, entry, change):
    assert status(entry, {**CALLS[entry], **change}) == ACCEPTED


@pytest.mark.parametrize("change,want", [
    (dict(X=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(R=None), ARG),
    (dict(h=None), ARG), (dict(tokens=0), ARG), (dict(tokens=-1), ARG), (dict(cols=0), ARG),
    (dict(cols=-32), ARG), (dict(cols=250), ARG), (dict(cols=240), ARG), (dict(group=8), ARG),
    (dict(group=128), ARG), (dict(group=0), ARG), (dict(cols=96, group=64), ARG),
    (dict(tokens=1 << 31, cols=32), ARG), (dict(tokens=1, cols=(1 << 40) + 32), ARG),
    (dict(tokens=2, cols=(1 << 39) + 32), ARG), (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(fmt=3, g=0.0), ARG),
    (dict(fmt=3, g=-1.0), ARG), (dict(fmt=3, g=float("nan")), ARG),
    (dict(fmt=3, g=float("inf")), ARG), (_off(NORM, "X", 8), ARG), (_off(NORM, "R", 8), ARG),
    (_off(NORM, "h", 8), ARG), (_off(NORM, "w", 8), ARG), (_off(NORM, "b", 8), ARG),
    (_off(NORM, "codes", 8), ARG), ({"fmt": 2, **_off(NORM, "codes", 4)}, ARG),
    ({**NVFP4, **_off(NORM, "codes", 4)}, ARG), ({"fmt": 0, **_off(NORM, "scales", 1)}, ARG),
    (dict(fmt=5), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED), (dict(xt=2), UNSUPPORTED),
    (dict(xt=-1), UNSUPPORTED), (dict(wt=2), UNSUPPORTED), (dict(wt=-1), UNSUPPORTED)])
@pytest.mark.parametrize("entry", NORMS)
def test_norm_refuses(status, entry, change, want):
    assert status(entry, {**CALLS[entry], **change}) == want


def test_norm_status_and_workspace(status):
    entry = "dq_norm_quantize_act_async"
    assert status(entry, {**NORM, "status": None}) == ARG
    for by, want in ((1, ARG), (2, ARG), (3, ARG), (4, ACCEPTED)):
        assert status(entry, {**NORM, **_off(NORM, "status", by)}) == want
    entry, call = "dq_norm_quantize_act", NORM_BLOCKING
    assert status(entry, {**call, "ws_bytes": 255}) == WORKSPACE
    assert status(entry, {**call, "ws_bytes": 0}) == WORKSPACE
    for by, want in ((16, ARG), (128, ARG), (256, ACCEPTED)):
        assert status(entry, {**call, **_off(call, "ws", by)}) == want
    assert status(entry, {**call, "ws": None, "ws_bytes": 0}) == ACCEPTED


# names of the weights' codes and scales and of the factors, and of the number of channels
WEIGHTS = {"dq_gemm_mx_epilogue": (["wc"], ["ws"], ["a", "bias"], "out"),
           "dq_gated_mx": (["gc", "uc"], ["gs", "us"], ["ag", "au"], "inner"),
           "dq_gated_mx_quantized": (["gc", "uc"], ["gs", "us"], ["ag", "au", "b"], "inner")}


@pytest.mark.parametrize("entry", PRODUCTS)
def test_products_accept(status, entry):
    call = CALLS[entry]
    codes, scales, factors, channels = WEIGHTS[entry]
    good = [{"tokens": 1}, {"tokens": 2 ** 31 - 1 - 256}, {"K": 1 << 22}, {"K": 1536},
            {channels: 32}, {channels: 1 << 22}, {"fmt": 4}, {"act": 4}]
    good += [{n: None} for n in factors]
    good += [_off(call, n, 4) for n in scales] + [_off(call, n, 16) for n in (*codes, *factors)]
    if entry != "dq_gated_mx_quantized":
        good += [{channels: 1}, {channels: 37}, {"yt": 0}, _off(call, "y", 2),
                 {"yt": 0, **_off(call, "y", 4)}]
    else:
        good += [{"qfmt": 2}, _off(call, "scales", 1), _off(call, "codes", 16)]
    if entry == "dq_gemm_mx_epilogue":
        good += [{"res": None}, {"res": call["y"]}, _off(call, "res", 2),
                 {"yt": 0, **_off(call, "res", 4)}]
    else:
        good += [{"uc": call["gc"], "us": call["gs"]}, {"au": call["ag"]}]
    for change in good:
        assert status(entry, {**call, **change}) == ACCEPTED, change


@pytest.mark.parametrize("entry", PRODUCTS)
def test_products_refuse(status, entry):
    call = CALLS[entry]
    codes, scales, factors, channels = WEIGHTS[entry]
    bad = [({"tokens": 0}, ARG), ({"tokens": -1}, ARG), ({"tokens": 2 ** 31 - 256}, ARG),
           ({"K": 0}, ARG), ({"K": -512}, ARG), ({"K": 256}, ARG), ({"K": 768}, ARG), ({"K": 544}, ARG),
           ({"K": (1 << 22) + 512}, ARG), ({channels: 0}, ARG), ({channels: -32}, ARG),
           ({channels: (1 << 22) + 32}, ARG), ({"fmt": 0}, UNSUPPORTED), ({"fmt": 1}, UNSUPPORTED),
           ({"fmt": 3}, UNSUPPORTED), ({"fmt": 5}, UNSUPPORTED), ({"act": 5}, UNSUPPORTED),
           ({"act": -1}, UNSUPPORTED)]
    bad += [({n: None}, ARG) for n in ("xc", "xs", *codes, *scales)]
    bad += [(_off(call, n, 8), ARG) for n in ("xc", "xs", *codes, *factors)]
    bad += [(_off(call, n, 2), ARG) for n in scales]
    if entry == "dq_gated_mx_quantized":
        bad += [({"codes": None}, ARG), ({"scales": None}, ARG), ({"inner": 48}, ARG),
                ({"inner": 31}, ARG), (_off(call, "codes", 8), ARG), ({"qfmt": 0}, UNSUPPORTED),
                ({"qfmt": 3}, UNSUPPORTED), ({"qfmt": 5}, UNSUPPORTED)]
    else:
        bad += [({"y": None}, ARG), (_off(call, "y", 1), ARG), ({"yt": 0, **_off(call, "y", 2)}, ARG),
                ({"yt": 2}, UNSUPPORTED), ({"yt": -1}, UNSUPPORTED),
                ({"yt": 0, "fmt": 4}, UNSUPPORTED)]  # fp32 results of MXFP8 activations
    if entry == "dq_gemm_mx_epilogue":
        bad += [(_off(call, "res", 1), ARG), ({"yt": 0, **_off(call, "res", 2)}, ARG)]
    for change, want in bad:
        assert status(entry, {**call, **change}) == want, change


def _bytes(entry, call):
    """The bytes of every array of a call of 4 tokens, with its sizes as above."""
    if entry in NORMS:
        x = 4 * 256 * (2 if call["xt"] else 4)
        return dict(X=x, R=x, h=x, w=256 * (2 if call["wt"] else 4), b=1024,
                    codes=4 * (256 if call["fmt"] == 4 else 128),
                    scales=4 * 8 * (2 if call["fmt"] == 0 else 1),
                    **({"ws": 256} if "ws" in call else {"status": 4}))
    n = dict(xc=4 * (512 if call["fmt"] == 4 else 256), xs=4 * 16)
    for k in ("wc", "gc", "uc"):
        n[k] = 64 * 256
    for k in ("ws", "gs", "us"):
        n[k] = 64 * 16
    for k in ("a", "bias", "ag", "au", "b"):
        n[k] = 64 * 4
    n["res"] = n["y"] = 4 * 64 * (2 if call.get("yt") else 4)
    n["codes"] = 4 * (64 if call.get("qfmt") == 4 else 32)
    if entry == "dq_gated_mx_quantized":
        n["scales"] = 4 * 2
    return {k: v for k, v in n.items() if k in call}


OUTPUTS = {"dq_gemm_mx_epilogue": ["y"], "dq_gated_mx": ["y"],
           "dq_gated_mx_quantized": ["codes", "scales"],
           NORMS[0]: ["codes", "scales", "h", "status"], NORMS[1]: ["codes", "scales", "h", "ws"]}


@pytest.mark.parametrize("entry,change", [(e, {}) for e in CALLS] + [
    (NORMS[0], dict(fmt=0)), (NORMS[0], dict(fmt=2)), (NORMS[0], dict(xt=0, wt=0)),
    (PRODUCTS[0], dict(yt=0)), (PRODUCTS[0], dict(fmt=4)), (PRODUCTS[1], dict(yt=0)),
    (PRODUCTS[1], dict(fmt=4)), (PRODUCTS[2], dict(qfmt=2, fmt=4))])
def test_an_output_overlaps_no_other_array(status, entry, change):
    # either array may end where the other begins, and neither may reach a byte into the other
    call = {**CALLS[entry], **change}
    size = _bytes(entry, call)
    for out in OUTPUTS[entry]:
        for other in size:
            if other == out:
                continue
            # steps that keep the output's alignment; sizes that are no whole steps reach over
            step = 256 if out == "ws" else 16
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


def test_an_in_place_output_may_not_reach_into_the_other_input(status):
    for entry in NORMS:
        call = CALLS[entry]
        for a, b in (("X", "R"), ("R", "X")):
            same = {**call, "h": call[a]}
            assert status(entry, {**same, b: call[a] + 32}) == ARG
            assert status(entry, {**same, b: call[a] + 2048}) == ACCEPTED
