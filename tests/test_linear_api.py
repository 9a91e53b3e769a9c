"""The projection with an epilogue and the products over tokens in segments, without a
GPU: every malformed argument is refused before anything is launched, with its reason."""

import ctypes

import pytest

import ggml_q2_quantized_gb300 as q2k
from ggml_q2_quantized_gb300 import build as q2k_build

INVALID = 1
L, G = q2k.LinearParams, q2k.GatedFfnParams
X, W, W2, BIAS, RES, Y, Z, OFF, WS, GATE, UP = (0x1000000 * i for i in range(1, 12))
OK = (20, 8, 256, 10, 1, 1, 0, 0)       # m, n, k, type, bf16, gelu, no segments
SEG = (20, 8, 256, 10, 1, 1, 3, 0)
NONE = (20, 8, 256, 10, 1, 2, 0, 0)     # no activation


@pytest.fixture(scope="module")
def lib():
    q2k_build.build()
    return q2k.load()


def refused(lib, status, fragment):
    assert status == INVALID
    assert fragment in lib.q2k_last_error().decode()


def _wb(p):
    return max(1, p.n_experts) * p.n * (p.k // 256) * 84


def linear(lib, p, path=0, flags=0, **kw):
    a = dict(x=X, xe=p.m * p.k, w=W, wb=_wb(p), bias=BIAS, res=RES, y=Y, ye=p.m * p.n, z=Z,
             off=OFF if p.n_experts else None, ws=WS, wsb=1 << 22)
    a.update(kw)
    return lib.q2k_linear(path, flags, a["x"], a["xe"], a["w"], a["wb"], a["bias"], a["res"], a["y"],
                          a["ye"], a["z"], a["off"], ctypes.byref(p), a["ws"], a["wsb"], None)


BAD_PARAMS = [
    ((0, 8, 256, 10, 1, 1, 0, 0), ">= 1"),
    ((20, 0, 256, 10, 1, 1, 0, 0), ">= 1"),
    ((20, 8, 0, 10, 1, 1, 0, 0), ">= 1"),
    ((20, 8, 128, 10, 1, 1, 0, 0), "multiple of 256"),
    ((20, 8, 256, 9, 1, 1, 0, 0), "not Q2_K"),
    ((20, 8, 256, 10, 3, 1, 0, 0), "unknown dtype"),
    ((20, 8, 256, 10, 1, 3, 0, 0), "unknown act"),
    ((20, 8, 256, 10, 1, 1, 4097, 0), "n_experts must be"),
    ((20, 8, 256, 10, 1, 1, 0, 5), "reserved"),
    (((1 << 20) + 1, 8, 256, 10, 1, 1, 0, 0), "m must be <="),
]


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS] + [
    (OK, {"path": 7}, "unknown path"),
    (OK, {"flags": 2}, "unknown flag bits"),
    (OK, {"x": None}, "non-NULL"),
    (OK, {"w": None}, "non-NULL"),
    (OK, {"y": None}, "non-NULL"),
    (OK, {"xe": 1}, "x has 1"),
    (OK, {"wb": 84}, "w has 84"),
    (SEG, {"wb": 8 * 84}, "w has 672"),
    (OK, {"ye": 161}, "y has 161"),
    (OK, {"off": OFF}, "offsets must be NULL"),
    (SEG, {"off": None}, "offsets must be non-NULL"),
    (SEG, {"off": OFF + 2}, "offsets must be 4-byte aligned"),
    (OK, {"x": X + 8}, "16-byte aligned"),
    (OK, {"bias": BIAS + 4}, "16-byte aligned"),
    (OK, {"res": RES + 2}, "16-byte aligned"),
    (OK, {"z": Z + 2}, "16-byte aligned"),
    (OK, {"w": W + 2}, "4-byte aligned"),
    (OK, {"y": X}, "y must not alias x"),
    (OK, {"y": RES}, "y must not alias residual"),
    (OK, {"y": BIAS + 16}, "y must not alias bias"),
    (OK, {"z": Y + 16}, "y must not alias z"),
    (OK, {"z": RES}, "z must not alias residual"),
    (SEG, {"y": OFF}, "y must not alias offsets"),
    (SEG, {"ws": None}, "workspace is NULL"),
    (SEG, {"wsb": 16}, "workspace has 16"),
    (SEG, {"ws": W}, "workspace must not alias w"),
])
def test_linear_refuses(lib, params, kw, fragment):
    refused(lib, linear(lib, L(*params), **kw), fragment)


def backward(lib, p, **kw):
    a = dict(dy=X, dye=p.m * p.n, z=Z if p.act != 2 else None, w=W, wb=_wb(p), dx=Y, dxe=p.m * p.k,
             dz=RES if p.act != 2 else None, db=BIAS, off=OFF if p.n_experts else None, ws=WS,
             wsb=1 << 22)
    a.update(kw)
    return lib.q2k_linear_backward(a["dy"], a["dye"], a["z"], a["w"], a["wb"], a["dx"], a["dxe"],
                                   a["dz"], a["db"], a["off"], ctypes.byref(p), a["ws"], a["wsb"],
                                   None)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS] + [
    ((20, 8, 256, 10, 0, 1, 0, 0), {}, "bf16 activations only"),
    (OK, {"dy": None}, "non-NULL"),
    (OK, {"dx": None}, "non-NULL"),
    (OK, {"z": None}, "z must be non-NULL"),
    (NONE, {"z": Z}, "must be NULL"),
    (NONE, {"dz": RES}, "must be NULL"),
    (OK, {"dye": 159}, "dy has 159"),
    (OK, {"dxe": 1}, "dx has 1"),
    (SEG, {"wb": 1}, "w has 1"),
    (OK, {"off": OFF}, "offsets must be NULL"),
    (SEG, {"off": None}, "offsets must be non-NULL"),
    (OK, {"dz": RES + 4}, "16-byte aligned"),
    (OK, {"db": BIAS + 4}, "16-byte aligned"),
    (OK, {"dx": X}, "dx must not alias dy"),
    (OK, {"dz": Z}, "dz must not alias z"),
    (OK, {"db": RES}, "dz must not alias dbias"),
    (SEG, {"db": OFF}, "dbias must not alias offsets"),
    (SEG, {"ws": None}, "workspace is NULL"),
    (SEG, {"wsb": 0}, "workspace has 0"),
])
def test_linear_backward_refuses(lib, params, kw, fragment):
    refused(lib, backward(lib, L(*params), **kw), fragment)


GOK = (20, 8, 256, 10, 1, 0)


def gated(lib, p, experts=3, path=0, **kw):
    wb = max(1, experts) * p.n * (p.k // 256) * 84
    a = dict(x=X, w=W, w2=W2, wb=wb, h=Y, gate=GATE, up=UP, off=OFF, ws=WS, wsb=1 << 22)
    a.update(kw)
    return lib.q2k_gated_ffn_experts(path, 0, a["x"], p.m * p.k, a["w"], a["wb"], a["w2"], a["wb"],
                                     a["h"], p.m * p.n, a["gate"], a["up"], a["off"], experts,
                                     ctypes.byref(p), a["ws"], a["wsb"], None)


def gated_backward(lib, p, experts=3, **kw):
    wb = max(1, experts) * p.n * (p.k // 256) * 84
    a = dict(dh=X, w=W, w2=W2, wb=wb, dx=Y, gate=GATE, up=UP, dg=Z, du=RES, off=OFF, ws=WS,
             wsb=1 << 22)
    a.update(kw)
    return lib.q2k_gated_ffn_experts_backward(a["dh"], a["gate"], a["up"], p.m * p.n, a["w"], a["wb"],
                                              a["w2"], a["wb"], a["dx"], p.m * p.k, a["dg"], a["du"],
                                              a["off"], experts, ctypes.byref(p), a["ws"], a["wsb"],
                                              None)


@pytest.mark.parametrize("params,kw,fragment", [
    ((20, 8, 255, 10, 1, 0), {}, "multiple of 256"),
    ((20, 8, 256, 10, 1, 2), {}, "unknown act"),
    (GOK, {"experts": 0}, "n_experts must be >= 1"),
    (GOK, {"experts": 5000}, "n_experts must be <="),
    (GOK, {"wb": 672}, "has 672"),
    (GOK, {"off": None}, "offsets must be non-NULL"),
    (GOK, {"off": OFF + 1}, "4-byte aligned"),
    (GOK, {"gate": OFF}, "gate must not alias offsets"),
    (GOK, {"ws": None}, "workspace is NULL"),
])
@pytest.mark.parametrize("call", [gated, gated_backward])
def test_gated_experts_refuse(lib, call, params, kw, fragment):
    if call is gated_backward and "gate" in kw:
        kw, fragment = {"dg": OFF}, "dgate must not alias offsets"
    refused(lib, call(lib, G(*params), **kw), fragment)


def test_gated_without_segments_takes_no_activation_none(lib):
    p = G(20, 8, 256, 10, 1, 2)
    assert lib.q2k_gated_ffn_workspace_bytes(0, ctypes.byref(p)) == 0
    assert lib.q2k_gated_ffn_experts_workspace_bytes(0, ctypes.byref(G(*GOK)), 0) == 0
    assert lib.q2k_gated_ffn_experts_backward_workspace_bytes(ctypes.byref(G(*GOK)), 4097) == 0


def test_null_params(lib):
    assert lib.q2k_linear(0, 0, X, 1, W, 1, None, None, Y, 1, None, None, None, None, 0, None) == INVALID
    assert lib.q2k_linear_backward(X, 1, Z, W, 1, Y, 1, None, None, None, None, None, 0, None) == INVALID
    assert lib.q2k_linear_workspace_bytes(0, None) == 0
    assert lib.q2k_linear_backward_workspace_bytes(None) == 0


def test_struct_layout():
    assert ctypes.sizeof(L) == 32 and L.n_experts.offset == 24


def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 256), torch.zeros(84, dtype=torch.uint8)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.linear(x, w, 1)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.linear_backward(x.bfloat16(), w, 256)
    routes = q2k.Routes(None, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        q2k.gated_ffn(x, w, w, 1, routes=routes)
