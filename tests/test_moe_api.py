"""The calls that move tokens to their experts and back, without a GPU: every
malformed argument is refused before anything is launched, with its reason."""

import ctypes

import pytest

import ggml_q2_quantized_gb300 as q2k
from ggml_q2_quantized_gb300 import build as q2k_build

INVALID = 1
P = q2k.MoeParams
X, XS, ROWS, ORDER, OFFSETS, WEIGHTS, RES, BAD, DW = (0x1000000 * i for i in range(1, 10))
OK = (6, 2, 5, 40, 1, 0)


@pytest.fixture(scope="module")
def lib():
    q2k_build.build()
    return q2k.load()


def refused(lib, status, fragment):
    assert status == INVALID
    assert fragment in lib.q2k_last_error().decode()


BAD_PARAMS = [
    ((0, 2, 5, 40, 1, 0), "n_tokens must be"),
    (((1 << 20) + 1, 2, 5, 40, 1, 0), "n_tokens must be"),
    ((6, 0, 5, 40, 1, 0), "top_k must be"),
    ((6, 257, 5, 40, 1, 0), "top_k must be"),
    ((6, 2, 0, 40, 1, 0), "n_experts must be"),
    ((6, 2, 4097, 40, 1, 0), "n_experts must be"),
    ((6, 2, 5, 40, 1, 1), "reserved"),
]
BAD_ROWS = [
    ((6, 2, 5, 0, 1, 0), "width must be"),
    ((6, 2, 5, (1 << 20) + 1, 1, 0), "width must be"),
    ((6, 2, 5, 40, 2, 0), "unknown dtype"),
]


def route(lib, p, **kw):
    a = dict(ids=X, n=p.n_tokens * p.top_k, rows=ROWS, order=ORDER, offsets=OFFSETS, bad=BAD)
    a.update(kw)
    return lib.q2k_moe_route(a["ids"], a["n"], a["rows"], a["order"], a["offsets"],
                             ctypes.byref(p), a["bad"], None)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS] + [
    (OK, {"ids": None}, "non-NULL"),
    (OK, {"order": None}, "non-NULL"),
    (OK, {"n": 11}, "ids has 11"),
    (OK, {"rows": ROWS + 2}, "4-byte aligned"),
    (OK, {"bad": BAD + 1}, "4-byte aligned"),
    (OK, {"rows": X + 4}, "rows must not alias ids"),
    (OK, {"order": ROWS}, "rows must not alias order"),
    (OK, {"offsets": ORDER + 44}, "order must not alias offsets"),
    (OK, {"bad": OFFSETS + 20}, "offsets must not alias bad_id_count"),
])
def test_route_refuses(lib, params, kw, fragment):
    refused(lib, route(lib, P(*params), **kw), fragment)


def sort(lib, p, name="q2k_moe_sort", **kw):
    narrow, wide = p.n_tokens * p.width, p.n_tokens * p.top_k * p.width
    a = dict(x=X, xe=narrow, rows=ROWS, offsets=OFFSETS, xs=XS, xse=wide)
    if name == "q2k_moe_sort_backward":
        a.update(x=XS, xe=wide, xs=X, xse=narrow)
    a.update(kw)
    return getattr(lib, name)(a["x"], a["xe"], a["rows"], a["offsets"], a["xs"], a["xse"],
                              ctypes.byref(p), None)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS + BAD_ROWS] + [
    (OK, {"x": None}, "non-NULL"),
    (OK, {"rows": None}, "non-NULL"),
    (OK, {"offsets": None}, "non-NULL"),
    (OK, {"xs": None}, "non-NULL"),
    (OK, {"xe": 239}, "x has 239"),
    (OK, {"xse": 481}, "xs has 481"),
    (OK, {"x": X + 1}, "aligned to their elements"),
    (OK, {"rows": ROWS + 2}, "4-byte aligned"),
    (OK, {"xs": X + 16}, "xs must not alias x"),
    (OK, {"xs": ROWS}, "xs must not alias rows"),
])
def test_sort_refuses(lib, params, kw, fragment):
    refused(lib, sort(lib, P(*params), **kw), fragment)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS + BAD_ROWS] + [
    (OK, {"x": None}, "dxs, rows, offsets and dx"),
    (OK, {"xe": 479}, "dxs has 479"),
    (OK, {"xse": 241}, "dx has 241"),
    (OK, {"xs": XS + 8}, "dx must not alias dxs"),
])
def test_sort_backward_refuses(lib, params, kw, fragment):
    refused(lib, sort(lib, P(*params), "q2k_moe_sort_backward", **kw), fragment)


def combine(lib, p, **kw):
    a = dict(ys=XS, yse=p.n_tokens * p.top_k * p.width, rows=ROWS, offsets=OFFSETS, w=WEIGHTS,
             res=RES, y=X, ye=p.n_tokens * p.width)
    a.update(kw)
    return lib.q2k_moe_combine(a["ys"], a["yse"], a["rows"], a["offsets"], a["w"], a["res"], a["y"],
                               a["ye"], ctypes.byref(p), None)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS + BAD_ROWS] + [
    (OK, {"ys": None}, "non-NULL"),
    (OK, {"y": None}, "non-NULL"),
    (OK, {"yse": 1}, "ys has 1"),
    (OK, {"ye": 1}, "y has 1"),
    (OK, {"res": RES + 1}, "aligned to their elements"),
    (OK, {"w": WEIGHTS + 2}, "4-byte aligned"),
    (OK, {"y": RES}, "y must not alias residual"),
    (OK, {"y": WEIGHTS}, "y must not alias weights"),
])
def test_combine_refuses(lib, params, kw, fragment):
    refused(lib, combine(lib, P(*params), **kw), fragment)


def combine_backward(lib, p, **kw):
    a = dict(dy=X, dye=p.n_tokens * p.width, ys=XS, yse=p.n_tokens * p.top_k * p.width, rows=ROWS,
             offsets=OFFSETS, w=WEIGHTS, dys=RES, dw=DW)
    a.update(kw)
    return lib.q2k_moe_combine_backward(a["dy"], a["dye"], a["ys"], a["yse"], a["rows"], a["offsets"],
                                        a["w"], a["dys"], a["dw"], ctypes.byref(p), None)


@pytest.mark.parametrize("params,kw,fragment", [(p, {}, f) for p, f in BAD_PARAMS + BAD_ROWS] + [
    (OK, {"w": None}, "non-NULL"),
    (OK, {"dw": None}, "non-NULL"),
    (OK, {"dye": 1}, "dy has 1"),
    (OK, {"yse": 1}, "ys has 1"),
    (OK, {"dys": RES + 1}, "aligned to their elements"),
    (OK, {"dw": DW + 2}, "4-byte aligned"),
    (OK, {"dys": XS}, "dys must not alias ys"),
    (OK, {"dw": RES + 4}, "dys must not alias dweights"),
    (OK, {"dw": WEIGHTS}, "dweights must not alias weights"),
])
def test_combine_backward_refuses(lib, params, kw, fragment):
    refused(lib, combine_backward(lib, P(*params), **kw), fragment)


def test_null_params(lib):
    assert lib.q2k_moe_route(X, 1, ROWS, ORDER, OFFSETS, None, BAD, None) == INVALID
    assert lib.q2k_moe_sort(X, 1, ROWS, OFFSETS, XS, 1, None, None) == INVALID


def test_struct_layout():
    assert ctypes.sizeof(P) == 24 and P.dtype.offset == 16


def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    ids = torch.zeros(2, 2, dtype=torch.int32)
    routes = q2k.Routes(ids, ids.view(-1), torch.zeros(4, dtype=torch.int32))
    assert routes.n_experts == 3
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.moe_route(ids, 3)
    for call in (q2k.moe_sort, q2k.moe_sort_backward, q2k.moe_combine):
        with pytest.raises(TypeError, match="CUDA"):
            call(x, routes)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.moe_combine_backward(x[:2], x, routes, torch.zeros(2, 2))
