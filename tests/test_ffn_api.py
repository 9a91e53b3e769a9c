"""The feed-forward calls without a GPU: every malformed argument is refused
before anything is launched, with its reason."""

import ctypes

import pytest

import ggml_q2_quantized_gb300 as q2k
from ggml_q2_quantized_gb300 import build as q2k_build

INVALID = 1
G, L = q2k.GatedFfnParams, q2k.LoraParams
X, W1, W2, H, GATE, UP, WS = (0x1000000 * i for i in range(1, 8))
A, B, IDS, SCALES, BAD = (0x1000000 * i for i in range(8, 13))


@pytest.fixture(scope="module")
def lib():
    q2k_build.build()
    return q2k.load()


def _wb(p):
    return p.n * (p.k // 256) * 84


def gated(lib, p, path=0, flags=0, **kw):
    a = dict(x=X, xe=p.m * p.k, wg=W1, wgb=_wb(p), wu=W2, wub=_wb(p), h=H, he=p.m * p.n, gate=None,
             up=None, ws=WS, wsb=1 << 22)
    a.update(kw)
    return lib.q2k_gated_ffn(path, flags, a["x"], a["xe"], a["wg"], a["wgb"], a["wu"], a["wub"],
                             a["h"], a["he"], a["gate"], a["up"], ctypes.byref(p), a["ws"],
                             a["wsb"], None)


def refused(lib, status, fragment):
    assert status == INVALID
    assert fragment in lib.q2k_last_error().decode()


OK = (20, 8, 256, 10, 1, 0)


@pytest.mark.parametrize("params,kw,fragment", [
    ((0, 8, 256, 10, 1, 0), {}, ">= 1"),
    ((1, 0, 256, 10, 1, 0), {}, ">= 1"),
    ((1, 8, 0, 10, 1, 0), {}, ">= 1"),
    ((1, 8, 255, 10, 1, 0), {}, "multiple of 256"),
    ((1, 8, 256, 11, 1, 0), {}, "not Q2_K"),
    ((1, 8, 256, 10, 2, 0), {}, "unknown dtype"),
    ((1, 8, 256, 10, 1, 2), {}, "unknown act"),
    (((1 << 20) + 1, 8, 256, 10, 1, 0), {}, "m must be <="),
    ((1, (1 << 20) + 1, 256, 10, 1, 0), {}, "m must be <="),
    (OK, {"path": 3}, "unknown path"),
    (OK, {"flags": 2}, "unknown flag bits"),
    (OK, {"x": None}, "non-NULL"),
    (OK, {"wu": None}, "non-NULL"),
    (OK, {"h": None}, "non-NULL"),
    (OK, {"gate": GATE}, "both be NULL"),
    (OK, {"xe": 20 * 256 - 1}, "x has 5119"),
    (OK, {"he": 161}, "h has 161"),
    (OK, {"wgb": 671}, "w_gate has 671"),
    (OK, {"wub": 673}, "w_up has 673"),
    (OK, {"x": X + 8}, "16-byte aligned"),
    (OK, {"h": H + 2}, "16-byte aligned"),
    (OK, {"wg": W1 + 2}, "4-byte aligned"),
    (OK, {"h": X + 16}, "h must not alias x"),
    (OK, {"h": W2}, "h must not alias w_up"),
    (OK, {"gate": GATE, "up": GATE + 16}, "gate must not alias up"),
    (OK, {"gate": H, "up": UP}, "h must not alias gate"),
    (OK, {"ws": None}, "workspace is NULL"),
    (OK, {"wsb": 16}, "workspace has 16"),
    (OK, {"ws": WS + 8}, "16-byte aligned"),
    (OK, {"ws": X, "path": 2}, "workspace must not alias x"),
])
def test_gated_refuses(lib, params, kw, fragment):
    p = G(*params)
    if "workspace" in fragment or "ws" in kw:
        if not lib.q2k_gated_ffn_workspace_bytes(kw.get("path", 0), ctypes.byref(p)):
            pytest.skip("this geometry takes no workspace")
    refused(lib, gated(lib, G(*params), **kw), fragment)


def test_gated_refuses_null_params(lib):
    assert lib.q2k_gated_ffn(0, 0, X, 1, W1, 1, W2, 1, H, 1, None, None, None, None, 0, None) == INVALID
    assert lib.q2k_gated_ffn_workspace_bytes(0, None) == 0


def backward(lib, p, **kw):
    a = dict(dh=X, gate=GATE, up=UP, he=p.m * p.n, wg=W1, wgb=_wb(p), wu=W2, wub=_wb(p), dx=H,
             dxe=p.m * p.k, dg=None, du=None, ws=WS, wsb=1 << 22)
    a.update(kw)
    return lib.q2k_gated_ffn_backward(a["dh"], a["gate"], a["up"], a["he"], a["wg"], a["wgb"],
                                      a["wu"], a["wub"], a["dx"], a["dxe"], a["dg"], a["du"],
                                      ctypes.byref(p), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("params,kw,fragment", [
    ((20, 8, 256, 10, 0, 0), {}, "bf16 activations only"),
    ((20, 8, 257, 10, 1, 0), {}, "multiple of 256"),
    (OK, {"dh": None}, "non-NULL"),
    (OK, {"dx": None}, "non-NULL"),
    (OK, {"dg": A}, "both be NULL"),
    (OK, {"he": 159}, "dh has 159"),
    (OK, {"dxe": 5121}, "dx has 5121"),
    (OK, {"wgb": 84}, "w_gate has 84"),
    (OK, {"dh": X + 4}, "16-byte aligned"),
    (OK, {"dg": A + 2, "du": B}, "16-byte aligned"),
    (OK, {"dx": GATE}, "dx must not alias gate"),
    (OK, {"dg": A, "du": A}, "dgate must not alias dup"),
    (OK, {"dg": X, "du": A}, "dgate must not alias dh"),
    (OK, {"ws": None}, "workspace is NULL"),
    (OK, {"wsb": 0}, "workspace has 0"),
])
def test_gated_backward_refuses(lib, params, kw, fragment):
    refused(lib, backward(lib, G(*params), **kw), fragment)


def lora(lib, p, path=0, flags=0, **kw):
    a = dict(x=X, xe=p.m * p.k, w=W1, wb=_wb(p), a=A, ae=p.n_adapters * p.rank * p.k, b=B,
             be=p.n_adapters * p.rank * p.n, s=SCALES, ids=IDS, y=H, ye=p.m * p.n, bad=BAD, ws=WS,
             wsb=1 << 22)
    a.update(kw)
    return lib.q2k_matmul_lora(path, flags, a["x"], a["xe"], a["w"], a["wb"], a["a"], a["ae"],
                               a["b"], a["be"], a["s"], a["ids"], a["y"], a["ye"], ctypes.byref(p),
                               a["bad"], a["ws"], a["wsb"], None)


LOK = (20, 8, 256, 10, 1, 8, 3, 0)


@pytest.mark.parametrize("params,kw,fragment", [
    ((0, 8, 256, 10, 1, 8, 3, 0), {}, ">= 1"),
    ((20, 8, 256, 10, 1, 0, 3, 0), {}, "rank = 0"),
    ((20, 8, 256, 10, 1, 12, 3, 0), {}, "rank = 12"),
    ((20, 8, 256, 10, 1, 264, 3, 0), {}, "rank = 264"),
    ((20, 8, 256, 10, 1, 8, 0, 0), {}, "n_adapters"),
    ((20, 8, 256, 10, 1, 8, 70000, 0), {}, "n_adapters"),
    ((20, 8, 256, 10, 1, 8, 3, 1), {}, "reserved"),
    (LOK, {"path": 9}, "unknown path"),
    (LOK, {"flags": 4}, "unknown flag bits"),
    (LOK, {"a": None}, "non-NULL"),
    (LOK, {"ids": None}, "non-NULL"),
    (LOK, {"ae": 3 * 8 * 256 + 1}, "a has 6145"),
    (LOK, {"be": 3 * 8 * 8 - 1}, "b has 191"),
    (LOK, {"ye": 1}, "y has 1"),
    (LOK, {"wb": 1}, "w has 1"),
    (LOK, {"b": B + 8}, "16-byte aligned"),
    (LOK, {"ids": IDS + 2}, "4-byte aligned"),
    (LOK, {"y": B}, "y must not alias b"),
    (LOK, {"bad": IDS}, "bad_id_count must not alias ids"),
    (LOK, {"bad": H}, "y must not alias bad_id_count"),
    (LOK, {"ws": None}, "workspace is NULL"),
    (LOK, {"wsb": 4}, "workspace has 4"),
])
def test_lora_refuses(lib, params, kw, fragment):
    refused(lib, lora(lib, L(*params), **kw), fragment)


def test_struct_layouts(lib):
    assert ctypes.sizeof(G) == 24 and ctypes.sizeof(L) == 32
    assert G.act.offset == 20 and L.reserved.offset == 28


def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(1, 256), torch.zeros(84, dtype=torch.uint8)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.gated_ffn(x, w, w, 1)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.gated_ffn_backward(x.bfloat16(), x, x, w, w, 256)
    with pytest.raises(TypeError, match="CUDA"):
        q2k.matmul_lora(x, w, 1, x, x, x)
