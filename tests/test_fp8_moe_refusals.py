"""Arguments that the 8-bit and routing calls refuse, without a GPU: the C ABI before any
launch, the binding before it calls the library."""
import ctypes

import pytest

from post_weight_quantization_03_amd import gptq

torch = pytest.importorskip("torch")
BAD, OK, WS = gptq.GPTQ_ERR_INVALID_ARG, gptq.GPTQ_OK, gptq.GPTQ_ERR_WORKSPACE
F32, BF16, F16, E4M3, E8M0 = 0, 1, 2, 3, 4


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(rows=-1), dict(cols=0), dict(cols=24), dict(xt=E4M3), dict(xt=7), dict(X=None), dict(X=17),
    dict(ldx=112), dict(br=64), dict(st=BF16), dict(Q=None), dict(Q=8), dict(S=None), dict(S=18), dict(lsr=0),
    dict(lsb=0), dict(batch=2, bsx=100), dict(batch=2, bss=0)])
def test_quantize_refusals(change):
    a = dict(batch=1, rows=4, cols=128, xt=BF16, X=16, ldx=128, bsx=512, br=1, st=F32, Q=16, S=16, lsr=1, lsb=4,
             bss=4, stream=None)
    assert gptq.lib().gptq_fp8_quantize(*{**a, **change}.values()) == BAD
    if "rows" not in change:
        assert gptq.lib().gptq_fp8_quantize(*{**a, "rows": 0}.values()) == OK     # nothing to do


MATMUL = dict(m=4, n=64, k=128, xt=E4M3, X=16, ldx=128, st=F32, xs=16, xsr=1, xsb=4, W=16, ws=16, yt=BF16, Y=16,
              ldy=64, wsp=None, wsb=0, stream=None)


@pytest.mark.parametrize("change", [
    dict(m=-1), dict(n=0), dict(k=0), dict(k=120), dict(xt=F32), dict(xt=E8M0), dict(X=None), dict(X=24),
    dict(ldx=112), dict(ldx=136), dict(st=BF16), dict(xs=None), dict(xs=18), dict(xsr=0), dict(xsb=0), dict(W=None),
    dict(W=8), dict(ws=None), dict(ws=2), dict(yt=E4M3), dict(Y=None), dict(Y=17), dict(ldy=63),
    dict(yt=F32, Y=18), dict(xt=BF16, X=17), dict(xt=BF16, wsp=8)])
def test_matmul_refusals(change):
    assert gptq.lib().gptq_fp8_matmul(*{**MATMUL, **change}.values()) == BAD


def test_matmul_workspace_and_empty():
    L = gptq.lib()
    for x in (BF16, F16):
        need = gptq.workspace_size(gptq.WS_FP8_MATMUL, 1, 64, 128, 4)
        assert need >= 4 * 128 + 4 * 4
        assert L.gptq_fp8_matmul(*{**MATMUL, "xt": x, "wsp": 16, "wsb": need - 1}.values()) == WS
        assert L.gptq_fp8_matmul(*{**MATMUL, "xt": x}.values()) == WS
    assert L.gptq_fp8_matmul(*{**MATMUL, "m": 0, "X": None, "xs": None}.values()) == OK
    for args in ((0, 64, 128, 4), (1, 0, 128, 4), (1, 64, 120, 4), (1, 64, 128, -1)):
        assert gptq.workspace_size(gptq.WS_FP8_GROUPED, *args) == 0
    assert gptq.workspace_size(gptq.WS_FP8_GROUPED, 8, 64, 128, 0) > 0


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(xr=-1), dict(rows=-1), dict(off=None), dict(off=12), dict(idx=18), dict(W=None), dict(X=None),
    dict(ldx=120), dict(ldy=8), dict(k=24)])
def test_grouped_refusals(change):
    a = dict(batch=2, xr=4, rows=8, n=64, k=128, xt=E4M3, X=16, ldx=128, st=F32, xs=16, xsr=1, xsb=4, W=16, ws=16,
             off=16, idx=16, yt=BF16, Y=16, ldy=64, wsp=None, wsb=0, stream=None)
    assert gptq.lib().gptq_fp8_matmul_grouped(*{**a, **change}.values()) == BAD
    assert gptq.lib().gptq_fp8_matmul_grouped(*{**a, "rows": 0}.values()) == OK


@pytest.mark.parametrize("change", [
    dict(t=-1), dict(e=0), dict(e=1025), dict(lt=E4M3), dict(l=None), dict(l=18), dict(ldl=60), dict(b=18),
    dict(ids=None), dict(ids=18), dict(w=None), dict(w=18), dict(scoring=2), dict(n_groups=0), dict(n_groups=5),
    dict(n_groups=128), dict(top_groups=0), dict(top_groups=9), dict(group_score=2), dict(top_k=0), dict(top_k=33),
    dict(top_k=17, top_groups=2), dict(scale=float("inf")), dict(scale=float("nan"))])
def test_route_refusals(change):
    p = dict(scoring=0, n_groups=8, top_groups=8, group_score=0, top_k=6, renormalize=1, scale=1.0)
    a = dict(t=4, e=64, lt=F32, l=16, ldl=64, b=None, p=None, ids=16, w=16, stream=None)
    for k, v in change.items():
        (p if k in p else a)[k] = v
    a["p"] = ctypes.byref(gptq._RouteParams(*p.values()))
    assert gptq.lib().gptq_moe_route(*a.values()) == BAD
    a["p"] = None
    assert gptq.lib().gptq_moe_route(*a.values()) == BAD


@pytest.mark.parametrize("change", [
    dict(t=-1), dict(k=0), dict(e=0), dict(e=1025), dict(t=2 ** 30, k=2), dict(ids=None), dict(off=None),
    dict(off=12), dict(rows=None), dict(place=None), dict(ids=18), dict(wsp=8)])
def test_group_refusals(change):
    a = dict(t=4, k=2, e=8, ids=16, off=16, rows=16, place=16, wsp=None, wsb=0, stream=None)
    assert gptq.lib().gptq_moe_group_tokens(*{**a, **change}.values()) == BAD


def test_group_workspace():
    assert gptq.lib().gptq_moe_group_tokens(40000, 8, 64, 16, 16, 16, 16, None, 0, None) == WS
    assert gptq.workspace_size(gptq.WS_MOE_GROUP, 1, 64, 8, 40000) > 256
    assert gptq.workspace_size(gptq.WS_MOE_GROUP, 1, 2000, 8, 40) == 0
    assert gptq.workspace_size(gptq.WS_MOE_GROUP, 1, 64, 0, 40) == 0
    assert gptq.workspace_size(gptq.WS_MOE_GROUP, 1, 64, 8, 2 ** 40) == 0


@pytest.mark.parametrize("change", [
    dict(t=-1), dict(k=0), dict(rows=-1), dict(d=0), dict(yt=E4M3), dict(Y=None), dict(Y=17), dict(ldy=60),
    dict(place=None), dict(place=18), dict(w=None), dict(w=18), dict(out=None), dict(out=17), dict(ldo=60)])
def test_combine_refusals(change):
    a = dict(t=4, k=2, rows=8, d=64, yt=BF16, Y=16, ldy=64, place=16, w=16, out=16, ldo=64, stream=None)
    assert gptq.lib().gptq_moe_combine(*{**a, **change}.values()) == BAD


def refused(error, call, *args, **kw):
    with pytest.raises(error):
        call(*args, **kw)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x, f8 = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(64, 128).to(torch.float8_e4m3fn)
    s, x8 = torch.ones(1, 1), torch.zeros(4, 128).to(torch.float8_e4m3fn)
    refused(ValueError, gptq.fp8_quantize, x)                                     # not on a GPU
    refused(TypeError, gptq.fp8_quantize, x.to(torch.int32))
    refused(TypeError, gptq.fp8_quantize, x, 1, torch.float16)
    refused(ValueError, gptq.fp8_quantize, x, 64)
    refused(ValueError, gptq.fp8_quantize, x[:, :100])
    refused(ValueError, gptq.fp8_quantize, x.t())
    refused(ValueError, gptq.fp8_quantize, x[0])
    refused(ValueError, gptq.fp8_matmul, x, f8, s)                                # not on a GPU
    refused(TypeError, gptq.fp8_matmul, x.float(), f8, s)
    refused(TypeError, gptq.fp8_matmul, x, f8.float(), s)
    refused(TypeError, gptq.fp8_matmul, x, f8, s.half())
    refused(TypeError, gptq.fp8_matmul, x, f8, s, out_dtype=torch.float64)
    refused(TypeError, gptq.fp8_matmul, x, f8, s, torch.ones(4, 1))               # scales of 16-bit rows
    refused(TypeError, gptq.fp8_matmul, x8, f8, s)                                # 8-bit rows without scales
    refused(TypeError, gptq.fp8_matmul, x8, f8, s, torch.ones(4, 1).to(torch.float8_e8m0fnu))
    refused(ValueError, gptq.fp8_matmul, x8, f8, s, torch.ones(3, 1))
    refused(ValueError, gptq.fp8_matmul, x8, f8, s, torch.ones(1, 1).expand(4, 1))
    refused(ValueError, gptq.fp8_matmul, x[:, :64], f8, s)
    refused(ValueError, gptq.fp8_matmul, x, f8, torch.ones(2, 1))
    refused(ValueError, gptq.fp8_matmul, x, f8[None], s[None])
    refused(ValueError, gptq.fp8_matmul, x, f8, s, out=torch.zeros(4, 65, dtype=torch.bfloat16))
    refused(ValueError, gptq.fp8_matmul, x, f8, s, out=torch.zeros(4, 64))
    refused(ValueError, gptq.fp8_matmul, x, f8, s, out=torch.zeros(1, 64, dtype=torch.bfloat16).expand(4, 64))
    off = torch.zeros(2, dtype=torch.int64)
    refused(ValueError, gptq.fp8_matmul_grouped, x, f8[None], s[None], off)       # not on a GPU
    refused(ValueError, gptq.fp8_matmul_grouped, x, f8, s, off)
    refused(ValueError, gptq.fp8_matmul_grouped, x, f8[None], s[None], off.int())
    refused(ValueError, gptq.fp8_matmul_grouped, x, f8[None], s[None], torch.zeros(3, dtype=torch.int64))
    refused(ValueError, gptq.fp8_matmul_grouped, x, f8[None], s[None], off, torch.zeros(3, dtype=torch.int64))


def test_binding_refuses_bad_routing_arguments():
    l, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    refused(ValueError, gptq.moe_route, l, 2)                                     # not on a GPU
    refused(TypeError, gptq.moe_route, l.double(), 2)
    refused(TypeError, gptq.moe_route, l, 2, torch.zeros(8).half())
    refused(ValueError, gptq.moe_route, l, 2, torch.zeros(7))
    refused(ValueError, gptq.moe_route, l, 2, scoring="relu")
    refused(ValueError, gptq.moe_route, l, 2, group_score="mean")
    refused(ValueError, gptq.moe_route, l.t(), 2)
    refused(ValueError, gptq.moe_route, l[0], 2)
    refused(ValueError, gptq.moe_group_tokens, ids, 8)                            # not on a GPU
    refused(TypeError, gptq.moe_group_tokens, ids.long(), 8)
    refused(ValueError, gptq.moe_group_tokens, ids, 0)
    refused(ValueError, gptq.moe_group_tokens, ids, 1025)
    refused(ValueError, gptq.moe_group_tokens, ids.t(), 8)
    y, w = torch.zeros(8, 16), torch.zeros(4, 2)
    refused(ValueError, gptq.moe_combine, y, ids, w)                              # not on a GPU
    refused(TypeError, gptq.moe_combine, y.double(), ids, w)
    refused(TypeError, gptq.moe_combine, y, ids.long(), w)
    refused(TypeError, gptq.moe_combine, y, ids, w.half())
    refused(ValueError, gptq.moe_combine, y, ids, w[:3])
    refused(ValueError, gptq.moe_combine, y.t(), ids, w)
    refused(ValueError, gptq.moe_combine, y, ids, w, out=torch.zeros(4, 15))


def test_grouped_rows_past_the_activations():
    # without an index output row p reads row p of X
    a = dict(batch=2, xr=4, rows=5, n=64, k=128, xt=E4M3, X=16, ldx=128, st=F32, xs=16, xsr=1, xsb=4, W=16, ws=16,
             off=16, idx=None, yt=BF16, Y=16, ldy=64, wsp=None, wsb=0, stream=None)
    assert gptq.lib().gptq_fp8_matmul_grouped(*a.values()) == BAD
    assert gptq.lib().gptq_fp8_matmul_grouped(*{**a, "xr": 2 ** 31, "rows": 2 ** 31 + 1}.values()) == BAD


def test_binding_refuses_a_workspace_with_less_memory_than_elements():
    ws = torch.empty(1, dtype=torch.uint8).expand(1 << 24)
    q, s = torch.empty(64, 128, dtype=torch.float8_e4m3fn), torch.empty(1, 1)
    with pytest.raises(ValueError, match="workspace"):
        gptq.fp8_matmul(torch.empty(4, 128, dtype=torch.bfloat16), q, s, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        gptq.moe_group_tokens(torch.zeros(20000, 2, dtype=torch.int32), 8, workspace=ws)


def test_group_workspace_tells_whether_it_is_used():
    # 256 bytes mean that the call keeps nothing there: the binding then passes none
    for experts in (1, 2, 3, 4, 7, 8, 63, 64, 1024):
        for slots in (0, 1, 8192):
            assert gptq.workspace_size(gptq.WS_MOE_GROUP, 1, experts, 1, slots) == 256
        for slots in (8193, 9216, 16384, 32768, 2 ** 31 - 1):
            need = gptq.workspace_size(gptq.WS_MOE_GROUP, 1, experts, 1, slots)
            assert need > 256
            assert gptq.lib().gptq_moe_group_tokens(slots, 1, experts, 16, 16, 16, 16, None, 0, None) == WS
            assert gptq.lib().gptq_moe_group_tokens(slots, 1, experts, 16, 16, 16, 16, 16, need - 1, None) == WS


def test_too_many_tiles_are_refused_before_anything_is_enqueued():
    # 16-bit rows are rounded by a launch of its own: without a GPU it would fail with another error
    UNS, big = gptq.GPTQ_ERR_UNSUPPORTED, 1 << 62
    for x, y in ((E4M3, BF16), (BF16, BF16), (F16, F32)):
        for m in (1 << 25, 1 << 40):
            a = {**MATMUL, "m": m, "n": 1 << 20, "k": 16, "ldx": 16, "xt": x, "yt": y, "ldy": 1 << 20, "wsp": 16, "wsb": big}
            assert gptq.lib().gptq_fp8_matmul(*a.values()) == UNS
    a = dict(batch=1024, xr=1 << 20, rows=1 << 20, n=1 << 24, k=16, xt=BF16, X=16, ldx=16, st=F32, xs=None, xsr=0,
             xsb=0, W=16, ws=16, off=16, idx=None, yt=BF16, Y=16, ldy=1 << 24, wsp=16, wsb=big, stream=None)
    assert gptq.lib().gptq_fp8_matmul_grouped(*a.values()) == UNS
