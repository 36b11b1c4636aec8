"""Arguments that the 4-bit microscaled calls refuse, without a GPU: the C ABI before any launch, the
binding before it calls the library."""
import pytest

from post_weight_quantization_03_amd import gptq

torch = pytest.importorskip("torch")
BAD, OK, WS, UNS = gptq.GPTQ_ERR_INVALID_ARG, gptq.GPTQ_OK, gptq.GPTQ_ERR_WORKSPACE, gptq.GPTQ_ERR_UNSUPPORTED
F32, BF16, F16, E4M3, E8M0, E2M1 = 0, 1, 2, 3, 4, 5


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(rows=-1), dict(cols=0), dict(cols=48), dict(xt=E4M3), dict(xt=E2M1), dict(X=None), dict(X=17),
    dict(xt=F32, X=18), dict(ldx=96), dict(scaling=2), dict(scaling=-1), dict(Q=None), dict(Q=8), dict(S=None),
    dict(batch=2, bsx=500)])
def test_quantize_refusals(change):
    a = dict(batch=1, rows=4, cols=128, xt=BF16, X=16, ldx=128, bsx=512, scaling=0, Q=16, S=16, stream=None)
    assert gptq.lib().gptq_mxfp4_quantize(*{**a, **change}.values()) == BAD
    if "rows" not in change:
        assert gptq.lib().gptq_mxfp4_quantize(*{**a, "rows": 0}.values()) == OK     # nothing to do


def test_quantize_and_dequantize_too_large():
    L = gptq.lib()
    assert L.gptq_mxfp4_quantize(1, 1 << 24, 2048, BF16, 16, 2048, 0, 0, 16, 16, None) == UNS
    assert L.gptq_mxfp4_quantize(65536, 1, 32, BF16, 16, 32, 32, 0, 16, 16, None) == UNS
    assert L.gptq_mxfp4_quantize(1, 1 << 31, 32, BF16, 16, 32, 0, 0, 16, 16, None) == UNS
    assert L.gptq_mxfp4_dequantize(1 << 24, 2048, 16, 16, BF16, 16, None) == UNS


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(cols=40), dict(Q=None), dict(Q=8), dict(S=None), dict(yt=E2M1), dict(yt=E8M0),
    dict(Y=None), dict(Y=8)])
def test_dequantize_refusals(change):
    a = dict(rows=4, cols=128, Q=16, S=3, yt=BF16, Y=16, stream=None)
    assert gptq.lib().gptq_mxfp4_dequantize(*{**a, **change}.values()) == BAD
    assert gptq.lib().gptq_mxfp4_dequantize(*{**a, "rows": 0}.values()) == OK


MATMUL = dict(m=4, n=64, k=128, xt=E2M1, X=16, ldx=64, xs=3, xsr=4, W=16, ws=3, yt=BF16, Y=16, ldy=64, wsp=None, wsb=0,
              stream=None)
SHARED = [dict(n=0), dict(k=0), dict(k=112), dict(xt=F32), dict(xt=E4M3), dict(X=None), dict(X=24), dict(ldx=48),
          dict(ldx=72), dict(xs=None), dict(xsr=3), dict(W=None), dict(W=8), dict(ws=None), dict(yt=E4M3), dict(Y=None),
          dict(Y=17), dict(ldy=63), dict(yt=F32, Y=18), dict(xt=BF16, ldx=120), dict(xt=F16, ldx=132)]


@pytest.mark.parametrize("change", [dict(m=-1), dict(wsp=8)] + SHARED)
def test_matmul_refusals(change):
    assert gptq.lib().gptq_mxfp4_matmul(*{**MATMUL, **change}.values()) == BAD


def test_matmul_workspace_and_empty():
    L = gptq.lib()
    assert L.gptq_mxfp4_matmul(*{**MATMUL, "m": 0, "X": None, "Y": None}.values()) == OK
    need = gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 4096, 14336, 64)      # shares the inputs among workgroups
    assert need > 256
    for xt, ldx in ((E2M1, 7168), (BF16, 14336), (F16, 14336)):
        a = {**MATMUL, "m": 64, "n": 4096, "k": 14336, "xt": xt, "ldx": ldx, "xsr": 448, "ldy": 4096}
        assert L.gptq_mxfp4_matmul(*a.values()) == WS
        assert L.gptq_mxfp4_matmul(*{**a, "wsp": 16, "wsb": 255}.values()) == WS
    assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 4096, 14336, 8192) > 256       # scales by stage
    assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 4096, 14336, 1) == 256
    assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 4096, 14336, 0) == 256
    for bad in ((2, 64, 128, 4), (1, 0, 128, 4), (1, 64, 100, 4), (1, 64, 128, -1)):
        assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, *bad) == 0


def test_a_workspace_for_more_rows_may_be_too_small_for_fewer():
    # sizes go by the kernel that m takes: the largest of them serves all, the last does not
    size = lambda m: gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 4096, 14336, m)
    assert size(1024) == 256 < size(128)
    a = {**MATMUL, "n": 4096, "k": 14336, "xt": BF16, "ldx": 14336, "ldy": 4096}
    assert gptq.lib().gptq_mxfp4_matmul(*{**a, "m": 128, "wsp": 16, "wsb": size(1024)}.values()) == WS
    assert gptq.lib().gptq_mxfp4_matmul(*{**a, "m": 128, "wsp": 16, "wsb": size(128) // 2 - 1}.values()) == WS


def test_too_many_tiles_are_refused():
    for xt, ldx in ((E2M1, 16), (BF16, 32), (F16, 32)):
        for m in (1 << 25, 1 << 40):
            a = {**MATMUL, "m": m, "n": 1 << 20, "k": 32, "xt": xt, "ldx": ldx, "ldy": 1 << 20}
            assert gptq.lib().gptq_mxfp4_matmul(*a.values()) == UNS


@pytest.mark.parametrize("rows", [(1 << 30) + 1, 1 << 62, (1 << 63) - 40, (1 << 63) - 1])
def test_rows_up_to_the_end_of_int64_are_refused(rows):
    L = gptq.lib()
    for xt, ldx in ((E2M1, 64), (BF16, 128), (F16, 128)):
        for n in (1, 64, 1 << 20):
            a = {**MATMUL, "m": rows, "n": n, "xt": xt, "ldx": ldx, "ldy": 1 << 20, "wsp": 16, "wsb": 1 << 62}
            assert L.gptq_mxfp4_matmul(*a.values()) == UNS
        for batch, idx in ((1, None), (2, 16), (1024, 16)):
            a = {**GROUPED, "batch": batch, "xr": rows, "rows": rows, "xt": xt, "ldx": ldx, "idx": idx, "wsp": 16, "wsb": 1 << 62}
            assert L.gptq_mxfp4_matmul_grouped(*a.values()) == UNS
    for cols in (32, 64, 4096):
        assert L.gptq_mxfp4_quantize(1, rows, cols, BF16, 16, cols, 0, 0, 16, 16, None) == UNS
        assert L.gptq_mxfp4_dequantize(rows, cols, 16, 16, BF16, 16, None) == UNS
    assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 64, 128, rows) == 256
    assert gptq.workspace_size(gptq.WS_MXFP4_GROUPED, 64, 64, 128, rows) == 256


GROUPED = dict(batch=2, xr=8, rows=5, n=64, k=128, xt=E2M1, X=16, ldx=64, xs=3, xsr=4, W=16, ws=3, off=16, idx=None,
               yt=BF16, Y=16, ldy=64, wsp=None, wsb=0, stream=None)


@pytest.mark.parametrize("change", [dict(batch=0), dict(xr=-1), dict(rows=-1), dict(off=None), dict(off=12), dict(idx=6),
                                    dict(xr=4)] + SHARED)
def test_grouped_refusals(change):
    assert gptq.lib().gptq_mxfp4_matmul_grouped(*{**GROUPED, **change}.values()) == BAD


def test_grouped_empty_and_too_large():
    assert gptq.lib().gptq_mxfp4_matmul_grouped(*{**GROUPED, "rows": 0}.values()) == OK
    a = {**GROUPED, "batch": 1 << 20, "xr": 1 << 16, "rows": 1 << 16}
    assert gptq.lib().gptq_mxfp4_matmul_grouped(*a.values()) == UNS
    need = gptq.workspace_size(gptq.WS_MXFP4_GROUPED, 4, 4096, 2048, 8192)
    a = {**GROUPED, "batch": 4, "xr": 8192, "rows": 8192, "n": 4096, "k": 2048, "ldx": 1024, "xsr": 64, "ldy": 4096}
    assert need > 256 and gptq.lib().gptq_mxfp4_matmul_grouped(*a.values()) == WS
    assert gptq.lib().gptq_mxfp4_matmul_grouped(*{**a, "wsp": 16, "wsb": need - 1}.values()) == WS
    assert gptq.workspace_size(gptq.WS_MXFP4_GROUPED, 4, 4096, 2048, 0) == 256
    assert gptq.workspace_size(gptq.WS_MXFP4_MATMUL, 1, 2 ** 31 - 1, 2048, 4) == 256     # refused by the call
    a = {**GROUPED, "n": 2 ** 31 - 1, "ldy": 2 ** 31}
    assert gptq.lib().gptq_mxfp4_matmul_grouped(*a.values()) == UNS
    for bad in ((0, 64, 128, 4), (2, 0, 128, 4), (2, 64, 100, 4), (2, 64, 128, -1)):
        assert gptq.workspace_size(gptq.WS_MXFP4_GROUPED, *bad) == 0


MLP = dict(tokens=4, k=2, experts=8, d=64, inner=96, xt=BF16, X=16, ldx=64, ids=16, w=16, W1=16, s1=16, W2=16, s2=16, act=0,
           out=16, ldo=64, wsp=16, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(k=0), dict(k=33), dict(experts=0), dict(experts=1025), dict(d=0), dict(d=80), dict(inner=0),
    dict(inner=48), dict(xt=F32), dict(xt=E2M1), dict(X=None), dict(X=24), dict(ldx=56), dict(ldx=68), dict(ids=None), dict(ids=18),
    dict(w=None), dict(w=18), dict(W1=None), dict(W1=8), dict(s1=None), dict(s1=8), dict(W2=None), dict(W2=8), dict(s2=None), dict(s2=4),
    dict(act=2), dict(act=-1), dict(out=None), dict(out=17), dict(ldo=63), dict(wsp=8)])
def test_mlp_refusals(change):
    assert gptq.lib().gptq_mxfp4_moe_mlp(*{**MLP, **change}.values()) == BAD


def test_mlp_limits_and_workspace():
    L = gptq.lib()
    assert L.gptq_mxfp4_moe_mlp(*{**MLP, "tokens": 0, "X": None}.values()) == OK
    assert L.gptq_mxfp4_moe_mlp(*{**MLP, "tokens": 2049}.values()) == UNS
    assert L.gptq_mxfp4_moe_mlp(*{**MLP, "tokens": 1 << 40}.values()) == UNS
    need = gptq.workspace_size(gptq.WS_MXFP4_MOE_MLP, 1, 96, 64, 8)
    assert need >= 8 * 96 * 4
    assert L.gptq_mxfp4_moe_mlp(*{**MLP, "wsb": need - 1}.values()) == WS
    assert L.gptq_mxfp4_moe_mlp(*{**MLP, "wsp": None}.values()) == WS
    for bad in ((1, 48, 64, 8), (1, 96, 64, -1), (1, 96, 64, 4097)):
        assert gptq.workspace_size(gptq.WS_MXFP4_MOE_MLP, *bad) == 0


def refused(kind, fn, *a, **kw):
    with pytest.raises(kind):
        fn(*a, **kw)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    refused(ValueError, gptq.mxfp4_quantize, x)                                   # not on a GPU
    refused(TypeError, gptq.mxfp4_quantize, x.double())
    refused(ValueError, gptq.mxfp4_quantize, x, "even")
    refused(ValueError, gptq.mxfp4_quantize, x[0])
    refused(ValueError, gptq.mxfp4_quantize, x[:, :48])
    refused(ValueError, gptq.mxfp4_quantize, torch.zeros(64, 64).t()[:, ::2])
    refused(ValueError, gptq.mxfp4_dequantize, q, s)                              # not on a GPU
    refused(TypeError, gptq.mxfp4_dequantize, q.int(), s)
    refused(TypeError, gptq.mxfp4_dequantize, q, s.float())
    refused(TypeError, gptq.mxfp4_dequantize, q, s, torch.float64)
    refused(ValueError, gptq.mxfp4_dequantize, q, s[:, :1])
    refused(ValueError, gptq.mxfp4_dequantize, q[:, :24], s)
    refused(ValueError, gptq.mxfp4_dequantize, q[::2], s[::2])
    mm = gptq.mxfp4_matmul
    refused(ValueError, mm, x, q, s)                                              # not on a GPU
    refused(TypeError, mm, x.float(), q, s)
    refused(TypeError, mm, x, q.int(), s)
    refused(TypeError, mm, x, q, s.float())
    refused(TypeError, mm, x, q, s, out_dtype=torch.float64)
    refused(TypeError, mm, x, q, s, s[:4])                                        # 16-bit X has no scales
    refused(ValueError, mm, x[:, :32], q, s)
    refused(ValueError, mm, x, q[0], s[0])
    refused(ValueError, mm, x, q, s[:8])
    refused(ValueError, mm, x, q.t(), s)
    refused(ValueError, mm, x.t(), q, s)
    refused(ValueError, mm, q[:4], q, s, s[:3])
    refused(ValueError, mm, q[:4], q, s, s[:1].expand(4, 2))
    refused(TypeError, mm, q[:4], q, s)                                           # codes without scales
    refused(ValueError, mm, x, q, s, out=torch.zeros(4, 15, dtype=torch.bfloat16))
    gm, off = gptq.mxfp4_matmul_grouped, torch.zeros(3, dtype=torch.int64)
    W, WS3 = q.view(2, 8, 32), s.view(2, 8, 2)
    refused(ValueError, gm, x, W, WS3, off)                                       # not on a GPU
    refused(ValueError, gm, x, q, s, off)
    refused(ValueError, gm, x, W, WS3, off[:2])
    refused(ValueError, gm, x, W, WS3, off.int())
    refused(ValueError, gm, x, W, WS3, off, torch.zeros(4, dtype=torch.int64))
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w1, s1 = torch.zeros(3, 64, 32, dtype=torch.uint8), torch.zeros(3, 64, 2, dtype=torch.uint8)
    w2, s2 = torch.zeros(3, 64, 16, dtype=torch.uint8), torch.zeros(3, 64, 1, dtype=torch.uint8)
    mlp = gptq.mxfp4_moe_mlp
    refused(ValueError, mlp, x, ids, w, w1, s1, w2, s2)                           # not on a GPU
    refused(TypeError, mlp, x.float(), ids, w, w1, s1, w2, s2)
    refused(TypeError, mlp, x, ids.long(), w, w1, s1, w2, s2)
    refused(TypeError, mlp, x, ids, w.half(), w1, s1, w2, s2)
    refused(TypeError, mlp, x, ids, w, w1.int(), s1, w2, s2)
    refused(ValueError, mlp, x, ids, w, w1, s1, w2, s2, "relu")
    refused(ValueError, mlp, x, ids[:3], w[:3], w1, s1, w2, s2)
    refused(ValueError, mlp, x, ids, w[:3], w1, s1, w2, s2)
    refused(ValueError, mlp, x, ids.t().contiguous().t(), w, w1, s1, w2, s2)
    refused(ValueError, mlp, x[:, :32], ids, w, w1, s1, w2, s2)
    refused(ValueError, mlp, x, ids, w, w1[:2], s1[:2], w2, s2)
    refused(ValueError, mlp, x, ids, w, w1[:, :32], s1[:, :32], w2, s2)
    refused(ValueError, mlp, x, ids, w, w1, s1, w2[:, :32], s2[:, :32])
    refused(ValueError, mlp, x, ids, w, w1[0], s1[0], w2, s2)
    refused(ValueError, mlp, x, torch.zeros(4, 33, dtype=torch.int32), torch.zeros(4, 33), w1, s1, w2, s2)
    refused(ValueError, mlp, x, ids, w, w1, s1, w2, s2, out=torch.zeros(4, 63, dtype=torch.bfloat16))
    long = torch.zeros(5000, 64, dtype=torch.bfloat16)
    refused(ValueError, mlp, long, torch.zeros(5000, 1, dtype=torch.int32), torch.zeros(5000, 1), w1, s1, w2, s2)
