"""Every form that the 4-bit products and the expert layer take, by the sizes that choose it.

The choice goes by estimates, so it is pinned here without a GPU: a size that no longer takes the
form it stands for fails, and another has to stand in.  On the GPU each size runs against 64 bits with
the bounds of test_gpu_mx.py, with plain operands and with awkward ones: strided rows and scales that
start anywhere, an output without a scale, a row with a NaN and one with infinities, experts without
rows, rows without a token.
"""
import ctypes

import numpy as np
import pytest

import test_gpu_mx as T
from oracle import mx_ref as M
from post_weight_quantization_03_amd import gptq

torch = pytest.importorskip("torch")

FORMS = ["few", "32 x 128", "64 x 128", "64 x 64", "128 x 128", "256 x 256"]
KINDS = {"mx": 0, "bf16": 1, "f16": 2}


def form(m, n, k, x, experts=0):
    f = gptq.lib().gptq_internal_mxfp4_form
    f.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 4
    v = f(m, n, k, KINDS[x], experts)
    return FORMS[v & 7] + (" wide" if v & 8 else "") + (f" in {v >> 4 & 31}" if v >> 4 & 31 != 1 else "")


# form -> sizes (m, n, k) for each type of X; fp16 takes bf16's
DENSE = [
    ("few", "mx", (7, 1016, 4128)), ("few", "16", (3, 1016, 4128)),
    ("few wide", "mx", (9, 17000, 2080)), ("few wide", "16", (9, 17000, 2080)), ("few wide", "16", (5, 20011, 3104)),
    ("32 x 128", "16", (17, 16700, 1120)), ("32 x 128 in 4", "16", (19, 4150, 1568)),
    ("32 x 128 in 16", "16", (6, 1034, 6304)), ("32 x 128 in 8", "mx", (19, 4209, 7520)),
    ("64 x 64", "mx", (333, 1416, 2016)), ("64 x 64", "16", (333, 1416, 2016)), ("64 x 64 in 16", "mx", (24, 1000, 14336)),
    ("64 x 128", "16", (1027, 4096, 2080)), ("64 x 128 in 8", "16", (2159, 65, 3808)),
    ("128 x 128", "mx", (1027, 4096, 2080)), ("128 x 128", "16", (17789, 258, 1056)),
    ("256 x 256", "mx", (3600, 4180, 1056)), ("256 x 256", "16", (3600, 4180, 1056)), ("256 x 256", "16", (1990, 4050, 2112)),
]
# (rows, n, k, experts); rows in a range, of no token and behind the last range together
GROUPED = [
    ("few", "mx", (90, 200, 1056, 64)), ("few", "16", (61, 600, 2080, 8)),
    ("few wide", "mx", (30, 1400, 2080, 64)), ("few wide", "16", (96, 1400, 2080, 64)), ("few wide", "16", (384, 1400, 2080, 64)),
    ("32 x 128", "mx", (384, 1400, 2080, 64)), ("32 x 128", "mx", (1536, 1400, 2080, 64)), ("32 x 128", "16", (1536, 1400, 2080, 64)),
    ("64 x 64", "mx", (1000, 1400, 2080, 8)), ("64 x 64", "16", (1000, 1400, 2080, 8)),
    ("64 x 128", "16", (6144, 1400, 2080, 64)),
    ("128 x 128", "mx", (6144, 1400, 2080, 64)), ("128 x 128", "16", (14696, 279, 1120, 64)),
    ("256 x 256", "mx", (15331, 1841, 1056, 2)), ("256 x 256", "16", (15331, 1841, 1056, 2)),
]
# waves that share a tile's inputs in the two launches: tokens, choices, experts, d, inner
LAYERS = [
    ((1, 1), (32, 6, 64, 2048, 288)), ((2, 1), (64, 6, 64, 2048, 160)), ((2, 2), (16, 2, 8, 2048, 1056)),
    ((1, 1), (8, 6, 64, 2048, 416)), ((4, 4), (8, 2, 8, 1056, 512)), ((4, 1), (40, 3, 16, 4128, 64)),
    ((2, 4), (20, 2, 8, 1056, 1056)), ((1, 4), (24, 2, 4, 320, 4128)),
]


def spread(cases):
    return [(f, x, s) for f, types, s in cases for x in (["mx"] if types == "mx" else ["bf16", "f16"])]


@pytest.mark.parametrize("want,x,size", spread(DENSE) + spread(GROUPED))
def test_size_takes_its_form(want, x, size):
    assert form(*size[:3], x, *size[3:]) == want


def test_forms_that_all_types_of_rows_take_are_covered():
    for cases in (DENSE, GROUPED):
        for x in KINDS:
            have = {f.split(" in ")[0] for f, y, _ in spread(cases) if x == y}
            want = set(FORMS) | {"few wide"}
            assert have == (want - {"64 x 128"} if x == "mx" else want)      # never taken for 4-bit rows
    assert {w for pair, _ in LAYERS for w in enumerate(pair)} == {(h, w) for h in (0, 1) for w in (1, 2, 4)}


@pytest.mark.parametrize("want,size", LAYERS)
def test_layer_takes_its_form(want, size):
    tokens, k, experts, d, inner = size
    f = gptq.lib().gptq_internal_mxfp4_mlp_waves
    assert tuple(f(up, tokens * k, experts, d, inner) for up in (1, 0)) == want


# ------------------------------------------------------------------------------------ GPU


@pytest.fixture(autouse=True)
def announce(request):
    print(f"\n[gpu-case] {request.node.name}", flush=True)
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()


def wide(q, s):
    """Operands in 64 bits, a scale of 255 as NaN."""
    v = T.wide(q, s)
    return v if s is None else v.masked_fill((s == 255).repeat_interleave(32, -1), float("nan"))


def strided(q, s):
    """The same rows 32 bytes apart, and scales that start anywhere with rows of odd length."""
    raw = q.view(torch.uint8)
    store = torch.zeros(raw.shape[0], raw.shape[1] + 32, dtype=torch.uint8, device="cuda")
    store[:, 16:16 + raw.shape[1]] = raw
    q = store.view(q.dtype)[:, 16 // q.element_size():][:, :q.shape[1]]
    if s is not None:
        store = torch.full((s.shape[0], s.shape[1] + 4 + s.shape[1] % 2 + 1), 255, dtype=torch.uint8, device="cuda")
        store[:, 3:3 + s.shape[1]] = s
        s = store[:, 3:3 + s.shape[1]]
    return q, s


def spoil(q, s, ws):
    """A NaN in one row of X, infinities in another, and an output without a scale in the last expert."""
    ws[..., -1, ws.shape[-2] // 2, ws.shape[-1] - 1] = 255
    m = q.shape[0]
    if s is not None:
        s[m // 3, s.shape[1] - 1] = 255
    else:
        q[m // 3, q.shape[1] - 1] = float("nan")
        if m > 1:
            q[m - 1, 5], q[m - 1, q.shape[1] - 7] = float("inf"), float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("awkward", [False, True])
@pytest.mark.parametrize("want,x,size", spread(DENSE))
def test_products_of_every_form(want, x, size, awkward):
    m, n, k = size
    q, s = T.random_operand(m + n, m, k, x)
    w, ws = T.random_operand(n + k, n, k, "mx")
    if awkward:
        spoil(q, s, ws[None])
    vq, vs = strided(q, s) if awkward else (q, s)
    for out in ("bf16", "f32"):
        Y = T.lib().mxfp4_matmul(vq, w, ws, vs, out_dtype=T.DT[out])
        print("worst / bound", T.check_large(Y, wide(q, s), wide(w, ws), k, x, out), flush=True)
        assert torch.equal(torch.nan_to_num(Y, nan=3.0), torch.nan_to_num(T.lib().mxfp4_matmul(vq, w, ws, vs, out_dtype=T.DT[out]), nan=3.0))
        assert bool(Y.isnan().any()) == awkward


def ranges(total, experts, seed):
    """Offsets of ranges in `total` rows, three before the first and two behind the last; some experts are far more
    popular than others, and about one of five has no row."""
    rng = np.random.default_rng(seed)
    p = np.exp(0.7 * rng.standard_normal(experts)) * (rng.random(experts) > 0.2)
    p[-1] = 1.0
    return 3 + np.concatenate([[0], np.cumsum(rng.multinomial(total - 5, p / p.sum()))]).astype(np.int64)


def check_grouped(Y, offsets, rows, x, w, ws, k, kind, out):
    assert bool((Y[:3] == 2.5).all()) and bool((Y[int(offsets[-1]):] == 2.5).all())
    idx = T.cuda(rows.astype(np.int64))
    ok = (idx >= 0) & (idx < x.shape[0])
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            here = ok[lo:hi]
            assert bool((Y[lo:hi][~here] == 0).all())
            T.check_large(Y[lo:hi][here], x[idx[lo:hi][here]], wide(w[e], ws[e]), k, kind, out)


@pytest.mark.gpu
@pytest.mark.parametrize("awkward", [False, True])
@pytest.mark.parametrize("want,x,size", spread(GROUPED))
def test_grouped_products_of_every_form(want, x, size, awkward):
    total, n, k, experts = size
    tokens = total // 6 + 37
    q, s = T.random_operand(total + n, tokens, k, x)
    w, ws = T.random_operand(n + k, n, k, "mx", (experts,))
    offsets = ranges(total, experts, n)
    rows = np.random.default_rng(k).integers(0, tokens, total).astype(np.int32)
    rows[[4, total // 2, int(offsets[-1]) - 1]] = -1, tokens, -2 ** 31
    if awkward:
        spoil(q, s, ws)
    vq, vs = strided(q, s) if awkward else (q, s)
    for out in ("bf16", "f32"):
        Y = torch.full((total, n), 2.5, dtype=T.DT[out], device="cuda")
        T.lib().mxfp4_matmul_grouped(vq, w, ws, T.cuda(offsets), T.cuda(rows), vs, out_dtype=T.DT[out], out=Y)
        check_grouped(Y, offsets, rows, wide(q, s), w, ws, k, x, out)


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["mx", "bf16"])
def test_largest_tiles_of_rows_too_far_apart_for_them(x):
    # indexed rows of X over more than 2^31 bytes: the largest tiles' offsets do not reach, others take the product
    total, n, k, experts = 15331, 1841, 1056, 2
    assert form(total, n, k, x, experts) == "256 x 256"
    tokens, apart = 2600, 1 << 20
    q, s = T.random_operand(7, tokens, k, x)
    w, ws = T.random_operand(8, n, k, "mx", (experts,))
    size = q.element_size()
    far = torch.empty(tokens * (apart // size), dtype=q.dtype, device="cuda").as_strided(q.shape, (apart // size, 1))
    far.copy_(q)
    assert tokens * apart > 2 ** 31
    offsets = ranges(total, experts, 3)
    rows = np.random.default_rng(4).integers(0, tokens, total).astype(np.int32)
    Y = torch.full((total, n), 2.5, dtype=torch.bfloat16, device="cuda")
    T.lib().mxfp4_matmul_grouped(far, w, ws, T.cuda(offsets), T.cuda(rows), s, out=Y)
    check_grouped(Y, offsets, rows, wide(q, s), w, ws, k, x, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("x,size", [("mx", (646, 16553, 1088)), ("bf16", (1990, 4050, 2112))])
def test_largest_tiles_of_dense_rows_too_far_apart_for_them(x, size):
    m, n, k = size
    assert form(m, n, k, x) == "256 x 256"
    q, s = T.random_operand(9, m, k, x)
    w, ws = T.random_operand(10, n, k, "mx")
    apart = ((1 << 31) // 256 + 4096) // q.element_size()
    far = torch.empty(m * apart, dtype=q.dtype, device="cuda").as_strided(q.shape, (apart, 1))
    far.copy_(q)
    T.check_large(T.lib().mxfp4_matmul(far, w, ws, s), wide(q, s), wide(w, ws), k, x, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("want,size", LAYERS)
def test_layers_of_every_form(want, size, dtype):
    tokens, k, experts, d, inner = size
    rng = np.random.default_rng(tokens + inner)
    x, ids, p, w, xv, wv = T.layer(rng, tokens, k, experts, d, inner, dtype, spare=0.05)
    if tokens > 16:      # an expert that all tokens choose: more of them than fit at a time
        ids[:, 1:][ids[:, 1:] == 1] = -1
        ids[:, 0] = 1
    act = "silu" if dtype == "bf16" else "gelu_tanh"
    out = T.lib().mxfp4_moe_mlp(x, T.cuda(ids), T.cuda(p), *w, activation=act)
    print("worst / bound", T.check_layer(out, xv, ids, p, *wv, act, dtype), flush=True)
    for _ in range(3):
        assert torch.equal(out, T.lib().mxfp4_moe_mlp(x, T.cuda(ids), T.cuda(p), *w, activation=act))
