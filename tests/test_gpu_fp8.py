"""8-bit numbers on the GPU: codes and scales bit for bit, products element by element against float64.

A product's bound: every e4m3 x e4m3 product is exact in fp32, so what is left are the additions of d_in terms, each
off by at most one step (the matrix unit may cut where fp32 rounds), 2^-23 of a partial sum below sum |x| |w|, and
half a step of the output's type (relative, or of its smallest number).  For 16-bit outputs the unit's 8-bit products
come on top: of eight consecutive ones, seven are off by less than 2^-13 of the largest."""
import numpy as np
import pytest

from oracle import fp8 as F
from tests import answer_data as D
from tests.gpu_run import log

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def values(rows, cols, dtype, seed, spread=1.0):
    """Rows and columns of different sizes, some zero."""
    r = np.random.default_rng([51, seed])
    x = r.standard_normal((rows, cols)) * np.exp(spread * r.standard_normal((rows, 1)))
    x *= np.exp(spread * r.standard_normal((1, cols)))
    x[:, r.random(cols) < 0.05] = 0
    return D.store(x, dtype)


def place(xs, dtype, ld=None, offset=0):
    """The rows in a buffer with row stride ld, `offset` elements in."""
    import torch
    x = D.to_torch(xs, dtype)
    n, w = x.shape
    ld = ld or w
    buf = torch.full((offset + n * ld,), 77.0, dtype=x.dtype, device="cuda")
    view = buf.as_strided((n, w), (ld, 1), offset)
    view.copy_(x)
    return view


def bytes_of(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def codes_to_torch(codes):
    import torch
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)


def scales_to_torch(b):
    import torch
    return torch.from_numpy(b).cuda().view(torch.float8_e8m0fnu)


# (rows, columns, type, tiles, row stride or None, first element): one element, ends inside a block of lanes and a
# block, rows that start anywhere, several workgroups
QUANT = [
    (1, 1, "f32", False, None, 0), (1, 7, "f16", False, None, 1), (3, 127, "bf16", False, 129, 3),
    (5, 128, "f32", False, None, 0), (2, 129, "bf16", False, None, 0), (37, 1000, "f16", False, 1001, 5),
    (300, 2056, "bf16", False, None, 0), (129, 4100, "f32", False, 4101, 1), (1000, 135, "f16", False, None, 0),
    (1, 1, "bf16", True, None, 0), (7, 130, "f32", True, 133, 1), (128, 128, "f16", True, None, 0),
    (129, 127, "bf16", True, 129, 1), (200, 1000, "f32", True, None, 0), (513, 520, "f16", True, 521, 3),
    (1000, 2048, "bf16", True, None, 0),
]


@pytest.mark.parametrize("rows,cols,dtype,tiles,ld,offset", QUANT)
def test_codes_and_scales(rows, cols, dtype, tiles, ld, offset):
    from post_weight_quantization_08_amd import pipeline as P
    xs = values(rows, cols, dtype, rows + cols, 2.0 if dtype != "f16" else 1.0)
    out = P.fp8_quantize(place(xs, dtype, ld, offset), tiles=tiles)
    codes, b = F.fp8_quantize(D.exact(xs, dtype), tiles)
    np.testing.assert_array_equal(bytes_of(out["scales"]), b)
    got = bytes_of(out["codes"])
    assert got.shape == codes.shape
    np.testing.assert_array_equal(got, codes)
    if tiles:
        turned = np.zeros((cols, -(-rows // 128) * 128), dtype=np.uint8)
        turned[:, :rows] = codes[:, :cols].T
        np.testing.assert_array_equal(bytes_of(out["codes_t"]), turned)
        np.testing.assert_array_equal(bytes_of(out["scales_t"]), b.T)


@pytest.mark.parametrize("tiles", [False, True])
def test_borders_of_blocks(tiles):
    """Ties, the largest code and the step above it, zeros, subnormal and huge numbers, NaN and infinities."""
    from post_weight_quantization_08_amd import pipeline as P
    x = np.zeros((260, 128), dtype=np.float32)
    x[0, :4] = [448, 17, 19, -17]
    x[1, :3] = [np.nextafter(np.float32(448), np.float32(500)), 447, 432]
    x[2, :3] = [1.75, 1.7500001, 2.0 ** -12]
    x[3, 0] = 3.4028235e38
    x[4, :2] = [2.0 ** -140, 2.0 ** -149]
    x[5, :2] = [2.0 ** -92, 2.0 ** -101]
    x[6, :2] = [-0.0, 1]
    if not tiles:
        x[7, 5], x[8, 5], x[9, 5] = np.nan, np.inf, -np.inf
    else:
        x[130, 5], x[259, 5] = -np.inf, np.nan
    out = P.fp8_quantize(place(x, "f32"), tiles=tiles)
    codes, b = F.fp8_quantize(x.astype(np.float64), tiles)
    np.testing.assert_array_equal(bytes_of(out["scales"]), b)
    np.testing.assert_array_equal(bytes_of(out["codes"]), codes)


def test_given_outputs_keep_what_is_around_them():
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    xs = values(70, 300, "bf16", 3)
    buf = torch.full((72, 448), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((70, 3), 9, dtype=torch.uint8, device="cuda")
    out = {"codes": buf.view(torch.float8_e4m3fn)[1:71, 16:400], "scales": scales.view(torch.float8_e8m0fnu)}
    P.fp8_quantize(place(xs, "bf16"), out=out)
    codes, b = F.fp8_quantize(D.exact(xs, "bf16"))
    whole = np.full((72, 448), 9, dtype=np.uint8)
    whole[1:71, 16:400] = codes
    np.testing.assert_array_equal(buf.cpu().numpy(), whole)
    np.testing.assert_array_equal(scales.cpu().numpy(), b)
    # tiles without the transpose
    t = {"codes": torch.empty(70, 384, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
         "scales": torch.empty(1, 3, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)}
    P.fp8_quantize(place(xs, "bf16"), tiles=True, out=t)
    codes, b = F.fp8_quantize(D.exact(xs, "bf16"), True)
    np.testing.assert_array_equal(bytes_of(t["codes"]), codes)
    np.testing.assert_array_equal(bytes_of(t["scales"]), b)


def operands(M, d_in, d_out, seed):
    W = values(d_out, d_in, "f32", seed + 1, 0.7).astype(np.float64) / np.sqrt(d_in)
    wc, wb = F.fp8_quantize(W, tiles=True)
    return wc, wb, F.fp8_values(wc, wb, tiles=True)


def check(got, x, w, dtype, what):
    want = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    bound = x.shape[1] * 2.0 ** -23 * size
    if dtype != "f32":
        some = np.linspace(0, x.shape[0] - 1, min(x.shape[0], 100)).astype(int)   # these tokens' bound takes time
        got, want, x = got[some], want[some], x[some]
        bound = bound[some]
        wa = np.abs(w)
        for m in range(len(x)):
            p = wa * np.abs(x[m])
            eights = np.pad(p, ((0, 0), (0, -p.shape[1] % 8))).reshape(p.shape[0], -1, 8)
            bound[m] += 7 * 2.0 ** -13 * eights.max(2).sum(1)
    bound += (np.abs(want) + bound) * HALF[dtype] + LEAST[dtype]
    bad = np.abs(got - want) > bound
    assert np.array_equal(np.isnan(got), np.isnan(want)) and not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
    log(f"[gpu] fp8 product {what}: error in norm {rel:.2e}")
    return rel


# (M, d_in, d_out, x, y, stride of x, stride of y, first element): one token to several tiles of every kernel, sums
# that end inside a block, few blocks and split sums, outputs that end inside four, a tile of 128 and a tile of 256
MATMUL = [
    (1, 1, 1, "f32", "f32", None, None, 0), (1, 128, 16, "e4m3", "f32", None, None, 0),
    (1, 4096, 300, "f16", "f16", None, None, 0), (2, 1000, 257, "bf16", "bf16", 1003, 260, 1),
    (16, 2048, 130, "f32", "f32", 2049, 131, 1), (15, 1152, 64, "e4m3", "bf16", 1168, None, 0),
    (17, 640, 200, "f16", "f32", None, None, 0), (32, 3200, 100, "e4m3", "f16", None, 103, 1),
    (33, 130, 515, "bf16", "bf16", 131, None, 1), (48, 2176, 1000, "bf16", "bf16", None, None, 0),
    (64, 100, 129, "f32", "f32", None, None, 0), (64, 1280, 48, "e4m3", "f32", None, None, 0),
    (65, 384, 130, "bf16", "f32", None, None, 0), (100, 8200, 260, "f16", "bf16", 8201, 263, 3),
    (129, 128, 127, "e4m3", "f32", None, None, 0), (200, 2100, 700, "f32", "f16", None, 701, 1),
    (300, 4224, 129, "e4m3", "bf16", 4240, None, 0), (777, 1100, 401, "f32", "f32", None, None, 0),
    (4100, 256, 4099, "e4m3", "bf16", None, None, 0), (4097, 300, 4001, "bf16", "f32", None, 4003, 1),
]


@pytest.mark.parametrize("M,d_in,d_out,xt,yt,ld_x,ld_y,offset", MATMUL)
def test_products(M, d_in, d_out, xt, yt, ld_x, ld_y, offset):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    wc, wb, w = operands(M, d_in, d_out, M)
    if xt == "e4m3":
        xc, xb = F.fp8_quantize(values(M, d_in, "f32", M, 0.7).astype(np.float64))
        buf = torch.zeros(M, ld_x or d_in, dtype=torch.uint8, device="cuda")
        buf[:, :d_in] = torch.from_numpy(xc).cuda()
        X, xs = buf.view(torch.float8_e4m3fn)[:, :d_in], scales_to_torch(xb)
    else:
        stored = values(M, d_in, xt, M, 0.7)
        xc, xb = F.fp8_quantize(D.exact(stored, xt))
        X, xs = place(stored, xt, ld_x, offset), None
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[yt]
    ld_y = ld_y or d_out
    buf = torch.full((offset + M * ld_y + 5,), 7.0, dtype=dt, device="cuda")
    Y = buf.as_strided((M, d_out), (ld_y, 1), offset)
    P.fp8_matmul(X, codes_to_torch(wc), scales_to_torch(wb), x_scales=xs, Y=Y)
    torch.cuda.synchronize()
    got = Y.double().cpu().numpy()
    check(got, F.fp8_values(xc, xb), w, yt, f"{M}x{d_in}x{d_out} {xt}->{yt}")
    around = torch.ones_like(buf, dtype=torch.bool)
    around.as_strided((M, d_out), (ld_y, 1), offset).fill_(False)
    assert bool((buf[around] == 7.0).all())              # nothing beside the outputs is written


@pytest.mark.parametrize("M", [3, 40, 150, 2100])
def test_every_way_to_hand_in_x_gives_the_same_bits(M):
    """Values quantized in the call, and their codes from fp8_quantize, on every kernel."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    d_in, d_out = 1111, 8200 if M > 1000 else 333
    wc, wb, _ = operands(M, d_in, d_out, 5)
    W, ws = codes_to_torch(wc), scales_to_torch(wb)
    X = place(values(M, d_in, "bf16", 6), "bf16")
    q = P.fp8_quantize(X)
    a, b = P.fp8_matmul(X, W, ws), P.fp8_matmul(q["codes"], W, ws, x_scales=q["scales"])
    assert torch.equal(a, b)
    assert torch.equal(P.fp8_matmul(X.float(), W, ws), a)
    assert torch.equal(P.fp8_matmul(X, W, ws), a)        # and again


@pytest.mark.parametrize("M,d_out", [(5, 40), (40, 300), (130, 200), (2100, 8200)])
def test_nan_stays_in_its_row(M, d_out):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    d_in = 400
    xs = values(M, d_in, "f32", 9)
    xs[1, 7], xs[M - 2, 300] = np.nan, np.inf
    wc, wb, w = operands(M, d_in, d_out, 5)
    wc[d_out - 1, 3] = 0x7F                               # one NaN weight: one column of outputs
    got = P.fp8_matmul(place(xs, "f32"), codes_to_torch(wc), scales_to_torch(wb)).cpu().numpy()
    nan = np.zeros((M, d_out), dtype=bool)
    nan[[1, M - 2]] = True
    nan[:, d_out - 1] = True
    np.testing.assert_array_equal(np.isnan(got), nan)
    xc, xb = F.fp8_quantize(D.exact(xs, "f32"))
    rows = np.setdiff1d(np.arange(M), [1, M - 2])
    check(got[rows][:, :-1].astype(np.float64), F.fp8_values(xc[rows], xb[rows]), w[:-1], "f32", f"{M} beside NaN")


@pytest.mark.parametrize("M", [4, 40, 140])
def test_scales_far_apart(M):
    """Blocks of very different sizes in one sum, weights as well; scale bytes from the lowest to near the highest."""
    from post_weight_quantization_08_amd import pipeline as P
    r = np.random.default_rng([61, M])
    d_in, d_out = 1024, 256
    x = r.standard_normal((M, d_in)) * 2.0 ** np.repeat(r.integers(-40, 40, (M, 8)), 128, 1)
    w = r.standard_normal((d_out, d_in)) * np.repeat(np.repeat(2.0 ** r.integers(-40, 40, (2, 8)), 128, 1), 128, 0)
    x = x.astype(np.float32).astype(np.float64)
    xc, xb = F.fp8_quantize(x)
    wc, wb = F.fp8_quantize(w, tiles=True)
    got = P.fp8_matmul(place(x.astype(np.float32), "f32"), codes_to_torch(wc), scales_to_torch(wb)).double().cpu().numpy()
    check(got, F.fp8_values(xc, xb), F.fp8_values(wc, wb, tiles=True), "f32", f"{M} scales far apart")


def test_gradient_of_the_input_by_differences():
    """The transposed weights give the gradient of sum(Y G) with respect to what X's codes stand for: the product is
    linear in X, so a difference of two products is the gradient times the step (one column changed by a power of two)."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    M, d_in, d_out = 70, 256, 384
    W = place(values(d_out, d_in, "f32", 4, 0.3) / np.float32(16), "f32")
    q = P.fp8_quantize(W, tiles=True)
    wc, wb = bytes_of(q["codes"]), bytes_of(q["scales"])
    G = place(values(M, d_out, "bf16", 8, 0.3), "bf16")
    g = P.fp8_quantize(G)
    dX = P.fp8_matmul(G, q["codes_t"], q["scales_t"]).double().cpu().numpy()
    gv = F.fp8_values(bytes_of(g["codes"]), bytes_of(g["scales"]))
    wv = F.fp8_values(wc, wb, tiles=True)
    check(dX, gv, wv.T.copy(), "f32", "input gradient")
    x = np.ones((M, d_in), dtype=np.float32)
    for col in (0, 100, 255):
        x2 = x.copy()
        x2[:, col] = 1.5
        y = [P.fp8_matmul(place(v, "f32"), q["codes"], q["scales"]).double().cpu().numpy() for v in (x, x2)]
        diff = ((y[1] - y[0]) * gv).sum(1) / 0.5
        # two fp32 products of 256 terms each, over a step of 0.5
        bound = 4 * 256 * 2.0 ** -23 * (np.abs(gv) @ np.abs(wv).sum(1)) + 256 * 2.0 ** -23 * (np.abs(gv) @ np.abs(wv[:, col]))
        assert np.all(np.abs(diff - dX[:, col]) <= bound)


def test_empty_batches_and_single_rows():
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    wc, wb, w = operands(1, 256, 40, 1)
    W, ws = codes_to_torch(wc), scales_to_torch(wb)
    assert P.fp8_matmul(torch.empty(0, 256, device="cuda"), W, ws).shape == (0, 40)
    q = P.fp8_quantize(torch.empty(0, 256, device="cuda"))
    assert q["codes"].shape == (0, 256) and P.fp8_quantize(torch.empty(0, 200, device="cuda"), tiles=True)["codes_t"].shape == (200, 0)
    one = P.fp8_quantize(torch.ones(5, 300, device="cuda"))["codes"][3:4]
    assert one.shape == (1, 384)
    x = torch.randn(3, 512, device="cuda")[1:2, 100:356]         # a row alone, any stride
    got = P.fp8_matmul(x, W, ws).double().cpu().numpy()
    xc, xb = F.fp8_quantize(x.double().cpu().numpy())
    check(got, F.fp8_values(xc, xb), w, "f32", "one row of a view")


def test_wrappers_refuse():
    import torch
    import post_weight_quantization_08_amd as G
    from post_weight_quantization_08_amd import pipeline as P
    wc, wb, _ = operands(4, 256, 40, 1)
    W, ws = codes_to_torch(wc), scales_to_torch(wb)
    x = torch.randn(4, 256, device="cuda")
    q = P.fp8_quantize(x)
    for bad in (lambda: P.fp8_matmul(x[:, :100], W, ws), lambda: P.fp8_matmul(x, W, ws.view(torch.uint8)),
                lambda: P.fp8_matmul(x, W.view(torch.uint8), ws), lambda: P.fp8_matmul(q["codes"], W, ws),
                lambda: P.fp8_matmul(x, W, ws, x_scales=q["scales"]), lambda: P.fp8_matmul(x, W, ws[:, :1]),
                lambda: P.fp8_matmul(x, W, ws, Y=torch.empty(4, 39, device="cuda")),
                lambda: P.fp8_matmul(q["codes"][:, 8:136], W[:, :128], ws[:, :1].contiguous(), x_scales=q["scales"][:, :1].contiguous()),
                lambda: P.fp8_quantize(x.t()), lambda: P.fp8_quantize(x[0]),
                lambda: P.fp8_quantize(x, out={"codes": q["codes"], "scales": q["scales"].view(torch.uint8)})):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(G.GptqError):
        P.fp8_quantize(x.double())
    with pytest.raises(G.GptqError):
        P.fp8_matmul(x, W, ws, y_dtype=torch.float64)


@pytest.mark.parametrize("M", [1, 40, 200])
def test_captured_and_on_another_stream(M):
    """A captured call on new inputs, replayed, and calls on two streams with buffers of their own."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    wc, wb, _ = operands(M, 2048, 520, 2)
    W, ws = codes_to_torch(wc), scales_to_torch(wb)
    X = torch.randn(M, 2048, device="cuda").bfloat16()
    Y, work = P.fp8_matmul_buffers(X, W)
    out = P.fp8_quantize_buffers(X)
    P.fp8_matmul(X, W, ws, Y=Y, ws=work)
    P.fp8_quantize(X, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.fp8_quantize(X, out=out)
        P.fp8_matmul(out["codes"], W, ws, x_scales=out["scales"], Y=Y, ws=work)
    for _ in range(3):
        X.copy_(torch.randn(M, 2048, device="cuda"))
        want = P.fp8_matmul(X, W, ws)
        Y.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = P.fp8_matmul(X, W, ws, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
