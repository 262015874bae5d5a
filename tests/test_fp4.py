"""Microscaled 4-bit quantisation and product against their definition in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_ref as ref
import w8a8_post_quantization_sq_b200 as sq

FMTS = [sq.SQ_NVFP4, sq.SQ_MXFP4]
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def L():
    from w8a8_post_quantization_sq_b200 import build

    build.build()
    return sq.lib()


def data(M, K, dt, seed=0, loud=True):
    g = torch.Generator().manual_seed(seed + 131 * M + K)
    x = torch.randn((M, K), generator=g)
    if loud:
        x[:, :: max(1, K // 7)] *= 30.0
    return x.to(dt)


def random_fp4(rows, K, fmt, seed):
    """Codes, scale bytes, row scales of a quantised random matrix (numpy)."""
    return ref.quantise(data(rows, K, torch.float32, seed).double().numpy(), fmt)


# ---------------------------------------------------------------- without a GPU
def test_reference_formats():
    """The reference's own conversions at every value, midpoint and the ends."""
    t = np.array([0, 0.25, 0.2500001, 0.5, 0.75, 0.7499999, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.0, -0.25, -5.0, -1e9])
    want = [0, 0, 1, 1, 2, 1, 2, 4, 4, 6, 6, 7, 7, 8, 14, 15]
    assert ref.e2m1(t).tolist() == want
    b = np.arange(0x7F, dtype=np.uint8)
    assert np.array_equal(ref.e4m3_byte(ref.e4m3_value(b)), b)
    mid = (ref.e4m3_value(b[:-1]) + ref.e4m3_value(b[1:])) / 2
    assert np.array_equal(ref.e4m3_byte(mid), np.where(b[:-1] % 2 == 0, b[:-1], b[1:]))
    assert ref.e4m3_byte(np.array([448.0, 1e6, 2.0**-10, 2.0**-10 * 1.01])).tolist() == [0x7E, 0x7E, 0, 1]
    x = torch.tensor(np.random.default_rng(0).uniform(0, 448, 4096), dtype=torch.float32)
    assert np.array_equal(ref.e4m3_byte(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_bytes(L):
    assert sq.sq_fp4_scale_bytes(sq.SQ_NVFP4, 1, 32) == 512
    assert sq.sq_fp4_scale_bytes(sq.SQ_NVFP4, 129, 4096) == 2 * 64 * 512
    assert sq.sq_fp4_scale_bytes(sq.SQ_MXFP4, 128, 4096) == 32 * 512
    assert sq.sq_fp4_scale_bytes(sq.SQ_MXFP4, 1, 160) == 2 * 512
    assert sq.sq_fp4_scale_bytes(7, 1, 32) == sq.sq_fp4_scale_bytes(0, 0, 32) == 0


def test_refusals(L):
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)

    def expect(status, code, text):
        assert status == code and text in L.sq_last_error_string().decode(), L.sq_last_error_string()

    qa = L.sq_quantize_act_fp4
    expect(qa(p, 3, 4, 32, 32, None, 0, 1, None, p, p, p, None), 1, "dtype")
    expect(qa(p, 2, 4, 32, 32, None, 5, 1, None, p, p, p, None), 1, "format")
    expect(qa(p, 2, 4, 48, 48, None, 0, 1, None, p, p, p, None), 2, "multiple of 32")
    expect(qa(p, 2, 4, 32, 16, None, 0, 1, None, p, p, p, None), 2, "stride")
    expect(qa(p, 2, -1, 32, 32, None, 0, 1, None, p, p, p, None), 2, "need")
    expect(qa(None, 2, 4, 32, 32, None, 0, 1, None, p, p, p, None), 1, "null")
    expect(qa(p, 2, 4, 32, 32, None, 0, 1, None, p, p, None, None), 1, "row scales")
    expect(qa(p, 2, 4, 32, 32, None, 1, 1, None, p, p, p, None), 1, "no row scales")
    expect(qa(p, 2, 4, 32, 32, None, 0, 0, None, p, p, p, None), 1, "static_qs")
    expect(qa(odd, 2, 4, 32, 32, None, 0, 1, None, p, p, p, None), 3, "aligned")
    expect(qa(p, 2, 4, 32, 36, None, 0, 1, None, p, p, p, None), 3, "aligned")
    assert qa(None, 2, 0, 32, 32, None, 0, 1, None, None, None, None, None) == 0
    qw = L.sq_quantize_weight_fp4
    expect(qw(p, 2, 4, 32, odd, 0, p, p, p, None), 3, "aligned")
    dq = L.sq_dequantize_fp4
    expect(dq(p, p, 0, 4, 32, p, 1, 4, p, 32, None), 1, "dtype")
    expect(dq(p, p, 0, 4, 32, p, 1, 2, p, 36, None), 3, "aligned")
    expect(dq(p, None, 0, 4, 32, p, 1, 2, p, 32, None), 1, "null")
    gm = L.sq_gemm_fp4
    ok = [p, p, p, p, 0, 16, 16, 32, p, 1, p, 1, None, 2, p, 16, p, 256, None]
    for at, v, code, text in [(0, None, 1, "null"), (3, None, 1, "null"), (4, 2, 1, "format"), (6, 0, 2, "N > 0"),
                              (7, 48, 2, "multiple of 32"), (13, 3, 1, "dtype"), (15, 8, 2, "ldy"), (0, odd, 3, "aligned"),
                              (1, odd, 3, "aligned"), (16, None, 1, "workspace"), (17, 128, 1, "workspace"),
                              (5, 1 << 30, 2, "2^30")]:
        bad = list(ok)
        bad[at] = v
        expect(gm(*bad), code, text)
    assert gm(None, None, None, None, 0, 0, 16, 32, None, 0, None, 0, None, 2, None, 16, None, 0, None) == 0


def test_binding_refusals():
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError, match="codes"):
        sq.sq_quantize_act_fp4(torch.empty(4, 64), None, 0, True, None, u8(4, 64), u8(512), torch.empty(4))
    with pytest.raises(ValueError, match="block scales"):
        sq.sq_quantize_act_fp4(torch.empty(129, 64), None, 0, True, None, u8(129, 32), u8(512), torch.empty(129))
    with pytest.raises(ValueError, match="format"):
        sq.sq_quantize_act_fp4(torch.empty(4, 64), None, 9, True, None, u8(4, 32), u8(512), torch.empty(4))
    with pytest.raises(ValueError, match="codes"):
        sq.sq_gemm_fp4(u8(4, 32), u8(512), u8(8, 16), u8(512), 0, None, None, None, torch.empty(4, 8), u8(256))


# ---------------------------------------------------------------- quantisation
def quantise_gpu(x, fmt, s=None, weight=False, static=None):
    M, K = x.shape
    codes, scales, qs = sq.fp4_buffers(M, K, fmt)
    scales.fill_(0xAA)
    if static is not None:
        qs = torch.empty(1, device="cuda")
    if weight:
        sq.sq_quantize_weight_fp4(x, s, fmt, codes, scales, qs)
    else:
        sq.sq_quantize_act_fp4(x, s, fmt, static is None, static, codes, scales, qs)
    return codes, scales, qs


def check_quant(x, fmt, s=None, weight=False, static=None):
    codes, scales, qs = quantise_gpu(x.cuda(), fmt, None if s is None else s.cuda(), weight,
                                     None if static is None else torch.tensor([static], device="cuda"))
    v = x.double().numpy()
    if s is not None:
        with np.errstate(invalid="ignore"):
            v = ref.f32(v * s.double().numpy() if weight else v / s.double().numpy())
    c, b, q = ref.quantise(v, fmt, static)
    got = codes.cpu().numpy()
    want = ref.pack(c)
    # the sign of a zero code says nothing
    zero = lambda p: np.where(p & 0x7, p, p & 0xF0) & np.where(p & 0x70, 0xFF, 0x0F)  # noqa: E731
    assert np.array_equal(zero(got), zero(want)), np.argwhere(zero(got) != zero(want))[:4]
    assert np.array_equal(scales.cpu().numpy(), ref.tile(b))
    if fmt == sq.SQ_NVFP4:
        assert np.array_equal(qs.cpu().double().numpy(), q if static is None else q[:1])
    return codes, scales, qs, c, b, q


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (130, 96), (129, 4096), (7, 1056), (5, 12288), (2, 40000), (33, 544), (2000, 2048), (700, 20480), (3, 49152), (3, 65536)])
def test_quantise(M, K, dt, fmt):
    check_quant(data(M, K, dt), fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("dt", DTYPES)
def test_quantise_smoothed(fmt, weight, dt):
    s = torch.rand(1120, generator=torch.Generator().manual_seed(3)) + 0.25
    check_quant(data(37, 1120, dt), fmt, s, weight)


@pytest.mark.gpu
@pytest.mark.parametrize("static", [2.0**5, 3.7, 1e4])
def test_quantise_static(static):
    check_quant(data(19, 512, torch.bfloat16), sq.SQ_NVFP4, static=float(np.float32(static)))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", DTYPES)
def test_quantise_edges(fmt, dt):
    """Zero rows, zero blocks, subnormal and largest values, NaN and infinities, ties."""
    x = data(12, 256, torch.float32, loud=False).to(dt)
    x[0] = 0
    x[1, 32:96] = 0
    x[2] *= torch.finfo(dt).tiny
    x[3] = torch.finfo(dt).max
    x[4, 5] = float("nan")
    x[5, 77] = float("inf")
    x[6, 200] = -float("inf")
    x[7] = float("nan")
    x[8] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5] * 32, dtype=dt)
    x[9] = torch.tensor([-6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5] * 32, dtype=dt)
    x[10, :128] *= 1e-4
    x[11, ::32] *= 300
    check_quant(x, fmt)


@pytest.mark.gpu
def test_quantise_strided_rows():
    x = data(21, 768, torch.bfloat16)
    base = torch.zeros((21, 1024), dtype=torch.bfloat16)
    base[:, 64:832] = x
    view = base.cuda()[:, 64:832]
    a = quantise_gpu(view, sq.SQ_NVFP4)
    b = quantise_gpu(x.cuda(), sq.SQ_NVFP4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (131, 160), (9, 4128)])
def test_dequantise(M, K, dt, fmt):
    codes, scales, qs, c, b, q = check_quant(data(M, K, torch.float32), fmt)
    y = torch.full((M, K + 8), -1.0, dtype=dt, device="cuda")
    sq.sq_dequantize_fp4(codes, scales, fmt, qs, y[:, :K])
    v = ref.f32(ref.values(c, b, fmt)) / (q[:, None] if q is not None else 1.0)
    want = torch.from_numpy(v).to(dt)
    assert torch.equal(y[:, :K].cpu().double(), want.double())
    assert bool((y[:, K:] == -1).all())


@pytest.mark.gpu
def test_dequantise_nan_and_one_scale():
    x = data(4, 64, torch.float32)
    x[2, 40] = float("inf")
    for fmt in FMTS:
        codes, scales, _ = quantise_gpu(x.cuda(), fmt)
        y = torch.empty((4, 64), device="cuda")
        sq.sq_dequantize_fp4(codes, scales, fmt, torch.tensor([4.0], device="cuda"), y)
        bad = torch.zeros((4, 64), dtype=torch.bool)
        bad[2, 32:48 if fmt == sq.SQ_NVFP4 else 64] = True
        assert torch.equal(y.isnan().cpu(), bad)


# ---------------------------------------------------------------- product
def operand(rows, K, fmt, seed):
    c, b, q = random_fp4(rows, K, fmt, seed)
    dev = (torch.from_numpy(ref.pack(c)).cuda(), torch.from_numpy(ref.tile(b)).cuda(),
           None if q is None else torch.from_numpy(q).float().cuda())
    v = ref.values(c, b, fmt) / (q[:, None] if q is not None else 1.0)
    return dev, torch.from_numpy(v).cuda()


def check_gemm(y, xv, wv, bias, K):
    """|y - exact| within the fp32 sum's bound (K 2^-23 sum |a b|, as for the other GEMMs of the library), two fp32
    roundings of the scale factor and one of the bias (3 x 2^-24), and half a step of the output type."""
    want = xv @ wv.T
    mass = xv.abs() @ wv.abs().T
    if bias is not None:
        want = want + bias.double()
        mass = mass + bias.double().abs()
    half = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}[y.dtype]
    tol = (K + 4) * 2.0**-23 * mass + half * want.abs() + 2.0**-25 * (y.dtype == torch.float16)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SHAPES = [(1, 8, 32), (16, 128, 64), (128, 128, 256), (5, 129, 96), (333, 1001, 1056), (130, 257, 544),
          (16, 4096, 4096), (1, 1024, 8192), (64, 384, 2080), (257, 640, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, fmt):
    (xq, xs, qx), xv = operand(M, K, fmt, 1)
    (wq, wsc, qw), wv = operand(N, K, fmt, 2)
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(5)).cuda()
    for dt, b in ((torch.float32, None), (torch.bfloat16, bias), (torch.float16, None)):
        y = torch.empty((M, N), dtype=dt, device="cuda")
        sq.sq_gemm_fp4(xq, xs, wq, wsc, fmt, qx, qw, b, y, ws)
        check_gemm(y, xv, wv, b, K)
    sq.sq_workspace_status(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2048, 2560, 512), (2100, 2344, 1120), (4096, 4096, 256), (1000, 5000, 2048),
                                   (3000, 6000, 320)])
def test_gemm_many_tiles(M, N, K, fmt):
    """Shapes of several tiles per SM, whose accumulators follow one another."""
    (xq, xs, qx), xv = operand(M, K, fmt, 3)
    (wq, wsc, qw), wv = operand(N, K, fmt, 4)
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    for dt in (torch.bfloat16, torch.float32):
        y = torch.empty((M, N), dtype=dt, device="cuda")
        sq.sq_gemm_fp4(xq, xs, wq, wsc, fmt, qx, qw, None, y, ws)
        check_gemm(y, xv, wv, None, K)
    sq.sq_workspace_status(ws)


def random_operand(rows, K, fmt, seed):
    """Any codes, any block scales of moderate size, row scales for NVFP4; and what they stand for."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (rows, K), dtype=np.uint8)
    byte = g.integers(0x28, 0x50, (rows, K // ref.BLOCK[fmt])) if fmt == 0 else g.integers(122, 131, (rows, K // 32))
    q = 2.0 ** g.integers(-3, 4, rows) if fmt == 0 else None
    byte = byte.astype(np.uint8)
    dev = (torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(ref.tile(byte)).cuda(),
           None if q is None else torch.from_numpy(q).float().cuda())
    v = torch.tensor(ref.GRID, device="cuda")[torch.from_numpy(codes & 7).cuda().int()]
    v = torch.where(torch.from_numpy(codes & 8).cuda() > 0, -v, v)
    v *= torch.from_numpy(ref.scale_value(byte, fmt)).cuda().repeat_interleave(ref.BLOCK[fmt], 1)
    return dev, v if q is None else v / torch.from_numpy(q).cuda()[:, None]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2560, 2560, 12288), (2500, 2490, 12320), (1024, 7168, 16384)])
def test_gemm_split_last_wave(M, N, K, fmt):
    """Shapes whose last wave is cut by k-blocks: with and without room for it, twice, and counters zero again."""
    (xq, xs, qx), xv = random_operand(M, K, fmt, 1)
    (wq, wsc, qw), wv = random_operand(N, K, fmt, 2)
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    assert ws.numel() > 256
    bias = torch.randn(N, generator=torch.Generator().manual_seed(5)).cuda()
    for dt, b in ((torch.bfloat16, bias), (torch.float32, None)):
        ys = []
        for use in (ws, ws, ws[:256]):
            y = torch.empty((M, N), dtype=dt, device="cuda")
            sq.sq_gemm_fp4(xq, xs, wq, wsc, fmt, qx, qw, b, y, use)
            ys.append(y)
        check_gemm(ys[0], xv, wv, b, K)
        check_gemm(ys[2], xv, wv, b, K)
        assert torch.equal(ys[0], ys[1])
        assert int(ws[: 256 + 128 * 2 * 8 * 4].sum()) == int(ws[12:16].sum())  # only the region's size is noted
    sq.sq_workspace_status(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("ldy", [1008, 1003])
def test_gemm_strided_output(dt, ldy):
    M, N, K = 70, 1000, 512
    (xq, xs, qx), xv = operand(M, K, 0, 1)
    (wq, wsc, qw), wv = operand(N, K, 0, 2)
    full = torch.full((M + 2, ldy), 7.0, dtype=dt, device="cuda")
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    sq.sq_gemm_fp4(xq, xs, wq, wsc, 0, qx, qw, None, full[1 : M + 1, :N], ws)
    check_gemm(full[1 : M + 1, :N], xv, wv, None, K)
    assert bool((full[0] == 7).all() and (full[-1] == 7).all() and (full[:, N:] == 7).all())


@pytest.mark.gpu
def test_gemm_scale_forms():
    """One scale for all rows, none, and per row give the same product up to the factor."""
    M, N, K = 33, 300, 256
    (xq, xs, _), xv = operand(M, K, 1, 1)
    (wq, wsc, _), wv = operand(N, K, 1, 2)
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    one = torch.tensor([4.0], device="cuda")
    y0, y1, y2 = (torch.empty((M, N), device="cuda") for _ in range(3))
    sq.sq_gemm_fp4(xq, xs, wq, wsc, 1, None, None, None, y0, ws)
    sq.sq_gemm_fp4(xq, xs, wq, wsc, 1, one, one, None, y1, ws)
    sq.sq_gemm_fp4(xq, xs, wq, wsc, 1, one.expand(M).contiguous(), one.expand(N).contiguous(), None, y2, ws)
    check_gemm(y0, xv, wv, None, K)
    assert torch.equal(y0 / 16, y1) and torch.equal(y1, y2)


@pytest.mark.gpu
def test_gemm_nan_stays_in_its_row():
    for fmt in FMTS:
        M, N, K = 200, 256, 512
        x = data(M, K, torch.float32, 1)
        x[77, 100] = float("nan")
        w = data(N, K, torch.float32, 2)
        w[9, 3] = float("inf")
        a, b = quantise_gpu(x.cuda(), fmt), quantise_gpu(w.cuda(), fmt)
        y = torch.empty((M, N), device="cuda")
        sq.sq_gemm_fp4(a[0], a[1], b[0], b[1], fmt, a[2], b[2], None, y, sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K))
        bad = torch.zeros((M, N), dtype=torch.bool)
        bad[77] = True
        bad[:, 9] = True
        assert torch.equal(y.isnan().cpu(), bad)


@pytest.mark.gpu
def test_gemm_workspace_and_repeats():
    """One workspace for shapes with and without a split, in turn; equal bits every time; a small workspace."""
    shapes = [(16, 4096, 4096), (1, 1024, 8192), (300, 512, 1024), (2560, 2560, 12288), (8, 128, 16384),
              (16, 4096, 4096)]
    ws = torch.zeros(max(sq.sq_workspace_size(sq.SQ_OP_GEMM_FP4, *s) for s in shapes), dtype=torch.uint8, device="cuda")
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for M, N, K in shapes:
        (xq, xs, qx), xv = random_operand(M, K, 0, 1)
        (wq, wsc, qw), wv = random_operand(N, K, 0, 2)
        ys = []
        for use in (ws, ws, small):
            y = torch.empty((M, N), device="cuda")
            sq.sq_gemm_fp4(xq, xs, wq, wsc, 0, qx, qw, None, y, use)
            check_gemm(y, xv, wv, None, K)
            ys.append(y)
        assert torch.equal(ys[0], ys[1])
        assert int(ws[256 : 256 + 8192].sum()) == 0  # counters are zero again
        sq.sq_workspace_status(ws)


@pytest.mark.gpu
def test_graph_and_streams():
    """Quantise and multiply captured once, replayed on new inputs, on a stream of their own."""
    M, N, K = 24, 1024, 2048
    x = data(M, K, torch.bfloat16, 1).cuda()
    (wq, wsc, qw), _ = operand(N, K, 0, 2)
    codes, scales, qs = sq.fp4_buffers(M, K, 0)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)

    def step():
        sq.sq_quantize_act_fp4(x, None, 0, True, None, codes, scales, qs)
        sq.sq_gemm_fp4(codes, scales, wq, wsc, 0, qs, qw, None, y, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for seed in (5, 6):
        x.copy_(data(M, K, torch.bfloat16, seed))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        assert torch.equal(got, y)


@pytest.mark.gpu
def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    w = torch.randn(8, 64).cuda()
    wq, wsc, qw = quantise_gpu(w, 0, weight=True)
    sq.sq_quantize_act_fp4(torch.empty((0, 64), device="cuda"), None, 0, True, None, e(0, 32), e(0), torch.empty(0).cuda())
    sq.sq_gemm_fp4(e(0, 32), e(0), wq, wsc, 0, None, qw, None, torch.empty((0, 8), device="cuda"),
                   sq.workspace(sq.SQ_OP_GEMM_FP4, 0, 8, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("smooth", [False, True])
def test_quantise_static_past_the_largest(dt, smooth):
    """A static scale under which finite values pass fp32's largest: they saturate, and so does their block's scale."""
    static = float(np.float32(1e36 if dt == torch.float16 else 1e30))
    x = data(8, 256, torch.float32)
    top = torch.finfo(dt).max / (4 if smooth else 1)  # (the quotient by s is still finite)
    x[0] = top
    x[1, 5] = -top
    x[2, ::7] = top
    x[3] *= 1e-3 if dt == torch.float16 else 1e-27
    x[3, ::16] = -top  # beside values of a few hundred times the largest code
    x[4, 9] = float("inf")
    x[5, 40] = float("nan")
    x[6] = 0
    x[6, 100] = top
    s = torch.rand(256, generator=torch.Generator().manual_seed(3)) + 0.5 if smooth else None
    check_quant(x.to(dt), sq.SQ_NVFP4, s, static=static)


def exact_operand(rows, K, fmt, seed):
    """Any codes, block scales 1, 2 and 4, row scales powers of two: products are multiples of 1/4."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (rows, K), dtype=np.uint8)
    step = g.integers(0, 3, (rows, K // ref.BLOCK[fmt]))
    byte = (0x38 + 8 * step if fmt == 0 else 127 + step).astype(np.uint8)
    q = 2.0 ** g.integers(-3, 4, rows) if fmt == 0 else None
    dev = (torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(ref.tile(byte)).cuda(),
           None if q is None else torch.from_numpy(q).float().cuda())
    v = torch.tensor(ref.GRID, device="cuda")[torch.from_numpy(codes & 7).cuda().int()]
    v = torch.where(torch.from_numpy(codes & 8).cuda() > 0, -v, v)
    v *= torch.from_numpy(2.0**step).cuda().repeat_interleave(ref.BLOCK[fmt], 1)
    return dev, v, q


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 1024, 8192), (16, 4096, 4096), (64, 384, 2080), (333, 1001, 1056), (2100, 2344, 1120),
                                   (2560, 2560, 12288), (2500, 2490, 12320), (1024, 7168, 16384)])
def test_gemm_exact(M, N, K, fmt):
    """Sums that fp32 holds exactly in any order (multiples of 1/4 whose absolute sum stays below 2^22, 24 bits): the
    product to the last bit, in parts of a k-loop, whole tiles and the last wave's pieces."""
    (xq, xs, qx), xv, rx = exact_operand(M, K, fmt, 1)
    (wq, wsc, qw), wv, rw = exact_operand(N, K, fmt, 2)
    assert float((xv.abs() @ wv.abs().T).max()) < 2.0**22
    want = xv @ wv.T
    if fmt == 0:
        want = want / torch.from_numpy(rx).cuda()[:, None] / torch.from_numpy(rw).cuda()
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty((M, N), dtype=dt, device="cuda")
        sq.sq_gemm_fp4(xq, xs, wq, wsc, fmt, qx, qw, None, y, ws)
        assert torch.equal(y, want.float().to(dt))
    sq.sq_workspace_status(ws)


def test_refuses_an_unaligned_workspace(L):
    """Its counters and sums are accessed up to 16 bytes at a time: host error, no launch."""
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
    status = L.sq_gemm_fp4(p, p, p, p, 0, 16, 16, 32, p, 1, p, 1, None, 2, p, 16, odd, 256, None)
    assert status == 3 and "workspace must be 16-byte aligned" in L.sq_last_error_string().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,N,K,ldy", [(60, 957, 128, 968), (300, 41, 96, 48), (2778, 959, 128, 960), (2500, 2489, 12320, 2496)])
def test_gemm_rows_that_end_inside_16_bytes(M, N, K, ldy, dt):
    """Widths that are no multiple of 8 in rows that start on 16-byte boundaries (Y a part of a wider matrix): the
    columns behind Y, up to the next boundary too, keep what they hold."""
    (xq, xs, qx), xv, rx = exact_operand(M, K, 0, 1)
    (wq, wsc, qw), wv, rw = exact_operand(N, K, 0, 2)
    want = (xv @ wv.T) / torch.from_numpy(rx).cuda()[:, None] / torch.from_numpy(rw).cuda()
    big = torch.full((M + 1, ldy), 7.0, dtype=dt, device="cuda")
    ws = sq.workspace(sq.SQ_OP_GEMM_FP4, M, N, K)
    sq.sq_gemm_fp4(xq, xs, wq, wsc, 0, qx, qw, None, big[:M, :N], ws)
    sq.sq_workspace_status(ws)
    assert torch.equal(big[:M, :N], want.float().to(dt))
    assert bool((big[:, N:] == 7).all() and (big[M:] == 7).all())
