"""Matrices in 8 bits with block scales: the quantisation bit for bit, the
product against the 64-bit form, exactly on integers."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
import norm_fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _u8(t):
    return t.cpu().view(torch.uint8)


def _values(R, C, dtype, seed):
    """Rows of very different sizes, rows of zeros, negative zeros, denormals."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, C), generator=g) * torch.exp(2 * torch.randn((R, 1), generator=g))
    x[2::5] = 0
    x[4::11] = -0.0
    x[3::7] *= 1e-30
    x[6::13] *= 1e-39
    return x.to(dtype)


SHAPES = [(1, 1), (1, 128), (128, 1), (3, 7), (127, 129), (128, 128), (130, 136), (257, 1000),
          (64, 2304), (1029, 999), (2048, 1088)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_quant_bits(R, C, dtype, block_rows):
    print("[case] fp8_quant", R, C, dtype, block_rows, flush=True)
    x = _values(R, C, dtype, R + C)
    xg = x.to(DEV)
    want, want_t = ref.quant(x, block_rows), ref.quant(x.t(), block_rows)
    for layout in ("rows", "cols", "both"):
        o, t = tw.fp8_quant(xg, block_rows=block_rows, layout=layout)
        torch.cuda.synchronize()
        for got, w in ((o, want), (t, want_t)):
            if got is not None:
                assert torch.equal(got.scale.cpu(), w[1])
                # the sign of a zero is not part of the value
                a, b = got.q.cpu().float(), w[0].float()
                assert torch.equal(a, b), int((a != b).sum())
        assert (o is None) == (layout == "cols") and (t is None) == (layout == "rows")


def test_quant_every_bf16_ratio():
    """Every bfloat16 significand against several amaxes: quotients on and
    next to the ties between e4m3 values."""
    m = torch.arange(128, 256, dtype=torch.float32)
    rows = []
    for top in range(128, 256):
        for k in range(0, 11, 2):
            row = torch.zeros(256)
            row[:128] = m * 2.0 ** -k
            row[:128] = torch.where(row[:128] > top, torch.zeros(1), row[:128])
            row[127] = top
            row[128:] = -row[:128] * 2.0 ** 20
            rows.append(row)
    x = torch.stack(rows).to(BF)
    o, _ = tw.fp8_quant(x.to(DEV))
    q, s = ref.quant(x, 1)
    assert torch.equal(o.scale.cpu(), s) and torch.equal(o.q.cpu().float(), q.float())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_nan_and_infinity(block_rows):
    x = _values(200, 300, F32, 5)
    x[140, 130], x[20, 290] = float("nan"), -float("inf")
    o, t = tw.fp8_quant(x.to(DEV), block_rows=block_rows, layout="both")
    for got, src in ((o.float().cpu(), x), (t.float().cpu(), x.t())):
        r = torch.arange(src.shape[0])[:, None] // block_rows
        c = torch.arange(src.shape[1])[None, :] // 128
        bad = torch.zeros(src.shape, dtype=torch.bool)
        for i, j in (~src.isfinite()).nonzero().tolist():
            bad |= (r == i // block_rows) & (c == j // 128)
        assert got[bad].isnan().all() and got[~bad].isfinite().all()


def test_quant_strided_source():
    x = _values(300, 523, BF, 3)
    buf = torch.full((300, 530), float("nan"), dtype=BF, device=DEV)
    v = buf[:, 3:526]
    v.copy_(x)
    o, t = tw.fp8_quant(v, layout="both")
    assert torch.equal(o.q.cpu().float(), ref.quant(x, 1)[0].float())
    assert torch.equal(t.q.cpu().float(), ref.quant(x.t(), 1)[0].float())


def test_quant_offsets_past_32_bits():
    R, C = 66000, 65664
    x = torch.zeros((R, C), dtype=BF, device=DEV)  # 8.7 GB, q 4.3 GB
    tail = _values(150, C, BF, 9)
    x[-150:] = tail.to(DEV)
    o, t = tw.fp8_quant(x, layout="both")
    torch.cuda.synchronize()
    q, s = ref.quant(tail, 1)
    assert torch.equal(o.q[-150:].cpu().float(), q.float())
    assert torch.equal(o.scale[:, -150:].cpu(), s)
    # the transpose's last block of 80 columns of R (66000 = 515 * 128 + 80)
    q, s = ref.quant(tail[-80:].t(), 1)
    assert torch.equal(t.q[:, 515 * 128:].cpu().float(), q.float())
    assert torch.equal(t.scale[515:].cpu(), s)


# ---------------------------------------------------------------- product
LARGE = [(2049, 4097, 1160), (2000, 5801, 392), (3001, 2305, 2312)]  # the large tiles, ragged


def _fp8(rows, cols, block_rows, seed, integers=False):
    """A matrix on the CPU: (q, scale), zeros past cols."""
    g = torch.Generator().manual_seed(seed)
    cb, rb = -(-cols // 128), -(-rows // block_rows)
    if integers:  # |q| <= 2 and scales 1/2, 1, 2: every sum is exact in float32
        q = torch.randint(-2, 3, (rows, cb * 128), generator=g).float()
        s = 2.0 ** torch.randint(-1, 2, (cb, rb), generator=g).float()
    else:
        q = torch.randn((rows, cb * 128), generator=g) * 60
        s = torch.exp(torch.randn((cb, rb), generator=g)) * 0.01
    q[:, cols:] = 0
    return q.to(E4), s


def _up(m, cols, block_rows):
    """On the GPU, with NaN bytes right after the last row."""
    q, s = m
    buf = torch.full((q.numel() + 4096,), 0x7F, dtype=torch.uint8, device=DEV)
    v = buf[:q.numel()].view(E4).view(q.shape)
    v.view(torch.uint8).copy_(q.view(torch.uint8))
    return tw.Fp8(v, s.to(DEV), cols, block_rows)


MM = [  # M, N, K
    (1, 1, 1), (1, 6144, 2304), (3, 17, 130), (16, 128, 256), (17, 100, 128), (31, 2304, 1000),
    (33, 64, 4096), (64, 96, 384), (65, 130, 200), (100, 1, 640), (1, 333, 6144),
    (128, 128, 128), (129, 257, 136), (255, 256, 1088), (256, 512, 2048), (257, 2811, 576),
    (1029, 515, 1088), (640, 1000, 64), (2048, 130, 384), (1000, 1000, 1000), (300, 260, 8192),
]


@pytest.mark.parametrize("ra,rb", [(1, 128), (1, 1), (128, 128), (128, 1)])
@pytest.mark.parametrize("M,N,K", MM)
def test_product_integers(M, N, K, ra, rb):
    print("[case] fp8_matmul integers", M, N, K, ra, rb, flush=True)
    a, b = _fp8(M, K, ra, 1, True), _fp8(N, K, rb, 2, True)
    want = ref.dequant(*a, ra) @ ref.dequant(*b, rb).t()
    A, B = _up(a, K, ra), _up(b, K, rb)
    got = tw.fp8_matmul(A, B, out_dtype=F32)
    half = tw.fp8_matmul(A, B)
    fast = tw.fp8_matmul(A, B, out_dtype=F32, fast_sums=True)
    fast_half = tw.fp8_matmul(A, B, fast_sums=True)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu().double(), want)
    assert torch.equal(fast, got) and torch.equal(fast_half, half)
    assert torch.equal(half.cpu(), want.float().to(BF))


def test_every_kernel_on_integers():
    """Sizes that between them take every kernel, whole and split
    contractions, each result exact."""
    names = set()
    timer = tw.KernelTimer()
    for M, N, K in ((1, 300, 700), (1, 4100, 300), (4100, 16, 300), (4100, 20, 1000),
                    (4100, 100, 700), (2049, 1000, 700), (2000, 4100, 700), (2000, 6000, 700),
                    (1, 16, 70000), (520, 20, 40000), (130, 6000, 8192)):
        for rb in (128, 1):
            a, b = _fp8(M, K, 1, 1, True), _fp8(N, K, rb, 2, True)
            # float32 is exact here too: |sum| < 70000 * 16, in quarters
            da, db = ref.dequant(*a, 1).float().to(DEV), ref.dequant(*b, rb).float().to(DEV)
            want = da @ db.t()
            A, B = _up(a, K, 1), _up(b, K, rb)
            for fast in (False, True):
                print("[case] fp8_matmul kernels", M, N, K, rb, fast, flush=True)
                need = tw.fp8_matmul_workspace_bytes(M, N, K)
                ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN
                got = tw.fp8_matmul(A, B, out_dtype=F32, fast_sums=fast, workspace=ws)
                half = tw.fp8_matmul(A, B, fast_sums=fast, timing=timer)
                torch.cuda.synchronize()
                names |= {(n, fast, rb) for n, _ in timer.collect()}
                assert torch.equal(got, want)
                assert torch.equal(half, want.to(BF))
    seen = {n for n, _, _ in names}
    assert seen == {"fp8_mm_rows_1x1", "fp8_mm_rows_1x2", "fp8_mm_rows_2x2", "fp8_mm_rows_2x2_8",
                    "fp8_mm_tile64", "fp8_mm_tile128", "fp8_mm_tile192", "fp8_mm_tile256",
                    "fp8_mm_join"}, seen
    for fast, rb in ((True, 1), (True, 128), (False, 128)):
        assert ("fp8_mm_tile256", fast, rb) in names, (fast, rb)


@pytest.mark.parametrize("out", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("ra,rb", [(1, 128), (1, 1)])
@pytest.mark.parametrize("M,N,K", MM)
def test_product(M, N, K, ra, rb, out):
    print("[case] fp8_matmul", M, N, K, ra, rb, out, flush=True)
    a, b = _fp8(M, K, ra, 3), _fp8(N, K, rb, 4)
    da, db = ref.dequant(*a, ra), ref.dequant(*b, rb)
    want, mag = da @ db.t(), da.abs() @ db.abs().t()
    got = tw.fp8_matmul(_up(a, K, ra), _up(b, K, rb), out_dtype=out)
    again = tw.fp8_matmul(_up(a, K, ra), _up(b, K, rb), out_dtype=out)
    torch.cuda.synchronize()
    k = 128 + 2 + -(-K // 128) + 64
    ref.assert_within(got, want, k * ref.U32 * mag + ref.ustore(out) * want.abs(), "product")
    assert torch.equal(got, again)


@pytest.mark.parametrize("out", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("ra,rb", [(1, 128), (1, 1)])
@pytest.mark.parametrize("M,N,K", MM)
def test_product_fast_sums(M, N, K, ra, rb, out):
    print("[case] fp8_matmul fast", M, N, K, ra, rb, out, flush=True)
    a, b = _fp8(M, K, ra, 3), _fp8(N, K, rb, 4)
    da, db = ref.dequant(*a, ra), ref.dequant(*b, rb)
    want, mag = da @ db.t(), da.abs() @ db.abs().t()
    A, B = _up(a, K, ra), _up(b, K, rb)
    got = tw.fp8_matmul(A, B, out_dtype=out, fast_sums=True)
    again = tw.fp8_matmul(A, B, out_dtype=out, fast_sums=True)
    torch.cuda.synchronize()
    k = 128 + 2 + -(-K // 128) + 64
    ref.assert_within(got, want, (k * ref.U32 + ref.FAST) * mag + ref.ustore(out) * want.abs(),
                      "product")
    assert torch.equal(got, again)


@pytest.mark.parametrize("fast", [False, True], ids=["full", "fast"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (300, 77, 384), (515, 1029, 640)])
@pytest.mark.parametrize("out", [F32, BF], ids=["f32", "bf16"])
def test_product_into_a_slice(M, N, K, out, fast):
    """out's rows any distance apart, at any element; nothing else is written."""
    a, b = _fp8(M, K, 1, 1, True), _fp8(N, K, 128, 2, True)
    buf = torch.full((M + 2, N + 13), float("nan"), dtype=out, device=DEV)
    v = buf[1:M + 1, 3:N + 3]
    tw.fp8_matmul(_up(a, K, 1), _up(b, K, 128), out=v, out_dtype=out, fast_sums=fast)
    torch.cuda.synchronize()
    want = (ref.dequant(*a, 1) @ ref.dequant(*b, 128).t()).float().to(out)
    assert torch.equal(v.cpu(), want)
    v.fill_(float("nan"))
    assert buf.isnan().all()


@pytest.mark.parametrize("fast", [False, True], ids=["full", "fast"])
@pytest.mark.parametrize("M", [4, 40, 300])
def test_product_nan_stays_in_its_row(M, fast):
    N, K = 260, 640
    a, b = _fp8(M, K, 1, 1, True), _fp8(N, K, 128, 2, True)
    A, B = _up(a, K, 1), _up(b, K, 128)
    clean = tw.fp8_matmul(A, B, out_dtype=F32, fast_sums=fast)
    A.q.view(torch.uint8)[1, 200] = 0x7F  # NaN
    A.scale[2, 2] = float("inf")
    got = tw.fp8_matmul(A, B, out_dtype=F32, fast_sums=fast)
    torch.cuda.synchronize()
    assert got[1].isnan().all() and not got[2].isfinite().any()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])


def test_product_empty():
    A, B = tw.empty_fp8(0, 256, 1, DEV), _up(_fp8(30, 256, 128, 1), 256, 128)
    assert tw.fp8_matmul(A, B).shape == (0, 30)
    assert tw.fp8_matmul(B, A).shape == (30, 0)
    Z = tw.empty_fp8(5, 0, 1, DEV)  # no columns: sums of nothing
    out = torch.full((5, 5), float("nan"), device=DEV)
    tw.fp8_matmul(Z, Z, out=out, out_dtype=F32)
    torch.cuda.synchronize()
    assert not out.any()


def test_product_offsets_past_32_bits():
    M, N, K = 530000, 16, 8192  # a 4.3 GB
    q = torch.zeros((M, K), dtype=torch.uint8, device=DEV)
    a, b = _fp8(40, K, 1, 1, True), _fp8(N, K, 128, 2, True)
    q[-40:] = a[0].view(torch.uint8).to(DEV)
    s = torch.ones((64, M), device=DEV)
    s[:, -40:] = a[1].to(DEV)
    got = tw.fp8_matmul(tw.Fp8(q.view(E4), s, K, 1), _up(b, K, 128), out_dtype=F32)
    torch.cuda.synchronize()
    assert not got[:-40].any()
    assert torch.equal(got[-40:].cpu().double(), ref.dequant(*a, 1) @ ref.dequant(*b, 128).t())


def test_product_backward_by_quantised_products():
    """dx and dW of y = x W^T by two more products, against the 64-bit
    gradients of the values the operands stand for."""
    T, N, K = 257, 300, 392
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn((T, K), generator=g), torch.randn((N, K), generator=g) / K ** 0.5
    dy = torch.randn((T, N), generator=g)
    up = lambda t: t.to(DEV)
    xq, xt = tw.fp8_quant(up(x), layout="both")
    wq, wt = tw.fp8_quant(up(w), block_rows=128, layout="both")
    gq, gt = tw.fp8_quant(up(dy), layout="both")
    for got, a, b in ((tw.fp8_matmul(xq, wq, out_dtype=F32), xq, wq),
                      (tw.fp8_matmul(gq, wt, out_dtype=F32), gq, wt),
                      (tw.fp8_matmul(gt, xt, out_dtype=F32), gt, xt)):
        da = ref.dequant(a.q.cpu(), a.scale.cpu(), a.block_rows)
        db = ref.dequant(b.q.cpu(), b.scale.cpu(), b.block_rows)
        mag = da.abs() @ db.abs().t()
        k = 128 + 2 + a.scale.shape[0] + 64
        ref.assert_within(got, da @ db.t(), (k + 1) * ref.U32 * mag, "gradient")
    # and each is the true gradient up to the quantisation: e4m3 rounds to
    # 2^-4, so a product of two is within 2 * 2^-4 + 2^-8 of its terms' sum
    wtrue = dy.double().t() @ x.double()
    mag = dy.double().abs().t() @ x.double().abs()
    got = tw.fp8_matmul(gt, xt, out_dtype=F32).cpu().double()
    assert ((got - wtrue).abs() <= (2.0 ** -3 + 2.0 ** -8) * mag + 1e-2).all()


def test_streams_and_graph():
    """A block's steps on a stream of their own, then captured: every replay,
    with other work and synchronisations between, equals the eager results."""
    T, d, N = 130, 520, 300
    g = torch.Generator().manual_seed(1)
    x, res = torch.randn((T, d), generator=g).to(DEV), torch.randn((T, d), generator=g).to(DEV, BF)
    gain = torch.ones(d, device=DEV)
    w, _ = tw.fp8_quant(torch.randn((N, d), generator=g).to(DEV), block_rows=128)
    n8, h = tw.empty_fp8(T, d, 1, DEV), torch.empty_like(res)
    y, dh = torch.empty((T, N), device=DEV, dtype=BF), torch.empty((T, d), device=DEV)
    dg = torch.empty(d, device=DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    ws = torch.empty(tw.rmsnorm_bwd_workspace_bytes(T, d), **u8)
    mws = torch.empty(max(16, tw.fp8_matmul_workspace_bytes(T, N, d)), **u8)
    yt = tw.empty_fp8(N, T, 1, DEV)

    def step():
        tw.rmsnorm_fwd(x, gain, residual=res, h=h, out=n8, out_dtype=E4)
        tw.fp8_matmul(n8, w, out=y, workspace=mws)
        tw.fp8_quant(y, layout="cols", out_t=yt)
        tw.rmsnorm_bwd(x, h, gain, dh=dh, dgain=dg, workspace=ws)

    outs = lambda: [h, n8.q.view(torch.uint8), n8.scale, y, yt.q.view(torch.uint8), yt.scale, dh, dg]
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs()]
    side = torch.cuda.Stream()
    for t in outs():
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outs(), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in outs():
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(), want))


@pytest.mark.parametrize("rb", [128, 1])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_product_large(M, N, K, rb):
    print("[case] fp8_matmul large", M, N, K, rb, flush=True)
    a, b = _fp8(M, K, 1, 3), _fp8(N, K, rb, 4)
    da, db = ref.dequant(*a, 1).to(DEV), ref.dequant(*b, rb).to(DEV)
    want, mag = da @ db.t(), da.abs() @ db.abs().t()
    A, B = _up(a, K, 1), _up(b, K, rb)
    k = 128 + 2 + -(-K // 128) + 64
    for out in (F32, BF):
        for fast in (False, True):
            got = tw.fp8_matmul(A, B, out_dtype=out, fast_sums=fast)
            tol = (k * ref.U32 + (ref.FAST if fast else 0)) * mag + ref.ustore(out) * want.abs()
            ref.assert_within(got, want, tol, f"product {out} {fast}")


@pytest.mark.parametrize("rb", [128, 1])
@pytest.mark.parametrize("M,N,K,shift", [(4173, 4226, 64, 0), (4173, 4226, 300, 3),
                                         (8192, 5632, 128, 0), (2500, 16390, 1025, 1),
                                         (24577, 513, 640, 5)])
def test_product_of_many_tiles(M, N, K, shift, rb):
    """More large tiles than the chip has CUs, so that workgroups go on to
    further ones, whole and cut; sums that are exact in float32, results in a
    slice of a wider matrix that keeps what is around them."""
    print("[case] fp8_matmul many tiles", M, N, K, shift, rb, flush=True)
    a, b = _fp8(M, K, 1, 5, True), _fp8(N, K, rb, 6, True)
    want = ref.dequant(*a, 1).to(DEV) @ ref.dequant(*b, rb).to(DEV).t()
    A, B = _up(a, K, 1), _up(b, K, rb)
    for out in (F32, BF):
        for fast in (False, True):
            wide = torch.full((M, N + 2 * shift), 7.0, dtype=out, device=DEV)
            got = tw.fp8_matmul(A, B, out=wide[:, shift:shift + N], out_dtype=out, fast_sums=fast)
            assert torch.equal(got, want.to(F32).to(out)), (out, fast)
            assert bool((wide[:, :shift] == 7).all()) and bool((wide[:, shift + N:] == 7).all())
