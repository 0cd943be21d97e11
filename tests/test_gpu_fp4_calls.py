"""The calls on weights in 4 bits as a program makes them: every kernel that the
sizes choose between, strided and unaligned rows, outputs given, infinities and
NaN, offsets past 32 bits, streams, graphs, workspaces; the gradient against
differences; a block served from them."""
import pytest
import torch

import fp4_ref as ref
from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32, GROUPS, gen, quantised, weights, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def acts(T, K, seed, dtype=BF):
    return torch.randn(T, K, generator=gen(seed)).to(dtype)


def coded(N, K, group, seed, spread=4):
    """A matrix of any codes, scales of powers of two: (Fp4, its float64 values), on
    the GPU."""
    g = torch.Generator(DEV).manual_seed(seed)
    kp = -(-K // 128) * 128
    q = torch.randint(0, 256, (N, kp // 2), generator=g, device=DEV, dtype=torch.uint8)
    if K < kp:
        q[:, (K + 1) // 2:] = 0
        if K % 2:
            q[:, K // 2] &= 15
    e = torch.randint(-spread, spread + 1, (kp // group, N), generator=g, device=DEV)
    w4 = tw.Fp4(q, torch.exp2(e.float()).to(BF), K, group)
    return w4, w4.float().double()


def check(call, x, w4, w, T, n, K):
    """call(x, w4) against x w^T (w given with the contraction last), 64 bits on the GPU."""
    t = tw.KernelTimer()
    got = call(x, w4, out_dtype=F32, timing=t)
    x = x.double()
    want, mag = x @ w.t().contiguous(), x.abs() @ w.t().abs().contiguous()
    assert got.shape == (T, n)
    d = (got.double() - want).abs() - ref.terms(K) * ref.U32 * mag
    assert bool((d <= 0).all()), f"off by {float(d.max()):.3e} past the tolerance"
    return [name for name, _ in t.collect()]


# ---------------------------------------------------------------- kernels and sizes
# few tokens: rows of each width class, contractions longer than the scales staged
# at once, several tiles of tokens
ROWS = [(1, 4097, 256, 32), (3, 16400, 128, 64), (16, 16385, 130, 32), (2, 40, 9000, 32),
        (16, 24, 17000, 128), (12, 4200, 640, 64), (40, 200, 4500, 32), (70, 300, 900, 32),
        (32, 4300, 520, 128)]
# many: tiles of each size, the contraction in parts, and longer than the scales
# staged at once, edges cut; with how many tokens
TILES = [(100, 2811, 2304, 32), (60, 33000, 2200, 32), (500, 5632, 2200, 32), (333, 2811, 1090, 64),
         (2048, 4096, 520, 64), (640, 4090, 2048, 128), (1030, 4101, 1000, 128), (4200, 4100, 2200, 32), (8200, 2050, 136, 128)]


@pytest.mark.parametrize("T,N,K,group", ROWS)
def test_matmul_few_tokens(T, N, K, group):
    print("[case] fp4_matmul", T, N, K, group, flush=True)
    w4, w = coded(N, K, group, N)
    for dtype in (BF, F32):
        check(tw.fp4_matmul, acts(T, K, 5, dtype).to(DEV), w4, w, T, N, K)


@pytest.mark.parametrize("dtype", (BF, F32))
def test_matmul_tiles(dtype):
    seen = set()
    for T, N, K, group in TILES:
        print("[case] fp4_matmul", T, N, K, group, dtype, flush=True)
        w4, w = coded(N, K, group, N)
        seen |= set(check(tw.fp4_matmul, acts(T, K, 5, dtype).to(DEV), w4, w, T, N, K))
    assert {"fp4_tile64", "fp4_tile128", "fp4_tile256", "fp4_join"} <= seen


@pytest.mark.parametrize("dtype", (BF, F32))
def test_matmul_dx_kernels(dtype):
    seen = set()
    for T, K, N, group in TILES + [(1, 5000, 130, 32), (17, 600, 2000, 64), (33, 300, 7000, 128),
                                   (30, 40000, 300, 64), (20, 384, 513, 64), (5, 70, 600, 32)]:
        print("[case] fp4_matmul_dx", T, N, K, group, dtype, flush=True)
        w4, w = coded(N, K, group, N)
        seen |= set(check(tw.fp4_matmul_dx, acts(T, N, 5, dtype).to(DEV), w4, w.t(), T, K, N))
    assert {"fp4_cols", "fp4_tile64", "fp4_tile128", "fp4_tile256", "fp4_join"} <= seen


@pytest.mark.parametrize("T,d,f,group", [(64, 2304, 6144, 32), (40, 1024, 16384, 128), (34, 4096, 4224, 64)])
@pytest.mark.parametrize("dtype", (BF, F32))
def test_layer_of_many_tokens(T, d, f, group, dtype):
    """The gates and up products as tiles, their contraction in parts."""
    x = acts(T, d, 1)
    x[:, 0] = 1
    ms = []
    for i in range(3):
        m = torch.randn(f, d, generator=gen(10 + i)) / (f if i == 2 else d) ** 0.5
        if i == 0:
            m[:, 0] = -2
        w4 = tw.fp4_quant(m.to(DEV), group=group)
        ms.append((w4, w4.float().double().cpu()))
    x = x.to(dtype)
    t = tw.KernelTimer()
    y = tw.fp4_decode_fwd(x.to(DEV), *(m for m, _ in ms), timing=t)
    want, tol = ref.layer(x, *(v for _, v in ms))
    within(y, want, tol)
    assert [n for n, _ in t.collect()][-3:] == ["fp4_gates", "fp4_act", "fp4_down"]


@pytest.mark.parametrize("T", (1, 3, 5, 17))
def test_layer_of_many_weights(T):
    """Few tokens by the most weights that the layer is given here."""
    d, f, group = 4096, 16512, 64
    for dtype in (BF, F32):
        g = gen(3)
        x = torch.randn(T, d, generator=g)
        x[:, 0] = 1
        x = x.to(dtype)
        w = []
        for i in range(3):
            q = torch.randint(0, 256, (f, d // 2), generator=g, dtype=torch.uint8)
            s = torch.full((d // group, f), 2.0 ** -7).to(BF)
            if i == 0:
                q[:, 0] = (q[:, 0] & 0xf0) | 15  # -6 times its scale, 0.5
                s[0] = 0.5
                q[:, 1:group // 2] = 0
            w.append((tw.Fp4(q.to(DEV), s.to(DEV), d, group), ref.values(q, s, d, group)))
        want, tol = ref.layer(x, *(v for _, v in w))
        got = tw.fp4_decode_fwd(x.to(DEV), *(m for m, _ in w))
        within(got, want, tol)


def test_quantise_past_a_launch():
    """More rows than tiles of one launch, rows of a few columns."""
    R = (1 << 25) + 37
    w = torch.randint(-3, 4, (R, 2), generator=torch.Generator(DEV).manual_seed(1), device=DEV,
                      dtype=torch.int32).to(BF)
    w4 = tw.fp4_quant(w, group=128)
    back = tw.fp4_dequant(w4)
    # 3, 2 and 1 over a scale near 0.5, 1/3 and 1/6 are within a half step of a value
    assert float((back - w).abs().max()) <= 0.25
    sample = torch.cat((torch.arange(40), torch.arange(R - 40, R)))
    q, s = ref.quant(w[sample].cpu(), 128)
    assert torch.equal(w4.q[sample].cpu(), q) and torch.equal(w4.scale[0, sample].cpu(), s[0])


# ---------------------------------------------------------------- strides and places
@pytest.mark.parametrize("T", (1, 4, 30, 150))
@pytest.mark.parametrize("dtype", (F32, BF))
def test_rows_any_stride_apart(T, dtype):
    """x a slice of columns from an odd one on, results into a slice; what lies
    around them stays."""
    N, K = 131, 260
    w4, w = quantised(N, K, 64, 1)
    for dx in (False, True):
        a, b = (N, K) if dx else (K, N)
        big = acts(T, a + 9, 3, dtype).to(DEV)
        x = big[:, 3:3 + a]
        out = torch.full((T + 2, b + 7), 5.0, dtype=dtype, device=DEV)
        res = out[1:T + 1, 5:5 + b]
        call = tw.fp4_matmul_dx if dx else tw.fp4_matmul
        assert call(x, w4, out=res, out_dtype=dtype) is res
        want, mag = ref.matmul(x, w.t() if dx else w)
        within(res, want, ref.bound(mag, want, a, dtype))
        res.fill_(5.0)
        assert bool((out == 5).all())


def test_layer_strided():
    d, f = 192, 256
    ms = [quantised(f, d, 32, i, 0.1) for i in range(3)]
    for T in (2, 20):
        x = acts(T, d + 5, 1).to(DEV)[:, 5:]
        want, tol = ref.layer(x, *(v for _, v in ms))
        y = torch.full((T, d), NAN, device=DEV)
        assert tw.fp4_decode_fwd(x, *(m for m, _ in ms), y=y) is y
        within(y, want, tol)


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes of codes: its last rows."""
    N = (1 << 26) + 300
    q = torch.zeros(N, 64, dtype=torch.uint8, device=DEV)
    s = torch.ones(1, N, dtype=BF, device=DEV)
    q[-300:] = torch.randint(0, 256, (300, 64), generator=gen(1), dtype=torch.uint8).to(DEV)
    w4 = tw.Fp4(q, s, 128, 128)
    w = ref.values(q[-300:].cpu(), s[:, -300:].cpu(), 128, 128)
    x = torch.randint(-2, 3, (1, 128), generator=gen(2)).to(BF)
    out = tw.fp4_matmul(x.to(DEV), w4, out_dtype=F32)
    assert torch.equal(out[:, -300:].cpu().double(), x.double() @ w.t())
    assert not bool(out[:, :-300].any())
    back = tw.fp4_dequant(w4)
    assert torch.equal(back[-300:].cpu().double(), w)


# ---------------------------------------------------------------- not finite
@pytest.mark.parametrize("T", (2, 33, 140))
@pytest.mark.parametrize("dtype", (F32, BF))
def test_infinities_and_nan_go_where_they_belong(T, dtype):
    N, K = 150, 300
    w4, w = quantised(N, K, 64, 1)
    x = acts(T, K, 2, dtype)
    x[0, 5], x[1, 299] = INF, NAN
    got = tw.fp4_matmul(x.to(DEV), w4, out_dtype=F32).cpu()
    want, mag = ref.matmul(x, w)
    assert torch.equal(got[:2].isnan(), want[:2].isnan())
    assert torch.equal(got[0].isinf(), want[0].isinf())
    within(got[2:], want[2:], ref.bound(mag, want, K, F32)[2:])
    dy = acts(T, N, 2, dtype)
    dy[0, 5], dy[1, 149] = INF, NAN
    got = tw.fp4_matmul_dx(dy.to(DEV), w4, out_dtype=F32).cpu()
    want, mag = ref.matmul(dy, w.t())
    assert torch.equal(got[:2].isnan(), want[:2].isnan())
    assert torch.equal(got[0].isinf(), want[0].isinf())
    within(got[2:], want[2:], ref.bound(mag, want, N, F32)[2:])


@pytest.mark.parametrize("T", (2, 33, 140))
def test_a_group_of_nan(T):
    """A weight's NaN spoils its row of the product, its group's columns of the
    gradient, and nothing else."""
    N, K, group = 150, 300, 64
    raw = weights(N, K, 4)
    raw[7, 130] = NAN
    w4 = tw.fp4_quant(raw.to(DEV), group=group)
    x = acts(T, K, 2)
    got = tw.fp4_matmul(x.to(DEV), w4, out_dtype=F32).cpu()
    bad = torch.zeros(N, dtype=torch.bool)
    bad[7] = True
    assert got[:, bad].isnan().all() and got[:, ~bad].isfinite().all()
    got = tw.fp4_matmul_dx(acts(T, N, 2).to(DEV), w4, out_dtype=F32).cpu()
    bad = torch.zeros(K, dtype=torch.bool)
    bad[128:192] = True
    assert got[:, bad].isnan().all() and got[:, ~bad].isfinite().all()


@pytest.mark.parametrize("T", (1, 20))
def test_layer_nan_and_no_gate(T):
    d, f = 128, 256
    (g, gv), (u, uv), (w, wv) = (quantised(f, d, 64, i, 0.1) for i in range(3))
    x = acts(T, d, 1)
    # every gate closed: zeros
    shut = tw.Fp4(torch.full_like(g.q, 0xaa), torch.ones_like(g.scale), d, 64)  # -1
    y = tw.fp4_decode_fwd(x.abs().to(DEV), shut, u, w)
    assert torch.equal(y.cpu(), torch.zeros(T, d))
    x[0, 3] = NAN  # opens every gate of its token
    y = tw.fp4_decode_fwd(x.to(DEV), g, u, w).cpu()
    assert y[0].isnan().all() and y[1:].isfinite().all()


def test_sizes_of_numbers():
    """Activations and scales over the range that the documentation gives."""
    K = 256
    q, _ = ref.quant(weights(40, K, 1), 64)
    for es, ex in ((-66, -40), (-66, 100), (60, -100), (0, 110), (100, 0)):
        s = torch.full((K // 64, 40), 2.0 ** es).to(BF)
        w4, w = tw.Fp4(q.to(DEV), s.to(DEV), K, 64), ref.values(q, s, K, 64)
        for T in (3, 100):
            for dtype in (BF, F32):
                x = (acts(T, K, 1).clamp(-1, 1).double() * 2.0 ** ex).to(dtype)
                want, mag = ref.matmul(x, w)
                within(tw.fp4_matmul(x.to(DEV), w4, out_dtype=F32), want,
                       ref.bound(mag, want, K, F32))


# ---------------------------------------------------------------- gradient
@pytest.mark.parametrize("T", (4, 100))
def test_gradient_against_differences(T):
    """The product is linear in x: <dy, (x + e) W^T - x W^T> = <dX, e>, on whole
    numbers, exactly."""
    N, K = 96, 200
    g = gen(T)
    code = torch.randint(0, 16, (N, 256), generator=g).to(torch.uint8)
    code[:, K:] = 0
    w4 = tw.Fp4((code[:, ::2] + 16 * code[:, 1::2]).to(DEV),
                torch.full((4, N), 2.0, dtype=BF, device=DEV), K, 64)
    x, e, dy = (torch.randint(-3, 4, (T, n), generator=g).to(BF).to(DEV) for n in (K, K, N))
    diff = tw.fp4_matmul(x + e, w4, out_dtype=F32) - tw.fp4_matmul(x, w4, out_dtype=F32)
    dx = tw.fp4_matmul_dx(dy, w4, out_dtype=F32)
    assert float((dy.double() * diff.double()).sum()) == float((dx.double() * e.double()).sum())


# ---------------------------------------------------------------- streams, graphs, workspaces
def _calls():
    """Calls that take each path, as (name, function of nothing, its eager result)."""
    w4, _ = quantised(300, 520, 64, 1)
    ms = [quantised(256, 192, 32, i, 0.1)[0] for i in range(3)]
    out = []
    for T in (1, 14, 40, 200):
        for dtype in (BF, F32):
            x, dy = acts(T, 520, T, dtype).to(DEV), acts(T, 300, T, dtype).to(DEV)
            out.append((f"matmul {T} {dtype}", lambda x=x: tw.fp4_matmul(x, w4, out_dtype=F32)))
            out.append((f"dx {T} {dtype}", lambda d=dy: tw.fp4_matmul_dx(d, w4, out_dtype=F32)))
            if T <= 64:
                h = acts(T, 192, T, dtype).to(DEV)
                out.append((f"layer {T} {dtype}", lambda h=h: tw.fp4_decode_fwd(h, *ms)))
    raw = weights(90, 300, 2).to(DEV)
    out.append(("quant", lambda: tw.fp4_quant(raw, group=32).q))
    out.append(("dequant", lambda: tw.fp4_dequant(w4)))
    return [(n, f, f()) for n, f in out]


def test_results_repeat_bit_for_bit():
    for name, f, want in _calls():
        for _ in range(3):
            assert torch.equal(f(), want), name


def test_two_streams_at_once():
    calls = _calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for name, f, want in calls:
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append((name, f(), want))
    torch.cuda.synchronize()
    for res in got:
        for name, y, want in res:
            assert torch.equal(y, want), name


def test_graph_replays():
    """Captured, then replayed between eager calls: every replay as the eager result."""
    calls = _calls()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = [f() for _, f, _ in calls]
    for _ in range(4):
        for o in outs:
            o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        for (name, f, want), o in zip(calls, outs):
            assert torch.equal(o, want), name
            assert torch.equal(f(), want), name


def test_given_workspaces():
    """A workspace of the documented size is enough and is all that is written; a
    smaller one is refused."""
    w4, w = quantised(300, 520, 64, 1)
    for dx, call, size in ((False, tw.fp4_matmul, tw.fp4_matmul_workspace_bytes),
                           (True, tw.fp4_matmul_dx, tw.fp4_matmul_dx_workspace_bytes)):
        for T in (1, 14, 40, 200):
            for dtype, dt in ((BF, tw.TWELL_BF16), (F32, tw.TWELL_F32)):
                x = acts(T, 300 if dx else 520, T, dtype).to(DEV)
                need = size(dt, T, 300, 520)
                buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device=DEV)
                got = call(x, w4, out_dtype=F32, workspace=buf[256:256 + need])
                assert torch.equal(got, call(x, w4, out_dtype=F32))
                assert bool((buf[:256] == 0x5a).all()) and bool((buf[256 + need:] == 0x5a).all())
                if T == 200 and dtype == F32:
                    with pytest.raises(tw.TwellError, match="workspace"):
                        call(x, w4, workspace=buf[256:256 + need // 16 * 8])
    ms = [quantised(256, 192, 32, i, 0.1)[0] for i in range(3)]
    for T in (1, 14, 40):
        x = acts(T, 192, 1).to(DEV)
        need = tw.fp4_decode_workspace_bytes(tw.TWELL_BF16, T, 192, 256)
        buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device=DEV)
        got = tw.fp4_decode_fwd(x, *ms, workspace=buf[256:256 + need])
        assert torch.equal(got, tw.fp4_decode_fwd(x, *ms))
        assert bool((buf[:256] == 0x5a).all()) and bool((buf[256 + need:] == 0x5a).all())
        with pytest.raises(tw.TwellError, match="workspace"):
            tw.fp4_decode_fwd(x, *ms, workspace=buf[256:256 + need - 16])


def test_nothing_to_do():
    w4, _ = quantised(30, 200, 64, 1)
    assert tw.fp4_matmul(torch.empty(0, 200, device=DEV), w4).shape == (0, 30)
    assert tw.fp4_matmul_dx(torch.empty(0, 30, device=DEV), w4).shape == (0, 200)
    none = tw.empty_fp4(0, 200, 64, DEV)
    for T in (3, 100):
        assert tw.fp4_matmul(torch.ones(T, 200, device=DEV), none).shape == (T, 0)
        y = tw.fp4_matmul_dx(torch.empty(T, 0, device=DEV), none, out_dtype=F32)
        assert torch.equal(y, torch.zeros(T, 200, device=DEV))  # a sum of nothing
        y = tw.fp4_matmul(torch.empty(T, 0, device=DEV), tw.empty_fp4(30, 0, 64, DEV), out_dtype=F32)
        assert torch.equal(y, torch.zeros(T, 30, device=DEV))
    ms = [quantised(128, 64, 32, i, 0.1)[0] for i in range(3)]
    assert tw.fp4_decode_fwd(torch.empty(0, 64, device=DEV), *ms).shape == (0, 64)
    assert tw.fp4_quant(torch.empty(0, 5, device=DEV)).rows == 0
    assert tw.fp4_dequant(none).shape == (0, 200)


def test_sums_of_nothing_for_many_tokens():
    """No columns, and more tokens than a launch of the few-token kernels has workgroups for."""
    for T, dtype in ((300, BF), (5 * (1 << 22) + 7, F32)):
        x, w4 = torch.empty(T, 0, device=DEV, dtype=dtype), tw.empty_fp4(2, 0, 64, DEV)
        out = torch.full((T, 2), 7.0, device=DEV, dtype=dtype)
        tw.fp4_matmul(x, w4, out=out, out_dtype=dtype)
        assert not bool(out.any())


def test_kernels_are_timed():
    t, seen = tw.KernelTimer(), {}
    w4, ms = coded(300, 520, 64, 1)[0], [coded(256, 192, 32, i)[0] for i in range(3)]
    x = acts(40, 520, 1, F32).to(DEV)
    for call in (lambda: tw.fp4_matmul(x, w4, timing=t),
                 lambda: tw.fp4_matmul_dx(x[:2, :300], w4, timing=t),
                 lambda: tw.fp4_decode_fwd(x[:2, :192], *ms, timing=t),
                 lambda: tw.fp4_quant(x, timing=t), lambda: tw.fp4_dequant(w4, timing=t)):
        call()
        torch.cuda.synchronize()
        t.add(seen)
    assert {"fp4_pack", "fp4_rows", "fp4_cols", "fp4_dequant", "fp4_quant", "fp4_gate_up",
            "fp4_down"} <= set(seen)
    assert all(0 < ms < 10 for ms in seen.values())


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("T", (1, 6, 40))
@pytest.mark.parametrize("group", GROUPS)
def test_block_in_four_bits(T, group):
    """Norm, sparse layer, norm, projection, all weights in 4 bits, each stage
    against its formula on what the stage before gave."""
    d, f, n = 320, 640, 200
    g = gen(1)
    w = {"g": torch.randn(f, d, generator=g) / d ** 0.5, "u": torch.randn(f, d, generator=g) / d ** 0.5,
         "d": torch.randn(f, d, generator=g) / f ** 0.5, "p": torch.randn(n, d, generator=g) / d ** 0.5}
    w["g"][:, 0] = -1.5
    w4 = {k: tw.fp4_quant(v.to(DEV), group=group) for k, v in w.items()}
    v = {k: ref.values(*ref.quant(m, group), d, group) for k, m in w.items()}
    gain = torch.ones(d, device=DEV)
    h0 = torch.randn(T, d, generator=g)
    h0[:, 0] = 1
    n1, h1 = tw.rmsnorm_fwd(torch.zeros(T, d, device=DEV), gain, residual=h0.to(DEV))
    y = tw.fp4_decode_fwd(n1, w4["g"], w4["u"], w4["d"])
    want, tol = ref.layer(n1, v["g"], v["u"], v["d"])
    within(y, want, tol)
    n2, _ = tw.rmsnorm_fwd(y, gain, residual=h1)
    out = tw.fp4_matmul(n2, w4["p"])
    want, mag = ref.matmul(n2, v["p"])
    within(out, want, ref.bound(mag, want, d, BF))
    dn = tw.fp4_matmul_dx(out, w4["p"], out_dtype=F32)
    want, mag = ref.matmul(out, v["p"].t())
    within(dn, want, ref.bound(mag, want, n, F32))
    # a long prefill multiplies by the values themselves
    long = tw.fp4_dequant(w4["g"])
    assert torch.equal(long.cpu().double(), v["g"])


def test_the_example_serves_from_four_bits():
    """One token, several and a prefill: the calls it makes, on what the stages give."""
    from test_gpu_prenorm_block import _example
    block, a, h0 = _example().make_case(150, 256, 512, 136, density=0.05)
    block.freeze(64)
    w = block.w4
    for T in (1, 20, 150):
        out, h2 = block.serve_fp4(a[:T], h0[:T])
        block.check()
        n1, h1 = tw.rmsnorm_fwd(a[:T], block.master["g1"], residual=h0[:T], eps=block.eps)
        v = [w[k].float().double().cpu() for k in ("wg", "wu", "wd")]
        y, tol = ref.layer(n1, *v)
        # the prefill's layer rounds the gates to bfloat16, half a step of each
        if T > tw.DECODE_T:
            n = n1.double().cpu()
            h = (n @ v[0].t()).clamp(min=0)
            tol = tol + ref.UBF * ((h * (n @ v[1].t())).abs() @ v[2].abs())
        within(h2, h1.double().cpu() + y, tol + ref.U32 * (h1.double().cpu().abs() + y.abs()))
        n2, _ = tw.rmsnorm_fwd(h2, block.master["g2"], eps=block.eps)
        want, mag = ref.matmul(n2, w["proj"].float().double().cpu())
        # n2 of the stored h2 is a step of bfloat16 from the example's at most
        within(out, want, ref.bound(mag, want, 256, BF) + 2 * ref.UBF * mag)
