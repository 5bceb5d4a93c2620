"""GPU: the GEMM with bias, activation and residual in its epilogue and its gradient, the norms around a block, and
the balance loss, against 64-bit forms, and a run of them together.

Bounds count roundings: half a step of the output's type (2^-8 of the value for bf16, 2^-4 for e4m3, or 2^-10 of the
scale below its normal range), plus what FP32 arithmetic can have moved the value by (`noise`), each derived where it
is used.  u below is 2^-24.  Casts behind such a value may round the other way: what code and scale stand for must
lie within half a step plus twice the noise.
"""
import math

import pytest
import torch

from tests.test_gpu_moe import near, scale_near, values

pytestmark = pytest.mark.gpu

BLOCK = 128
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dgm():
    from moe_grouped_gemm_weight_b200 import build
    build.build()
    import moe_grouped_gemm_weight_b200 as dg
    dg.dg_set_num_sms(0)
    assert dg.dg_get_device_error() == 0
    return dg


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def framed(*shape, dtype=torch.bfloat16):
    """A tensor with 128 marked elements before and behind it, and a check that they are still there."""
    n = math.prod(shape)
    buf = torch.full((n + 256,), 9, device="cuda").to(dtype) if dtype != torch.uint8 else torch.full((n + 256,), 0x5A, dtype=dtype, device="cuda")
    mark = buf[0].clone()
    t = buf[128:128 + n].view(*shape)
    return t, lambda: bool((buf[:128] == mark).all() and (buf[128 + n:] == mark).all())


def inside(got, want, tol, what):
    """|got - want| <= tol; NaN where want is NaN; equal where want is infinite."""
    got = got.double()
    nan = want.isnan()
    assert bool((got.isnan() == nan).all()), f"{what}: NaN elsewhere"
    inf = want.isinf()
    assert bool((got[inf] == want[inf]).all()), f"{what}: infinities"
    far = ((got - want).abs() - tol)[~(nan | inf)]
    assert far.numel() == 0 or not bool((far > 0).any()), f"{what}: off by {float(far.max())} beyond the bound"


def cast1x128(x):
    R, K = x.shape
    b = x.float().view(R, K // BLOCK, BLOCK)
    amax = b.abs().amax(dim=2, keepdim=True).clamp_min(1e-4)
    q = (b * (torch.full_like(amax, 448.0) / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(R, K), (amax / 448.0)[:, :, 0].t().contiguous()


def cast128x128(x):
    R, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, 0, 0, -R % BLOCK)).view(-1, BLOCK, K // BLOCK, BLOCK)
    amax = b.abs().amax(dim=(1, 3), keepdim=True).clamp_min(1e-4)
    q = (b * (torch.full_like(amax, 448.0) / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(-1, K)[:R], (amax / 448.0)[:, 0, :, 0].contiguous()


# --------------------------------------------------------------------------------------------- activations

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
C2 = math.sqrt(8 / math.pi)


def number(dg, act):
    return getattr(dg, "DG_ACT_" + act.upper())


def act64(z, act):
    """Value, slope, and the largest part of 2^-24 that FP32 steps may have added to each (sums of the terms'
    magnitudes times their count of roundings)."""
    if act == "none":
        return z, torch.ones_like(z), 0 * z, 0 * z
    if act == "relu":
        return torch.where(z.isnan(), z, z.clamp_min(0)), (z > 0).double(), 0 * z, 0 * z
    if act == "gelu":
        # the tail 7.2 units from the fit and its Horner sums, the exponential 3 and its exponent's two roundings 1.2 z^2, the
        # product 1; then one product, and for positive z one subtraction
        q = 0.5 * torch.special.erfc(z.abs() / math.sqrt(2))
        phi = torch.where(z > 0, 1 - q, q)
        dens = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        ez = 1.2 * (z * z).clamp(max=300.0)
        return (z * phi, phi + z * dens, z.abs() * ((16 + ez) * q + 2 * phi),
                (16 + ez) * q + 2 * phi + (10 + ez) * (z * dens).abs())
    g = C2 * (z + 0.044715 * z ** 3) if act == "gelu_tanh" else z
    up = C2 * (1 + 3 * 0.044715 * z * z) if act == "gelu_tanh" else torch.ones_like(z)
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    # the sigmoid 8 units, and of its argument the roundings times its slope: 1.3 |g| units of the exponent, 4 |g| before that
    # (gelu_tanh)
    arg = (5.3 if act == "gelu_tanh" else 1.3) * g.abs()
    rel, rel_c = 8 + arg * c, 8 + arg * s
    value, slope = z * s, s + z * up * s * c
    return value, slope, value.abs() * (rel + 2), (s * (rel + 2) + (z * up * s * c).abs() * (rel + rel_c + 6))


# ------------------------------------------------------------------------------------ GEMM with an epilogue


class Gemm:
    def __init__(self, dg, M, N, K, seed, bias=True, residual=True):
        g = gen(seed)
        self.M, self.N, self.K, self.act = M, N, K, None
        self.A, sa = cast1x128(randn(g, M, K))
        self.stride = dg.dg_get_tma_aligned_size(M, 4) + 4
        self.sa = torch.full((K // BLOCK, self.stride), NAN, device="cuda")
        self.sa[:, :M] = sa
        self.B, self.sb = cast128x128(randn(g, N, K) * (1.5 / math.sqrt(K)))
        self.bias = 0.5 * randn(g, N) if bias else None
        self.residual = randn(g, M, N).bfloat16() if residual else None

    def exact(self, act):
        """z, v and their noise."""
        a = self.A.double() * self.sa[:, :self.M].double().t().repeat_interleave(BLOCK, dim=1)
        b = self.B.double() * self.sb.double().repeat_interleave(BLOCK, dim=0)[:self.N].repeat_interleave(BLOCK, dim=1)
        z, mag = a @ b.t(), a.abs() @ b.abs().t()
        # each K block: four steps of 32 products whose sum the tensor core may cut at 2^-22 of the largest of them;
        # its scaling 2 roundings; one addition per block and per slice of a split K
        noise = (4 * 4 + 2 + self.K // BLOCK + 8) * U * mag
        if self.bias is not None:
            z = z + self.bias.double()
            noise = noise + U * z.abs()
        v, slope, units, _ = act64(z, act)
        # no activation's slope passes 1.2 in size; v itself, and its sum with the residual, rounded
        nv = 1.2 * noise + U * (units + v.abs())
        if self.residual is not None:
            v = v + self.residual.double()
            nv = nv + U * v.abs()
        return z, v, noise, nv

    def check(self, dg, act, outs, in_place=False):
        M, N = self.M, self.N
        D, d_ok = framed(M, N)
        Z, z_ok = framed(M, N)
        Q, q_ok = framed(M, N, dtype=torch.uint8)
        sq = torch.full((max(N // BLOCK, 1), self.stride), -7.0, device="cuda")
        res = self.residual
        if in_place:
            D.copy_(res)
            res = D
        dg.dg_fp8_gemm_nt_epilogue(D if "D" in outs else None, self.A, self.sa, self.stride, self.B, self.sb,
                                   bias=self.bias, act=number(dg, act), residual=res, Z=Z if "Z" in outs else None,
                                   Q=Q if "Q" in outs else None, sq=sq if "Q" in outs else None, sq_stride=self.stride)
        z, v, noise, nv = self.exact(act)
        assert d_ok() and z_ok() and q_ok()
        if "D" in outs:
            inside(D, v, 2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * nv, "D")
        else:
            assert bool((D == 9).all())
        if "Z" in outs:
            inside(Z, z, 2.0 ** -8 * z.abs() + (1 + 2.0 ** -8) * noise, "Z")
        if "Q" in outs:
            tile = lambda x: x.reshape(M, -1, BLOCK)  # noqa: E731
            scale_near(sq[:, :M].t(), tile(v), tile(nv), (2,), "sq")
            near(Q, sq[:, :M].t().repeat_interleave(BLOCK, dim=1), v, nv, "Q")
            assert bool((sq[:, M:] == -7).all())
        assert dg.dg_get_device_error() == 0
        return D, Z, Q, sq


# Few rows: one and several tiles, split over clusters and not; many rows: each tile width, ragged edges, a short K
# (the epilogue staged at once), a K-split last wave.
SHAPES = [(1, 8, 128), (1, 2112, 7168), (7, 24, 256), (33, 520, 2048), (64, 4096, 1024), (128, 256, 384), (100, 24576, 256),
          (129, 8, 128), (150, 264, 512), (300, 2048, 512), (1001, 2112, 1536), (700, 2048, 4096), (1500, 4096, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_epilogue_shapes(dgm, M, N, K):
    for i, act in enumerate(ACTS):
        G = Gemm(dgm, M, N, K, seed=M + N + i, bias=i != 1, residual=i != 2)
        G.check(dgm, act, ["DZ", "D", "Z", "DZ", "D"][i])


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (5, 256, 2048), (64, 4096, 1024), (127, 2048, 256), (100, 24576, 256),
                                   (129, 128, 128), (300, 640, 512), (700, 2048, 4096), (1300, 4096, 4096),
                                   (257, 24576, 256)])
def test_gemm_epilogue_cast(dgm, M, N, K):
    for i, act in enumerate(ACTS):
        G = Gemm(dgm, M, N, K, seed=M + N + i, bias=i != 3, residual=i % 2 == 0)
        G.check(dgm, act, ["Q", "QZ", "DQ", "DQZ", "QZ"][i])


@pytest.mark.parametrize("M,N,K", [(3, 264, 256), (300, 264, 512), (1500, 4096, 4096)])
def test_gemm_epilogue_adds_to_the_residual_in_place(dgm, M, N, K):
    G = Gemm(dgm, M, N, K, seed=1)
    G.check(dgm, "gelu", "DZ", in_place=True)


@pytest.mark.parametrize("K", [128, 256, 512, 640, 1024, 1152, 1536, 2048, 2176, 2304])
@pytest.mark.parametrize("M,N", [(2500, 2056), (4100, 520), (2500, 2048)])
def test_gemm_epilogue_residual_over_several_tiles(dgm, M, N, K):
    # more tiles than SMs, of one group of K blocks up to more than the scale ring holds
    G = Gemm(dgm, M, N, K, seed=K)
    first = [t.clone() for t in G.check(dgm, "none", "D" if N % BLOCK else "DQ")]
    for _ in range(3):  # the same again: what comes early in shared memory does not show
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, G.check(dgm, "none", "D" if N % BLOCK else "DQ")))
    G.check(dgm, "silu", "DZ", in_place=True)


@pytest.mark.parametrize("M", [2, 200])
@pytest.mark.parametrize("act", ACTS)
def test_gemm_epilogue_extreme_values(dgm, M, act):
    G = Gemm(dgm, M, 256, 128, seed=3, residual=False)
    special = [0.0, -0.0, 1e30, -1e30, 3e38, -3e38, 50.0, -50.0, 88.0, -88.0, -12.9, -13.4, -100.0, -127.0, NAN, INF, 1e-30, -5.0, 1.5, NAN]
    G.B.view(torch.uint8).zero_()  # z is the bias
    G.bias = torch.zeros(256, device="cuda")
    G.bias[:len(special)] = torch.tensor(special, device="cuda")
    D, Z, Q, sq = framed(M, 256)[0], framed(M, 256)[0], torch.zeros(M, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, G.stride, device="cuda")
    dgm.dg_fp8_gemm_nt_epilogue(D, G.A, G.sa, G.stride, G.B, G.sb, bias=G.bias, act=number(dgm, act), Z=Z, Q=Q, sq=sq,
                                sq_stride=G.stride)
    z = G.bias.double().expand(M, 256)
    want, _, units, _ = act64(z, act)
    # a sigmoid or tail below 2^-126 is zero
    flush = 2.0 ** -126 * z.abs().nan_to_num(posinf=0.0)
    inside(D, want, 2.0 ** -8 * want.abs() + U * units.nan_to_num(posinf=0.0) + flush, "D")
    inside(Z, z, 2.0 ** -8 * z.abs(), "Z")
    assert bool(((Q[:, 14] & 0x7F) == 0x7F).all())  # NaN stays one, in the cast too
    # ... and does not reach the second tile, whose scale is the least one
    assert bool((sq[1, :M] * 448 == torch.tensor(1e-4, device="cuda") / 448 * 448).all() or (sq[1, :M] > 0).all())
    assert bool((Q[:, 128:] & 0x7F == 0).all())


def test_gemm_epilogue_is_the_gemm(dgm):
    """Without bias, activation and residual D is dg_fp8_gemm_nt's, bit for bit."""
    for M, N, K in [(1, 2112, 7168), (64, 4096, 1024), (300, 264, 512), (1500, 4096, 4096)]:
        G = Gemm(dgm, M, N, K, seed=5)
        D, D2 = framed(M, N)[0], framed(M, N)[0]
        dgm.dg_fp8_gemm_nt_epilogue(D, G.A, G.sa, G.stride, G.B, G.sb)
        dgm.dg_fp8_gemm_nt(D2, G.A, G.sa, G.stride, G.B, G.sb)
        assert torch.equal(D.view(torch.int16), D2.view(torch.int16))


# ------------------------------------------------------------------------------------- its gradient


@pytest.mark.parametrize("M,N", [(1, 128), (127, 256), (128, 128), (129, 640), (300, 2048), (1001, 384), (4096, 128), (640, 7168)])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_gradient(dgm, M, N, act):
    g = gen(M + N)
    dD = (0.02 * randn(g, M, N)).bfloat16()
    Z = (1.5 * randn(g, M, N)).bfloat16()
    Z[0, :10] = torch.tensor([0.0, -0.0, 40.0, -40.0, 88.0, -100.0, 1e30, -1e30, 13.5, -13.5], device="cuda").bfloat16()
    if act not in ("none", "relu") and M > 1:  # a NaN is its own element's alone
        one = Z.clone()
        one[1, 4] = NAN
        outs = [torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(-(-M // 128) * 128, N, dtype=torch.uint8, device="cuda")]
        dgm.dg_epilogue_bwd(outs[0], torch.zeros(N // BLOCK, M, device="cuda"), M, outs[1], torch.zeros(-(-M // 128), N, device="cuda"), N,
                            dD, Z=one, act=number(dgm, act))
        for q in outs:
            nan = torch.nonzero((q & 0x7F) == 0x7F).tolist()
            assert nan == [[1, 4]]
    R = -(-M // BLOCK) * BLOCK
    Qr, qr_ok = framed(M, N, dtype=torch.uint8)
    Qc, qc_ok = framed(R, N, dtype=torch.uint8)
    sr, sc = torch.full((N // BLOCK, M + 5), -7.0, device="cuda"), torch.full((R // BLOCK, N + 3), -7.0, device="cuda")
    dbias, b_ok = framed(N, dtype=torch.float32)
    ws, ws_ok = framed(dgm.dg_get_bias_workspace(M, N), dtype=torch.float32)
    ws.fill_(NAN)
    dgm.dg_epilogue_bwd(Qr, sr, M + 5, Qc, sc, N + 3, dD, Z=None if act == "none" else Z, act=number(dgm, act), dbias=dbias, ws=ws)
    assert qr_ok() and qc_ok() and b_ok() and ws_ok()
    _, slope, _, units = act64(Z.double(), act)
    dz = dD.double() * slope
    # past the bounds of the argument the slope is off by up to 2^-45
    noise = dD.double().abs() * (U * (units + slope.abs()) + 2.0 ** -45) + 2.0 ** -100
    tile = lambda x: x.reshape(M, -1, BLOCK)  # noqa: E731
    scale_near(sr[:, :M].t(), tile(dz), tile(noise), (2,), "sr")
    near(Qr, sr[:, :M].t().repeat_interleave(BLOCK, dim=1), dz, noise, "Qr")
    assert bool((sr[:, M:] == -7).all() and (sc[:, N:] == -7).all())
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, R - M)).reshape(R // BLOCK, BLOCK, N)  # noqa: E731
    scale_near(sc[:, :N], pad(dz), pad(noise), (1,), "sc")
    near(Qc, sc[:, :N].repeat_interleave(BLOCK, dim=0), pad(dz).reshape(R, N), pad(noise).reshape(R, N), "Qc")
    assert bool((Qc[M:] & 0x7F == 0).all())
    # at most 8 + 9 additions in a row block, and one per block
    inside(dbias, dz.sum(dim=0), noise.sum(dim=0) + (20 + R // BLOCK) * U * dz.abs().sum(dim=0), "dbias")
    # without the bias, the same casts
    Qr2, Qc2, sr2, sc2 = torch.zeros_like(Qr), torch.zeros_like(Qc), torch.full_like(sr, -7.0), torch.full_like(sc, -7.0)
    dgm.dg_epilogue_bwd(Qr2, sr2, M + 5, Qc2, sc2, N + 3, dD, Z=Z, act=number(dgm, act))
    assert torch.equal(Qr, Qr2) and torch.equal(Qc, Qc2) and torch.equal(sr, sr2) and torch.equal(sc, sc2)


@pytest.mark.parametrize("act", ACTS[2:])
def test_activation_slopes_against_differences(act):
    z = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    h = 1e-5
    num = (act64(z + h, act)[0] - act64(z - h, act)[0]) / (2 * h)
    # the third derivatives stay below 3: h^2 / 6 of that, and the difference's rounding
    assert float((act64(z, act)[1] - num).abs().max()) < 3 * h * h + 1e-9


def test_epilogue_gradient_without_rows(dgm):
    dbias = torch.full((256,), 3.0, device="cuda")
    none = torch.zeros(0, 256, dtype=torch.uint8, device="cuda")
    sr, sc = torch.zeros(2, 4, device="cuda"), torch.zeros(0, 256, device="cuda")
    dD = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    dgm.dg_epilogue_bwd(none, sr, 4, none, sc, 256, dD, dbias=dbias, ws=torch.zeros(0, device="cuda"))
    assert bool((dbias == 0).all())
    A, sa, B, sb = none[:, :128].contiguous(), torch.zeros(1, 4, device="cuda"), torch.zeros(256, 128, dtype=torch.uint8, device="cuda"), torch.zeros(2, 1, device="cuda")
    dgm.dg_fp8_gemm_nt_epilogue(dD, A, sa, 4, B, sb, bias=dbias, Z=dD, Q=none, sq=sr, sq_stride=4)
    dgm.dg_norm_residual(dD, dD, dD, H=dD, Q=none, sq=sr, sq_stride=4)


# -------------------------------------------------------------------------------------------- norms


def stream(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else U


# roundings of a sum over a row: 17 products a thread, their halves, two shuffles of 5 steps, the join, the mean and eps
ROW = 17 + 1 + 5 + 5 + 1 + 3


class Norm:
    def __init__(self, T, N, dtype, post_norm, gate=True, wpost=True, wpre=True, X=True, Y=True, seed=0):
        g = gen(seed + T + N)
        self.T, self.N, self.dtype, self.post_norm, self.scale, self.eps = T, N, dtype, post_norm, 0.7, 1e-5
        self.X = (2 * randn(g, T, N)).to(stream(dtype)) if X else None
        self.Y = randn(g, T, N).bfloat16() if Y else None
        self.w_post = 1 + 0.3 * randn(g, N) if wpost else None
        self.w_pre = 1 + 0.3 * randn(g, N) if wpre else None
        self.gate = randn(g, T) if gate else None
        self.dU = (0.1 * randn(g, T, N)).to(stream(dtype))
        self.dH = (0.1 * randn(g, T, N)).bfloat16()

    def inputs(self):
        return dict(w_post=self.w_post, gate=self.gate, w_pre=self.w_pre, post_norm=self.post_norm, scale=self.scale)

    def wide(self):
        one = lambda t, n: torch.ones(n, dtype=torch.float64, device="cuda") if t is None else t.double()  # noqa: E731
        zero = torch.zeros(self.T, self.N, dtype=torch.float64, device="cuda")
        x = zero if self.X is None else self.X.double()
        y = zero if self.Y is None else self.Y.double()
        return x, y, one(self.w_post, self.N), one(self.gate, self.T)[:, None], one(self.w_pre, self.N)

    def exact(self):
        x, y, wp, gt, wn = self.wide()
        ry = (y.square().mean(dim=1, keepdim=True) + self.eps).rsqrt() if self.post_norm and self.Y is not None else torch.ones_like(gt)
        z = self.scale * gt * wp * ry * y
        u = x + z
        # the reciprocal root halves its argument's error; k = scale r gate, k y, the fused product and sum
        nu = (ROW / 2 + 5) * U * z.abs() + U * u.abs()
        ru = (u.square().mean(dim=1, keepdim=True) + self.eps).rsqrt()
        rel_r = (ROW / 2 + 1) * U + nu.square().mean(dim=1, keepdim=True).sqrt() * ru
        h = u * ru * wn
        nh = ru * wn.abs() * nu + h.abs() * (rel_r + 2 * U)
        return dict(ry=ry, ru=ru, u=u, h=h, nu=nu, nh=nh, rel_r=rel_r, z=z)


def run_norm(dg, n, out="UHQR"):
    T, N = n.T, n.N
    U_, u_ok = framed(T, N, dtype=stream(n.dtype))
    H, h_ok = framed(T, N)
    Q, q_ok = framed(T, N, dtype=torch.uint8)
    stride = T + 3
    sq = torch.full((max(N // BLOCK, 1), stride), -7.0, device="cuda")
    rstd, r_ok = framed(T, 2, dtype=torch.float32)
    dg.dg_norm_residual(U_ if "U" in out else None, n.X, n.Y, H=H if "H" in out else None, Q=Q if "Q" in out else None,
                        sq=sq if "Q" in out else None, sq_stride=stride, rstd=rstd if "R" in out else None, eps=n.eps, **n.inputs())
    assert u_ok() and h_ok() and q_ok() and r_ok()
    return U_, H, Q, sq, rstd


NORM_SIZES = [(1, 8), (3, 24), (5, 128), (64, 7168), (33, 8200), (7, 16384), (301, 2120), (1000, 640), (2, 8192), (9, 8320)]


@pytest.mark.parametrize("T,N", NORM_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("post_norm", [False, True])
def test_norm_residual(dgm, T, N, dtype, post_norm):
    for i in range(4):
        n = Norm(T, N, dtype, post_norm, gate=i != 1, wpost=i != 2, wpre=i != 3, X=i != 2 or dtype == "fp32", seed=i)
        if i == 3 and T > 2:  # rows of zeros and of very different sizes
            n.X[0], n.Y[0] = 0, 0
            n.X[1] *= 1e-4
            n.Y[2] *= 1e4
        out = "UHR" + ("Q" if N % BLOCK == 0 else "")
        dt = dtype if n.X is not None or dtype == "bf16" else "bf16"
        n.dtype = dt
        U_, H, Q, sq, rstd = run_norm(dgm, n, out)
        w = n.exact()
        inside(U_, w["u"], half_step(dt) * w["u"].abs() + 2 * w["nu"], "U")
        inside(H, w["h"], 2.0 ** -8 * w["h"].abs() + 2 * w["nh"] + 2.0 ** -133, "H")
        inside(rstd[:, :1], w["ry"], (ROW / 2 + 1) * U * w["ry"], "r_y")
        inside(rstd[:, 1:], w["ru"], w["rel_r"] * w["ru"] + U * w["ru"], "r_u")
        if "Q" in out:
            tile = lambda x: x.reshape(T, -1, BLOCK)  # noqa: E731
            scale_near(sq[:, :T].t(), tile(w["h"]), tile(w["nh"]), (2,), "sq")
            near(Q, sq[:, :T].t().repeat_interleave(BLOCK, dim=1), w["h"], w["nh"], "Q")
            assert bool((sq[:, T:] == -7).all())


def test_norm_alone_in_place_and_single_outputs(dgm):
    n = Norm(37, 256, "fp32", False, Y=False)
    U_, H, Q, sq, rstd = run_norm(dgm, n)
    assert torch.equal(U_, n.X) and bool((rstd[:, 0] == 1).all())
    n = Norm(37, 256, "bf16", True)
    U_, H, Q, sq, rstd = run_norm(dgm, n)
    for out, i in (("U", 0), ("H", 1), ("Q", 2), ("R", 4)):
        assert torch.equal(run_norm(dgm, n, out)[i].view(torch.uint8), (U_, H, Q, sq, rstd)[i].view(torch.uint8)), out
    x = n.X.clone()
    dgm.dg_norm_residual(x, x, n.Y, eps=n.eps, **n.inputs())
    assert torch.equal(x, U_)


def test_norm_of_values_at_the_limits(dgm):
    n = Norm(5, 256, "fp32", True)
    n.X[0, 3] = INF
    n.X[1, 4] = NAN
    n.Y[2, 5] = NAN
    n.X[3] = 1e25   # squares leave FP32
    n.Y[4] = 0      # a block without output
    U_, H, Q, sq, rstd = run_norm(dgm, n)
    assert U_[0, 3] == INF and bool(H[0, 3].isnan()) and bool((H[0, :3] == 0).all())
    assert bool(H[1].isnan().all() and U_[1].isnan().sum() == 1)
    assert bool(U_[2].isnan().all())
    assert bool((H[3] == 0).all() and (rstd[3, 1] == 0))
    assert torch.equal(U_[4], n.X[4])
    w = n.exact()
    inside(H[4:], w["h"][4:], 2.0 ** -8 * w["h"][4:].abs() + 2 * w["nh"][4:], "H")


class NormGrad:
    """The gradient's formula in 64 bits from a call's inputs, with its noise."""

    def __init__(self, n, U_, rstd, dU, dH, parts):
        _, y, wp, gt, wn = n.wide()
        zero = torch.zeros(n.T, n.N, dtype=torch.float64, device="cuda")
        dU = zero if dU is None else dU.double()
        dH = zero if dH is None else dH.double()
        ry, ru = rstd[:, :1].double(), rstd[:, 1:].double()
        a, b, g, k = U_.double() * ru, y * ry, wn * dH, n.scale * gt
        mean, size = (a * g).mean(dim=1, keepdim=True), (a * g).abs().mean(dim=1, keepdim=True)
        self.du = dU + ru * (g - a * mean)
        # the mean 2 roundings a term and the row's sum; then the difference, the product and the sum
        ndu = U * (self.du.abs() + 3 * ru * (g.abs() + (a * mean).abs()) + ru * a.abs() * (ROW + 4) * size)
        d = k * self.du
        self.dw_pre = (dH * a).sum(dim=0)
        steps = -(-n.T // parts) + -(-parts // 8) + 16  # a part's rows, every eighth part, the join
        self.npre = (steps + 2) * U * (dH * a).abs().sum(dim=0)
        self.dw_post = (d * b).sum(dim=0)
        self.npost = (k * b).abs().mul(ndu).sum(dim=0) + (steps + 4) * U * (d * b).abs().sum(dim=0)
        # sum(du w b) as sum(e w b) - r m sum(a w b), e = dU + r w_pre dH: each a row's sum of terms with 5 roundings, then r m
        # with the mean's error and two roundings, and their difference
        e, rm, wb = dU + ru * g, ru * mean, wp * b
        dot = (self.du * wb).sum(dim=1)
        left, right = (e * wb).abs().sum(dim=1), (a * wb).abs().sum(dim=1)
        ndot = (ROW + 5) * U * (left + rm[:, 0].abs() * right) + ((ROW + 4) * ru * size)[:, 0] * U * right + 3 * U * (left + rm[:, 0].abs() * right)
        del e, wb
        self.dgate, self.ngate = n.scale * dot, n.scale * ndot + U * (n.scale * dot).abs()
        self.dY = wp * d
        self.ny = wp.abs() * k.abs() * ndu + 3 * U * self.dY.abs()
        if n.post_norm:
            sub = k * b * dot[:, None] / n.N
            self.ny = ry * (self.ny + (k * b).abs() * ndot[:, None] / n.N + 6 * U * (self.dY.abs() + sub.abs()))
            self.dY = ry * (self.dY - sub)
        self.ndu = ndu


def run_norm_bwd(dg, n, U_, rstd, dU, dH, out="XYGPN"):
    T, N = n.T, n.N
    bufs = dict(X=framed(T, N, dtype=stream(n.dtype)), Y=framed(T, N), G=framed(T, dtype=torch.float32),
                P=framed(N, dtype=torch.float32), N=framed(N, dtype=torch.float32))
    t = {k: v[0] if k in out else None for k, v in bufs.items()}
    ws, ws_ok = framed(dg.dg_get_norm_workspace(T, N), dtype=torch.float32)
    ws.fill_(NAN)
    dg.dg_norm_residual_bwd(t["X"], dU, dH, U_, n.Y, rstd, dY=t["Y"], dgate=t["G"], dw_post=t["P"], dw_pre=t["N"],
                            ws=ws if "P" in out or "N" in out else None, **n.inputs())
    assert ws_ok() and all(v[1]() for v in bufs.values())
    return t


@pytest.mark.parametrize("T,N", NORM_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("post_norm", [False, True])
def test_norm_gradient(dgm, T, N, dtype, post_norm):
    for i in range(4):
        n = Norm(T, N, dtype, post_norm, gate=i != 1, wpost=i != 2, wpre=i != 3, seed=10 + i)
        if i == 3 and T > 2:
            n.X[0], n.Y[0] = 0, 0
            n.Y[1] *= 1e-3
        w = n.exact()
        U_, rstd = w["u"].to(stream(dtype)), torch.cat([w["ry"], w["ru"]], dim=1).float()
        dU, dH = (None if i == 1 else n.dU), (None if i == 2 else n.dH)
        t = run_norm_bwd(dgm, n, U_, rstd, dU, dH)
        e = NormGrad(n, U_, rstd, dU, dH, min(T, 148))
        inside(t["X"], e.du, half_step(dtype) * e.du.abs() + 2 * e.ndu, "dX")
        inside(t["Y"], e.dY, 2.0 ** -8 * e.dY.abs() + 2 * e.ny + 2.0 ** -133, "dY")
        inside(t["G"], e.dgate, e.ngate, "dgate")
        inside(t["P"], e.dw_post, e.npost, "dw_post")
        inside(t["N"], e.dw_pre, e.npre, "dw_pre")


def test_norm_gradient_parts_and_in_place(dgm):
    n = Norm(300, 384, "fp32", True)
    w = n.exact()
    U_, rstd = w["u"].float(), torch.cat([w["ry"], w["ru"]], dim=1).float()
    every = run_norm_bwd(dgm, n, U_, rstd, n.dU, n.dH)
    for out in ("X", "Y", "G", "P", "N", "XN", "YP"):
        t = run_norm_bwd(dgm, n, U_, rstd, n.dU, n.dH, out)
        for k in out:
            assert torch.equal(t[k], every[k]), (out, k)
    d = n.dU.clone()
    dgm.dg_norm_residual_bwd(d, d, n.dH, U_, n.Y, rstd, **n.inputs())
    assert torch.equal(d, every["X"])
    # without the block's output: the stream's norm alone
    n.Y = None
    t = run_norm_bwd(dgm, n, U_, rstd, n.dU, n.dH, "XN")
    assert torch.equal(t["X"], every["X"]) and torch.equal(t["N"], every["N"])
    # without tokens the sums are zero
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    a, b = torch.ones(384, device="cuda"), torch.ones(384, device="cuda")
    dgm.dg_norm_residual_bwd(z(0, 384), z(0, 384), None, z(0, 384), z(0, 384, dt=torch.bfloat16), z(0, 2), dw_post=a, dw_pre=b, ws=z(0))
    assert bool((a == 0).all() and (b == 0).all())


@pytest.mark.parametrize("post_norm", [False, True])
def test_norm_gradient_against_differences(dgm, post_norm):
    # <dU, U> + <dH, H> in 64 bits as a function of each input.  Steps of 1e-4 leave 1e-8 of third derivatives and 1e-11
    # of rounding; the inputs of the gradient are in FP32 (r as rounded: 2^-24), its dY in bf16.
    n = Norm(4, 16, "fp32", post_norm)
    x, y, wp, gt, wn = n.wide()
    leaves = dict(x=x.clone(), y=y.clone(), wp=wp.clone(), gt=gt.clone(), wn=wn.clone())

    def loss(v):
        ry = (v["y"].square().mean(dim=1, keepdim=True) + n.eps).rsqrt() if post_norm else 1.0
        u = v["x"] + n.scale * v["gt"] * v["wp"] * ry * v["y"]
        h = u * (u.square().mean(dim=1, keepdim=True) + n.eps).rsqrt() * v["wn"]
        return float((n.dU.double() * u).sum() + (n.dH.double() * h).sum())

    w = n.exact()
    t = run_norm_bwd(dgm, n, w["u"].float(), torch.cat([w["ry"], w["ru"]], dim=1).float(), n.dU, n.dH)
    got = dict(x=t["X"], y=t["Y"], wp=t["P"], gt=t["G"][:, None], wn=t["N"])
    for name, leaf in leaves.items():
        flat = leaf.view(-1)
        for i in range(flat.numel()):
            old = float(flat[i])
            flat[i] = old + 1e-4
            up = loss(leaves)
            flat[i] = old - 1e-4
            num = (up - loss(leaves)) / 2e-4
            flat[i] = old
            g = float(got[name].reshape(-1)[i])
            assert abs(g - num) <= (2.0 ** -8 if name == "y" else 0) * abs(num) + 2e-6, (name, i, g, num)


# ------------------------------------------------------------------------------------- balance loss


class Balance:
    def __init__(self, T, E, k, S, pad, score, dtype, seed=0, offsets=None):
        g = gen(seed + T + E)
        self.T, self.E, self.k, self.S, self.score = T, E, k, S, score
        self.coef = 0.3
        self.logits = (2 * randn(g, T, E) + randn(g, E)).to(stream(dtype))
        self.dtype = dtype
        self.idx = torch.topk(self.logits.float(), k, dim=1).indices.int()
        if T > 3:
            self.idx[1] = -1
            self.idx[2, 0] = E  # no expert
        if offsets is None and (S > 1 or pad):
            cut = torch.sort(torch.randint(0, T - pad + 1, (S - 1,), generator=g, device="cuda")).values.tolist()
            offsets = [0] + cut + [T - pad]
        self.cut = offsets or [0, T]
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def number(self, dg):
        return dg.DG_SCORE_SOFTMAX if self.score == "softmax" else dg.DG_SCORE_SIGMOID

    def exact(self, dloss=1.0, add=None):
        x = self.logits.double()
        T, E, k, S = self.T, self.E, self.k, self.S
        low = x == -INF
        if self.score == "softmax":
            m = x.amax(dim=1, keepdim=True)
            far = (x - m.nan_to_num(neginf=0.0)).nan_to_num(neginf=0.0)
            e = torch.where(low, 0.0, torch.exp(x - m.nan_to_num(neginf=0.0)))
            # the difference's rounding, the exponential 5, the quotient and sum
            slope, units = torch.ones_like(x), far.abs() + 8
        else:
            e, slope, units = torch.sigmoid(x), torch.sigmoid(-x), torch.full_like(x, 12.0)
        total = e.sum(dim=1, keepdim=True)
        p = torch.where(total > 0, e / total, torch.zeros_like(e))
        p = torch.where(total.isnan(), torch.full_like(e, NAN), p)
        # of p: its own units, those of the sum (weighted by p), and the sum's order (1 + 32 + 5 additions)
        np_ = U * p * (units + (p * units).nan_to_num().sum(dim=1, keepdim=True) + 40) + 2.0 ** -126
        L = self.cut[S] - self.cut[0]
        counts = torch.zeros(S, E, dtype=torch.int64, device="cuda")
        P, nP = (torch.zeros(S, E, dtype=torch.float64, device="cuda") for _ in range(2))
        d, nd = torch.zeros_like(x), torch.zeros_like(x)
        loss, nloss = 0.0, 0.0
        for s in range(S):
            a, b = self.cut[s], self.cut[s + 1]
            if a >= b:
                continue
            i = self.idx[a:b].long().reshape(-1)
            counts[s] = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
            P[s] = p[a:b].mean(dim=0)
            # a warp adds at most 1/8 of a chunk's tokens, then warps and chunks, the mean
            nP[s] = np_[a:b].mean(dim=0) + U * P[s] * (T // 296 // 8 + 1 + 8 + 300)
            f = counts[s].double() * E / (k * (b - a))
            loss += self.coef * (b - a) / L * float((f * P[s]).sum())
            nloss += self.coef * (b - a) / L * float((f * nP[s]).sum())
            n = counts[s].double()
            pp, pn, sl = p[a:b], np_[a:b], slope[a:b]
            best = pp.nan_to_num().argmax(dim=1, keepdim=True)
            # distances to the likeliest expert's count where it has more than half (or might), else to the mean load
            rel = torch.where(pp.nan_to_num().gather(1, best) > 0.5, n[None, :] - n[best[:, 0]][:, None], n[None, :] - float(k * (b - a) // E))
            mean = (pp * rel).sum(dim=1, keepdim=True)
            nmean = (pn * rel.abs()).sum(dim=1, keepdim=True) + 40 * U * (pp * rel.abs()).sum(dim=1, keepdim=True)
            K = self.coef * dloss / L * E / (k * (b - a))
            d[a:b] = K * pp * sl * (rel - mean)
            # p's noise, the sigmoid's 12 units, 4 products, the difference
            nd[a:b] = abs(K) * sl * (pn * (rel - mean).abs() + pp * nmean + pp * U * (18 * (rel - mean).abs() + rel.abs() + mean.abs()))
        if add is not None:
            d = d + add.double()
            nd = nd + U * d.abs()
        return dict(counts=counts, P=P, nP=nP, loss=loss, nloss=nloss + 4 * U * abs(loss), d=d, nd=nd)


def run_balance(dg, b, dloss=None, add=None):
    T, E, S = b.T, b.E, b.S
    loss, l_ok = framed(1, dtype=torch.float32)
    counts, c_ok = framed(S, E, dtype=torch.int32)
    probs, p_ok = framed(S, E, dtype=torch.float32)
    ws, ws_ok = framed(dg.dg_get_balance_workspace(T, E, S), dtype=torch.float32)
    ws.fill_(NAN)
    d, d_ok = framed(T, E, dtype=stream(b.dtype))
    dg.dg_balance_loss(loss, counts, probs, b.logits, b.idx, ws, seq_offsets=b.offsets, score=b.number(dg), coef=b.coef)
    dg.dg_balance_loss_bwd(d, b.logits, counts, b.k, dloss=None if dloss is None else torch.tensor([dloss], device="cuda"),
                           add=add, seq_offsets=b.offsets, score=b.number(dg), coef=b.coef)
    assert l_ok() and c_ok() and p_ok() and ws_ok() and d_ok()
    return loss, counts, probs, d


def check_balance(dg, b, dloss=None, add=None):
    loss, counts, probs, d = run_balance(dg, b, dloss, add)
    e = b.exact(1.0 if dloss is None else dloss, add)
    assert torch.equal(counts.long(), e["counts"])
    inside(probs, e["P"], e["nP"] + 2 * U * e["P"], "probs")
    assert math.isnan(e["loss"]) == math.isnan(float(loss)) and (math.isnan(e["loss"]) or abs(float(loss) - e["loss"]) <= e["nloss"]), (float(loss), e["loss"])
    inside(d, e["d"], half_step(b.dtype) * e["d"].abs() + 2 * e["nd"] + 2.0 ** -126, "dlogits")
    return loss, counts, probs, d


@pytest.mark.parametrize("T,E,k,S,pad", [(1, 1, 1, 1, 0), (1, 4, 2, 1, 0), (7, 31, 3, 2, 1), (64, 33, 8, 1, 0), (300, 60, 4, 5, 20),
                                         (4097, 256, 8, 1, 0), (5000, 256, 8, 37, 65), (1000, 65, 2, 1000, 0), (200, 513, 8, 3, 9),
                                         (333, 1024, 16, 4, 100), (20000, 16, 2, 7, 1234)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_balance(dgm, T, E, k, S, pad, score, dtype):
    b = Balance(T, E, k, S, pad, score, dtype)
    check_balance(dgm, b)
    add = randn(gen(1), T, E).to(b.logits.dtype)
    _, _, _, d = check_balance(dgm, b, dloss=-2.5, add=add)
    out = add.clone()  # in place
    counts = b.exact()["counts"].int()
    dgm.dg_balance_loss_bwd(out, b.logits, counts, k, dloss=torch.tensor([-2.5], device="cuda"), add=out, seq_offsets=b.offsets,
                            score=b.number(dgm), coef=b.coef)
    assert torch.equal(out, d)
    assert dgm.dg_get_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_masks(dgm, score):
    b = Balance(200, 64, 4, 3, 0, score, "fp32", offsets=[10, 10, 120, 190])  # an empty sequence, padding on both sides
    b.logits[20, 5:] = -INF
    b.logits[21] = -INF                       # nothing left
    b.logits[30] = torch.finfo(torch.float32).min  # no mask
    b.logits[31, :32] = torch.finfo(torch.float32).min
    b.logits[0] = NAN                         # outside of every sequence
    b.logits[199] = INF
    b.logits[40] = 0
    b.logits[41, 3] = 60.0                    # one expert has nearly all
    if score == "sigmoid":
        b.logits[30] = -90.0                  # every sigmoid below 2^-126: none left
        b.logits[30, :] = -INF
    loss, counts, probs, d = check_balance(dgm, b)
    assert bool((d[:10] == 0).all() and (d[190:] == 0).all() and (d[21] == 0).all())
    assert bool((counts[0] == 0).all() and (probs[0] == 0).all())
    assert bool((d[20, 5:] == 0).all())
    b.logits[50, 7] = NAN
    loss, counts, probs, d = run_balance(dgm, b)
    assert bool(loss.isnan().all() and probs[1].isnan().all() and not probs[2].isnan().any())
    assert bool(d[50].isnan().all() and d.isnan().any(dim=1).sum() == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [60, 64, 1024])
def test_balance_of_low_sigmoids(dgm, E, dtype):
    # tokens whose sigmoids are small, or below FP32, still divide their sum; a token's differences of logits are exact
    # (they lie within a factor of two)
    b = Balance(70, E, 4, 2, 3, "sigmoid", dtype)
    for row, base in ((5, 25.0), (6, 60.0), (7, 87.0), (8, 100.0), (9, 400.0), (69, 100.0)):
        b.logits[row] -= base
    b.logits[10] = -100.0
    b.logits[10, 3] = -60.0
    b.logits[11] = -INF
    b.logits[11, :2] = -95.0
    b.logits[12] = -100.0
    b.logits[12, 1] = NAN
    b.cut = [0, 12, 67]
    b.offsets = torch.tensor(b.cut, dtype=torch.int32, device="cuda")
    check_balance(dgm, b)


@pytest.mark.parametrize("offsets", [[0, 0], [5, 5], [8, 8]])
def test_balance_without_tokens(dgm, offsets):
    b = Balance(8, 6, 2, 1, 0, "softmax", "fp32", offsets=offsets)
    loss, counts, probs, d = run_balance(dgm, b)
    assert float(loss) == 0 and not bool(counts.any() or probs.any() or d.any())
    if offsets == [0, 0]:
        b = Balance(0, 6, 2, 1, 0, "softmax", "fp32")
        loss, counts, probs, d = run_balance(dgm, b)
        assert float(loss) == 0 and not bool(counts.any() or probs.any())


def test_balance_reports_bad_offsets(dgm):
    for offsets in ([0, 9, 8], [0, 4, 9], [-1, 4, 8], [0, 100, 8]):
        b = Balance(8, 6, 2, 2, 0, "softmax", "fp32", offsets=offsets)
        run_balance(dgm, b)
        assert dgm.dg_get_device_error() == dgm.DG_DEVERR_BAD_SEQ_OFFSET
    assert dgm.dg_get_device_error() == 0


def test_balance_of_even_loads_is_coef(dgm):
    # every expert chosen as often, equal logits: f = 1 and P = 1 / E
    T, E, k = 512, 32, 4
    b = Balance(T, E, k, 1, 0, "softmax", "fp32")
    b.logits.zero_()
    b.idx = (torch.arange(T * k, device="cuda") % E).int().view(T, k)
    loss, counts, probs, d = run_balance(dgm, b)
    assert abs(float(loss) - b.coef) <= 4 * U and bool((counts == T * k // E).all()) and not bool(d.any())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(dgm, score):
    # the counts stand still; steps of 1e-3 leave 1e-6 of third derivatives (all below coef E / k / L)
    b = Balance(6, 5, 2, 2, 0, score, "fp32", offsets=[0, 4, 6])
    _, _, _, d = run_balance(dgm, b)
    bound = b.coef * b.E / b.k / 6 * 1e-6 + 1e-7
    for t in range(6):
        for e in range(5):
            old = b.logits[t, e].clone()
            vals = []
            for h in (1e-3, -1e-3):
                b.logits = b.logits.double()
                b.logits[t, e] = float(old) + h
                vals.append(b.exact()["loss"])
                b.logits[t, e] = float(old)
                b.logits = b.logits.float()
            assert abs(float(d[t, e]) - (vals[0] - vals[1]) / 2e-3) <= bound


# --------------------------------------------------------------------------------- streams, graphs, runs


class Block:
    """A post- and pre-normed dense block and a router, forward and backward, with buffers that a program keeps."""

    def __init__(self, dg, T, N, F, E, seed=0):
        g = gen(seed)
        self.dg, self.T, self.N, self.F, self.E = dg, T, N, F, E
        self.R = R = -(-T // 128) * 128
        self.ld = dg.dg_get_tma_aligned_size(T, 4)
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.X, self.dOut = randn(g, T, N), 0.05 * randn(g, T, N)
        self.w1, self.w2 = (1 + 0.1 * randn(g, N) for _ in range(2))
        self.W1, self.s1 = cast128x128(randn(g, F, N) * (1.5 / math.sqrt(N)))
        self.W2, self.s2 = cast128x128(randn(g, N, F) * (1.5 / math.sqrt(F)))
        self.b1, self.b2 = 0.2 * randn(g, F), 0.2 * randn(g, N)
        self.gate = torch.sigmoid(randn(g, T))
        self.Wr = (randn(g, E, N) / math.sqrt(N)).bfloat16()
        self.H, self.Q, self.sq, self.r0 = bf(T, N), u8(T, N), f32(N // 128, self.ld), f32(T, 2)
        self.logits, self.idx, self.wt = bf(T, E), torch.zeros(T, 2, dtype=torch.int32, device="cuda"), f32(T, 2)
        self.loss, self.counts, self.probs = f32(1), torch.zeros(1, E, dtype=torch.int32, device="cuda"), f32(1, E)
        self.bws, self.dlogits = f32(dg.dg_get_balance_workspace(T, E, 1)), bf(T, E)
        self.Z, self.Q1, self.sq1 = bf(T, F), u8(T, F), f32(F // 128, self.ld)
        self.Y, self.Out, self.r1 = bf(T, N), f32(T, N), f32(T, 2)
        self.dYm, self.dX1, self.dgate, self.dw2, self.dw1 = bf(T, N), f32(T, N), f32(T), f32(N), f32(N)
        self.nws = f32(dg.dg_get_norm_workspace(T, N))
        self.d2r, self.d2s, self.d2c, self.d2t = u8(T, N), f32(N // 128, self.ld), u8(R, N), f32(R // 128, N)
        self.db2, self.ws2 = f32(N), f32(dg.dg_get_bias_workspace(T, N))
        self.dA1 = bf(T, F)
        self.d1r, self.d1s, self.d1c, self.d1t = u8(T, F), f32(F // 128, self.ld), u8(R, F), f32(R // 128, F)
        self.db1, self.ws1 = f32(F), f32(dg.dg_get_bias_workspace(T, F))
        self.dH, self.dX = bf(T, N), f32(T, N)

    def step(self):
        dg, ld = self.dg, self.ld
        dg.dg_norm_residual(None, self.X, H=self.H, Q=self.Q, sq=self.sq, sq_stride=ld, rstd=self.r0, w_pre=self.w1)
        torch.mm(self.H, self.Wr.t(), out=self.logits)
        dg.dg_route_topk(self.idx, self.wt, self.logits)
        dg.dg_balance_loss(self.loss, self.counts, self.probs, self.logits, self.idx, self.bws, coef=0.01)
        dg.dg_fp8_gemm_nt_epilogue(None, self.Q, self.sq, ld, self.W1, self.s1, bias=self.b1, act=dg.DG_ACT_GELU_TANH, Z=self.Z,
                                   Q=self.Q1, sq=self.sq1, sq_stride=ld)
        dg.dg_fp8_gemm_nt_epilogue(self.Y, self.Q1, self.sq1, ld, self.W2, self.s2, bias=self.b2)
        dg.dg_norm_residual(self.Out, self.X, self.Y, rstd=self.r1, w_post=self.w2, gate=self.gate, post_norm=True, scale=0.5)
        # backward
        dg.dg_norm_residual_bwd(self.dX1, self.dOut, None, self.Out, self.Y, self.r1, dY=self.dYm, dgate=self.dgate,
                                dw_post=self.dw2, ws=self.nws, w_post=self.w2, gate=self.gate, post_norm=True, scale=0.5)
        dg.dg_epilogue_bwd(self.d2r, self.d2s, ld, self.d2c, self.d2t, self.N, self.dYm, dbias=self.db2, ws=self.ws2)
        dg.dg_fp8_gemm_nn(self.dA1, self.d2r, self.d2s, ld, self.W2, self.s2.t().contiguous())
        dg.dg_epilogue_bwd(self.d1r, self.d1s, ld, self.d1c, self.d1t, self.F, self.dA1, Z=self.Z, act=dg.DG_ACT_GELU_TANH,
                           dbias=self.db1, ws=self.ws1)
        dg.dg_fp8_gemm_nn(self.dH, self.d1r, self.d1s, ld, self.W1, self.s1.t().contiguous())
        dg.dg_balance_loss_bwd(self.dlogits, self.logits, self.counts, 2, coef=0.01)
        self.dH.addmm_(self.dlogits, self.Wr)
        dg.dg_norm_residual_bwd(self.dX, self.dX1, self.dH, self.X, None, self.r0, dw_pre=self.dw1, ws=self.nws, w_pre=self.w1)

    OUT = ("H", "Q", "sq", "logits", "idx", "loss", "counts", "probs", "Z", "Q1", "sq1", "Y", "Out", "dYm", "dgate", "dw2", "db2",
           "dA1", "db1", "dH", "dX", "dw1", "dlogits", "d1c", "d1t", "d2c", "d2t")

    def out(self, n):  # without the gap behind a row of scales
        t = getattr(self, n)
        return t[:, :self.T].contiguous() if n in ("sq", "sq1") else t

    def snapshot(self):
        return {n: self.out(n).clone() for n in self.OUT}

    def wipe(self):
        for n in self.OUT:
            getattr(self, n).view(torch.uint8).fill_(0x5B)
        for n in ("bws", "nws", "ws1", "ws2"):
            getattr(self, n).fill_(NAN)

    def same(self, want):
        for n, t in want.items():
            assert torch.equal(self.out(n).view(torch.uint8), t.view(torch.uint8)), n


def test_a_block_forward_and_backward(dgm):
    """The run against 64-bit autograd of the same block with the casts left out: e4m3 operands carry half a step, 2^-4, of
    each value at random, so vectors agree to a few percent in norm (3 casts behind one another on the longest path: sums of
    independent roundings of 2^-4 / sqrt(3) each, 4 % a cast, 10 % in all)."""
    b = Block(dgm, 200, 256, 384, 8)
    b.step()
    assert dgm.dg_get_device_error() == 0
    leaf = {n: getattr(b, n).double().requires_grad_() for n in ("X", "w1", "w2", "b1", "b2", "gate")}
    W1 = b.W1.double() * b.s1.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    W2 = b.W2.double() * b.s2.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    norm = lambda v: v * (v.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    h = norm(leaf["X"]) * leaf["w1"]
    z = h @ W1.t() + leaf["b1"]
    y = act64(z, "gelu_tanh")[0] @ W2.t() + leaf["b2"]
    out = leaf["X"] + 0.5 * leaf["gate"][:, None] * leaf["w2"] * norm(y)
    p = torch.softmax(h @ b.Wr.double().t(), dim=1)
    f = b.counts[0].double() * b.E / (2 * b.T)
    loss = 0.01 * (f * p.mean(dim=0)).sum()
    ((out * b.dOut.double()).sum() + loss).backward()

    def agree(got, want, share, what):
        off = float((got.double() - want).detach().norm() / want.detach().norm())
        assert off < share, (what, off)

    agree(b.H, h, 0.01, "H")
    agree(b.Z, z, 0.10, "Z")
    agree(b.Y, y, 0.10, "Y")
    agree(b.Out, out, 0.10, "Out")
    assert abs(float(b.loss) - float(loss.detach())) < 0.01 * float(loss.detach())
    for got, n in ((b.dX, "X"), (b.dw1, "w1"), (b.dw2, "w2"), (b.db1, "b1"), (b.db2, "b2"), (b.dgate, "gate")):
        agree(got, leaf[n].grad, 0.10, n)


@pytest.mark.parametrize("T", [3, 200])
def test_a_block_repeats_in_graphs_and_on_streams(dgm, T):
    b = Block(dgm, T, 256, 384, 8)
    b.step()
    want = b.snapshot()
    b.wipe()
    b.step()
    b.same(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.step()  # the stream's own workspaces exist before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        b.step()
    for _ in range(2):
        b.wipe()
        graph.replay()
        torch.cuda.synchronize()
        b.same(want)
    # new inputs in the same buffers
    b.X.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = b.snapshot()
    b.wipe()
    b.step()
    b.same(got)
    # two at once on streams of their own
    c = Block(dgm, T, 256, 384, 8, seed=1)
    c.step()
    want_c = c.snapshot()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in (b, c):
        x.wipe()
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s in zip((b, c), streams):
            with torch.cuda.stream(s):
                x.step()
    torch.cuda.synchronize()
    b.same(got)
    c.same(want_c)
    assert dgm.dg_get_device_error() == 0


@pytest.mark.parametrize("sms", [1, 5, 100])
def test_results_under_an_sm_cap(dgm, sms):
    b = Block(dgm, 200, 256, 384, 8)
    b.step()
    want = b.snapshot()
    n = Norm(300, 384, "fp32", True)
    w = n.exact()
    U_, rstd = w["u"].float(), torch.cat([w["ry"], w["ru"]], dim=1).float()
    dgm.dg_set_num_sms(sms)
    try:
        b.wipe()
        b.step()
        torch.cuda.synchronize()
        t = run_norm_bwd(dgm, n, U_, rstd, n.dU, n.dH)
    finally:
        dgm.dg_set_num_sms(0)
    # sums over tokens run in another order; everything else is the same
    for name, x in want.items():
        if name in ("dw1", "dw2"):
            assert torch.allclose(getattr(b, name), x, rtol=1e-4, atol=1e-5), name
        else:
            assert torch.equal(b.out(name).view(torch.uint8), x.view(torch.uint8)), name
    e = NormGrad(n, U_, rstd, n.dU, n.dH, min(sms, 148))
    inside(t["P"], e.dw_post, e.npost, "dw_post")
    inside(t["N"], e.dw_pre, e.npre, "dw_pre")


def test_a_block_without_programmatic_launch_and_with_given_streams(dgm):
    b = Block(dgm, 130, 256, 384, 8)
    b.step()
    want = b.snapshot()
    dgm.dg_set_pdl(False)
    try:
        b.wipe()
        b.step()
        torch.cuda.synchronize()
    finally:
        dgm.dg_set_pdl(None)
    b.same(want)
    # a call on a stream that is not the current one
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    Out, r1, dX, dw = (torch.empty_like(t) for t in (b.Out, b.r1, b.dX1, b.dw2))
    dgm.dg_norm_residual(Out, b.X, b.Y, rstd=r1, w_post=b.w2, gate=b.gate, post_norm=True, scale=0.5, stream=s)
    dgm.dg_norm_residual_bwd(dX, b.dOut, None, Out, b.Y, r1, dw_post=dw, ws=b.nws, w_post=b.w2, gate=b.gate, post_norm=True, scale=0.5,
                             stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(Out, b.Out) and torch.equal(dX, b.dX1) and torch.equal(dw, b.dw2)


@pytest.mark.parametrize("sms", [1, 20])
def test_gemm_epilogue_under_an_sm_cap(dgm, sms):
    # many tiles a CTA, and the K-split of a last wave
    dgm.dg_set_num_sms(sms)
    try:
        for M, N, K in [(300, 2048, 512), (700, 2048, 4096), (40, 640, 1024)]:
            G = Gemm(dgm, M, N, K, seed=sms)
            G.check(dgm, "gelu_tanh", "DQZ")
            G.check(dgm, "none", "D", in_place=True)
    finally:
        dgm.dg_set_num_sms(0)


def test_gemm_epilogue_graphs_of_one_stream_run_at_once(dgm):
    # sizes whose last wave is split along K where the stream's workspace may be used: not in a graph, which may run
    # beside another one of the same stream
    side = torch.cuda.Stream()
    gemms = [Gemm(dgm, M, N, K, seed=M) for M, N, K in [(1300, 4096, 4096), (1500, 4096, 4096)]]
    outs = [torch.empty(G.M, G.N, dtype=torch.bfloat16, device="cuda") for G in gemms]

    def call(G, D):
        dgm.dg_fp8_gemm_nt_epilogue(D, G.A, G.sa, G.stride, G.B, G.sb, bias=G.bias, act=dgm.DG_ACT_GELU, residual=G.residual)

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    graphs = []
    for G, D in zip(gemms, outs):
        assert dgm.dg_make_plan(0, G.M, G.N, G.K, 1, sms)["tail_split"] > 1
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(G, D)  # the stream has its workspace
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            for _ in range(4):
                call(G, D)
    want = []
    for G, D, graph in zip(gemms, outs, graphs):
        D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _, v, _, nv = G.exact("gelu")
        inside(D, v, 2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * nv, "D")
        want.append(D.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    eager = [torch.empty_like(D) for D in outs]
    for _ in range(5):
        for D in outs + eager:
            D.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(side):
            call(gemms[0], eager[0])
            call(gemms[1], eager[1])
        torch.cuda.synchronize()
        for G, D, E, w in zip(gemms, outs, eager, want):
            assert torch.equal(D, w)
            _, v, _, nv = G.exact("gelu")
            inside(E, v, 2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * nv, "split")
    assert dgm.dg_get_device_error() == 0


def test_rows_past_31_bits_of_bytes(dgm):
    """Rows whose elements lie past 2^31: the first and the last rows of a long stream."""
    N = 8192
    T = (1 << 31) // N + 300
    X = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    pick = torch.tensor([0, 1, T - 200, T - 1], device="cuda")
    X[pick] = randn(gen(2), 4, N).bfloat16()
    H = torch.empty_like(X)
    rstd = torch.empty(T, 2, device="cuda")
    dgm.dg_norm_residual(None, X, H=H, rstd=rstd)
    ref = torch.empty(4, N, dtype=torch.bfloat16, device="cuda")
    dgm.dg_norm_residual(None, X[pick].contiguous(), H=ref)
    assert torch.equal(H[pick], ref) and bool((H[2] == 0).all() and (H[T - 2] == 0).all())
    dX = torch.empty_like(X)
    dw = torch.empty(N, device="cuda")
    dgm.dg_norm_residual_bwd(dX, None, H, X, None, rstd, dw_pre=dw, ws=torch.empty(dgm.dg_get_norm_workspace(T, N), device="cuda"))
    dref = torch.empty(4, N, dtype=torch.bfloat16, device="cuda")
    dgm.dg_norm_residual_bwd(dref, None, ref, X[pick].contiguous(), None, rstd[pick].contiguous())
    assert torch.equal(dX[pick], dref)


def test_values_helper_reads_codes():
    assert float(values(torch.tensor([0x7E], dtype=torch.uint8))) == 448.0
