"""GPU: dispatch, combine and the gated activation with its 8-bit checkpoints,
against plain forms, and a whole MoE layer's step made of them.

Casts of given values (dispatch, the checkpoint, the casts of dY = w dout, the
recast) take every decision in single precision, so codes and scales are
compared bit for bit with the same steps in torch on the CPU.  Where the value
that is cast comes out of exp (the activation and its gradient), the value may
differ by `noise` from the 64-bit one, and a code may round the other way: what
code and scale stand for must lie within half an e4m3 step (2^-4 of the value,
or 2^-10 of the scale below the normal range) plus twice the noise.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_route import layout64

pytestmark = pytest.mark.gpu

BLOCK = 128


@pytest.fixture(scope="module")
def dgm():
    from moe_grouped_gemm_weight_b200 import build
    build.build()
    import moe_grouped_gemm_weight_b200 as dg
    dg.dg_set_num_sms(0)
    assert dg.dg_get_device_error() == 0
    return dg


class Layout:
    """Random experts for T tokens, some slots dropped, and their layout (host-made)."""

    def __init__(self, dg, T, k, E, max_rows=0, seed=0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.k, self.E, self.max_rows = T, k, E, max_rows
        idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
        idx[torch.rand(T, k, generator=g) < 0.1] = -1
        if T > 2:
            idx[2] = -1               # a token without an expert
        self.idx = idx
        self.rows = E * max_rows or dg.dg_get_layout_rows(T, k, E) + extra
        out = layout64(idx.numpy(), E, self.rows, max_rows)
        self.row_of, self.m_indices, self.slot_of, self.offsets, self.counts = (torch.from_numpy(a) for a in out)
        self.held = self.m_indices >= 0
        self.blocks = self.held[:self.rows // 128 * 128].view(-1, 128).any(dim=1)


def cast(x, dims):
    """The cast's steps in FP32 (torch, CPU): codes and scales, tiles spanning `dims` of x."""
    x = x.float()
    amax = x.abs().nan_to_num(nan=0.0, posinf=float("inf")).amax(dim=dims, keepdim=True).clamp_min(1e-4)
    q = (x * (torch.full_like(amax, 448.0) / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, amax / 448.0


def cast_rows(x):
    R, K = x.shape
    q, s = cast(x.reshape(R, K // BLOCK, BLOCK), (2,))
    return q.reshape(R, K).view(torch.uint8), s.reshape(R, K // BLOCK).t().contiguous()


def cast_cols(x):
    R, K = x.shape
    q, s = cast(x.reshape(R // BLOCK, BLOCK, K), (1,))
    return q.reshape(R, K).view(torch.uint8), s.reshape(R // BLOCK, K).contiguous()


def cast_blocks(x):
    R, K = x.shape
    q, s = cast(x.reshape(R // BLOCK, BLOCK, K // BLOCK, BLOCK), (1, 3))
    return q.reshape(R, K).view(torch.uint8), s.reshape(R // BLOCK, K // BLOCK).t().contiguous()


def codes(*shape):
    return torch.full(shape, 0x5A, dtype=torch.uint8, device="cuda")


def scales(*shape):
    return torch.full(shape, -7.0, device="cuda")


def values(q):
    return q.view(torch.float8_e4m3fn).double()


def same(a, b):
    return torch.equal(a.cpu(), b.cpu())


# ------------------------------------------------------------------- dispatch

@pytest.mark.parametrize("T,k,E,K,max_rows", [(1, 1, 1, 128, 0), (3, 2, 4, 256, 0), (33, 6, 16, 640, 0),
                                              (200, 8, 64, 1024, 0), (1000, 3, 9, 896, 0), (64, 8, 32, 7168, 64),
                                              (7, 2, 5, 384, 3), (50, 20, 40, 256, 50), (2500, 8, 16, 512, 0)])
def test_dispatch_is_the_cast_of_each_slots_token(dgm, T, k, E, K, max_rows):
    L = Layout(dgm, T, k, E, max_rows, seed=T + K)
    X = (torch.randn(T, K, generator=torch.Generator().manual_seed(K)) * 3).bfloat16()
    X[0, :128] = 0
    if T > 1:
        X[1, 5] = float("nan")
        X[1, 130 % K] = 1e30
    stride = dgm.dg_get_tma_aligned_size(max_rows, 4) + 4 if max_rows else L.rows + 8
    Q, sa = codes(L.rows, K), scales(E if max_rows else 1, K // BLOCK, stride)
    dgm.dg_dispatch_fp8_1x128(Q, sa, stride, X.cuda(), L.row_of.cuda(), group_rows=max_rows)
    q, s = cast_rows(X)
    want_q, want_s = codes(L.rows, K).cpu(), scales(*sa.shape).cpu()
    for r in range(L.rows):
        slot = int(L.slot_of[r])
        if slot >= 0:
            t = slot // k
            want_q[r] = q[t]
            if max_rows:
                want_s[r // max_rows, :, r % max_rows] = s[:, t]
            else:
                want_s[0, :, r] = s[:, t]
    nan = (want_q & 0x7F) == 0x7F
    assert same(Q.cpu() & 0x7F | torch.where(nan, 0, Q.cpu() & 0x80), want_q & 0x7F | torch.where(nan, 0, want_q & 0x80))
    assert same(sa, want_s)


def test_dispatch_rows_out_of_range_are_not_written(dgm):
    X = torch.randn(2, 256, device="cuda").bfloat16()
    Q, sa = codes(4, 256), scales(2, 4)
    row_of = torch.tensor([[0, 4], [-3, 2]], dtype=torch.int32, device="cuda")
    dgm.dg_dispatch_fp8_1x128(Q, sa, 4, X, row_of)
    q, s = cast_rows(X.cpu())
    assert same(Q[0], q[0]) and same(Q[2], q[1]) and bool((Q[1] == 0x5A).all() and (Q[3] == 0x5A).all())
    assert bool((sa[:, 1] == -7).all() and (sa[:, 3] == -7).all())


# -------------------------------------------------------------------- combine

@pytest.mark.parametrize("T,k,E,N,max_rows", [(1, 1, 1, 8, 0), (5, 3, 4, 24, 0), (33, 6, 16, 1000, 0),
                                              (100, 8, 64, 7168, 0), (64, 8, 32, 2056, 64), (40, 17, 20, 136, 0)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(dgm, T, k, E, N, max_rows, weighted):
    L = Layout(dgm, T, k, E, max_rows, seed=N)
    g = torch.Generator().manual_seed(T)
    Y = torch.randn(L.rows, N, generator=g).bfloat16()
    Y[~L.held] = float("nan")          # rows without a slot are not read
    w = torch.randn(T, k, generator=g) if weighted else None
    if weighted:
        w[L.row_of < 0] = float("inf")  # nor are the weights of slots without a row
    buf = torch.full((T * N + 256,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[128:128 + T * N].view(T, N)
    dgm.dg_combine(out, Y.cuda(), L.row_of.cuda(), None if w is None else w.cuda())
    assert bool((buf[:128] == 9).all() and (buf[-128:] == 9).all())
    want, mag = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if L.row_of[t, j] >= 0:
                part = Y[L.row_of[t, j].long()].double() * (1.0 if w is None else w[t, j].double())
                want[t] += part
                mag[t] += part.abs()
    # k sums and products in FP32, one rounding to bf16
    tol = 2.0 ** -8 * want.abs() + 2 * k * 2.0 ** -24 * mag
    assert bool(((out.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T,k,E,N", [(1, 1, 1, 128), (3, 2, 4, 256), (33, 6, 16, 640), (300, 8, 12, 1152),
                                     (700, 4, 5, 7168)])
def test_combine_gradient(dgm, T, k, E, N):
    L = Layout(dgm, T, k, E, seed=N, extra=256)
    g = torch.Generator().manual_seed(T)
    dout = (0.01 * torch.randn(T, N, generator=g)).bfloat16()
    Y = torch.randn(L.rows, N, generator=g).bfloat16()
    Y[~L.held] = float("nan")
    w = torch.rand(T, k, generator=g)
    w[L.row_of < 0] = float("nan")
    dw = torch.full((T, k), 5.0, device="cuda")
    sr_stride, sc_stride = L.rows + 4, N + 4
    Qr, sr, Qc, sc = codes(L.rows, N), scales(N // BLOCK, sr_stride), codes(L.rows, N), scales(L.rows // BLOCK, sc_stride)
    dgm.dg_combine_bwd(dw, Qr, sr, sr_stride, Qc, sc, sc_stride, dout.cuda(), Y.cuda(), L.row_of.cuda(),
                       L.slot_of.cuda(), w.cuda())
    dY = torch.zeros(L.rows, N)
    want, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for r in torch.nonzero(L.held)[:, 0].tolist():
        t, j = divmod(int(L.slot_of[r]), k)
        dY[r] = dout[t].float() * w[t, j]
        prod = dout[t].double() * Y[r].double()
        want[t, j], mag[t, j] = prod.sum(), prod.abs().sum()
    # at most N / 16 sums in a row in one lane, then a few joins
    assert bool(((dw.cpu().double() - want).abs() <= (N / 16 + 32) * 2.0 ** -24 * mag).all())
    inside = L.blocks.repeat_interleave(128)
    q, s = cast_rows(dY)
    assert same(Qr.cpu()[inside], q[inside]) and same(sr.cpu()[:, :L.rows][:, inside], s[:, inside])
    assert bool((Qr.cpu()[~inside] == 0x5A).all() and (sr.cpu()[:, :L.rows][:, ~inside] == -7).all())
    assert bool((sr.cpu()[:, L.rows:] == -7).all() and (sc.cpu()[:, N:] == -7).all())
    q, s = cast_cols(dY)
    assert same(Qc.cpu()[inside], q[inside]) and same(sc.cpu()[L.blocks][:, :N], s[L.blocks])
    assert bool((Qc.cpu()[~inside] == 0x5A).all() and (sc.cpu()[~L.blocks] == -7).all())


@pytest.mark.parametrize("sms", [1, 4, 0])
def test_results_do_not_depend_on_the_sm_cap(dgm, sms):
    # Fewer SMs: longer runs of the persistent kernels, other splits of combine's gradient (the sums of dw are
    # joined in another order: 2^-24 of their terms' magnitudes a join).
    L = Layer(dgm, 300, 4, 9, 1152, 384, seed=3)
    for t in (L.Hid, L.Y, L.dA, L.dXr):
        t.zero_()
    L.forward()
    L.backward()
    keep = ("idx", "wt", "row_of", "mi", "slot_of", "off", "cnt", "Q", "sa", "Q2", "sa2", "C", "cs", "dYr", "sr", "dYc",
            "sc", "dHr", "shr", "dHc", "shc", "Qa", "sb", "Xb", "sx", "dX", "dlogits")
    ops = {n: getattr(L, n).clone() for n in keep}
    dw = L.dw.clone()
    dgm.dg_set_num_sms(sms)
    try:
        dgm.dg_route_topk(L.idx, L.wt, L.logits, L.bias, score=dgm.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
        dgm.dg_route_layout(L.row_of, L.mi, L.slot_of, L.off, L.cnt, L.idx)
        dgm.dg_dispatch_fp8_1x128(L.Q, L.sa, L.R, L.X, L.row_of)
        dgm.dg_swiglu_fp8(L.Q2, L.sa2, L.R, L.Hid, L.C, L.cs, L.R, m_indices=L.mi)
        dgm.dg_combine_bwd(L.dw, L.dYr, L.sr, L.R, L.dYc, L.sc, L.H, L.dout, L.Y, L.row_of, L.slot_of, L.wt)
        dgm.dg_swiglu_fp8_bwd(L.dHr, L.shr, L.R, L.dHc, L.shc, 2 * L.F, L.Qa, L.sb, L.dA, L.C, L.cs, L.R, m_indices=L.mi)
        dgm.dg_fp8_1x128_to_128x128(L.Xb, L.sx, L.Q, L.sa, L.R, m_indices=L.mi)
        dgm.dg_combine(L.dX, L.dXr, L.row_of)
        dgm.dg_route_topk_bwd(L.dlogits, dw, L.logits, L.idx, score=dgm.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
        torch.cuda.synchronize()
    finally:
        dgm.dg_set_num_sms(0)
    for n in keep:
        assert torch.equal(getattr(L, n).view(torch.uint8), ops[n].view(torch.uint8)), n
    mag = torch.zeros_like(dw)
    for t in range(L.T):
        for j in range(L.k):
            mag[t, j] = (L.dout[t].float() * L.Y[int(L.row_of[t, j])].float()).abs().sum()
    assert bool(((L.dw - dw).abs() <= 2 * (1152 / 16 + 32) * 2.0 ** -24 * mag).all())


def test_combine_gradient_against_differences(dgm):
    # dw is the derivative of <dout, combine(Y, w)>, which is linear in w.
    T, k, E, N = 6, 3, 5, 256
    L = Layout(dgm, T, k, E, seed=1)
    g = torch.Generator().manual_seed(8)
    dout, Y = torch.randn(T, N, generator=g).bfloat16(), torch.randn(L.rows, N, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g)

    def loss(w64):
        out = torch.zeros(T, N, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                if L.row_of[t, j] >= 0:
                    out[t] += w64[t, j] * Y[L.row_of[t, j].long()].double()
        return (out * dout.double()).sum()

    dw = torch.empty(T, k, device="cuda")
    dgm.dg_combine_bwd(dw, codes(L.rows, N), scales(2, L.rows), L.rows, codes(L.rows, N), scales(L.rows // 128, N), N,
                       dout.cuda(), Y.cuda(), L.row_of.cuda(), L.slot_of.cuda(), w.cuda())
    for t in range(T):
        for j in range(k):
            step = torch.zeros(T, k, dtype=torch.float64)
            step[t, j] = 0.5
            num = loss(w.double() + step) - loss(w.double() - step)
            assert abs(float(dw[t, j]) - float(num)) <= 1e-4 * (1 + abs(float(num)))


# ------------------------------------------------------- gated activation

def near(q, s, want, noise, what):
    """Codes q with scales s (both broadcast to q) stand for `want` within the module's bound."""
    got = values(q) * s.double()
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s.double()) * (1 + 2.0 ** -20) + 2 * noise
    far = (got - want).abs() - tol
    assert not bool((far > 0).any()), f"{what}: off by {float(far.max())} beyond the bound"


def scale_near(s, want, noise, dims, what):
    """A scale is amax / 448 with amax off by the tile's largest noise and two roundings."""
    amax = want.abs().amax(dim=dims).clamp_min(1e-4)
    tol = noise.amax(dim=dims) + 2.0 ** -22 * amax
    assert bool(((s.double() * 448 - amax).abs() <= tol).all()), what


@pytest.mark.parametrize("T,k,E,F,max_rows", [(1, 1, 1, 128, 0), (5, 2, 4, 256, 0), (100, 6, 16, 640, 0),
                                              (700, 3, 5, 2048, 0), (64, 8, 32, 2048, 64), (7, 2, 5, 384, 3)])
@pytest.mark.parametrize("checkpoint", [True, False])
def test_swiglu(dgm, T, k, E, F, max_rows, checkpoint):
    L = Layout(dgm, T, k, E, max_rows, seed=F)
    H = (2.5 * torch.randn(L.rows, 2 * F, generator=torch.Generator().manual_seed(T))).bfloat16()
    H[~L.held] = float("nan")
    first = int(torch.nonzero(L.held)[0]) if bool(L.held.any()) else 0
    H[first, :8] = torch.tensor([0.0, -0.0, 200.0, -200.0, 88.0, -88.0, 1e-30, -1e-30]).bfloat16()
    stride = (max_rows or L.rows) + 4
    nG, nfb = (E if max_rows else 1), F // BLOCK
    Q, sa = codes(L.rows, F), scales(nG, nfb, stride)
    C, cs = (codes(L.rows, 2 * F), scales(nG, 2 * nfb, stride)) if checkpoint else (None, None)
    dgm.dg_swiglu_fp8(Q, sa, stride, H.cuda(), C, cs, stride, m_indices=L.m_indices.cuda(), group_rows=max_rows)

    def by_row(s):  # [groups, blocks, stride] -> [rows, blocks]
        s = s.cpu()
        return s[:, :, :max_rows].permute(0, 2, 1).reshape(L.rows, -1) if max_rows else s[0, :, :L.rows].t()

    held = L.held
    assert bool((Q.cpu()[~held] == 0x5A).all() and (by_row(sa)[~held] == -7).all())
    assert bool((sa.cpu()[:, :, (max_rows or L.rows):] == -7).all())
    h = H[held].double()
    gate, up = h[:, :F], h[:, F:]
    a = gate / (1 + torch.exp(-gate)) * up
    # exp: 2 ulp plus its argument's rounding (|g| 2^-24), quotient 2 ulp, sums and products 2^-24 each
    noise = a.abs() * (gate.abs() + 24) * 2.0 ** -24
    tile = lambda x: x.reshape(x.shape[0], -1, BLOCK)  # noqa: E731
    s = by_row(sa)[held]
    near(Q.cpu()[held], s.repeat_interleave(BLOCK, dim=1), a, noise, "activation")
    scale_near(s, tile(a), tile(noise), (2,), "activation scale")
    if checkpoint:
        q, sq = cast_rows(H[held])
        assert same(C.cpu()[held], q) and same(by_row(cs)[held], sq.t())
        assert bool((C.cpu()[~held] == 0x5A).all() and (by_row(cs)[~held] == -7).all())


def test_swiglu_without_a_mask(dgm):
    H = torch.randn(37, 512, generator=torch.Generator().manual_seed(4)).bfloat16()
    Q, sa = codes(37, 256), scales(2, 40)
    dgm.dg_swiglu_fp8(Q, sa, 40, H.cuda())
    Q2, sa2 = codes(37, 256), scales(2, 40)
    dgm.dg_swiglu_fp8(Q2, sa2, 40, H.cuda(), m_indices=torch.zeros(37, dtype=torch.int32, device="cuda"))
    assert same(Q, Q2) and same(sa, sa2) and not bool((Q == 0x5A).all(dim=1).any())


def swiglu_bwd64(gate, up, dA):
    s = 1 / (1 + torch.exp(-gate))
    return dA * up * s * (1 + gate * (1 - s)), dA * gate * s, gate * s * up


def checkpoint_of(H):
    q, s = cast_rows(H)
    return q, s


@pytest.mark.parametrize("T,k,E,F,masked", [(1, 1, 1, 128, True), (5, 2, 4, 256, True), (100, 6, 16, 640, True),
                                            (700, 3, 5, 2048, True), (90, 2, 3, 384, False)])
def test_swiglu_gradient(dgm, T, k, E, F, masked):
    L = Layout(dgm, T, k, E, seed=F, extra=128)
    g = torch.Generator().manual_seed(T)
    H = 2.5 * torch.randn(L.rows, 2 * F, generator=g)
    H[0, :4] = torch.tensor([30.0, -30.0, 0.0, -1.2784])
    C, cs = checkpoint_of(H.bfloat16())
    dA = (0.01 * torch.randn(L.rows, F, generator=g)).bfloat16()
    held = L.held if masked else torch.ones_like(L.held)
    blocks = L.blocks if masked else torch.ones_like(L.blocks)
    if masked:
        C[~held] = 0x7F
        dA[~held] = float("nan")
    R, sr_stride, cs_stride, sc_stride = L.rows, L.rows + 4, L.rows + 8, 2 * F + 4
    csg = scales(2 * F // BLOCK, cs_stride)
    csg[:, :R] = cs.cuda()
    if masked:
        csg[:, :R][:, ~held.cuda()] = float("nan")
    Qr, sr = codes(R, 2 * F), scales(2 * F // BLOCK, sr_stride)
    Qc, sc = codes(R, 2 * F), scales(R // BLOCK, sc_stride)
    Qa, sb = codes(R, F), scales(F // BLOCK, R // BLOCK)
    dgm.dg_swiglu_fp8_bwd(Qr, sr, sr_stride, Qc, sc, sc_stride, Qa, sb, dA.cuda(), C.cuda(), csg, cs_stride,
                          m_indices=L.m_indices.cuda() if masked else None)
    h = values(C).nan_to_num(0) * cs.t().double().repeat_interleave(BLOCK, dim=1)
    h[~held] = 0
    d = dA.double().nan_to_num(0)
    d[~held] = 0
    gate, up = h[:, :F], h[:, F:]
    dgate, dup, a = swiglu_bwd64(gate, up, d)
    dH = torch.cat([dgate, dup], dim=1)
    # every factor is good to (|g| + 24) 2^-24; s + silu (1 - s) is a sum of terms that may cancel
    s = 1 / (1 + torch.exp(-gate))
    rel = (gate.abs() + 32) * 2.0 ** -24
    noise = torch.cat([(d * up).abs() * (s + (gate * s).abs() * (1 - s + 2.0 ** -2)) * rel, dup.abs() * rel], dim=1)
    inside = blocks.repeat_interleave(128)
    Qr, sr, Qc, sc, Qa, sb = (x.cpu() for x in (Qr, sr, Qc, sc, Qa, sb))
    for x in (Qr, Qc, Qa):
        assert bool((x[~inside] == 0x5A).all())
    assert bool((sr[:, :R][:, ~inside] == -7).all() and (sr[:, R:] == -7).all())
    assert bool((sc[~blocks] == -7).all() and (sc[:, 2 * F:] == -7).all() and (sb[:, ~blocks] == -7).all())
    tile = lambda x: x.reshape(x.shape[0], -1, BLOCK)  # noqa: E731
    near(Qr[inside], sr[:, :R].t()[inside].repeat_interleave(BLOCK, dim=1), dH[inside], noise[inside], "dH rows")
    scale_near(sr[:, :R].t()[inside], tile(dH[inside]), tile(noise[inside]), (2,), "dH row scales")
    near(Qc[inside], sc[blocks][:, :2 * F].repeat_interleave(128, dim=0), dH[inside], noise[inside], "dH columns")
    col = lambda x: x.reshape(-1, 128, x.shape[1])  # noqa: E731
    scale_near(sc[blocks][:, :2 * F], col(dH[inside]), col(noise[inside]), (1,), "dH column scales")
    na = a.abs() * rel
    near(Qa[inside], sb[:, blocks].t().repeat_interleave(128, dim=0).repeat_interleave(BLOCK, dim=1), a[inside],
         na[inside], "activation")
    sq = lambda x: x.reshape(-1, 128, F // BLOCK, BLOCK)  # noqa: E731
    scale_near(sb[:, blocks].t(), sq(a[inside]), sq(na[inside]), (1, 3), "activation scales")


def test_swiglu_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    gate, up, dA = (torch.randn(50, generator=g, dtype=torch.float64) * 3 for _ in range(3))
    f = lambda x, y: x / (1 + torch.exp(-x)) * y * dA  # noqa: E731
    dg_, du, _ = swiglu_bwd64(gate, up, dA)
    h = 1e-5
    assert torch.allclose((f(gate + h, up) - f(gate - h, up)) / (2 * h), dg_, rtol=1e-7, atol=1e-8)
    assert torch.allclose((f(gate, up + h) - f(gate, up - h)) / (2 * h), du, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("T,k,E,K,masked", [(1, 1, 1, 128, True), (5, 2, 4, 256, True), (301, 6, 16, 1152, True),
                                            (200, 3, 5, 7168, False)])
def test_recast(dgm, T, k, E, K, masked):
    L = Layout(dgm, T, k, E, seed=K, extra=128)
    g = torch.Generator().manual_seed(T)
    Q, sa = cast_rows(torch.randn(L.rows, K, generator=g) * torch.exp(torch.randn(L.rows, 1, generator=g)))
    held = L.held if masked else torch.ones_like(L.held)
    blocks = L.blocks if masked else torch.ones_like(L.blocks)
    Q[int(torch.nonzero(held)[0]), 7] = 0xFF      # a NaN stays one and is no maximum
    stride = L.rows + 4
    sag = scales(K // BLOCK, stride)
    sag[:, :L.rows] = sa.cuda()
    if masked:
        Q[~held] = 0x7E
        sag[:, :L.rows][:, ~held.cuda()] = float("inf")
    Qb, sb = codes(L.rows, K), scales(K // BLOCK, L.rows // BLOCK)
    dgm.dg_fp8_1x128_to_128x128(Qb, sb, Q.cuda(), sag, stride, m_indices=L.m_indices.cuda() if masked else None)
    x = Q.view(torch.float8_e4m3fn).float() * sa.t().repeat_interleave(BLOCK, dim=1)
    x[~held] = 0
    q, s = cast_blocks(x)
    inside = blocks.repeat_interleave(128)
    nan = (q & 0x7F) == 0x7F
    got = Qb.cpu()
    assert same(torch.where(nan, got & 0x7F, got)[inside], torch.where(nan, q & 0x7F, q)[inside])
    assert same(sb.cpu()[:, blocks], s[:, blocks])
    assert bool((got[~inside] == 0x5A).all() and (sb.cpu()[:, ~blocks] == -7).all())


# --------------------------------------------------------- together: a layer

class Layer:
    """One MoE layer's forward and backward step through the library, buffers made once."""

    def __init__(self, dg, T, k, E, H, F, seed=0):
        self.dg, self.T, self.k, self.E, self.H, self.F = dg, T, k, E, H, F
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.X, self.logits = r(T, H).bfloat16(), r(T, E)
        self.bias = 0.1 * r(E)
        self.dout = (0.05 * r(T, H)).bfloat16()
        self.W1, self.W2 = (H ** -0.5 * r(E, 2 * F, H)).bfloat16(), (F ** -0.5 * r(E, H, F)).bfloat16()
        self.w = {}
        for name, W in (("1", self.W1), ("2", self.W2), ("1t", self.W1.transpose(1, 2).contiguous()),
                        ("2t", self.W2.transpose(1, 2).contiguous())):
            q, s = torch.empty_like(W, dtype=torch.uint8), torch.empty(E, -(-W.shape[1] // 128), W.shape[2] // 128, device="cuda")
            for e in range(E):
                dg.dg_to_fp8_128x128(q[e], s[e], W[e])
            self.w[name] = (q, s)
        R = self.R = dg.dg_get_layout_rows(T, k, E)
        i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        u = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        b = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.idx, self.wt, self.row_of = i(T, k), f(T, k), i(T, k)
        self.mi, self.slot_of, self.off, self.cnt = i(R), i(R), i(E + 1), i(E)
        self.Q, self.sa, self.Hid = u(R, H), f(H // 128, R), b(R, 2 * F)
        self.Q2, self.sa2, self.C, self.cs = u(R, F), f(F // 128, R), u(R, 2 * F), f(2 * F // 128, R)
        self.Y, self.out = b(R, H), b(T, H)
        self.dw, self.dYr, self.sr, self.dYc, self.sc = f(T, k), u(R, H), f(H // 128, R), u(R, H), f(R // 128, H)
        self.dA = b(R, F)
        self.dHr, self.shr, self.dHc, self.shc = u(R, 2 * F), f(2 * F // 128, R), u(R, 2 * F), f(R // 128, 2 * F)
        self.Qa, self.sb, self.Xb, self.sx = u(R, F), f(F // 128, R // 128), u(R, H), f(H // 128, R // 128)
        self.dXr, self.dX = b(R, H), b(T, H)
        self.dW1, self.dW2, self.dlogits = b(E, 2 * F, H), b(E, H, F), f(T, E)

    def forward(self):
        dg, R = self.dg, self.R
        dg.dg_route_topk(self.idx, self.wt, self.logits, self.bias, score=dg.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
        dg.dg_route_layout(self.row_of, self.mi, self.slot_of, self.off, self.cnt, self.idx)
        dg.dg_dispatch_fp8_1x128(self.Q, self.sa, R, self.X, self.row_of)
        dg.dg_grouped_contiguous_nt(self.Hid, self.Q, self.sa, R, *self.w["1"], self.mi)
        dg.dg_swiglu_fp8(self.Q2, self.sa2, R, self.Hid, self.C, self.cs, R, m_indices=self.mi)
        dg.dg_grouped_contiguous_nt(self.Y, self.Q2, self.sa2, R, *self.w["2"], self.mi)
        dg.dg_combine(self.out, self.Y, self.row_of, self.wt)

    def backward(self):
        dg, R, H, F = self.dg, self.R, self.H, self.F
        dg.dg_combine_bwd(self.dw, self.dYr, self.sr, R, self.dYc, self.sc, H, self.dout, self.Y, self.row_of,
                          self.slot_of, self.wt)
        dg.dg_grouped_contiguous_nt(self.dA, self.dYr, self.sr, R, *self.w["2t"], self.mi)
        dg.dg_swiglu_fp8_bwd(self.dHr, self.shr, R, self.dHc, self.shc, 2 * F, self.Qa, self.sb, self.dA, self.C,
                             self.cs, R, m_indices=self.mi)
        dg.dg_k_grouped_fp8_gemm_tn(self.dW2, self.dYc, self.sc, H, self.Qa, self.sb, self.off)
        dg.dg_grouped_contiguous_nt(self.dXr, self.dHr, self.shr, R, *self.w["1t"], self.mi)
        dg.dg_fp8_1x128_to_128x128(self.Xb, self.sx, self.Q, self.sa, R, m_indices=self.mi)
        dg.dg_k_grouped_fp8_gemm_tn(self.dW1, self.dHc, self.shc, 2 * F, self.Xb, self.sx, self.off)
        dg.dg_combine(self.dX, self.dXr, self.row_of)
        dg.dg_route_topk_bwd(self.dlogits, self.dw, self.logits, self.idx, score=dg.DG_SCORE_SIGMOID, renorm=True,
                             scale=2.0)

    def results(self):
        return dict(out=self.out, dX=self.dX, dW1=self.dW1, dW2=self.dW2, dlogits=self.dlogits, dw=self.dw)

    def exact(self):
        """The layer's formulas in 64 bits, nothing cast to 8 bits, the choice as made; through autograd."""
        d = lambda t: t.double().requires_grad_(True)  # noqa: E731
        X, l, W1, W2 = d(self.X), d(self.logits), d(self.W1), d(self.W2)
        w = torch.sigmoid(l).gather(1, self.idx.long())
        w = 2.0 * w / (w.sum(1, keepdim=True) + 1e-20)
        out = torch.zeros(self.T, self.H, dtype=torch.float64, device="cuda")
        for e in range(self.E):
            t, j = torch.nonzero(self.idx == e, as_tuple=True)
            h = X[t] @ W1[e].t()
            a = torch.nn.functional.silu(h[:, :self.F]) * h[:, self.F:]
            out = out.index_add(0, t, (a @ W2[e].t()) * w[t, j][:, None])
        gX, gl, g1, g2 = torch.autograd.grad((out * self.dout.double()).sum(), (X, l, W1, W2))
        return dict(out=out.detach(), dX=gX, dW1=g1, dW2=g2, dlogits=gl)


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


# What the 8-bit casts can cost, as relative 2-norms: rounding to e4m3 is off by at most 2^-4 of each
# value.  A product of two cast operands is off by at most 2 * 2^-4 + 2^-8 of the sum of magnitudes if all
# roundings conspire; they are independent, so the 2-norm of a long sum's error is that of one term:
# about sqrt(2) * 2^-4 / sqrt(3) = 0.051 of the result's.  The forward pass has two products and one cast
# between; out: 0.051 * sqrt(2) + the activation's response (at most about 2x) < 0.16.  The gradients add
# up to three more casts and the checkpoint's: < 0.25.  A wrong row, scale or weight is off by 1.
CASTS = dict(out=0.16, dX=0.25, dW1=0.25, dW2=0.25, dlogits=0.25)


@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 2, 256, 128), (50, 2, 4, 256, 256), (300, 4, 9, 512, 384)])
def test_layer_step(dgm, T, k, E, H, F):
    L = Layer(dgm, T, k, E, H, F, seed=T)
    for t in (L.Q, L.Q2, L.C, L.dYr, L.dYc, L.dHr, L.dHc, L.Qa, L.Xb):
        t.fill_(0x7F)   # rows that no call writes hold NaN
    for t in (L.Hid, L.Y, L.dA, L.dXr):
        t.fill_(float("nan"))
    L.forward()
    L.backward()
    want, got = L.exact(), L.results()
    for name, bound in CASTS.items():
        # With k = 1 a renormalised weight is scale s / (s + 1e-20), a constant to 1e-20, so the logits'
        # gradient is the difference of two equal terms, each at most scale |dw| (1 - s) <= 2 |dw|: both sides
        # are rounding noise there (FP32: 2^-24 per operation; 64 bits: 2^-53), and a relative error says nothing.
        floor = 2.0 ** -20 * float(got["dw"].norm()) if name == "dlogits" else 0.0
        off = float((got[name].double() - want[name].double()).norm())
        assert off < bound * float(want[name].norm()) + floor, (name, rel(got[name], want[name]))
    assert dgm.dg_get_device_error() == 0


def test_layer_under_graph_replay_and_on_other_streams(dgm):
    # Captured once, replayed with other inputs; and two layers at once on two streams: the same bits.
    A, B = Layer(dgm, 200, 3, 6, 256, 256, seed=1), Layer(dgm, 200, 3, 6, 256, 256, seed=2)
    for L in (A, B):
        for t in (L.Hid, L.Y, L.dA, L.dXr):
            t.zero_()
        L.forward()
        L.backward()
    torch.cuda.synchronize()
    ra, rb = ({n: t.clone() for n, t in L.results().items()} for L in (A, B))

    dgm.dg_set_pdl(False)  # launches that do not overlap their predecessors: the same
    try:
        A.forward()
        A.backward()
        torch.cuda.synchronize()
    finally:
        dgm.dg_set_pdl(None)
    assert all(torch.equal(t, ra[n]) for n, t in A.results().items())

    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for L in (A, B):
        for t in L.results().values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, L in ((s1, A), (s2, B)):
            with torch.cuda.stream(s):
                L.forward()
                L.backward()
    torch.cuda.synchronize()
    for L, want in ((A, ra), (B, rb)):
        assert all(torch.equal(t, want[n]) for n, t in L.results().items())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.forward()
        A.backward()
    for name in ("X", "logits", "bias", "dout"):
        getattr(A, name).copy_(getattr(B, name))
    for n, (q, s) in A.w.items():
        q.copy_(B.w[n][0])
        s.copy_(B.w[n][1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, rb[n]) for n, t in A.results().items())
    assert dgm.dg_get_device_error() == 0


def test_decoding_through_the_masked_layout(dgm):
    T, k, E, H, F = 24, 2, 6, 256, 256
    L = Layer(dgm, T, k, E, H, F, seed=4)
    M = 24
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    row_of, mi, slot_of, off, cnt = i(T, k), i(E * M), i(E * M), i(E + 1), i(E)
    Q, sa = torch.full((E, M, H), 0x7F, dtype=torch.uint8, device="cuda"), torch.zeros(E, H // 128, M, device="cuda")
    Hid = torch.full((E, M, 2 * F), float("nan"), dtype=torch.bfloat16, device="cuda")
    Q2, sa2 = torch.full((E, M, F), 0x7F, dtype=torch.uint8, device="cuda"), torch.zeros(E, F // 128, M, device="cuda")
    Y = torch.full((E, M, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgm.dg_route_topk(L.idx, L.wt, L.logits, L.bias, score=dgm.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
    dgm.dg_route_layout(row_of, mi, slot_of, off, cnt, L.idx, max_rows=M)
    dgm.dg_dispatch_fp8_1x128(Q, sa, M, L.X, row_of, group_rows=M)
    dgm.dg_grouped_masked_nt(Hid, Q, sa, M, *L.w["1"], cnt)
    dgm.dg_swiglu_fp8(Q2, sa2, M, Hid, m_indices=mi, group_rows=M)
    dgm.dg_grouped_masked_nt(Y, Q2, sa2, M, *L.w["2"], cnt)
    dgm.dg_combine(L.out, Y, row_of, L.wt)
    assert rel(L.out, L.exact()["out"]) < CASTS["out"]
    assert dgm.dg_get_device_error() == 0
