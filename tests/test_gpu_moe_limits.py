"""GPU: the calls around the grouped GEMMs where FP32, 31 bits, a cap or a second host thread can go wrong."""
import ctypes
import math
import subprocess
import threading

import pytest
import torch

from tests.test_gpu_moe import Layer, codes, scales
from tests.test_gpu_route import check_route, scores64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of FP32, relative


@pytest.fixture(scope="module")
def dgm():
    from moe_grouped_gemm_weight_b200 import build
    build.build()
    import moe_grouped_gemm_weight_b200 as dg
    dg.dg_set_num_sms(0)
    assert dg.dg_get_device_error() == 0
    return dg


HAMMER = """
typedef int (*layout_fn)(void *, void *, void *, void *, void *, const void *, int, int, int, int, int, void *);
int hammer(layout_fn f, void **p, int T, int k, int E, int rows, void *stream, int n) {
    int failed = 0;
    for (int i = 0; i < n; ++i) failed += f(p[0], p[1], p[2], p[3], p[4], p[5], T, k, E, rows, 0, stream) != 0;
    return failed;
}
"""


def test_layouts_of_different_sizes_from_two_host_threads(dgm, tmp_path):
    # 8192 slots over 512 and over 600 experts take 80 and 94 KiB of shared memory, above what a kernel may have
    # without asking: a call must not lower what another thread has just asked for.
    (tmp_path / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-o", str(tmp_path / "hammer.so"), str(tmp_path / "hammer.c")],
                   check=True)
    hammer = ctypes.CDLL(str(tmp_path / "hammer.so")).hammer  # without the interpreter lock
    fn = ctypes.cast(dgm.lib().dg_route_layout, ctypes.c_void_p)
    T, k = 1024, 8
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    failed, outs = {}, {}

    def make(E):
        rows = dgm.dg_get_layout_rows(T, k, E)
        idx = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(E)).int().cuda()
        return i(T, k), i(rows), i(rows), i(E + 1), i(E), idx

    def work(E):
        args = outs[E]
        ptrs = (ctypes.c_void_p * 6)(*(t.data_ptr() for t in args))
        stream = torch.cuda.Stream()
        failed[E] = hammer(fn, ptrs, T, k, E, args[1].numel(), ctypes.c_void_p(stream.cuda_stream), 5000)
        stream.synchronize()

    for E in (512, 600):
        outs[E] = make(E)
        dgm.dg_route_layout(*outs[E])
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(E,)) for E in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == {512: 0, 600: 0}
    for E, args in outs.items():
        again = make(E)
        dgm.dg_route_layout(*again)
        assert all(torch.equal(a, b) for a, b in zip(args, again)), E


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (60, 5), (1020, 20)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_group_whose_sum_leaves_fp32_is_no_masked_group(dgm, E, groups, sigmoid, dtype):
    # The sum of two choice values at the lowest finite float is below every float, but the group has experts:
    # it stays behind the others, before masked ones.  Three experts of one group are ordinary, one group is masked.
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(7, E, generator=g).to(dtype)
    n = E // groups
    bias = torch.full((E,), torch.finfo(torch.float32).min)
    bias[n:2 * n] = -math.inf
    bias[2 * n:2 * n + 3] = 0.1
    bias[2 * n + 3:3 * n] = -math.inf
    check_route(dgm, logits, bias, k=8, groups=groups, keep=3, gtop=2, sigmoid=sigmoid, renorm=True, scale=1.0)
    check_route(dgm, logits, bias, k=8, groups=groups, keep=groups - 1, gtop=2, sigmoid=sigmoid)


def test_masked_layout_whose_ranks_pass_31_bits(dgm):
    # The last group starts three million rows below 2^31, and more slots ask for it than there are numbers left.
    E, k = 1024, 1
    M = 0x7FF00000 // E
    T = (1 << 31) - (E - 1) * M + 70000
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    idx = torch.full((T, k), E - 1, dtype=torch.int32, device="cuda")
    row_of, m_indices, slot_of, off, cnt = i(T, k), i(E * M), i(E * M), i(E + 1), i(E)
    dgm.dg_route_layout(row_of, m_indices, slot_of, off, cnt, idx, max_rows=M)
    want = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    want[:M] = torch.arange(M, dtype=torch.int32, device="cuda") + (E - 1) * M
    assert torch.equal(row_of.view(-1), want)
    assert int(cnt[-1]) == M and int(cnt[:-1].sum()) == 0 and int(off[-1]) == E * M
    assert bool((m_indices[:(E - 1) * M] == -1).all() and (m_indices[(E - 1) * M:] == E - 1).all())
    assert torch.equal(slot_of[(E - 1) * M:], torch.arange(M, dtype=torch.int32, device="cuda"))
    assert dgm.dg_get_device_error() == 0


@pytest.mark.parametrize("sms", [1, 3, 7])
def test_nothing_is_left_out_under_an_sm_cap(dgm, sms):
    # Every output starts from the same bytes with and without the cap; what a call leaves, it leaves in both.  The
    # GEMMs' results stay.  dw's partial sums may be joined in another order: one rounding for each of the 1152 / 16
    # products of a lane and the joins, of the terms' magnitudes, in both runs.
    L = Layer(dgm, 300, 4, 9, 1152, 384, seed=3)
    for t in (L.Hid, L.Y, L.dA, L.dXr):
        t.zero_()
    L.forward()
    L.backward()
    made = [n for n, t in vars(L).items() if torch.is_tensor(t) and n not in
            ("X", "logits", "bias", "dout", "W1", "W2", "Hid", "Y", "dA", "dXr", "dW1", "dW2")]
    given = L.dw.clone()

    def step():
        for n in made:
            getattr(L, n).view(torch.uint8).fill_(0x11)
        dgm.dg_route_topk(L.idx, L.wt, L.logits, L.bias, score=dgm.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
        dgm.dg_route_layout(L.row_of, L.mi, L.slot_of, L.off, L.cnt, L.idx)
        dgm.dg_dispatch_fp8_1x128(L.Q, L.sa, L.R, L.X, L.row_of)
        dgm.dg_swiglu_fp8(L.Q2, L.sa2, L.R, L.Hid, L.C, L.cs, L.R, m_indices=L.mi)
        dgm.dg_combine(L.out, L.Y, L.row_of, L.wt)
        dgm.dg_combine_bwd(L.dw, L.dYr, L.sr, L.R, L.dYc, L.sc, L.H, L.dout, L.Y, L.row_of, L.slot_of, L.wt)
        dgm.dg_swiglu_fp8_bwd(L.dHr, L.shr, L.R, L.dHc, L.shc, 2 * L.F, L.Qa, L.sb, L.dA, L.C, L.cs, L.R, m_indices=L.mi)
        dgm.dg_fp8_1x128_to_128x128(L.Xb, L.sx, L.Q, L.sa, L.R, m_indices=L.mi)
        dgm.dg_combine(L.dX, L.dXr, L.row_of)
        dgm.dg_route_topk_bwd(L.dlogits, given, L.logits, L.idx, score=dgm.DG_SCORE_SIGMOID, renorm=True, scale=2.0)
        torch.cuda.synchronize()
        return {n: getattr(L, n).clone() for n in made}

    want = step()
    assert all(bool((want[n].view(torch.uint8) != 0x11).any()) for n in made)
    dgm.dg_set_num_sms(sms)
    try:
        got = step()
    finally:
        dgm.dg_set_num_sms(0)
    for n in made:
        if n != "dw":
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n
    row = L.row_of.long()
    mag = (L.dout.float()[:, None] * L.Y[row.clamp_min(0)].float()).abs().sum(2) * (row >= 0)
    assert bool(((got["dw"] - want["dw"]).abs() <= 2 * (1152 / 16 + 32) * U * mag).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid_gradient_where_the_score_is_nearly_one(dgm, dtype):
    # s (1 - s) with 1 - s for itself: 1 / (1 + e) and e / (1 + e), an exponential of 2 ulp (4 U), an addition, a
    # quotient, a product each; scale dw and two more: at most 2 (4 + 1 + 1) + 4 half steps, and the type's rounding.
    l = torch.cat([torch.arange(-80, 80, 0.625), torch.tensor([16.0, 17.0, 18.0, 40.0, 80.0])]).to(dtype)
    T, E = l.numel(), 5
    logits = torch.zeros(T, E, dtype=dtype)
    logits[:, 3] = l
    dw = torch.linspace(0.5, 2.0, T)[:, None]
    d = torch.empty(T, E, dtype=dtype, device="cuda")
    dgm.dg_route_topk_bwd(d, dw.cuda(), logits.cuda(), torch.full((T, 1), 3, dtype=torch.int32, device="cuda"),
                          score=dgm.DG_SCORE_SIGMOID, scale=1.0)
    x = l.double()
    want = dw[:, 0].double() * torch.sigmoid(x) * torch.sigmoid(-x)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    got = d.cpu().double()[:, 3]
    assert bool(((got - want).abs() <= (16 * U + half) * want).all()), float(((got - want).abs() / want).max())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [8, 60, 256, 1024])
def test_softmax_gradient_of_a_dominant_expert(dgm, E, renorm):
    # ds_e - sum_j ds_j s_j is (1 - s_e) ds_e - sum over the other experts' slots, and 1 - s_e a sum of other
    # scores.  k = 1: dl_e = s_e dw (1 - s_e), dl_i = -s_i s_e dw.  Logits are multiples of 1/8, so their
    # differences are exact: a score is an exponential (5 U), a sum of E of them (5 U + at most 37 U), quotient and
    # product; dl has two scores and a few products: 2 (5 + 42 + 2) + 6 half steps.
    g = torch.Generator().manual_seed(E)
    logits = (-10 - torch.randint(0, 400, (40, E), generator=g).float() / 8)
    top = torch.randint(0, E, (40,), generator=g)
    logits[torch.arange(40), top] = torch.arange(40).float() / 4
    k = 2 if renorm else 1
    idx = torch.stack([top, (top + 1) % E], dim=1)[:, :k].int().contiguous()
    dw = torch.randn(40, k, generator=g)
    d = torch.empty(40, E, device="cuda")
    dgm.dg_route_topk_bwd(d, dw.cuda(), logits.cuda(), idx.cuda(), renorm=renorm)
    s = scores64(logits, False)
    w = dw.double()
    if not renorm:
        rest = torch.where(torch.arange(E) == top[:, None], 0.0, s).sum(1)  # 1 - s_e without cancellation
        se = s.gather(1, top[:, None])[:, 0]
        want = -s * (se * w[:, 0])[:, None]
        want[torch.arange(40), top] = se * w[:, 0] * rest
        tol = 105 * U * want.abs() + 1e-37
    else:
        s1, s2 = s.gather(1, idx.long()).unbind(1)
        S = s1 + s2 + 1e-20
        want = torch.zeros_like(s)
        # w1 = s1 / S: dL = (dw1 - dw2) s1 s2 / S^2 (dl1 - dl2), up to 1e-20
        x = (w[:, 0] - w[:, 1]) * s1 * s2 / S ** 2
        want[torch.arange(40), idx[:, 0].long()] = x
        want[torch.arange(40), idx[:, 1].long()] = -x
        mag = (w.abs().sum(1) * 1e-20 / S)[:, None] * s
        tol = 250 * U * want.abs() + 4 * mag + 1e-37  # four scores of 49, and products
    far = (d.cpu().double() - want).abs() - tol
    assert not bool((far > 0).any()), float(((d.cpu().double() - want).abs() / want.abs().clamp_min(1e-300)).max())


@pytest.mark.parametrize("g_range", [(-80.0, -20.0), (-20.0, 0.0), (0.0, 80.0)])
def test_gated_activation_is_good_to_fp32(dgm, g_range):
    # One value to a tile, whose scale shows it in FP32: a = 448 sa.  Exponential 2^-22.5 and two roundings (5 U),
    # 1 + e, quotient (1 ulp: 2 U), product with the gate, up a power of two (exact), / 448: 10 half steps.
    F, rows = 128 * 16, 64
    lo, hi = g_range
    gate = (lo + (hi - lo) * torch.rand(rows, F // 128, generator=torch.Generator().manual_seed(1))).bfloat16()
    gate[0, 0], gate[0, 1] = lo or 0.5, hi or -0.5
    x = gate.double()
    silu = x / (1 + torch.exp(-x))
    up = torch.exp2(torch.round(-torch.log2(silu.abs().clamp_min(1e-300))))  # a about 1
    H = torch.zeros(rows, 2 * F)
    H[:, ::128][:, :F // 128], H[:, ::128][:, F // 128:] = gate.float(), up.float()
    Q, sa = codes(rows, F), scales(F // 128, rows)
    dgm.dg_swiglu_fp8(Q, sa, rows, H.bfloat16().cuda())
    want = (silu * up).abs() / 448
    off = (sa.cpu().t().double() - want).abs() / want
    assert bool((off <= 11 * U).all()), float(off.max() / U)


@pytest.mark.parametrize("g_range", [(-80.0, -20.0), (-20.0, -3.0), (0.0, 80.0)])
def test_gradient_of_the_gated_activation_is_good_to_fp32(dgm, g_range):
    # As above: code 1 times the scale is the gate itself, one value to a tile, the gradient's scales show it.
    # s as above without the product (8 U); d up = dA silu: 9 + 1 + 1.  d gate = dA up (s + silu (1 - s)): silu 9 U;
    # 1 - s loses U and 8 U s; their product U; the sum U; two products and / 448.
    F, rows = 128 * 16, 128
    lo, hi = g_range
    gate = lo + (hi - lo) * torch.rand(rows, F // 128, generator=torch.Generator().manual_seed(2))
    x = gate.double()
    s = 1 / (1 + torch.exp(-x))
    silu, one = x * s, 1 / (1 + torch.exp(x))
    t = s + silu * one
    big = torch.exp2(torch.round(-torch.log2(torch.minimum(silu.abs(), t.abs()))))
    C = torch.zeros(rows, 2 * F, dtype=torch.uint8)
    C[:, ::128] = 0x38                                         # 1.0
    cs = torch.cat([gate, torch.ones_like(gate)], dim=1).t().contiguous()
    dA = torch.zeros(rows, F)
    dA[:, ::128] = big.float()
    out = (codes(rows, 2 * F), scales(2 * F // 128, rows), codes(rows, 2 * F), scales(1, 2 * F), codes(rows, F),
           scales(F // 128, 1))
    dgm.dg_swiglu_fp8_bwd(out[0], out[1], rows, out[2], out[3], 2 * F, out[4], out[5], dA.bfloat16().cuda(), C.cuda(),
                          cs.cuda(), rows)
    sr = out[1].cpu().t().double()
    dgate, dup = (t * big).abs() / 448, (silu * big).abs() / 448
    bound_t = (8 * s + (9 + 1) * (silu * one).abs() + silu.abs() * (1 + 8 * s) + t.abs()) / t.abs() + 3
    off_u = (sr[:, F // 128:] - dup).abs() / dup
    off_g = (sr[:, :F // 128] - dgate).abs() / dgate
    assert bool((off_u <= 12 * U).all()), float(off_u.max() / U)
    assert bool((off_g <= (bound_t + 1) * U).all()), float((off_g / bound_t).max() / U)


@pytest.mark.parametrize("E", [8, 60, 256])
def test_softmax_scores_far_below_the_largest(dgm, E):
    # In the gradient too a score is an exponential good to 5 U however far its logit lies below the largest
    # (multiples of 1/8: the difference is exact): dl_i = -s_i s_e dw, counted as above.
    g = torch.Generator().manual_seed(3)
    logits = -torch.randint(0, 640, (64, E), generator=g).float() / 8
    logits[:, 2] = 0.0
    dw = torch.ones(64, 1)
    d = torch.empty(64, E, device="cuda")
    dgm.dg_route_topk_bwd(d, dw.cuda(), logits.cuda(), torch.full((64, 1), 2, dtype=torch.int32, device="cuda"))
    s = scores64(logits, False)
    want = s * s[:, 2:3]
    off = (d.cpu().double().neg() - want).abs() / want
    off[:, 2] = 0
    n = 2 * (5 + 5 + 5 + (E + 31) // 32 + 2) + 3
    assert bool((off <= n * U).all()), (float(off.max() / U), n)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_the_renormalised_weight_of_one_expert_is_one(dgm, sigmoid):
    # s / (s + 1e-20), the sum s itself in FP32 (s > 1e-12): a quotient rounded to nearest is 1.
    g = torch.Generator().manual_seed(8)
    logits = (20 * torch.rand(5000, 24, generator=g) - 20).cuda()
    idx, w = torch.empty(5000, 1, dtype=torch.int32, device="cuda"), torch.empty(5000, 1, device="cuda")
    dgm.dg_route_topk(idx, w, logits, score=int(sigmoid), renorm=True)
    assert bool((w == 1.0).all()), int((w != 1.0).sum())
