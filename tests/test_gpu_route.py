"""GPU: routing, its gradient and the grouped layout against plain 64-bit forms.

Choices and layouts are whole numbers and compared exactly.  The weights'
tolerance counts roundings: the score's exponential and quotient are good to
2 ulp each (2^-22 relative) and a softmax argument l - max is rounded once,
which moves exp by |l - max| 2^-24 relative; sum, renormalisation and scale
add a few more roundings of 2^-24.  So rel = 2^-24 (|l - max| + 40), taken with
the row's largest |l - max|.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dgm():
    from moe_grouped_gemm_weight_b200 import build
    build.build()
    import moe_grouped_gemm_weight_b200 as dg
    dg.dg_set_num_sms(0)
    assert dg.dg_get_device_error() == 0
    return dg


GUARD = 64


def guarded(n, dtype, fill):
    """A buffer with a guard band on both sides: (whole, the n elements)."""
    buf = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + n]


def guard_ok(buf, fill):
    b = buf.cpu()
    return bool((b[:GUARD] == fill).all() and (b[-GUARD:] == fill).all())


def scores64(l, sigmoid):
    l = l.double()
    return torch.sigmoid(l) if sigmoid else torch.softmax(l, dim=1)


def route64(logits, bias, k, groups, keep, gtop, sigmoid, renorm, scale):
    """The definition in 64 bits, one token after the other."""
    T, E = logits.shape
    s = scores64(logits, sigmoid).numpy()
    l = logits.double().numpy()
    b = np.zeros(E) if bias is None else bias.double().numpy()
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        c = s[t] + b
        ok = (l[t] != -math.inf) & (b != -math.inf)
        key = c if bias is not None else l[t]
        if groups > 1:
            n = E // groups
            rate = []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * n, g * n + n) if ok[e]),
                              key=lambda x: math.inf if x != x else x, reverse=True)[:gtop]
                rate.append(sum(best) if best else -math.inf)
            live = [g for g in range(groups) if ok[g * n:g * n + n].any()]
            live.sort(key=lambda g: (-math.inf if rate[g] != rate[g] else -rate[g], g))
            kept = set(live[:keep])
            ok = ok & np.array([e // n in kept for e in range(E)])
        order = [e for e in range(E) if ok[e]]
        order.sort(key=lambda e: (0, 0, e) if key[e] != key[e] else (1, -key[e], e))
        chosen = order[:k]
        idx[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = s[t][chosen]
        if renorm:
            w[t] /= w[t].sum() + 1e-20
    return idx, w * scale


def run_route(dg, logits, bias, k, groups, keep, gtop, sigmoid, renorm, scale):
    T, E = logits.shape
    ib, idx = guarded(T * k, torch.int32, 77)
    wb, w = guarded(T * k, torch.float32, 7.5)
    dg.dg_route_topk(idx.view(T, k), w.view(T, k), logits.cuda(), None if bias is None else bias.cuda(),
                     n_groups=groups, topk_groups=keep, group_top=gtop,
                     score=dg.DG_SCORE_SIGMOID if sigmoid else dg.DG_SCORE_SOFTMAX, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    assert guard_ok(ib, 77) and guard_ok(wb, 7.5)
    return idx.view(T, k).cpu().numpy(), w.view(T, k).cpu().double().numpy()


def check_route(dg, logits, bias=None, k=4, groups=1, keep=1, gtop=1, sigmoid=False, renorm=False, scale=1.0):
    idx, w = run_route(dg, logits, bias, k, groups, keep, gtop, sigmoid, renorm, scale)
    want, ww = route64(logits, bias, k, groups, keep, gtop, sigmoid, renorm, scale)
    bad = np.argwhere(idx != want)
    assert bad.size == 0, f"{len(bad)} choices differ, first at {bad[0]}: {idx[bad[0][0]]} vs {want[bad[0][0]]}"
    assert np.array_equal(np.isnan(w), np.isnan(ww))
    fin = logits.double().numpy()
    fin = np.where(np.isfinite(fin), fin, 0.0)
    span = (fin.max(axis=1) - fin.min(axis=1))[:, None]
    far = np.abs(w - ww) - (2.0 ** -24 * (span + 40) * np.abs(ww) + 1e-37)
    assert not (far > 0).any(), f"weights off by {np.nanmax(far)} beyond the bound"


# (T, E, k, groups, keep, gtop): every instance of experts per lane, odd sizes, one token, one expert
SHAPES = [(1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (9, 17, 5, 1, 1, 1), (8, 32, 8, 4, 2, 2), (65, 60, 4, 1, 1, 1),
          (33, 64, 6, 8, 3, 1), (17, 100, 8, 10, 3, 2), (20, 128, 16, 32, 8, 2), (64, 256, 8, 8, 4, 2),
          (40, 250, 7, 5, 2, 2), (21, 384, 8, 3, 1, 1), (12, 512, 16, 16, 16, 2), (9, 1000, 10, 25, 6, 2),
          (7, 1024, 16, 31 + 1, 5, 1)]


@pytest.mark.parametrize("T,E,k,groups,keep,gtop", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_matches_the_definition(dgm, T, E, k, groups, keep, gtop, sigmoid, with_bias):
    g = torch.Generator().manual_seed(T * 131 + E)
    for dt in (torch.float32, torch.bfloat16):
        logits = (2 * torch.randn(T, E, generator=g)).to(dt)
        bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
        check_route(dgm, logits, bias, k, groups, keep, gtop, sigmoid, renorm=dt == torch.float32, scale=2.5)


@pytest.mark.parametrize("E,groups,gtop", [(31, 1, 1), (64, 8, 2), (256, 8, 2), (500, 10, 1), (1024, 16, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_choices_next_to_one_another(dgm, E, groups, gtop, sigmoid):
    # The bias makes every choice value 0.5 up to its own rounding (3e-8), so no
    # FP32 arithmetic orders them; the result must still be the exact one.
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(1, E, generator=g)
    bias = (0.5 - scores64(logits, sigmoid)[0]).float()
    check_route(dgm, logits, bias, min(8, E // groups), groups, max(1, groups // 2), gtop, sigmoid)


# (E, groups): groups that end inside a lane's equal share, one or several lanes to a group; 930, 990
# and 1020 experts would give a lane more than 32
GROUP_EDGES = [(12, 3), (60, 4), (62, 31), (96, 3), (150, 30), (231, 7), (408, 8), (510, 17), (930, 6), (992, 31),
               (990, 30), (1020, 20)]


@pytest.mark.parametrize("E,groups", GROUP_EDGES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("gtop", [1, 2])
def test_groups_that_are_not_equal_shares_of_the_lanes(dgm, E, groups, sigmoid, with_bias, gtop):
    g = torch.Generator().manual_seed(E + groups)
    keep = max(1, groups // 3)
    k = min(8, keep * (E // groups))
    for dt in (torch.float32, torch.bfloat16):
        logits = torch.randn(37, E, generator=g).to(dt)
        logits[3].view(groups, -1)[::2] = -math.inf  # whole groups without an expert
        logits[4].view(groups, -1)[:, 1:] = -math.inf  # one expert left in each
        logits[5] = -math.inf
        logits[6] = 0.25
        bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
        check_route(dgm, logits, bias, k, groups, keep, gtop, sigmoid, renorm=True, scale=1.5)


@pytest.mark.parametrize("E,groups", GROUP_EDGES)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_next_to_one_another(dgm, E, groups, sigmoid):
    # All values equal up to the bias's rounding, and groups whose best two
    # stand out by as much: no FP32 arithmetic orders the groups.
    g = torch.Generator().manual_seed(E * 7 + groups)
    logits = torch.randn(1, E, generator=g)
    bias = (0.5 - scores64(logits, sigmoid)[0]).float()
    ahead = bias.clone().view(groups, -1)
    ahead[:, -2:] += 0.125
    for b in (bias, ahead.reshape(-1)):
        check_route(dgm, logits, b, min(2, E // groups), groups, max(1, groups // 2), 2, sigmoid)


@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias_of", ["none", "zero", "steps"])
def test_equal_values_go_to_the_lower_index(dgm, groups, keep, sigmoid, bias_of):
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-2, 3, (50, 128), generator=g).bfloat16()
    logits[0] = 0
    logits[1] = -0.0
    logits[1, 5] = 0.0
    bias = {"none": None, "zero": torch.zeros(128), "steps": 0.25 * torch.randint(0, 3, (128,), generator=g)}[bias_of]
    check_route(dgm, logits, bias, 8, groups, keep, 2, sigmoid, renorm=True)


@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts_and_rows(dgm, groups, keep, sigmoid, with_bias):
    g = torch.Generator().manual_seed(11)
    logits = torch.randn(12, 40, generator=g)
    bias = 0.1 * torch.randn(40, generator=g) if with_bias else None
    inf = math.inf
    logits[0] = -inf                       # nothing left
    logits[1, :39] = -inf                  # one left
    logits[2, 10:] = -inf                  # one group left
    logits[3, 5:35] = -inf                 # groups with none, and with half, left
    logits[4] = torch.finfo(torch.float32).min  # the lowest value is not a mask
    logits[5, ::2] = torch.finfo(torch.float32).min
    logits[6] = -200.0
    logits[7, 3] = 300.0
    if with_bias:
        bias[20:32] = -inf
    check_route(dgm, logits, bias, 6, groups, keep, 2, sigmoid, renorm=True)
    check_route(dgm, logits, bias, 6, groups, keep, 1, sigmoid)


def test_nan_and_infinity_show(dgm):
    logits = torch.randn(4, 40, generator=torch.Generator().manual_seed(1))
    logits[0, 7] = math.nan
    logits[1, 9] = math.inf
    logits[2, 30] = math.nan
    logits[2, 3] = math.nan
    for sigmoid in (False, True):
        for bias in (None, torch.zeros(40)):
            idx, w = run_route(dgm, logits, bias, 4, 1, 1, 1, sigmoid, False, 1.0)
            want, ww = route64(logits, bias, 4, 1, 1, 1, sigmoid, False, 1.0)
            assert np.array_equal(np.isnan(w), np.isnan(ww)) and np.array_equal(idx, want)
            idx, _ = run_route(dgm, logits, bias, 4, 4, 2, 2, sigmoid, False, 1.0)
            assert np.array_equal(idx, route64(logits, bias, 4, 4, 2, 2, sigmoid, False, 1.0)[0])


def off_by_one(t, value=0):
    """The same tensor one element into a buffer: contiguous, aligned to its elements only."""
    buf = torch.full((t.numel() + 1,), value, dtype=t.dtype, device="cuda")
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("E", [64, 256, 1024])
def test_tensors_aligned_to_their_elements_only(dgm, E):
    # Whole lanes at aligned addresses take wide loads; elsewhere the same values must come out.
    g = torch.Generator().manual_seed(E)
    for dt in (torch.float32, torch.bfloat16):
        logits, bias = torch.randn(33, E, generator=g).to(dt).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
        dw = torch.randn(33, 6, generator=g).cuda()
        out = []
        for shift in (lambda t: t, off_by_one):
            l, b = shift(logits), shift(bias)
            idx, w = shift(torch.zeros(33, 6, dtype=torch.int32, device="cuda")), shift(torch.zeros(33, 6, device="cuda"))
            dgm.dg_route_topk(idx, w, l, b, n_groups=8, topk_groups=3, group_top=2, score=1, renorm=True)
            d = shift(torch.zeros_like(logits))
            dgm.dg_route_topk_bwd(d, shift(dw), l, idx, score=0, renorm=True)
            out.append((idx.clone(), w.clone(), d.clone()))
        assert all(torch.equal(a, b) for a, b in zip(*out))


def test_many_tokens(dgm):
    # Every choice of 20000 tokens, against a sort in 64 bits on the device.
    g = torch.Generator(device="cuda").manual_seed(9)
    T, E, k = 20000, 256, 8
    logits = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    bias = 0.05 * torch.randn(E, generator=g, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    for sigmoid in (False, True):
        dgm.dg_route_topk(idx, w, logits, bias, score=int(sigmoid))
        c = scores64(logits, sigmoid) + bias.double()
        want = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(idx.long(), want)


# ------------------------------------------------------------------- gradient

def route_bwd64(logits, idx, dw, sigmoid, renorm, scale):
    """From the formulas, 64 bits; slots outside [0, E) are absent."""
    T, E = logits.shape
    ok = (idx >= 0) & (idx < E)
    at = torch.where(ok, idx, torch.zeros_like(idx)).long()
    s = scores64(logits, sigmoid)
    s = torch.where((logits == -math.inf).all(dim=1, keepdim=True), torch.zeros_like(s), s)
    sj = torch.where(ok, s.gather(1, at), torch.zeros((), dtype=torch.float64))
    ds = torch.where(ok, dw.double() * scale, torch.zeros((), dtype=torch.float64))
    if renorm:
        tot = sj.sum(1, keepdim=True) + 1e-20
        ds = torch.where(ok, (ds - (ds * sj).sum(1, keepdim=True) / tot) / tot, torch.zeros((), dtype=torch.float64))
    full = torch.zeros(T, E, dtype=torch.float64).scatter_add(1, at, ds)
    if sigmoid:
        return full * s * (1 - s), (ds.abs().sum(1, keepdim=True) * torch.ones(1, E))
    dot = (full * s).sum(1, keepdim=True)
    return s * (full - dot), s * (full.abs() + (full.abs() * s).sum(1, keepdim=True))


def check_bwd(dg, logits, idx, dw, sigmoid, renorm, scale):
    T, E = logits.shape
    buf, d = guarded(T * E, logits.dtype, 3.0)
    dg.dg_route_topk_bwd(d.view(T, E), dw.cuda(), logits.cuda(), idx.cuda(), score=int(sigmoid), renorm=renorm,
                         scale=scale)
    torch.cuda.synchronize()
    assert guard_ok(buf, 3.0)
    want, mag = route_bwd64(logits, idx, dw, sigmoid, renorm, scale)
    got = d.view(T, E).cpu().double()
    # FP32 terms: each is a product of values good to (span + 40) 2^-24; with
    # renormalisation the terms under the difference are divided by the sum once
    # more.  `mag` sums the terms' magnitudes; the store rounds once (bf16 2^-8).
    fin = torch.where(logits.double().isfinite(), logits.double(), torch.zeros((), dtype=torch.float64))
    span = (fin.amax(1) - fin.amin(1)).clamp_max(100)[:, None]
    s = scores64(logits, sigmoid)
    extra = mag
    if renorm:
        ok = (idx >= 0) & (idx < E)
        at = torch.where(ok, idx, torch.zeros_like(idx)).long()
        sj = torch.where(ok, s.nan_to_num(0).gather(1, at), torch.zeros((), dtype=torch.float64))
        tot = sj.sum(1, keepdim=True) + 1e-20
        terms = (dw.double() * scale).abs().sum(1, keepdim=True) / tot * 2
        extra = (s.nan_to_num(0) if not sigmoid else s.nan_to_num(0) * (1 - s.nan_to_num(0)) + 2.0 ** -24 * s.nan_to_num(0)) * terms * 3
    elif sigmoid:
        # 1 - s is rounded at 2^-24 of 1, not of itself
        extra = (s.nan_to_num(0) * (1 - s.nan_to_num(0)) + s.nan_to_num(0)) * mag
    half = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 2.0 ** -24
    tol = 2.0 ** -24 * 2 * (span + 40) * extra + half * want.abs() + 1e-37
    far = (got - want).abs() - tol
    assert not (far > 0).any(), f"off by {float(far.max())} beyond the bound"


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (33, 60, 4), (64, 256, 8), (10, 100, 16), (7, 512, 5),
                                   (5, 1000, 8), (3, 1024, 16)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient(dgm, T, E, k, sigmoid, renorm):
    g = torch.Generator().manual_seed(T + 7 * E)
    for dt in (torch.float32, torch.bfloat16):
        logits = (2 * torch.randn(T, E, generator=g)).to(dt)
        idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
        check_bwd(dgm, logits, idx, torch.randn(T, k, generator=g), sigmoid, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_of_absent_and_repeated_slots(dgm, sigmoid, renorm):
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(6, 70, generator=g)
    idx = torch.randint(0, 70, (6, 4), generator=g).int()
    idx[0] = -1
    idx[1, 1:] = -1
    idx[2] = 33                      # the same expert in every slot
    idx[3, 0], idx[3, 1] = 70, -5    # outside [0, E)
    logits[4, 10:] = -math.inf       # masked experts have no gradient
    idx[4] = torch.tensor([0, 3, 9, 5])
    logits[5] = -math.inf            # nothing left
    idx[5] = -1
    check_bwd(dgm, logits, idx, torch.randn(6, 4, generator=g), sigmoid, renorm, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_renormalised_gradient_does_not_cancel(dgm, sigmoid):
    # One expert with nearly all the weight, and one expert alone (its weight is a constant up to 1e-20):
    # dw_j - sum_i dw_i s_i / S is a small difference of large terms, but every element is good to
    # (span + 40) 2^-24 of the sum of the magnitudes |dw_j - dw_i| s_i, which is what is left of it.
    g = torch.Generator().manual_seed(6)
    for k in (1, 2, 4):
        logits = torch.randn(20, 12, generator=g)
        logits[:, 0] += 9.0
        idx = torch.stack([torch.cat([torch.zeros(1, dtype=torch.int64), 1 + torch.randperm(11, generator=g)[:k - 1]])
                           for _ in range(20)]).int()
        dw = torch.randn(20, k, generator=g)
        d = torch.empty(20, 12, device="cuda")
        dgm.dg_route_topk_bwd(d, dw.cuda(), logits.cuda(), idx.cuda(), score=int(sigmoid), renorm=True)
        s = scores64(logits, sigmoid)
        sj, w = s.gather(1, idx.long()), dw.double()
        tot = sj.sum(1, keepdim=True) + 1e-20
        terms = (w[:, :, None] - w[:, None, :]) * sj[:, None, :]
        ds = (terms.sum(2) + 1e-20 * w) / tot ** 2
        mag = (terms.abs().sum(2) + 1e-20 * w.abs()) / tot ** 2
        full = torch.zeros_like(s).scatter_add(1, idx.long(), ds)
        most = torch.zeros_like(s).scatter_add(1, idx.long(), mag)
        if sigmoid:
            factor, rest = s * (1 - s), 0.0
        else:
            # sum_j ds_j s_j: the differences cancel in pairs, (w_j - w_i) s_i s_j + (w_i - w_j) s_j s_i = 0, which
            # leaves 1e-20 sum_j w_j s_j / S^2 (summed as it stands, 64 bits keep only its rounding, 1e-17)
            factor, rest = s, 1e-20 * (w * sj).sum(1, keepdim=True) / tot ** 2
        want = factor * (full - rest)
        span = (logits.amax(1) - logits.amin(1)).double()[:, None]
        tol = 2.0 ** -24 * 2 * (span + 40) * (s * (most + (abs(rest) if not sigmoid else 0.0))) + 1e-37
        assert bool(((d.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(dgm, sigmoid, renorm):
    # Central differences of the 64-bit weights, the choice held.  h = 1e-4: the
    # cubic term is h^2/6 times a third derivative that is at most a few times
    # the weights' scale (below 1e-7 here), cancellation 1e-16/h = 1e-12.
    g = torch.Generator().manual_seed(2)
    T, E, k, scale, h = 3, 24, 4, 1.5, 1e-4
    logits = torch.randn(T, E, generator=g)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    dw = torch.randn(T, k, generator=g)

    def loss(l):
        w = scores64(l, sigmoid).gather(1, idx.long())
        if renorm:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return (scale * w * dw.double()).sum(1)

    d = torch.empty(T, E, device="cuda")
    dgm.dg_route_topk_bwd(d, dw.cuda(), logits.cuda(), idx.cuda(), score=int(sigmoid), renorm=renorm, scale=scale)
    d = d.cpu().double()
    for e in range(E):
        step = torch.zeros(T, E, dtype=torch.float64)
        step[:, e] = h
        num = (loss(logits.double() + step) - loss(logits.double() - step)) / (2 * h)
        assert torch.allclose(d[:, e], num, rtol=1e-5, atol=2e-6), (e, d[:, e], num)


# --------------------------------------------------------------------- layout

def layout64(idx, E, rows, max_rows):
    T, k = idx.shape
    row_of = np.full((T, k), -1, np.int32)
    m_indices, slot_of = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32)
    lists = [[] for _ in range(E)]
    for s, e in enumerate(idx.reshape(-1)):
        if 0 <= e < E:
            lists[e].append(s)
    offsets, counts, at = [], [], 0
    for e in range(E):
        mine = lists[e][:max_rows] if max_rows else lists[e]
        offsets.append(at)
        counts.append(len(mine))
        for i, s in enumerate(mine):
            row_of.reshape(-1)[s] = at + i
            m_indices[at + i] = e
            slot_of[at + i] = s
        at += max_rows if max_rows else -(-len(mine) // 128) * 128
    return row_of, m_indices, slot_of, np.array(offsets + [at], np.int32), np.array(counts, np.int32)


def run_layout(dg, idx, E, rows, max_rows=0):
    T, k = idx.shape
    sizes = [T * k, rows, rows, E + 1, E]
    bufs = [guarded(n, torch.int32, 12345) for n in sizes]
    views = [v for _, v in bufs]
    dg.dg_route_layout(views[0].view(T, k), views[1], views[2], views[3], views[4], idx.cuda(), max_rows=max_rows)
    torch.cuda.synchronize()
    assert all(guard_ok(b, 12345) for b, _ in bufs)
    out = [v.cpu().numpy() for v in views]
    out[0] = out[0].reshape(T, k)
    return out


@pytest.mark.parametrize("T,k,E,extra,max_rows", [
    (0, 2, 5, 0, 0), (0, 2, 5, 256, 0), (0, 1, 4, 0, 16), (1, 1, 1, 0, 0), (1, 8, 256, 0, 0), (37, 3, 7, 128, 0),
    (500, 8, 8, 0, 0), (513, 8, 64, 384, 0), (1025, 4, 60, 0, 0), (4096, 8, 64, 0, 0), (9000, 5, 1024, 0, 0),
    (20001, 7, 33, 1280, 0), (33000, 8, 40, 0, 0), (40000, 8, 1024, 0, 0), (64, 8, 32, 0, 64), (64, 8, 32, 0, 5), (300, 6, 130, 0, 300), (5000, 8, 1000, 0, 3)])
def test_layout(dgm, T, k, E, extra, max_rows):
    g = torch.Generator().manual_seed(T + E)
    idx = torch.randint(-1, E, (T, k), generator=g).int()
    if T > 30:
        idx[5:T // 4] = E // 2        # a crowded expert
    rows = E * max_rows or dgm.dg_get_layout_rows(T, k, E) + extra
    got = run_layout(dgm, idx, E, rows, max_rows)
    want = layout64(idx.numpy(), E, rows, max_rows)
    for name, a, b in zip(("row_of", "m_indices", "slot_of", "group_offsets", "counts"), got, want):
        assert np.array_equal(a, b), name
    assert dgm.dg_get_device_error() == 0


def test_layout_flags_experts_out_of_range(dgm):
    idx = torch.tensor([[0, 3], [-1, 7], [2, -9]], dtype=torch.int32)
    rows = dgm.dg_get_layout_rows(3, 2, 3)
    got = run_layout(dgm, idx, 3, rows)
    want = layout64(idx.numpy(), 3, rows, 0)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert dgm.dg_get_device_error() == dgm.DG_DEVERR_BAD_EXPERT
    assert dgm.dg_get_device_error() == 0
