"""Host-side tests of the calls around the grouped GEMMs (no GPU needed): the C
ABI refuses bad sizes, strides, alignments and null pointers before any launch,
and the Python binding refuses tensors that the kernels would read or write
past, or of another type or shape."""
import pytest
import torch

import moe_grouped_gemm_weight_b200 as dg
from moe_grouped_gemm_weight_b200 import build as dgbuild

FAKE = 1 << 20  # never dereferenced: every call fails validation first, or has nothing to do
INV, UNS, MIS, OK = dg.DG_ERR_INVALID_ARG, dg.DG_ERR_UNSUPPORTED, dg.DG_ERR_MISALIGNED, dg.DG_OK


@pytest.fixture(scope="module", autouse=True)
def built_library():
    dgbuild.build()
    yield


def swapped(good, **changes):
    """Arguments `good` (an ordered dict) with some replaced."""
    return [changes.get(n, v) for n, v in good.items()]


ROUTE = dict(idx=FAKE, w=FAKE, logits=FAKE, dtype=0, bias=0, T=4, E=64, k=4, groups=8, keep=4, gtop=2, score=1,
             renorm=1, scale=1.0, stream=0)
ROUTE_BWD = dict(dlogits=FAKE, dw=FAKE, logits=FAKE, dtype=1, idx=FAKE, T=4, E=64, k=4, score=0, renorm=1, scale=1.0,
                 stream=0)
LAYOUT = dict(row_of=FAKE, m_indices=FAKE, slot_of=FAKE, offsets=FAKE, counts=FAKE, idx=FAKE, T=4, k=2, E=3,
              rows=384, max_rows=0, stream=0)
DISPATCH = dict(Q=FAKE, sa=FAKE, stride=384, X=FAKE, row_of=FAKE, T=4, k=2, K=256, rows=384, group_rows=0, stream=0)
COMBINE = dict(out=FAKE, Y=FAKE, row_of=FAKE, w=0, T=4, k=2, N=64, rows=384, stream=0)
COMBINE_BWD = dict(dw=FAKE, Qr=FAKE, sr=FAKE, sr_stride=384, Qc=FAKE, sc=FAKE, sc_stride=256, dout=FAKE, Y=FAKE,
                   row_of=FAKE, slot_of=FAKE, w=FAKE, T=4, k=2, N=256, rows=384, stream=0)
SWIGLU = dict(Q=FAKE, sa=FAKE, sa_stride=384, C=FAKE, cs=FAKE, cs_stride=384, H=FAKE, m_indices=0, rows=384, F=256,
              group_rows=0, stream=0)
SWIGLU_BWD = dict(Qr=FAKE, sr=FAKE, sr_stride=384, Qc=FAKE, sc=FAKE, sc_stride=512, Qa=FAKE, sb=FAKE, dA=FAKE, C=FAKE,
                  cs=FAKE, cs_stride=384, m_indices=0, rows=384, F=256, stream=0)
RECAST = dict(Qb=FAKE, sb=FAKE, Q=FAKE, sa=FAKE, sa_stride=384, m_indices=0, rows=384, K=256, stream=0)

REFUSALS = [
    ("dg_route_topk", ROUTE, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=65), INV), (dict(dtype=2), INV),
        (dict(score=2), INV), (dict(groups=7), INV), (dict(groups=0), INV), (dict(keep=0), INV), (dict(keep=9), INV),
        (dict(gtop=3), INV), (dict(gtop=0), INV), (dict(E=1032), UNS), (dict(k=17), UNS),
        (dict(E=64, groups=64, keep=2), UNS), (dict(T=1 << 30), UNS), (dict(idx=0), INV), (dict(w=0), INV),
        (dict(logits=0), INV), (dict(logits=FAKE + 1), MIS), (dict(dtype=1, logits=FAKE + 2), MIS),
        (dict(bias=FAKE + 2), MIS), (dict(idx=FAKE + 2), MIS), (dict(T=0, logits=0), OK)]),
    ("dg_route_topk_bwd", ROUTE_BWD, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(k=65), INV), (dict(dtype=-1), INV), (dict(score=-1), INV),
        (dict(E=1025), UNS), (dict(k=17), UNS), (dict(dlogits=0), INV), (dict(dw=0), INV), (dict(idx=0), INV),
        (dict(dlogits=FAKE + 2), MIS), (dict(dw=FAKE + 1), MIS), (dict(T=0, dw=0), OK)]),
    ("dg_route_layout", LAYOUT, [
        (dict(T=-1), INV), (dict(k=0), INV), (dict(k=33), UNS), (dict(E=0), INV), (dict(E=1025), UNS),
        (dict(rows=-128), INV), (dict(rows=385), INV), (dict(rows=256), INV), (dict(max_rows=-1), INV),
        (dict(max_rows=100), INV), (dict(T=1 << 30), UNS), (dict(T=(1 << 30) - 1, rows=2147483520), UNS), (dict(rows=0x7FF00080), UNS),
        (dict(T=0x3FF80000, k=2, E=1000), UNS),
        (dict(row_of=0), INV), (dict(m_indices=0), INV), (dict(slot_of=0), INV), (dict(offsets=0), INV),
        (dict(counts=0), INV), (dict(idx=0), INV), (dict(idx=FAKE + 2), MIS), (dict(counts=FAKE + 1), MIS)]),
    ("dg_dispatch_fp8_1x128", DISPATCH, [
        (dict(T=-1), INV), (dict(k=33), UNS), (dict(K=0), INV), (dict(K=192), UNS), (dict(K=(1 << 28) + 128), UNS),
        (dict(rows=0x7FF00080, stride=0x7FF00080), UNS), (dict(stride=383), INV),
        (dict(group_rows=-1), INV), (dict(group_rows=100), INV), (dict(group_rows=128, stride=127), INV),
        (dict(Q=0), INV), (dict(sa=0), INV), (dict(X=0), INV), (dict(row_of=0), INV), (dict(Q=FAKE + 8), MIS),
        (dict(X=FAKE + 8), MIS), (dict(sa=FAKE + 2), MIS), (dict(T=0, X=0), OK), (dict(rows=0, stride=0, Q=0), OK)]),
    ("dg_combine", COMBINE, [
        (dict(T=-1), INV), (dict(k=0), INV), (dict(k=40), UNS), (dict(N=0), INV), (dict(N=12), UNS), (dict(N=2147483640), UNS),
        (dict(rows=-1), INV), (dict(out=0), INV), (dict(Y=0), INV), (dict(row_of=0), INV), (dict(out=FAKE + 8), MIS),
        (dict(Y=FAKE + 2), MIS), (dict(w=FAKE + 2), MIS), (dict(T=0, out=0), OK)]),
    ("dg_combine_bwd", COMBINE_BWD, [
        (dict(T=-1), INV), (dict(k=33), UNS), (dict(N=64), UNS), (dict(N=0), INV), (dict(rows=300), INV),
        (dict(rows=-128), INV), (dict(rows=0), INV), (dict(sr_stride=383), INV), (dict(sc_stride=255), INV),
        (dict(dw=0), INV), (dict(Qr=0), INV), (dict(sr=0), INV), (dict(Qc=0), INV), (dict(sc=0), INV),
        (dict(dout=0), INV), (dict(Y=0), INV), (dict(row_of=0), INV), (dict(slot_of=0), INV), (dict(w=0), INV),
        (dict(Qc=FAKE + 8), MIS), (dict(dout=FAKE + 2), MIS), (dict(sc=FAKE + 2), MIS), (dict(T=0, dw=0), OK)]),
    ("dg_swiglu_fp8", SWIGLU, [
        (dict(rows=-1), INV), (dict(F=0), INV), (dict(F=64), UNS), (dict(F=(1 << 28) + 128), UNS), (dict(sa_stride=383), INV),
        (dict(cs_stride=383), INV), (dict(group_rows=-2), INV), (dict(group_rows=100), INV),
        (dict(group_rows=128, sa_stride=128, cs_stride=100), INV), (dict(Q=0), INV), (dict(sa=0), INV),
        (dict(H=0), INV), (dict(cs=0), INV), (dict(H=FAKE + 8), MIS), (dict(C=FAKE + 8), MIS),
        (dict(m_indices=FAKE + 2), MIS), (dict(rows=0, sa_stride=0, H=0), OK)]),
    ("dg_swiglu_fp8_bwd", SWIGLU_BWD, [
        (dict(rows=-128), INV), (dict(rows=200), INV), (dict(F=0), INV), (dict(F=100), UNS),
        (dict(sr_stride=383), INV), (dict(cs_stride=383), INV), (dict(sc_stride=511), INV), (dict(Qr=0), INV),
        (dict(Qc=0), INV), (dict(Qa=0), INV), (dict(sb=0), INV), (dict(dA=0), INV), (dict(C=0), INV),
        (dict(cs=0), INV), (dict(dA=FAKE + 8), MIS), (dict(sb=FAKE + 1), MIS), (dict(rows=0, Qr=0), OK)]),
    ("dg_fp8_1x128_to_128x128", RECAST, [
        (dict(rows=-128), INV), (dict(rows=200), INV), (dict(K=0), INV), (dict(K=100), UNS),
        (dict(sa_stride=383), INV), (dict(Qb=0), INV), (dict(sb=0), INV), (dict(Q=0), INV), (dict(sa=0), INV),
        (dict(Qb=FAKE + 8), MIS), (dict(sa=FAKE + 2), MIS), (dict(rows=0, Qb=0), OK)]),
]


@pytest.mark.parametrize("name,good,changes,want", [(n, g, c, w) for n, g, cs in REFUSALS for c, w in cs])
def test_bad_arguments_are_refused_before_any_launch(name, good, changes, want):
    L = dg.lib()
    assert getattr(L, name)(*swapped(good, **changes)) == want, L.dg_last_error_message()
    if want != OK:
        assert L.dg_last_error_message()


def test_calls_fail_loudly_without_the_extension(monkeypatch):
    import sys
    monkeypatch.setattr(dg, "_calls", None)
    monkeypatch.setitem(sys.modules, dg.__name__ + "._dgcall", None)
    monkeypatch.delattr(dg, "_dgcall", raising=False)
    with pytest.raises(RuntimeError, match="_dgcall"):
        dg.dg_route_topk(**BINDING["dg_route_topk"])


def test_marshalling_refuses_numbers_that_do_not_fit():
    c = dg._marshal()
    args = swapped(COMBINE, T=0)
    assert c.dg_combine(*args) == OK
    for bad in (1 << 31, -(1 << 31) - 1, 1 << 70):
        with pytest.raises(OverflowError):
            c.dg_combine(*swapped(COMBINE, T=0, N=bad))
    with pytest.raises(TypeError):
        c.dg_combine(*swapped(COMBINE, T=1.5))
    for bad in ("x", 1.5, [1], object()):
        with pytest.raises(TypeError):
            c.dg_combine(*swapped(COMBINE, out=bad))
        with pytest.raises(TypeError):
            c.dg_combine(*swapped(COMBINE, T=0, out=bad, k="y"))
    with pytest.raises(Exception):  # a tensor without memory behind it
        c.dg_combine(*swapped(COMBINE, T=0, out=torch.zeros(2, 2).to_sparse()))
    assert c.fits("x", 4, 1) == -1 and c.fits(torch.zeros(3), 4, 3) == -1 and c.fits(None, 4, 3) == -1
    for bad in ((), (torch.zeros(3), 4), (torch.zeros(3), "a", 3), (torch.zeros(3), 4, "a")):
        with pytest.raises(TypeError):
            c.fits(*bad)
    with pytest.raises(TypeError):
        c.dg_route_topk(*swapped(ROUTE, T=0, scale="z"))
    with pytest.raises(TypeError):
        c.dg_combine(*args[:-1])
    assert c.dg_combine(*swapped(COMBINE, T=0, w=None, stream=None)) == OK


def test_layout_rows():
    assert dg.dg_get_layout_rows(0, 8, 256) == 0
    assert dg.dg_get_layout_rows(1, 1, 256) == 128
    assert dg.dg_get_layout_rows(4, 2, 3) == (8 + 3 * 127) // 128 * 128
    assert dg.dg_get_layout_rows(4096, 8, 64) == (32768 + 64 * 127) // 128 * 128
    for bad in [(-1, 1, 1), (1, 0, 1), (1, 33, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 2, 1), ((1 << 30) - 1, 2, 1024)]:
        assert dg.dg_get_layout_rows(*bad) == -1
    # No choice of experts needs more: the segments of any counts are whole 128 rows.
    import random
    rng = random.Random(5)
    for _ in range(200):
        T, k, E = rng.randint(1, 300), rng.randint(1, 4), rng.randint(1, 40)
        counts = [0] * E
        for _ in range(T * k):
            counts[rng.randrange(E) if rng.random() < 0.7 else 0] += 1
        assert sum(-(-c // 128) * 128 for c in counts) <= dg.dg_get_layout_rows(T, k, E)


# ------------------------------------------------------------------ binding

def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(*shape)


T, E, K_, R, H, F = 5, 6, 2, 640, 256, 128
BINDING = {
    "dg_route_topk": dict(topk_idx=i32(T, K_), topk_w=f32(T, K_), logits=bf16(T, E), bias=f32(E)),
    "dg_route_topk_bwd": dict(dlogits=bf16(T, E), dw=f32(T, K_), logits=bf16(T, E), topk_idx=i32(T, K_)),
    "dg_route_layout": dict(row_of=i32(T, K_), m_indices=i32(R), slot_of=i32(R), group_offsets=i32(E + 1),
                            counts=i32(E), topk_idx=i32(T, K_)),
    "dg_dispatch_fp8_1x128": dict(Q=u8(R, H), sa=f32(2 * R), sa_stride=R, X=bf16(T, H), row_of=i32(T, K_)),
    "dg_combine": dict(out=bf16(T, H), Y=bf16(R, H), row_of=i32(T, K_), w=f32(T, K_)),
    "dg_combine_bwd": dict(dw=f32(T, K_), Qr=u8(R, H), sr=f32(2 * R), sr_stride=R, Qc=u8(R, H), sc=f32(R // 128 * H),
                           sc_stride=H, dout=bf16(T, H), Y=bf16(R, H), row_of=i32(T, K_), slot_of=i32(R), w=f32(T, K_)),
    "dg_swiglu_fp8": dict(Q=u8(R, F), sa=f32(R), sa_stride=R, H=bf16(R, 2 * F), C=u8(R, 2 * F), cs=f32(2 * R),
                          cs_stride=R, m_indices=i32(R)),
    "dg_swiglu_fp8_bwd": dict(Qr=u8(R, 2 * F), sr=f32(2 * R), sr_stride=R, Qc=u8(R, 2 * F), sc=f32(R // 128 * 2 * F),
                              sc_stride=2 * F, Qa=u8(R, F), sb=f32(R // 128), dA=bf16(R, F), C=u8(R, 2 * F),
                              cs=f32(2 * R), cs_stride=R, m_indices=i32(R)),
    "dg_fp8_1x128_to_128x128": dict(Qb=u8(R, H), sb=f32(2 * R // 128), Q=u8(R, H), sa=f32(2 * R), sa_stride=R,
                                    m_indices=i32(R)),
}


def refused(name, kwargs, match):
    with pytest.raises(dg.DGError) as ei:
        getattr(dg, name)(**kwargs)
    assert ei.value.status == INV and match in str(ei.value), str(ei.value)


@pytest.mark.parametrize("name", BINDING)
def test_valid_tensors_stop_only_at_the_device_check(name):
    refused(name, BINDING[name], "is not on a CUDA device")


TENSORS = [(n, a) for n, kw in BINDING.items() for a, v in kw.items() if torch.is_tensor(v)]


@pytest.mark.parametrize("name,arg", TENSORS)
def test_binding_refuses_short_strided_and_mistyped_tensors(name, arg):
    kw = BINDING[name]
    t = kw[arg]
    other = torch.float64 if t.dtype != torch.float64 else torch.float32
    refused(name, {**kw, arg: t.to(other)}, "")
    if t.dtype == torch.bfloat16:
        refused(name, {**kw, arg: t.half()}, "float16")
    if t.dtype == torch.int32:
        refused(name, {**kw, arg: t.float()}, "")
    short = t[:-1] if t.dim() == 1 else t[:, :-1].contiguous()
    refused(name, {**kw, arg: short}, "")
    if t.dim() == 2:
        wide = torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]
        refused(name, {**kw, arg: wide}, "contiguous")


@pytest.mark.parametrize("name,arg", [(n, a) for n, a in TENSORS if a in ("logits", "topk_idx", "X", "row_of", "dout", "Y", "dA", "Q")
                                      and BINDING[n][a].dim() == 2 and (n, a) not in (("dg_dispatch_fp8_1x128", "Q"), ("dg_swiglu_fp8", "Q"))
                                      and not (n == "dg_combine" and a == "Y")
                                      and not (n == "dg_route_layout" and a == "row_of")])
def test_tensors_whose_sizes_count_have_rank_two(name, arg):
    kw = BINDING[name]
    refused(name, {**kw, arg: kw[arg].reshape(-1)}, "rank 2")
    refused(name, {**kw, arg: None}, "rank 2")


def test_masked_scale_extents():
    # E groups of 8 rows, two K blocks each, stride 8: E * 2 * 8 scales.
    kw = dict(Q=u8(E, 8, H), sa=f32(E * 2 * 8), sa_stride=8, X=bf16(T, H), row_of=i32(T, K_), group_rows=8)
    refused("dg_dispatch_fp8_1x128", kw, "is not on a CUDA device")
    refused("dg_dispatch_fp8_1x128", {**kw, "sa": f32(E * 2 * 8 - 1)}, "sa holds")
    kw = dict(Q=u8(E, 8, F), sa=f32(E * 8), sa_stride=8, H=bf16(E, 8, 2 * F), group_rows=8)
    refused("dg_swiglu_fp8", kw, "is not on a CUDA device")
    refused("dg_swiglu_fp8", {**kw, "sa": f32(E * 8 - 1)}, "sa holds")
