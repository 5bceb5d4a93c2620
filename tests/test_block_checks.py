"""Host-side tests of the calls between a block's GEMMs and the rest of a transformer (no GPU needed): the C ABI
refuses bad sizes, strides, alignments and null pointers before any launch, and the Python binding refuses tensors
that the kernels would read or write past, or of another type or shape."""
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
    return [changes.get(n, v) for n, v in good.items()]


EPI = dict(D=FAKE, Z=FAKE * 2, Q=FAKE, sq=FAKE, sq_stride=200, A=FAKE, sa=FAKE, sa_stride=200, B=FAKE, sb=FAKE, bias=FAKE,
           act=2, residual=FAKE, M=200, N=256, K=384, stream=0)
EPI_BWD = dict(Qr=FAKE, sr=FAKE, sr_stride=200, Qc=FAKE, sc=FAKE, sc_stride=256, dbias=FAKE, ws=FAKE, dD=FAKE, Z=FAKE,
               act=2, M=200, N=256, stream=0)
NORM = dict(U=FAKE, H=FAKE, Q=FAKE, sq=FAKE, sq_stride=20, rstd=FAKE, X=FAKE, dtype=0, Y=FAKE, w_post=FAKE, gate=FAKE,
            w_pre=FAKE, T=20, N=256, post_norm=1, scale=1.0, eps=1e-6, stream=0)
NORM_BWD = dict(dX=FAKE, dY=FAKE, dgate=FAKE, dw_post=FAKE, dw_pre=FAKE, ws=FAKE, dU=FAKE, dH=FAKE, U=FAKE, dtype=1,
                Y=FAKE, rstd=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE, T=20, N=256, post_norm=1, scale=1.0, stream=0)
BALANCE = dict(loss=FAKE, counts=FAKE, probs=FAKE, ws=FAKE, logits=FAKE, dtype=0, idx=FAKE, offsets=FAKE, T=20, E=16, k=4,
               S=3, score=0, coef=0.01, stream=0)
BALANCE_BWD = dict(dlogits=FAKE, add=FAKE, dloss=FAKE, logits=FAKE, dtype=1, counts=FAKE, offsets=FAKE, T=20, E=16, k=4,
                   S=3, score=1, coef=0.01, stream=0)
INF, NAN = float("inf"), float("nan")

REFUSALS = [
    ("dg_fp8_gemm_nt_epilogue", EPI, [
        (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=200), UNS), (dict(N=260, Q=0), UNS),
        (dict(N=264), UNS), (dict(act=5), INV), (dict(act=-1), INV), (dict(D=0, Z=0, Q=0), INV), (dict(A=0), INV),
        (dict(sa=0), INV), (dict(B=0), INV), (dict(sb=0), INV), (dict(sq=0), INV), (dict(sq_stride=199), INV),
        (dict(sa_stride=196), INV), (dict(sa_stride=202), INV), (dict(D=FAKE + 8), MIS), (dict(Z=FAKE + 8), MIS),
        (dict(Q=FAKE + 8), MIS), (dict(bias=FAKE + 4), MIS), (dict(residual=FAKE + 2), MIS), (dict(sq=FAKE + 2), MIS),
        (dict(Z=FAKE), INV), (dict(D=0, Z=FAKE), INV), (dict(M=0, sa_stride=0), OK), (dict(M=0, D=0, Q=0), OK)]),
    ("dg_epilogue_bwd", EPI_BWD, [
        (dict(M=-1), INV), (dict(N=0), INV), (dict(N=200), UNS), (dict(N=(1 << 28) + 128, sc_stride=0x7FFFFFFF), UNS),
        (dict(M=0x7FF00080, sr_stride=0x7FF00080), UNS), (dict(act=9), INV), (dict(sr_stride=199), INV),
        (dict(sc_stride=255), INV), (dict(ws=0), INV), (dict(ws=FAKE + 2), MIS), (dict(dbias=FAKE + 1), MIS),
        (dict(Qr=0), INV), (dict(sr=0), INV), (dict(Qc=0), INV), (dict(sc=0), INV), (dict(dD=0), INV), (dict(Z=0), INV),
        (dict(Qr=FAKE + 8), MIS), (dict(Qc=FAKE + 8), MIS), (dict(dD=FAKE + 2), MIS), (dict(Z=FAKE + 2), MIS),
        (dict(sr=FAKE + 1), MIS), (dict(sc=FAKE + 2), MIS), (dict(M=1 << 30, sr_stride=1 << 30, N=1 << 20, sc_stride=1 << 20), UNS),
        (dict(M=0, dbias=0, Qr=0), OK)]),
    ("dg_norm_residual", NORM, [
        (dict(T=-1), INV), (dict(N=0), INV), (dict(N=12), UNS), (dict(N=16392), UNS), (dict(N=264), UNS),
        (dict(T=0x7FF00001, sq_stride=0x7FFFFFFF), UNS), (dict(dtype=2), INV), (dict(scale=INF), INV), (dict(scale=NAN), INV),
        (dict(eps=0.0), INV), (dict(eps=-1e-6), INV), (dict(eps=INF), INV), (dict(eps=NAN), INV),
        (dict(U=0, H=0, Q=0, rstd=0), INV), (dict(sq=0), INV), (dict(sq_stride=19), INV), (dict(X=0, Y=0), INV),
        (dict(U=FAKE + 8), MIS), (dict(H=FAKE + 2), MIS), (dict(Q=FAKE + 8), MIS), (dict(X=FAKE + 4), MIS),
        (dict(Y=FAKE + 2), MIS), (dict(w_post=FAKE + 4), MIS), (dict(w_pre=FAKE + 8), MIS), (dict(rstd=FAKE + 4), MIS),
        (dict(gate=FAKE + 2), MIS), (dict(sq=FAKE + 2), MIS), (dict(T=0, X=0, Y=0), OK)]),
    ("dg_norm_residual_bwd", NORM_BWD, [
        (dict(T=-1), INV), (dict(N=0), INV), (dict(N=12), UNS), (dict(N=16392), UNS), (dict(dtype=-1), INV),
        (dict(scale=NAN), INV), (dict(dX=0, dY=0, dgate=0, dw_post=0, dw_pre=0), INV), (dict(Y=0), INV),
        (dict(Y=0, dY=0, dgate=0), INV), (dict(ws=0), INV), (dict(dU=0, dH=0), INV), (dict(U=0), INV), (dict(rstd=0), INV),
        (dict(dX=FAKE + 8), MIS), (dict(dY=FAKE + 8), MIS), (dict(ws=FAKE + 8), MIS), (dict(dU=FAKE + 4), MIS),
        (dict(dH=FAKE + 2), MIS), (dict(U=FAKE + 4), MIS), (dict(Y=FAKE + 2), MIS), (dict(rstd=FAKE + 4), MIS),
        (dict(w_post=FAKE + 4), MIS), (dict(w_pre=FAKE + 4), MIS), (dict(gate=FAKE + 1), MIS), (dict(dgate=FAKE + 2), MIS),
        (dict(dw_pre=FAKE + 2), MIS), (dict(T=0, dw_post=0, dw_pre=0), OK)]),
    ("dg_balance_loss", BALANCE, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=17), INV), (dict(S=0), INV), (dict(dtype=2), INV),
        (dict(score=2), INV), (dict(coef=INF), INV), (dict(coef=NAN), INV), (dict(offsets=0), INV), (dict(E=1025), UNS),
        (dict(T=1 << 30, k=4), UNS), (dict(S=1 << 28), UNS), (dict(T=1 << 20, E=1024, S=1 << 20), UNS), (dict(loss=0), INV),
        (dict(counts=0), INV), (dict(logits=0), INV), (dict(idx=0), INV), (dict(ws=0), INV), (dict(logits=FAKE + 1), MIS),
        (dict(dtype=1, logits=FAKE + 2), MIS), (dict(idx=FAKE + 2), MIS), (dict(ws=FAKE + 2), MIS), (dict(loss=FAKE + 2), MIS),
        (dict(counts=FAKE + 1), MIS), (dict(probs=FAKE + 2), MIS), (dict(offsets=FAKE + 2), MIS)]),
    ("dg_balance_loss_bwd", BALANCE_BWD, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=17), INV), (dict(S=0), INV), (dict(dtype=2), INV),
        (dict(score=-1), INV), (dict(coef=NAN), INV), (dict(offsets=0), INV), (dict(E=1025), UNS), (dict(dlogits=0), INV),
        (dict(logits=0), INV), (dict(counts=0), INV), (dict(dlogits=FAKE + 2), MIS), (dict(add=FAKE + 2), MIS),
        (dict(logits=FAKE + 2), MIS), (dict(counts=FAKE + 2), MIS), (dict(dloss=FAKE + 2), MIS),
        (dict(offsets=FAKE + 2), MIS), (dict(T=0, logits=0), OK)]),
]


@pytest.mark.parametrize("name,good,change,status", [(n, g, c, s) for n, g, cs in REFUSALS for c, s in cs])
def test_c_abi_refuses_bad_arguments(name, good, change, status):
    L = dg.lib()
    assert set(change) <= set(good)
    assert getattr(L, name)(*swapped(good, **change)) == status
    if status != OK:
        assert L.dg_last_error_message()


def test_workspaces():
    assert dg.dg_get_bias_workspace(0, 256) == 0 and dg.dg_get_bias_workspace(129, 256) == 512
    assert dg.dg_get_norm_workspace(0, 64) == 0 and dg.dg_get_norm_workspace(3, 64) == 2 * 64 * 3
    assert dg.dg_get_norm_workspace(1 << 20, 16384) == dg.dg_get_norm_workspace(1 << 19, 16384) <= 1 << 23
    assert dg.dg_get_balance_workspace(1, 4, 1) == 2 * 4 * 2
    for T in (0, 1, 8, 9, 2368, 2369, 100000):
        # a part for each chunk and for each sequence that starts inside one
        assert dg.dg_get_balance_workspace(T, 4, 5) >= 2 * 4 * 5
        assert dg.dg_get_balance_workspace(T, 4, 5) <= 2 * 4 * (296 + 5)
    for f, bad in ((dg.dg_get_bias_workspace, [(-1, 8), (1, 0), (1 << 31, 8), (1 << 30, 1 << 20)]),
                   (dg.dg_get_norm_workspace, [(-1, 8), (1, 0), (1, 16385), (1 << 32, 8)]),
                   (dg.dg_get_balance_workspace, [(-1, 4, 1), (1, 0, 1), (1, 1025, 1), (1, 4, 0), (1, 1024, 1 << 21)])):
        for b in bad:
            assert f(*b) == -1, (f.__name__, b)


def test_marshalling_refuses_numbers_that_do_not_fit():
    c = dg._marshal()
    for name, good in (("dg_fp8_gemm_nt_epilogue", EPI), ("dg_norm_residual_bwd", NORM_BWD), ("dg_balance_loss", BALANCE),
                       ("dg_norm_residual", NORM), ("dg_epilogue_bwd", EPI_BWD), ("dg_balance_loss_bwd", BALANCE_BWD)):
        call = getattr(c, name)
        size = "M" if "M" in good else "T"
        with pytest.raises(OverflowError):
            call(*swapped(good, **{size: 1 << 31}))
        with pytest.raises(TypeError):
            call(*swapped(good, **{size: 1.5}))
        with pytest.raises(TypeError):
            call(*swapped(good)[:-1])
        for real in ("scale", "eps", "coef"):
            if real in good:
                with pytest.raises(TypeError):
                    call(*swapped(good, **{real: "z"}))


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(*shape)


M, N, K, T, E, KK, S = 200, 256, 384, 20, 6, 2, 3
BINDING = {
    "dg_fp8_gemm_nt_epilogue": dict(D=bf16(M, N), A=u8(M, K), sa=f32(3 * M), sa_stride=M, B=u8(N, K), sb=f32(6), bias=f32(N),
                                    act=1, residual=bf16(M, N), Z=bf16(M, N), Q=u8(M, N), sq=f32(2 * M), sq_stride=M),
    "dg_epilogue_bwd": dict(Qr=u8(M, N), sr=f32(2 * M), sr_stride=M, Qc=u8(256, N), sc=f32(2 * N), sc_stride=N,
                            dD=bf16(M, N), Z=bf16(M, N), act=1, dbias=f32(N), ws=f32(2 * N)),
    "dg_norm_residual": dict(U=bf16(T, N), X=bf16(T, N), Y=bf16(T, N), H=bf16(T, N), Q=u8(T, N), sq=f32(2 * T), sq_stride=T,
                             rstd=f32(T, 2), w_post=f32(N), gate=f32(T), w_pre=f32(N)),
    "dg_norm_residual_bwd": dict(dX=f32(T, N), dU=f32(T, N), dH=bf16(T, N), U=f32(T, N), Y=bf16(T, N), rstd=f32(T, 2),
                                 dY=bf16(T, N), dgate=f32(T), dw_post=f32(N), dw_pre=f32(N), ws=f32(2 * T * N),
                                 w_post=f32(N), gate=f32(T), w_pre=f32(N)),
    "dg_balance_loss": dict(loss=f32(1), counts=i32(S, E), probs=f32(S, E), logits=bf16(T, E), topk_idx=i32(T, KK),
                            ws=f32(2 * E * (3 + S)), seq_offsets=i32(S + 1)),
    "dg_balance_loss_bwd": dict(dlogits=bf16(T, E), logits=bf16(T, E), counts=i32(S, E), k=KK, dloss=f32(1),
                                add=bf16(T, E), seq_offsets=i32(S + 1)),
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
    refused(name, {**kw, arg: t.to(torch.float64)}, "")
    if t.dtype in (torch.bfloat16, torch.float32):
        refused(name, {**kw, arg: t.half()}, "float16")
    if t.dtype == torch.int32:
        refused(name, {**kw, arg: t.long()}, "")
    short = t[:-1] if t.dim() == 1 else t[:, :-1].contiguous()
    refused(name, {**kw, arg: short}, "")
    if t.dim() == 2:
        wide = torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]
        refused(name, {**kw, arg: wide}, "contiguous")


@pytest.mark.parametrize("name,arg", [("dg_fp8_gemm_nt_epilogue", "A"), ("dg_fp8_gemm_nt_epilogue", "B"),
                                      ("dg_epilogue_bwd", "dD"), ("dg_norm_residual", "X"), ("dg_norm_residual_bwd", "U"),
                                      ("dg_balance_loss", "logits"), ("dg_balance_loss", "topk_idx"),
                                      ("dg_balance_loss", "counts"), ("dg_balance_loss_bwd", "logits"),
                                      ("dg_balance_loss_bwd", "counts")])
def test_tensors_whose_sizes_count_have_rank_two(name, arg):
    kw = BINDING[name]
    refused(name, {**kw, arg: kw[arg].reshape(-1)}, "rank 2")
    refused(name, {**kw, arg: "x"}, "rank 2")
    if arg != "X":  # without a stream the sizes are Y's
        refused(name, {**kw, arg: None}, "rank 2")


def test_mixed_types_and_sizes_are_refused():
    kw = BINDING["dg_norm_residual"]
    refused("dg_norm_residual", {**kw, "U": f32(T, N)}, "float32")
    refused("dg_norm_residual", {**kw, "X": None, "Y": None}, "rank 2")
    refused("dg_norm_residual", {**kw, "X": u8(T, N)}, "stream is")
    kw = BINDING["dg_norm_residual_bwd"]
    refused("dg_norm_residual_bwd", {**kw, "dU": bf16(T, N)}, "bfloat16")
    kw = BINDING["dg_balance_loss_bwd"]
    refused("dg_balance_loss_bwd", {**kw, "dlogits": f32(T, E)}, "float32")
    refused("dg_balance_loss_bwd", {**kw, "counts": i32(S, E + 1)}, "E of counts")
    kw = BINDING["dg_balance_loss"]
    refused("dg_balance_loss", {**kw, "topk_idx": i32(T + 1, KK)}, "token count")
    kw = BINDING["dg_fp8_gemm_nt_epilogue"]
    refused("dg_fp8_gemm_nt_epilogue", {**kw, "B": u8(N, K + 128)}, "K of B")
    refused("dg_fp8_gemm_nt_epilogue", {**kw, "sq": None}, "is not on a CUDA device")
