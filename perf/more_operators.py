"""The operators that join a block's GEMMs and routing to the rest of a transformer, as cases to time and compare.

A case names one operator (``op``) and its sizes.  ``run`` computes it in plain torch operations, or, with
``own`` set, by the calls a user makes of this package.  The sizes are those of the package's own workloads
(hidden 7168, expert width 2048, the sweep's 4096, 2112 and 1536 columns, 64 and 4096 tokens, 8192-row groups)
and generic routings (256 experts with 8 per token; 60 with 4).

  gemm      e4m3 operands with their scales -> activation(A B^T + bias) + residual, as bf16, as the next GEMM's
            e4m3 operand or both, and what its gradient needs
  act_bwd   gradient of that result -> gradient of A B^T in both casts the backward GEMMs read, and of the bias
  norm      a block's output, normalised, gated and scaled, added to the residual stream, and the stream's own
            norm for the next block, as bf16 or as its e4m3 operand
  norm_bwd  gradients of the stream and of its norm -> of the stream before, the block's output, gate and weights
  balance   a router's logits and choices -> per-expert counts, balance loss and the loss's gradient
"""
import math

import torch

own = False

FP8_MAX = 448.0
HIDDEN, WIDTH = 7168, 2048
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases


def listed():
    """Twelve cases: single tokens and decoding steps, training steps, and odd sizes."""
    return [
        # one token through a projection in serving: the latency of one small call
        dict(name="gemm token", op="gemm", M=1, N=2112, K=HIDDEN, act="silu", bias=True, residual=False, out="D"),
        # a dense block's first product in training: pre-activation kept, result cast for the second product
        dict(name="gemm up train", op="gemm", M=4096, N=4096, K=HIDDEN, act="gelu_tanh", bias=True, residual=False,
             out="QZ"),
        # ... and its second product, added to the residual stream
        dict(name="gemm down train", op="gemm", M=4096, N=HIDDEN, K=WIDTH, act="none", bias=True, residual=True,
             out="D"),
        # a prompt of odd length through a product with everything on
        dict(name="gemm odd", op="gemm", M=1001, N=2112, K=1536, act="gelu", bias=True, residual=True, out="DZ"),
        # the first product's activation and bias in the backward pass
        dict(name="act bwd train", op="act_bwd", M=8192, N=4096, act="gelu_tanh", bias=True),
        # ... for a ragged number of tokens
        dict(name="act bwd odd", op="act_bwd", M=1001, N=WIDTH, act="gelu", bias=True),
        # between two blocks of a decoding step of 64 sequences, the stream in bf16
        dict(name="norm decode", op="norm", T=64, N=HIDDEN, dtype="bf16", post_norm=True, gate=False, out="HQ"),
        # ... of a training step, the stream in fp32, a gate per token
        dict(name="norm train", op="norm", T=8192, N=HIDDEN, dtype="fp32", post_norm=True, gate=True, out="H"),
        # its backward pass
        dict(name="norm bwd train", op="norm_bwd", T=8192, N=HIDDEN, dtype="fp32", post_norm=True, gate=True),
        # a ragged number of tokens of a narrower stream, no norm behind the block
        dict(name="norm bwd odd", op="norm_bwd", T=1001, N=2120, dtype="bf16", post_norm=False, gate=True),
        # a router's training step: loss, counts and gradient over one batch
        dict(name="balance train", op="balance", T=16384, E=256, k=8, S=1, pad=0, score="softmax", dtype="fp32"),
        # packed sequences of uneven length with padding behind them
        dict(name="balance packed", op="balance", T=4097, E=60, k=4, S=37, pad=65, score="sigmoid", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "act_bwd", "norm", "norm_bwd", "balance"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "gemm":
        out = rng.choice(["D", "DZ", "Q", "QZ", "DQ"])
        M = _log(rng, 1, 4096)
        K = 128 * _log(rng, 1, 56)
        most = min(HIDDEN, 4096 * 4096 * HIDDEN // (M * K))
        N = 128 * rng.randint(1, most // 128) if "Q" in out else 8 * rng.randint(1, most // 8)
        return dict(op=op, M=M, N=N, K=K, act=act, bias=rng.random() < 0.7, residual=rng.random() < 0.5, out=out)
    if op == "act_bwd":
        return dict(op=op, M=_log(rng, 1, 8192), N=128 * rng.randint(1, 32), act=act, bias=rng.random() < 0.7)
    if op in ("norm", "norm_bwd"):
        out = rng.choice(["H", "Q", "HQ"])
        wide = op == "norm" and "Q" in out
        case = dict(op=op, T=_log(rng, 1, 8192), N=128 * rng.randint(1, 56) if wide else 8 * rng.randint(1, 896),
                    dtype=rng.choice(["bf16", "fp32"]), post_norm=rng.random() < 0.6, gate=rng.random() < 0.5)
        if op == "norm":
            case["out"] = out
        return case
    E = rng.randint(4, 512)
    T = _log(rng, 1, min(32768, 16384 * 256 // E))
    pad = rng.choice([0, 0, rng.randint(0, T // 2)])
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=rng.choice([1, _log(rng, 1, 64)]), pad=pad,
                score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["bf16", "fp32"]))


def _blocks(n):
    return (n + 127) // 128


def work(case):
    c = case
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        moved = M * K + N * K + 4 * (M * K // 128 + _blocks(N) * K // 128)
        for o in c["out"]:
            moved += M * N + 4 * M * N // 128 if o == "Q" else 2 * M * N
        moved += (2 * M * N if c["residual"] else 0) + (4 * N if c["bias"] else 0)
        return dict(bytes=moved, flops=2 * M * N * K)
    if c["op"] == "act_bwd":
        M, N = c["M"], c["N"]
        read = (2 if c["act"] == "none" else 4) * M * N
        return dict(bytes=read + 2 * M * N + M * N // 16 + (4 * N if c["bias"] else 0), flops=30 * M * N)
    if c["op"] in ("norm", "norm_bwd"):
        T, N = c["T"], c["N"]
        e = 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "norm":
            out = (2 if "H" in c["out"] else 0) + (1 if "Q" in c["out"] else 0)
            return dict(bytes=T * N * (2 * e + 2 + out) + 8 * N + 8 * T, flops=12 * T * N)
        return dict(bytes=T * N * (3 * e + 6) + 16 * N + 16 * T, flops=24 * T * N)
    T, E = c["T"], c["E"]
    e = 2 if c["dtype"] == "bf16" else 4
    # logits in once and their gradient out once, although that has to wait for the counts of all tokens
    return dict(bytes=2 * T * E * e + 4 * T * c["k"] + 8 * c["S"] * E, flops=12 * T * E)


# --------------------------------------------------------------------------------------------- inputs


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def _stride(rows):
    """Scales of a K block take whole 16 bytes."""
    return (rows + 3) // 4 * 4


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case=c)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        A, sa = _cast_1x128(randn(M, K))
        held = _zeros(K // 128, _stride(M))
        held[:, :M] = sa
        B, sb = _cast_128x128(randn(N, K) * (1.3 / math.sqrt(K)))
        st.update(A=A, sa=held, B=B, sb=sb, bias=0.2 * randn(N) if c["bias"] else None,
                  residual=randn(M, N).bfloat16() if c["residual"] else None)
        if "D" in c["out"]:
            st["D"] = _zeros(M, N, dtype=torch.bfloat16)
        if "Z" in c["out"]:
            st["Z"] = _zeros(M, N, dtype=torch.bfloat16)
        if "Q" in c["out"]:
            st.update(Q=_codes(M, N), sq=_zeros(N // 128, _stride(M)))
    elif c["op"] == "act_bwd":
        M, N = c["M"], c["N"]
        R = 128 * _blocks(M)
        st.update(dD=(0.01 * randn(M, N)).bfloat16(), Z=None if c["act"] == "none" else (1.3 * randn(M, N)).bfloat16(),
                  Qr=_codes(M, N), sr=_zeros(N // 128, _stride(M)), Qc=_codes(R, N), sc=_zeros(R // 128, N))
        if c["bias"]:
            st["dbias"] = _zeros(N)
    elif c["op"] in ("norm", "norm_bwd"):
        T, N = c["T"], c["N"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st.update(w_pre=1 + 0.1 * randn(N), w_post=0.5 + 0.1 * randn(N),
                  gate=torch.sigmoid(randn(T)) if c["gate"] else None, Y=(0.7 * randn(T, N)).bfloat16())
        # the stream grows over a model's blocks, and a few of its columns grow more
        loud = torch.where(torch.rand(N, generator=g, device="cuda") < 0.01, 10.0, 1.0)
        stream = (2.0 * loud * randn(T, N)).to(dt)
        if c["op"] == "norm":
            st.update(X=stream, U=_zeros(T, N, dtype=dt), rstd=_zeros(T, 2))
            if "H" in c["out"]:
                st["H"] = _zeros(T, N, dtype=torch.bfloat16)
            if "Q" in c["out"]:
                st.update(Q=_codes(T, N), sq=_zeros(N // 128, _stride(T)))
        else:
            st.update(U=stream, dU=(0.01 * randn(T, N)).to(dt), dH=(0.01 * randn(T, N)).bfloat16(),
                      rstd=torch.stack([_rstd(st["Y"].float()) if c["post_norm"] else torch.ones(T, device="cuda"),
                                        _rstd(stream.float())], dim=1),
                      dX=_zeros(T, N, dtype=dt), dY=_zeros(T, N, dtype=torch.bfloat16),
                      dgate=_zeros(T) if c["gate"] else None, dw_post=_zeros(N), dw_pre=_zeros(N))
    else:
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["logits"] = (1.5 * randn(T, E) + 0.5 * randn(E)).to(dt)
        st["idx"] = st["logits"].float().argsort(dim=1, descending=True)[:, :k].int().contiguous()
        n = T - c["pad"]
        cuts = torch.sort(torch.randint(0, n + 1, (S - 1,), generator=g, device="cuda")).values
        ends = torch.tensor([0, n], device="cuda")
        st["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).int() if S > 1 or c["pad"] else None
        st.update(loss=_zeros(1), counts=_zeros(S, E, dtype=torch.int32), probs=_zeros(S, E),
                  dlogits=_zeros(T, E, dtype=dt))
    if own:
        _workspace(st)
    return st


def _workspace(st):
    """The call's workspace, which a program keeps from pass to pass."""
    import moe_grouped_gemm_weight_b200 as dg
    c = st["case"]
    if "ws" not in st and c["op"] == "norm_bwd":
        st["ws"] = _zeros(dg.dg_get_norm_workspace(c["T"], c["N"]))
    if "ws" not in st and c["op"] == "balance":
        st["ws"] = _zeros(dg.dg_get_balance_workspace(c["T"], c["E"], c["S"]))
    if "ws" not in st and st.get("dbias") is not None:
        st["ws"] = _zeros(dg.dg_get_bias_workspace(c["M"], c["N"]))
    return st.get("ws")


# -------------------------------------------------------------------------------------- plain forms

COEF = 0.01  # of the balance loss
SCALE = 0.8  # of a block's output on its way into the stream


def _quantised(x, amax):
    """Codes and scale of x for the largest magnitude amax of its tile."""
    amax = amax.clamp_min(1e-4)
    q = (x * (FP8_MAX / amax)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q, amax / FP8_MAX


def _cast_1x128(x):
    """A scale for each 128 columns of each row; scales [columns/128, rows]."""
    R, K = x.shape
    b = x.view(R, K // 128, 128)
    q, s = _quantised(b, b.abs().amax(dim=2, keepdim=True))
    return q.view(R, K), s[:, :, 0].t().contiguous()


def _cast_128x1(x):
    """A scale for each 128 rows of each column; scales [rows/128, columns]."""
    R, K = x.shape
    b = x.view(R // 128, 128, K)
    q, s = _quantised(b, b.abs().amax(dim=1, keepdim=True))
    return q.view(R, K), s[:, 0].contiguous()


def _cast_128x128(x):
    """A scale for each block of a weight matrix, its last rows' block perhaps short; scales [rows/128, columns/128]."""
    R, K = x.shape
    b = torch.nn.functional.pad(x, (0, 0, 0, -R % 128)).view(-1, 128, K // 128, 128)
    q, s = _quantised(b, b.abs().amax(dim=(1, 3), keepdim=True))
    return q.view(-1, K)[:R], s[:, 0, :, 0].contiguous()


def _padded(s, rows):
    """Scales with the gap behind the rows that the layout keeps."""
    return torch.nn.functional.pad(s, (0, _stride(rows) - rows))


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(dim=1) + EPS)


def _plain_gemm(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    a = st["A"].float() * st["sa"][:, :M].t().repeat_interleave(128, dim=1)
    b = st["B"].float() * st["sb"].repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)
    z = a @ b.t()
    if st["bias"] is not None:
        z = z + st["bias"]
    v = _act(z, c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    out = {}
    if "D" in c["out"]:
        out["D"] = v.bfloat16()
    if "Z" in c["out"]:
        out["Z"] = z.bfloat16()
    if "Q" in c["out"]:
        q, s = _cast_1x128(v)
        out.update(Q=q, sq=_padded(s, M))
    return out


def _plain_act_bwd(st):
    c = st["case"]
    M = c["M"]
    d = st["dD"].float()
    if c["act"] != "none":
        d = d * _act_slope(st["Z"].float(), c["act"])
    q, s = _cast_1x128(d)
    Qc, sc = _cast_128x1(torch.nn.functional.pad(d, (0, 0, 0, -M % 128)))
    out = dict(Qr=q, sr=_padded(s, M), Qc=Qc, sc=sc)
    if c["bias"]:
        out["dbias"] = d.sum(dim=0)
    return out


def _plain_norm(st):
    c = st["case"]
    y = st["Y"].float()
    ry = _rstd(y) if c["post_norm"] else torch.ones(c["T"], device=y.device)
    z = y * ry[:, None] * st["w_post"] * SCALE
    if st["gate"] is not None:
        z = z * st["gate"][:, None]
    u = st["X"].float() + z
    ru = _rstd(u)
    h = u * ru[:, None] * st["w_pre"]
    out = dict(U=u.to(st["X"].dtype), rstd=torch.stack([ry, ru], dim=1))
    if "H" in c["out"]:
        out["H"] = h.bfloat16()
    if "Q" in c["out"]:
        q, s = _cast_1x128(h)
        out.update(Q=q, sq=_padded(s, c["T"]))
    return out


def _plain_norm_bwd(st):
    c = st["case"]
    ry, ru = st["rstd"][:, :1], st["rstd"][:, 1:]
    u, y, dh = st["U"].float() * ru, st["Y"].float() * ry, st["dH"].float()
    g = dh * st["w_pre"]
    du = st["dU"].float() + ru * (g - u * (u * g).mean(dim=1, keepdim=True))
    out = dict(dX=du.to(st["U"].dtype), dw_pre=(dh * u).sum(dim=0))
    d = SCALE * du
    if st["gate"] is not None:
        out["dgate"] = (d * y * st["w_post"]).sum(dim=1)
        d = d * st["gate"][:, None]
    out["dw_post"] = (d * y).sum(dim=0)
    d = d * st["w_post"]
    if c["post_norm"]:
        d = ry * (d - y * (y * d).mean(dim=1, keepdim=True))
    out["dY"] = d.bfloat16()
    return out


def _plain_balance(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l, idx = st["logits"].float(), st["idx"].long()
    dev = l.device
    offsets = torch.tensor([0, T], device=dev) if st["offsets"] is None else st["offsets"].long()
    t = torch.arange(T, device=dev)
    # the sequence of each token; S: of none
    seq = (t[:, None] >= offsets[None, 1:]).sum(dim=1)
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        slope = torch.ones_like(e)
    else:
        e = 1 / (1 + torch.exp(-l))
        slope = 1 / (1 + torch.exp(l))
    p = e / e.sum(dim=1, keepdim=True)
    key = (seq[:, None] * E + idx).reshape(-1)
    counts = _zeros((S + 1) * E, dtype=torch.int64).index_add_(0, key, torch.ones_like(key)).view(S + 1, E)
    # 64 bits: sums over all tokens, and differences of loads that are nearly alike
    total = torch.zeros(S + 1, E, dtype=torch.float64, device=dev).index_add_(0, seq, p.double())[:S]
    length = (offsets[1:] - offsets[:-1]).double()[:, None]
    n = offsets[S] - offsets[0]
    probs = torch.where(length > 0, total / length.clamp_min(1), torch.zeros_like(total))
    f = counts[:S].double() * E / (k * length.clamp_min(1))
    loss = COEF * (length / n.clamp_min(1) * f * probs).sum()
    ft = torch.cat([f, torch.zeros(1, E, dtype=torch.float64, device=dev)])[seq]
    d = p * slope * (ft - (ft * p).sum(dim=1, keepdim=True)) * (COEF / n.clamp_min(1))
    d = torch.where((seq < S)[:, None], d, torch.zeros_like(d))
    return dict(loss=loss.float().view(1), counts=counts[:S].int(), probs=probs.float(),
                dlogits=d.to(st["logits"].dtype))


# ------------------------------------------------------------------------------- the package's calls


def _own(st):
    import moe_grouped_gemm_weight_b200 as dg
    c = st["case"]
    op = c["op"]
    if op in ("gemm", "act_bwd"):
        act = dict(none=dg.DG_ACT_NONE, relu=dg.DG_ACT_RELU, gelu=dg.DG_ACT_GELU, gelu_tanh=dg.DG_ACT_GELU_TANH,
                   silu=dg.DG_ACT_SILU)[c["act"]]
        m = _stride(c["M"])
        if op == "gemm":
            dg.dg_fp8_gemm_nt_epilogue(st.get("D"), st["A"], st["sa"], m, st["B"], st["sb"], bias=st["bias"], act=act,
                                       residual=st["residual"], Z=st.get("Z"), Q=st.get("Q"), sq=st.get("sq"),
                                       sq_stride=m)
            return {n: st[n] for n in ("D", "Z", "Q", "sq") if n in st}
        dg.dg_epilogue_bwd(st["Qr"], st["sr"], m, st["Qc"], st["sc"], c["N"], st["dD"], Z=st["Z"], act=act,
                           dbias=st.get("dbias"), ws=_workspace(st))
        return {n: st[n] for n in ("Qr", "sr", "Qc", "sc", "dbias") if n in st}
    if op == "norm":
        dg.dg_norm_residual(st["U"], st["X"], st["Y"], H=st.get("H"), Q=st.get("Q"), sq=st.get("sq"),
                            sq_stride=_stride(c["T"]), rstd=st["rstd"], w_post=st["w_post"], gate=st["gate"],
                            w_pre=st["w_pre"], post_norm=c["post_norm"], scale=SCALE, eps=EPS)
        return {n: st[n] for n in ("U", "rstd", "H", "Q", "sq") if n in st}
    if op == "norm_bwd":
        dg.dg_norm_residual_bwd(st["dX"], st["dU"], st["dH"], st["U"], st["Y"], st["rstd"], dY=st["dY"],
                                dgate=st["dgate"], dw_post=st["dw_post"], dw_pre=st["dw_pre"], ws=_workspace(st),
                                w_post=st["w_post"], gate=st["gate"], w_pre=st["w_pre"], post_norm=c["post_norm"],
                                scale=SCALE)
        return {n: st[n] for n in ("dX", "dw_pre", "dgate", "dw_post", "dY") if st[n] is not None}
    score = dg.DG_SCORE_SOFTMAX if c["score"] == "softmax" else dg.DG_SCORE_SIGMOID
    dg.dg_balance_loss(st["loss"], st["counts"], st["probs"], st["logits"], st["idx"], _workspace(st),
                       seq_offsets=st["offsets"], score=score, coef=COEF)
    dg.dg_balance_loss_bwd(st["dlogits"], st["logits"], st["counts"], c["k"], seq_offsets=st["offsets"], score=score,
                           coef=COEF)
    return {n: st[n] for n in ("loss", "counts", "probs", "dlogits")}


_PLAIN = dict(gemm=_plain_gemm, act_bwd=_plain_act_bwd, norm=_plain_norm, norm_bwd=_plain_norm_bwd,
              balance=_plain_balance)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- in 64 bits


def _exact_cast(x, dims):
    """Codes (as numbers) and scales of x, tiles spanning `dims`, by the nearest of all e4m3 numbers."""
    amax = x.abs().amax(dim=dims, keepdim=True).clamp_min(1e-4)
    y = x * (448 / amax)
    # e4m3: 3 bits behind the leading one, exponents from -6
    exponent = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = torch.exp2(exponent - 3)
    return torch.round(y / step) * step, amax / 448


def _exact_rows(x):
    """The cast per 1x128, scales in their layout of whole 16 bytes."""
    R, K = x.shape
    q, s = _exact_cast(x.reshape(R, K // 128, 128), (2,))
    full = torch.zeros(K // 128, R + -R % 4, dtype=torch.float64, device="cuda")
    full[:, :R] = s.reshape(R, K // 128).t()
    return q.reshape(R, K), full


def _exact_act(x, act):
    f = torch.nn.functional
    if act == "gelu_tanh":
        return x * torch.sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3))
    if act == "gelu":
        return x * torch.exp(torch.special.log_ndtr(x))
    return dict(none=lambda v: v, relu=f.relu, silu=f.silu)[act](x)


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        z = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        rows = torch.arange(N, device="cuda") // 128
        # one block of K after the other, as the scales are given
        for i in range(K // 128):
            part = st["A"][:, 128 * i:128 * i + 128].double() @ st["B"][:, 128 * i:128 * i + 128].double().t()
            z += part * st["sa"][i, :M].double()[:, None] * st["sb"][:, i].double()[rows][None, :]
        if c["bias"]:
            z += st["bias"].double()
        v = _exact_act(z, c["act"])
        if c["residual"]:
            v = v + st["residual"].double()
        out = {}
        if "D" in c["out"]:
            out["D"] = v
        if "Z" in c["out"]:
            out["Z"] = z
        if "Q" in c["out"]:
            out["Q"], out["sq"] = _exact_rows(v)
        return out
    if op == "act_bwd":
        M, N = c["M"], c["N"]
        if c["act"] == "none":
            d = st["dD"].double()
        else:
            x = st["Z"].double().requires_grad_()
            d, = torch.autograd.grad(_exact_act(x, c["act"]), x, st["dD"].double())
        out = {}
        out["Qr"], out["sr"] = _exact_rows(d)
        R = 128 * math.ceil(M / 128)
        tall = torch.zeros(R, N, dtype=torch.float64, device="cuda")
        tall[:M] = d
        q, s = _exact_cast(tall.reshape(R // 128, 128, N), (1,))
        out.update(Qc=q.reshape(R, N), sc=s[:, 0])
        if c["bias"]:
            out["dbias"] = d.sum(dim=0)
        return out
    if op == "norm":
        x, y = st["X"].double(), st["Y"].double()
        ry = y.square().mean(dim=1).add(EPS).rsqrt() if c["post_norm"] else torch.ones_like(y[:, 0])
        amount = SCALE * ry * (st["gate"].double() if c["gate"] else 1.0)
        u = torch.addcmul(x, amount[:, None], y * st["w_post"].double())
        ru = u.square().mean(dim=1).add(EPS).rsqrt()
        h = u * st["w_pre"].double() * ru[:, None]
        out = dict(U=u, rstd=torch.stack([ry, ru], dim=1))
        if "H" in c["out"]:
            out["H"] = h
        if "Q" in c["out"]:
            out["Q"], out["sq"] = _exact_rows(h)
        return out
    if op == "norm_bwd":
        # by differentiation of the operator, with the statistics that the call is given
        T, N = c["T"], c["N"]
        u, y, ry, ru = st["U"].double(), st["Y"].double(), st["rstd"][:, 0].double(), st["rstd"][:, 1].double()
        wu, wy = st["w_pre"].double(), st["w_post"].double()
        gate = st["gate"].double() if c["gate"] else torch.ones(T, dtype=torch.float64, device="cuda")
        dh = st["dH"].double()
        inner = torch.einsum("tn,tn,n->t", dh, u, wu)
        du = st["dU"].double() + dh * wu * ru[:, None] - u * (ru ** 3 * inner / N)[:, None]
        out = dict(dX=du, dw_pre=torch.einsum("tn,tn,t->n", dh, u, ru))
        if c["gate"]:
            out["dgate"] = SCALE * ry * torch.einsum("tn,tn,n->t", du, y, wy)
        k = SCALE * gate
        out["dw_post"] = torch.einsum("tn,tn,t->n", du, y, k * ry)
        dy = du * wy * (k * ry)[:, None]
        if c["post_norm"]:
            dy = dy - y * (k * ry ** 3 * torch.einsum("tn,tn,n->t", du, y, wy) / N)[:, None]
        out["dY"] = dy
        return out
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    x = st["logits"].double()
    cut = [0, T] if st["offsets"] is None else st["offsets"].tolist()
    n = max(cut[S] - cut[0], 1)
    probs = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    d = torch.zeros_like(x)
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    for s in range(S):
        a, b = cut[s], cut[s + 1]
        if a == b:
            continue
        share = torch.bincount(st["idx"][a:b].long().reshape(-1), minlength=E).double() * E / k / (b - a)
        part = x[a:b]
        if c["score"] == "softmax":
            p = torch.softmax(part, dim=1)
            local = torch.ones_like(p)
        else:
            one = torch.sigmoid(part)
            p = one / one.sum(dim=1, keepdim=True)
            local = torch.sigmoid(-part)
        probs[s] = p.mean(dim=0)
        loss += COEF * (b - a) / n * (share @ probs[s])
        d[a:b] = COEF / n * p * local * (share[None, :] - (p @ share)[:, None])
    return dict(loss=loss, counts=None, probs=probs, dlogits=d)
