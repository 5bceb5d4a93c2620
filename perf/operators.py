"""The operators around the grouped FP8 GEMMs of a mixture-of-experts layer, as cases to time and compare.

A case names one operator (``op``) and its sizes.  ``run`` computes it in plain torch operations, or, with
``own`` set, by the calls a user makes of this package.  The sizes are those of the package's own workloads
(hidden 7168, expert width 2048, 8192-row groups, 64 and 4096 tokens) and generic routings (256 experts in 8
groups with 8 per token; 60 experts with 4 per token).

  route       logits -> the k experts of each token and their weights
  route_bwd   gradient of the weights -> gradient of the logits
  dispatch    chosen experts -> the grouped layout, and the tokens cast to e4m3 into its rows
  combine     the experts' rows -> weighted sum per token (without weights: the backward of dispatch)
  combine_bwd gradient of that sum -> the rows' gradient in both casts a backward GEMM reads, and of the weights
  ckpt        gate and up rows -> the product's e4m3 operand, and the e4m3 checkpoint of gate and up
  ckpt_bwd    checkpoint and gradient -> gradient of gate and up in both casts, and the product again, per block
  recast      an e4m3 checkpoint with a scale for each 1x128 -> one with a scale for each 128x128
"""
import math

import torch

own = False

FP8_MAX = 448.0
HIDDEN, WIDTH = 7168, 2048


# ---------------------------------------------------------------------------------------------- cases


def listed():
    """Twelve cases: decoding with a handful of tokens, a training step's worth of tokens, and odd sizes."""
    return [
        # routing one decoding step of 64 sequences: the latency of one small call
        dict(name="route decode", op="route", T=64, E=256, k=8, groups=8, keep=4, gtop=2, score="sigmoid",
             bias=True, renorm=True, dtype="bf16"),
        # routing a training step
        dict(name="route train", op="route", T=16384, E=256, k=8, groups=8, keep=4, gtop=2, score="sigmoid",
             bias=True, renorm=True, dtype="fp32"),
        # a router with an odd number of experts and tokens and no groups
        dict(name="route odd", op="route", T=4097, E=60, k=4, groups=1, keep=1, gtop=1, score="softmax",
             bias=False, renorm=False, dtype="bf16"),
        # the router's gradient in that training step
        dict(name="route bwd", op="route_bwd", T=16384, E=256, k=8, score="softmax", renorm=True, dtype="fp32"),
        # one decoding step's tokens into the masked layout of the experts that one GPU holds
        dict(name="dispatch decode", op="dispatch", T=64, E=32, k=8, K=HIDDEN, max_rows=64, drop=False),
        # a training step's tokens into the contiguous layout: 32768 rows
        dict(name="dispatch train", op="dispatch", T=4096, E=64, k=8, K=HIDDEN, max_rows=0, drop=False),
        # the sum of a decoding step's expert rows
        dict(name="combine decode", op="combine", T=64, E=32, k=8, N=HIDDEN, drop=False, weighted=True),
        # ... and of a training step's, some slots dropped
        dict(name="combine train", op="combine", T=4096, E=64, k=8, N=HIDDEN, drop=True, weighted=True),
        # its backward pass
        dict(name="combine bwd", op="combine_bwd", T=4096, E=64, k=8, N=HIDDEN, drop=False),
        # gate and up of a training step's rows: the next GEMM's operand, and the checkpoint
        dict(name="ckpt train", op="ckpt", T=4096, E=64, k=8, F=WIDTH),
        # the checkpoint's use in the backward pass
        dict(name="ckpt bwd", op="ckpt_bwd", T=4096, E=64, k=8, F=WIDTH),
        # the dispatched input, as the weight gradient's operand; a ragged number of tokens
        dict(name="recast odd", op="recast", T=1001, E=16, k=6, K=HIDDEN),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine_bwd", "ckpt", "ckpt_bwd", "recast"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 512 // groups)
        T = _log(rng, 1, min(32768, 16384 * 256 // E))
        case = dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E // groups)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]))
        if op == "route":
            case.update(groups=groups, keep=rng.randint(1, groups), gtop=rng.choice([1, 2]), bias=rng.random() < 0.5)
        return case
    E, k = rng.randint(2, 128), rng.randint(1, 8)
    k = min(k, E)
    T = _log(rng, 1, 4096)
    if op in ("dispatch", "recast"):
        case = dict(op=op, T=T, E=E, k=k, K=128 * rng.randint(1, 56))
        if op == "dispatch":
            masked = T <= 256 and rng.random() < 0.7
            case.update(max_rows=T if masked else 0, drop=rng.random() < 0.3)
        return case
    if op == "combine":
        return dict(op=op, T=T, E=E, k=k, N=8 * rng.randint(8, 896), drop=rng.random() < 0.3,
                    weighted=rng.random() < 0.7)
    if op == "combine_bwd":
        return dict(op=op, T=T, E=E, k=k, N=128 * rng.randint(1, 56), drop=rng.random() < 0.3)
    return dict(op=op, T=T, E=E, k=k, F=128 * rng.randint(1, 16))


def _capacity(T, k, E):
    """Rows that any choice of T*k experts fits in, with segments of whole 128 rows."""
    n = min(E, T * k)
    return (T * k + 127 * n) // 128 * 128


def work(case):
    c = case
    T, E, k = c["T"], c["E"], c["k"]
    S = T * k
    if c["op"] in ("route", "route_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "route":
            return dict(bytes=T * E * e + 8 * S + (4 * E if c["bias"] else 0), flops=8 * T * E)
        read = T * E * e if c["score"] == "softmax" else S * e
        return dict(bytes=read + T * E * e + 8 * S, flops=8 * T * E)
    if c["op"] == "dispatch":
        rows = E * c["max_rows"] or _capacity(T, k, E)
        return dict(bytes=2 * T * c["K"] + S * (c["K"] + c["K"] // 32) + 8 * S + 8 * rows + 8 * E, flops=3 * T * c["K"])
    if c["op"] == "combine":
        return dict(bytes=2 * S * c["N"] + 2 * T * c["N"] + 8 * S, flops=2 * S * c["N"])
    if c["op"] == "combine_bwd":
        return dict(bytes=2 * S * c["N"] + 2 * T * c["N"] + 2 * S * c["N"] + S * c["N"] // 16 + 16 * S,
                    flops=8 * S * c["N"])
    if c["op"] == "ckpt":
        return dict(bytes=S * (7 * c["F"] + 3 * c["F"] // 32) + 4 * S, flops=16 * S * c["F"])
    if c["op"] == "ckpt_bwd":
        return dict(bytes=S * (9 * c["F"] + 6 * c["F"] // 32) + 4 * S, flops=30 * S * c["F"])
    return dict(bytes=S * (2 * c["K"] + c["K"] // 32) + 4 * S, flops=3 * S * c["K"])


# --------------------------------------------------------------------------------------------- inputs


def _chosen(T, E, k, drop, g):
    """k different experts for each token, some experts more popular than others; dropped slots are -1."""
    taste = torch.randn(E, generator=g, device="cuda")
    idx = (torch.randn(T, E, generator=g, device="cuda") + 0.5 * taste).argsort(dim=1, descending=True)[:, :k].int()
    if drop:
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, torch.full_like(idx, -1), idx)
    return idx.contiguous()


def _layout(idx, E, max_rows):
    """Rows of the slots, expert and slot of each row, segment starts and counts, in torch operations."""
    T, k = idx.shape
    S = T * k
    rows = E * max_rows or _capacity(T, k, E)
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).index_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, 0) - count  # of each expert in `order`
    rank = torch.empty_like(key)
    rank[order] = torch.arange(S, device=idx.device) - first[key[order]]
    count = count[:E]
    if max_rows:
        start = torch.arange(E + 1, device=idx.device) * max_rows
        count = count.clamp(max=max_rows)
    else:
        padded = (count + 127) // 128 * 128
        start = torch.cat([torch.zeros(1, dtype=torch.int64, device=idx.device), torch.cumsum(padded, 0)])
    row = start[key] + rank
    there = key < E
    if max_rows:
        there = there & (rank < max_rows)
    row = torch.where(there, row, torch.full_like(row, -1))
    to = torch.where(there, row, torch.full_like(row, rows))
    m_indices = torch.full((rows + 1,), -1, dtype=torch.int64, device=idx.device)
    slot_of = m_indices.clone()
    m_indices[to] = key
    slot_of[to] = torch.arange(S, device=idx.device)
    return dict(row_of=row.int().view(T, k), m_indices=m_indices[:rows].int(), slot_of=slot_of[:rows].int(),
                offsets=start.int(), counts=count.int(), rows=rows)


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    T, E, k = c["T"], c["E"], c["k"]
    st = dict(case=c)
    if c["op"] in ("route", "route_bwd"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["logits"] = (1.5 * randn(T, E)).to(dt)
        if c["op"] == "route":
            st["bias"] = 0.05 * randn(E) if c["bias"] else None
            st["idx"] = _zeros(T, k, dtype=torch.int32)
            st["w"] = _zeros(T, k)
        else:
            st["idx"] = _chosen(T, E, k, False, g)
            st["dw"] = randn(T, k)
            st["dlogits"] = _zeros(T, E, dtype=dt)
        return st
    idx = _chosen(T, E, k, c.get("drop", False), g)
    lay = _layout(idx, E, c.get("max_rows", 0))
    R = lay["rows"]
    if c["op"] == "dispatch":
        K, M = c["K"], c["max_rows"]
        stride = (M + 3) // 4 * 4 or R
        st.update(idx=idx, X=randn(T, K).bfloat16(), row_of=_zeros(T, k, dtype=torch.int32),
                  m_indices=_zeros(R, dtype=torch.int32), slot_of=_zeros(R, dtype=torch.int32),
                  offsets=_zeros(E + 1, dtype=torch.int32), counts=_zeros(E, dtype=torch.int32), Q=_codes(R, K),
                  sa=_zeros(E if M else 1, K // 128, stride), stride=stride)
        return st
    st.update(row_of=lay["row_of"], slot_of=lay["slot_of"], m_indices=lay["m_indices"])
    held = lay["m_indices"][:, None] >= 0
    w = torch.softmax(randn(T, k), dim=1)
    if c["op"] == "combine":
        st.update(Y=(0.5 * randn(R, c["N"])).bfloat16(), w=w if c["weighted"] else None,
                  out=_zeros(T, c["N"], dtype=torch.bfloat16))
    elif c["op"] == "combine_bwd":
        N = c["N"]
        st.update(Y=(0.5 * randn(R, N)).bfloat16(), w=w, dout=(0.01 * randn(T, N)).bfloat16(), dw=_zeros(T, k),
                  Qr=_codes(R, N), sr=_zeros(N // 128, R), Qc=_codes(R, N), sc=_zeros(R // 128, N))
    elif c["op"] == "ckpt":
        F = c["F"]
        st.update(H=(2.0 * randn(R, 2 * F)).bfloat16(), Q=_codes(R, F), sa=_zeros(F // 128, R), C=_codes(R, 2 * F),
                  cs=_zeros(2 * F // 128, R))
    elif c["op"] == "ckpt_bwd":
        F = c["F"]
        H = torch.where(held, 2.0 * randn(R, 2 * F), torch.zeros((), device="cuda")).bfloat16().float()
        C, cs = _cast_1x128(H)
        st.update(dA=(0.01 * randn(R, F)).bfloat16(), C=C, cs=cs, Qr=_codes(R, 2 * F), sr=_zeros(2 * F // 128, R),
                  Qc=_codes(R, 2 * F), sc=_zeros(R // 128, 2 * F), Qa=_codes(R, F), sb=_zeros(F // 128, R // 128))
    else:
        K = c["K"]
        Q, sa = _cast_1x128(torch.where(held, randn(R, K), torch.zeros((), device="cuda")))
        st.update(Q=Q, sa=sa, Qb=_codes(R, K), sb=_zeros(K // 128, R // 128))
    return st


# -------------------------------------------------------------------------------------- plain forms


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
    """A scale for each block; scales [columns/128, rows/128]."""
    R, K = x.shape
    b = x.view(R // 128, 128, K // 128, 128)
    q, s = _quantised(b, b.abs().amax(dim=(1, 3), keepdim=True))
    return q.view(R, K), s[:, 0, :, 0].t().contiguous()


def _only(held, q, s):
    """Codes and 1x128 scales (both by rows) only where `held`; elsewhere zeros."""
    q = torch.where(held[:, None], q.float(), torch.zeros((), device=q.device)).to(torch.float8_e4m3fn)
    return q, torch.where(held[None, :], s, torch.zeros_like(s))


def _values(q, s):
    """What e4m3 codes with 1x128 scales stand for."""
    return q.float() * s.t().repeat_interleave(128, dim=1)


def _plain_route(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    # 64 bits: choices lie next to one another
    l = st["logits"].double()
    s = torch.softmax(l, dim=1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-l))
    low = torch.full((), -math.inf, dtype=torch.float64, device=l.device)
    ok = l != low
    choice = s
    if st["bias"] is not None:
        choice = s + st["bias"].double()
        ok = ok & (st["bias"] != -math.inf)
    key = choice if st["bias"] is not None else l
    key = torch.where(ok, key, low)
    if c["groups"] > 1:
        by = torch.where(ok, choice, low).view(T, c["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :c["gtop"]]
        best = torch.where(best == low, torch.zeros_like(best), best).sum(dim=2)
        best = torch.where(ok.view(T, c["groups"], -1).any(dim=2), best, low)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(E // c["groups"], dim=1), key, low)
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    w = torch.where(top != low, torch.gather(s, 1, idx), torch.zeros_like(top)).float()
    idx = torch.where(top != low, idx, torch.full_like(idx, -1))
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    return dict(idx=idx.int(), w=w * SCALE)


SCALE = 2.5  # of the routing weights


def _plain_route_bwd(st):
    c = st["case"]
    l, idx, dw = st["logits"].float(), st["idx"].long(), st["dw"]
    s = torch.softmax(l, dim=1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-l))
    sj = torch.gather(s, 1, idx)
    ds = dw * SCALE
    if c["renorm"]:
        total = sj.sum(dim=1, keepdim=True) + 1e-20
        ds = (ds - (ds * sj).sum(dim=1, keepdim=True) / total) / total
    d = torch.zeros_like(s).scatter_add_(1, idx, ds)
    if c["score"] == "softmax":
        d = s * (d - (ds * sj).sum(dim=1, keepdim=True))
    else:
        d = d * s * (1 - s)
    return d.to(st["logits"].dtype)


def _plain_dispatch(st):
    c = st["case"]
    lay = _layout(st["idx"], c["E"], c["max_rows"])
    R, M, K = lay["rows"], c["max_rows"], c["K"]
    q, s = _cast_1x128(st["X"].float())
    held = lay["slot_of"] >= 0
    token = torch.where(held, lay["slot_of"], torch.zeros_like(lay["slot_of"])).long() // c["k"]
    Q, sr = _only(held, q.view(torch.uint8)[token].view(torch.float8_e4m3fn), s[:, token])
    sa = torch.zeros_like(st["sa"])
    if M:
        sa[:, :, :M] = sr.view(K // 128, c["E"], M).transpose(0, 1)
    else:
        sa[0, :, :R] = sr
    return dict(row_of=lay["row_of"], m_indices=lay["m_indices"], slot_of=lay["slot_of"], offsets=lay["offsets"],
                counts=lay["counts"], Q=Q, sa=sa)


def _plain_combine(st):
    row = st["row_of"].long()
    w = torch.ones_like(row, dtype=torch.float32) if st["w"] is None else st["w"]
    w = torch.where(row >= 0, w, torch.zeros_like(w))
    return (st["Y"][row.clamp_min(0)].float() * w[:, :, None]).sum(dim=1).bfloat16()


def _plain_combine_bwd(st):
    c = st["case"]
    slot, row = st["slot_of"].long(), st["row_of"].long()
    held = slot >= 0
    at = slot.clamp_min(0)
    zero = torch.zeros((), device=slot.device)
    d = torch.where(held[:, None], st["dout"].float()[at // c["k"]] * st["w"].reshape(-1)[at][:, None], zero)
    dw = (st["dout"].float()[:, None, :] * st["Y"][row.clamp_min(0)].float()).sum(dim=2)
    return dict(dw=torch.where(row >= 0, dw, zero), **_both(d, held))


def _blocks(held):
    """Rows of the 128-row blocks that hold a token."""
    return held.view(-1, 128).any(dim=1).repeat_interleave(128)


def _both(d, held):
    """The two casts of a gradient by rows; blocks without a token stay zero."""
    there = _blocks(held)
    Qr, sr = _only(there, *_cast_1x128(d))
    Qc, sc = _cast_128x1(d)
    sc = torch.where(there[::128, None], sc, torch.zeros_like(sc))
    return dict(Qr=Qr, sr=sr, Qc=Qc, sc=sc)


def _plain_ckpt(st):
    F = st["case"]["F"]
    held = st["m_indices"] >= 0
    H = st["H"].float()
    gate, up = H[:, :F], H[:, F:]
    Q, sa = _only(held, *_cast_1x128(gate / (1 + torch.exp(-gate)) * up))
    C, cs = _only(held, *_cast_1x128(H))
    return dict(Q=Q, sa=sa, C=C, cs=cs)


def _plain_ckpt_bwd(st):
    F = st["case"]["F"]
    held = st["m_indices"] >= 0
    zero = torch.zeros((), device=held.device)
    H = torch.where(held[:, None], _values(st["C"], st["cs"]), zero)
    dA = torch.where(held[:, None], st["dA"].float(), zero)
    gate, up = H[:, :F], H[:, F:]
    s = 1 / (1 + torch.exp(-gate))
    both = _both(torch.cat([dA * up * s * (1 + gate * (1 - s)), dA * gate * s], dim=1), held)
    Qa, sb = _cast_128x128(gate * s * up)
    sb = torch.where(_blocks(held)[None, ::128], sb, torch.zeros_like(sb))
    return dict(both, Qa=Qa, sb=sb)


def _plain_recast(st):
    held = st["m_indices"] >= 0
    x = torch.where(held[:, None], _values(st["Q"], st["sa"]), torch.zeros((), device=held.device))
    Qb, sb = _cast_128x128(x)
    return dict(Qb=Qb, sb=torch.where(_blocks(held)[None, ::128], sb, torch.zeros_like(sb)))


# ------------------------------------------------------------------------------- the package's calls


def _own(st):
    import moe_grouped_gemm_weight_b200 as dg
    c = st["case"]
    op = c["op"]
    if op in ("route", "route_bwd"):
        score = dg.DG_SCORE_SOFTMAX if c["score"] == "softmax" else dg.DG_SCORE_SIGMOID
        if op == "route":
            dg.dg_route_topk(st["idx"], st["w"], st["logits"], st["bias"], n_groups=c["groups"],
                             topk_groups=c["keep"], group_top=c["gtop"], score=score, renorm=c["renorm"], scale=SCALE)
            return dict(idx=st["idx"], w=st["w"])
        dg.dg_route_topk_bwd(st["dlogits"], st["dw"], st["logits"], st["idx"], score=score, renorm=c["renorm"],
                             scale=SCALE)
        return st["dlogits"]
    if op == "dispatch":
        dg.dg_route_layout(st["row_of"], st["m_indices"], st["slot_of"], st["offsets"], st["counts"], st["idx"],
                           max_rows=c["max_rows"])
        dg.dg_dispatch_fp8_1x128(st["Q"], st["sa"], st["stride"], st["X"], st["row_of"], group_rows=c["max_rows"])
        return {n: st[n] for n in ("row_of", "m_indices", "slot_of", "offsets", "counts", "Q", "sa")}
    R = st["m_indices"].numel()
    if op == "combine":
        dg.dg_combine(st["out"], st["Y"], st["row_of"], st["w"])
        return st["out"]
    if op == "combine_bwd":
        dg.dg_combine_bwd(st["dw"], st["Qr"], st["sr"], R, st["Qc"], st["sc"], c["N"], st["dout"], st["Y"],
                          st["row_of"], st["slot_of"], st["w"])
        return {n: st[n] for n in ("dw", "Qr", "sr", "Qc", "sc")}
    if op == "ckpt":
        dg.dg_swiglu_fp8(st["Q"], st["sa"], R, st["H"], st["C"], st["cs"], R, m_indices=st["m_indices"])
        return {n: st[n] for n in ("Q", "sa", "C", "cs")}
    if op == "ckpt_bwd":
        dg.dg_swiglu_fp8_bwd(st["Qr"], st["sr"], R, st["Qc"], st["sc"], 2 * c["F"], st["Qa"], st["sb"], st["dA"],
                             st["C"], st["cs"], R, m_indices=st["m_indices"])
        return {n: st[n] for n in ("Qr", "sr", "Qc", "sc", "Qa", "sb")}
    dg.dg_fp8_1x128_to_128x128(st["Qb"], st["sb"], st["Q"], st["sa"], R, m_indices=st["m_indices"])
    return dict(Qb=st["Qb"], sb=st["sb"])


_PLAIN = dict(route=_plain_route, route_bwd=_plain_route_bwd, dispatch=_plain_dispatch, combine=_plain_combine,
              combine_bwd=_plain_combine_bwd, ckpt=_plain_ckpt, ckpt_bwd=_plain_ckpt_bwd, recast=_plain_recast)


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
    R, K = x.shape
    q, s = _exact_cast(x.reshape(R, K // 128, 128), (2,))
    return q.reshape(R, K), s.reshape(R, K // 128).t()


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    op = c["op"]
    T, E, k = c["T"], c["E"], c["k"]
    if op in ("route", "route_bwd"):
        x = st["logits"].double()
        if c["score"] == "sigmoid":
            s = torch.sigmoid(x)
        else:
            s = (x - torch.logsumexp(x, dim=1, keepdim=True)).exp()
        if op == "route":
            p = s if st["bias"] is None else s + st["bias"].double()
            if c["groups"] > 1:
                per = p.reshape(T, c["groups"], E // c["groups"])
                rate = per.topk(min(c["gtop"], E // c["groups"]), dim=2).values.sum(dim=2)
                stay = torch.zeros_like(rate)
                stay[torch.arange(T, device="cuda")[:, None], (-rate).argsort(dim=1, stable=True)[:, :c["keep"]]] = 1
                p = torch.where(stay.unsqueeze(2) > 0, per, torch.full_like(per, -9.0)).reshape(T, E)
            w = s.gather(1, p.topk(k, dim=1).indices)
            if c["renorm"]:
                w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
            return dict(idx=None, w=2.5 * w)
        j, dw = st["idx"].long(), 2.5 * st["dw"].double()
        chosen = s.gather(1, j)
        if c["renorm"]:
            z = chosen.sum(dim=1, keepdim=True) + 1e-20
            up = dw / z - (dw * chosen).sum(dim=1, keepdim=True) / z ** 2
        else:
            up = dw
        full = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add(1, j, up)
        if c["score"] == "sigmoid":
            return full * s * torch.sigmoid(-x)
        return full * s - s * (full * s).sum(dim=1, keepdim=True)
    if op == "dispatch":
        q, s = _exact_rows(st["X"].double())
        slots = _layout(st["idx"], E, c["max_rows"])["slot_of"].long()
        where = torch.nonzero(slots >= 0)[:, 0]
        R, M, K = slots.numel(), c["max_rows"], c["K"]
        Q = torch.zeros(R, K, dtype=torch.float64, device="cuda")
        Q[where] = q[slots[where] // k]
        sa = torch.zeros(st["sa"].shape, dtype=torch.float64, device="cuda")
        vals = s[:, slots[where] // k]
        if M:
            sa[where // M, :, where % M] = vals.t()
        else:
            sa[0][:, where] = vals
        return dict(row_of=None, m_indices=None, slot_of=None, offsets=None, counts=None, Q=Q, sa=sa)
    if op == "combine":
        there = torch.nonzero(st["row_of"] >= 0)
        w = torch.ones(T, k, dtype=torch.float64, device="cuda") if st["w"] is None else st["w"].double()
        part = st["Y"][st["row_of"][there[:, 0], there[:, 1]].long()].double() * w[there[:, 0], there[:, 1]][:, None]
        return torch.zeros(T, c["N"], dtype=torch.float64, device="cuda").index_add_(0, there[:, 0], part)
    rows = st["m_indices"].numel()
    used = (st["m_indices"] >= 0).double()[:, None]
    block = torch.nonzero(used.reshape(-1, 128).sum(dim=1) > 0)[:, 0]  # 128-row blocks with a token
    inside = (block[:, None] * 128 + torch.arange(128, device="cuda")).reshape(-1)

    def placed(shape, dim, at, part):
        full = torch.zeros(shape, dtype=torch.float64, device="cuda")
        return full.index_copy_(dim, at, part)

    def two_casts(d):
        n = d.shape[1]
        qr, sr = _exact_rows(d[inside])
        qc, sc = _exact_cast(d.reshape(-1, 128, n)[block], (1,))
        return dict(Qr=placed((rows, n), 0, inside, qr), sr=placed((n // 128, rows), 1, inside, sr),
                    Qc=placed((rows, n), 0, inside, qc.reshape(-1, n)), sc=placed((rows // 128, n), 0, block, sc[:, 0]))

    def by_block(x):
        n = x.shape[1]
        q, s = _exact_cast(x.reshape(-1, 128, n // 128, 128)[block], (1, 3))
        return placed((rows, n), 0, inside, q.reshape(-1, n)), placed((n // 128, rows // 128), 1, block, s[:, 0, :, 0].t())

    if op == "combine_bwd":
        at = torch.nonzero(st["slot_of"] >= 0)[:, 0]
        slot = st["slot_of"][at].long()
        grad = st["dout"].double()[slot // k]
        d = torch.zeros(rows, c["N"], dtype=torch.float64, device="cuda")
        d[at] = grad * st["w"].double().reshape(-1)[slot][:, None]
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dw[slot] = torch.einsum("rn,rn->r", grad, st["Y"][at].double())
        return dict(dw=dw.reshape(T, k), **two_casts(d))
    if op == "ckpt":
        h = st["H"].double()
        h1, h2 = h.chunk(2, dim=1)
        q, s = _exact_rows(torch.nn.functional.silu(h1) * h2)
        qc, sc = _exact_rows(h)
        return dict(Q=q * used, sa=s * used.t(), C=qc * used, cs=sc * used.t())
    held = used[:, 0] > 0
    if op == "ckpt_bwd":
        h = st["C"].double() * st["cs"].double().t().repeat_interleave(128, dim=1) * used
        h1, h2 = h.chunk(2, dim=1)
        da = st["dA"].double() * used
        p = torch.sigmoid(h1)
        d = torch.cat([da * h2 * (p + h1 * p * torch.sigmoid(-h1)), da * h1 * p], dim=1)
        qa, sb = by_block(h1 * p * h2)
        return dict(two_casts(d), Qa=qa, sb=sb)
    x = torch.zeros(rows, c["K"], dtype=torch.float64, device="cuda")
    x[held] = st["Q"][held].double() * st["sa"].double().t()[held].repeat_interleave(128, dim=1)
    qb, sb = by_block(x)
    return dict(Qb=qb, sb=sb)
