"""Cases, plain forms and 64-bit values of the training operators: the backward
pass of the block-sparse attention, and the norm of queries and keys with the
position rotation, forward and backward.

``run`` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end), or, where ``own`` is true, makes the call that a
user makes of the framework.  ``exact`` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 64
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------
def _attn(name, B, N, H, D, routing="tau", tau=1.0, ratio=0.0, mode=0, prefix=0):
    return dict(name=name, op="attn_bwd", B=B, N=N, H=H, D=D, routing=routing, tau=tau, ratio=ratio, mode=mode,
                prefix=prefix)


def _rope(name, op, B, N, H, D, rot, interleaved, weights, layout="fused"):
    return dict(name=name, op=op, B=B, N=N, H=H, D=D, rot=rot, interleaved=interleaved, weights=weights,
                layout=layout)


def listed():
    return [
        # the tiny configuration: a unit-test or debugging step, where launches count
        _attn("attn_bwd_tiny", 1, 1024, 2, 64),
        # a ragged batch of two with a text prefix and the weighted summaries; odd block counts everywhere
        _attn("attn_bwd_ragged_n1000", 2, 1000, 3, 64, tau=0.5, mode=2, prefix=100),
        # a short clip, every head on one GPU
        _attn("attn_bwd_h56_n4096", 1, 4096, 56, 128),
        # the Top-K configuration with the compressed branch and the weighted summaries
        _attn("attn_bwd_spark_n8192", 1, 8192, 56, 128, routing="spark", ratio=0.2, mode=2),
        # the joint text/audio/video sequence with the log-mass bias: one GPU's heads of an eight-way head split
        _attn("attn_bwd_joint_n38247_h7", 1, 38247, 7, 128, mode=1, prefix=2407),
        # the benchmark's own sequence
        _attn("attn_bwd_h56_n32768", 1, 32768, 56, 128),
        # one new token for each of eight sequences (serving): launch latency
        _rope("norm_rope_token_b8", "norm_rope", 8, 1, 56, 128, 128, False, "bf16"),
        # an odd batch of the small head dimension, partial interleaved rotation
        _rope("norm_rope_n777_d64", "norm_rope", 2, 777, 3, 64, 32, True, "fp32"),
        # the benchmark's sequence, as strided views of the fused QKV projection
        _rope("norm_rope_h56_n32768", "norm_rope", 1, 32768, 56, 128, 128, False, "fp32"),
        # the tiny configuration's training step
        _rope("norm_rope_bwd_tiny", "norm_rope_bwd", 1, 1024, 2, 64, 64, False, "fp32"),
        # an odd length, interleaved pairs, separate (unfused) projections
        _rope("norm_rope_bwd_n4097", "norm_rope_bwd", 1, 4097, 56, 128, 128, True, "bf16", layout="separate"),
        # the benchmark's sequence
        _rope("norm_rope_bwd_h56_n32768", "norm_rope_bwd", 1, 32768, 56, 128, 128, False, "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_bwd", "attn_bwd", "norm_rope", "norm_rope_bwd"])
    B, D = rng.choice([1, 1, 2, 3]), rng.choice([64, 128, 128])
    H = _log(rng, 1, 56)
    if op == "attn_bwd":
        N = _log(rng, 1, 16384)
        while B * H * N > 56 * 16384:
            H = max(1, H // 2)
        routing = rng.choice(["tau", "tau", "spark", "drop"])
        return dict(op=op, B=B, N=N, H=H, D=D, routing=routing,
                    tau=round(rng.uniform(0.3, 2.0), 2) if routing == "tau" else 0.0,
                    ratio=0.0 if routing == "tau" else round(rng.uniform(0.05, 0.4), 3),
                    mode=0 if routing == "drop" else rng.choice([0, 1, 2]),
                    prefix=rng.choice([0, rng.randint(0, N // 8), rng.randint(0, min(N, 100))]))
    N = _log(rng, 1, 32768)
    while B * H * N > 56 * 32768:
        H = max(1, H // 2)
    rot = rng.choice([D, D, D // 2, 16 * rng.randint(0, D // 16)])
    return dict(op=op, B=B, N=N, H=H, D=D, rot=rot, interleaved=rng.random() < 0.5,
                weights=rng.choice(["fp32", "bf16"]), layout=rng.choice(["fused", "separate"]))


# ---- inputs -----------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * seed + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _topic_inputs(c, seed):
    """q, k, v (bf16 BTHD): video rows of a raster T x 32 x 32 grid whose 4x4x4 tiles share one of 128
    per-head unit topics (q, k = 2 topic + noise), prefix rows plain noise; dO plain noise."""
    g = _gen(seed)
    B, N, H, D, P = c["B"], c["N"], c["H"], c["D"], c["prefix"]
    topics = torch.nn.functional.normalize(_randn(g, H, 128, D), dim=-1)
    at = torch.arange(N - P, device=DEV)
    tile = (at // 4096) * 64 + (at // 128 % 8) * 8 + at // 4 % 8
    n_tiles = int(tile.max()) + 1 if N > P else 1
    topic = torch.randint(0, 128, (B, H, n_tiles), generator=g, device=DEV)
    mean = torch.zeros(B, N, H, D, device=DEV)
    mean[:, P:] = 2.0 * topics[torch.arange(H, device=DEV)[None, None, :], topic[:, :, tile].transpose(1, 2)]
    q = (mean + _randn(g, B, N, H, D)).bfloat16()
    k = (mean + _randn(g, B, N, H, D)).bfloat16()
    v = _randn(g, B, N, H, D).bfloat16()
    do = _randn(g, B, N, H, D).bfloat16()
    return q, k, v, do


def _blocks(x, nb):
    """[B, N, H, D] -> fp32 [B, H, nb, 64, D], rows past N zero."""
    B, N, H, D = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, nb * BLOCK - N))
    return x.view(B, nb, BLOCK, H, D).permute(0, 3, 1, 2, 4)


def _counts(N):
    nb = -(-N // BLOCK)
    return (N - BLOCK * torch.arange(nb, device=DEV)).clamp(max=BLOCK)


def _route(c, q, k):
    """Exact-block mask [B, H, nb, nb] of the case's routing (64-row query blocks)."""
    N, P = c["N"], c["prefix"]
    nb = -(-N // BLOCK)
    n = _counts(N).float()[:, None]
    qsum, kbar = _blocks(q, nb).sum(3), _blocks(k, nb).sum(3) / n
    s = 1.0 / math.sqrt(c["D"])
    if c["routing"] == "drop":   # 128-row query blocks: both halves share a row of scores
        pad = nb % 2
        qsum = torch.nn.functional.pad(qsum, (0, 0, 0, pad))
        n2 = torch.nn.functional.pad(n, (0, 0, 0, pad)).view(-1, 2).sum(1)
        qbar = qsum.view(*qsum.shape[:2], -1, 2, c["D"]).sum(3) / n2[:, None]
    else:
        qbar = qsum / n
    S = s * qbar @ kbar.transpose(-1, -2)
    if c["routing"] == "tau":
        sel = S > S.mean(-1, keepdim=True) + c["tau"] * S.std(-1, keepdim=True, unbiased=False)
    else:
        keep = max(1, min(nb, math.floor(c["ratio"] * nb + 0.5)))
        order = torch.sort(S, dim=-1, descending=True, stable=True).indices[..., :keep]
        sel = torch.zeros_like(S, dtype=torch.bool).scatter_(-1, order, True)
    if c["routing"] == "drop":
        sel[:, :, :-(-P // (2 * BLOCK))] = True
        return sel.repeat_interleave(2, dim=2)[:, :, :nb].contiguous()
    sel[..., :-(-P // BLOCK)] = True
    sel[:, :, :-(-P // BLOCK)] = True
    return sel


def _anchor(c, q):
    return q[:, c["prefix"]:].float().mean(1) if c["prefix"] < c["N"] else q.float().mean(1)


def _centroids(c, q, k, v):
    """fp32 centroid keys and values (rounded to bf16, as the attention reads them), the offset added to
    their logits, the anchor and the anchor's weights over each block's rows."""
    N, s = c["N"], 1.0 / math.sqrt(c["D"])
    nb = -(-N // BLOCK)
    n = _counts(N).float()
    K, V = _blocks(k, nb), _blocks(v, nb)
    a = _anchor(c, q)
    e = s * torch.einsum("bhd,bhjtd->bhjt", a, K)
    e = e.masked_fill(torch.arange(BLOCK, device=DEV)[None, :] >= n[:, None], -math.inf)
    w = torch.softmax(e, dim=-1)
    if c["mode"] == 2:
        kc, vc = torch.einsum("bhjt,bhjtd->bhjd", w, K), torch.einsum("bhjt,bhjtd->bhjd", w, V)
    else:
        kc, vc = K.sum(3) / n[:, None], V.sum(3) / n[:, None]
    if c["mode"] == 0:
        off = n.log().expand(c["B"], c["H"], nb)
    else:
        off = torch.logsumexp(e, -1) - s * torch.einsum("bhd,bhjd->bhj", a, kc)
    return kc.bfloat16(), vc.bfloat16(), off.contiguous(), a, w


def _plain_forward(c, q, k, v, sel, cent):
    """o (bf16) and lse of the given lists, one head at a time over its gathered block pairs."""
    N, s = c["N"], 1.0 / math.sqrt(c["D"])
    nb = sel.shape[-1]
    kc, vc, off = cent[0].float(), cent[1].float(), cent[2]
    Q, K, V = _blocks(q, nb), _blocks(k, nb), _blocks(v, nb)
    dead = torch.arange(nb * BLOCK, device=DEV).view(nb, 1, BLOCK) >= N
    o, lse = torch.empty_like(q), torch.empty(c["B"], c["H"], N, device=DEV)
    for b in range(c["B"]):
        for h in range(c["H"]):
            i, j = sel[b, h].nonzero(as_tuple=True)
            S = (s * Q[b, h, i] @ K[b, h, j].transpose(-1, -2)).masked_fill(dead[j], -math.inf)
            m = torch.full((nb, BLOCK), -math.inf, device=DEV)
            m = m.scatter_reduce(0, i[:, None].expand(-1, BLOCK), S.amax(-1), "amax")
            if c["routing"] != "drop":
                Sc = (s * Q[b, h] @ kc[b, h].T + off[b, h]).masked_fill(sel[b, h][:, None, :], -math.inf)
                m = torch.maximum(m, Sc.amax(-1))
            pr = torch.exp(S - m[i][..., None])
            z = torch.zeros(nb, BLOCK, device=DEV).index_add_(0, i, pr.sum(-1))
            out = torch.zeros(nb, BLOCK, c["D"], device=DEV).index_add_(0, i, pr @ V[b, h, j])
            if c["routing"] != "drop":
                pc = torch.exp(Sc - m[..., None])
                z, out = z + pc.sum(-1), out + pc @ vc[b, h]
            o[b, :, h] = (out / z[..., None]).view(-1, c["D"])[:N].bfloat16()
            lse[b, h] = (m + z.log()).view(-1)[:N]
    return o, lse


def _tables(c):
    """fp32 cos and sin [N, rot/2] of a video grid: the pairs are dealt to the axes (t, h, w) in thirds,
    angles position * 10000^(-i / pairs of the axis), in 64 bits."""
    half = c["rot"] // 2
    at = torch.arange(c["N"], device=DEV)
    pos = torch.stack([at // 1024, at // 32 % 32, at % 32]).double()
    third = half // 3
    pairs = [half - 2 * third, third, third]
    ang = [p[:, None] * 10000.0 ** (-torch.arange(m, device=DEV).double() / max(m, 1)) for p, m in zip(pos, pairs)]
    ang = torch.cat(ang, dim=1)
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def _rope_inputs(c, seed):
    g = _gen(seed)
    B, N, H, D = c["B"], c["N"], c["H"], c["D"]
    if c["layout"] == "fused":   # views of the fused projection, as the model's linear layer writes it
        q, k, _ = _randn(g, B, N, 3, H, D).bfloat16().unbind(2)
    else:
        q, k = _randn(g, B, N, H, D).bfloat16(), _randn(g, B, N, H, D).bfloat16()
    wt = torch.bfloat16 if c["weights"] == "bf16" else torch.float32
    qw, kw = ((1.0 + 0.1 * _randn(g, D)).to(wt) for _ in range(2))
    return q, k, qw, kw, g


def prepare(case, seed):
    c = case
    if c["op"] == "attn_bwd":
        q, k, v, do = _topic_inputs(c, seed)
        sel = _route(c, q, k)
        cent = _centroids(c, q, k, v)
        o, lse = _plain_forward(c, q, k, v, sel, cent)
        st = dict(c=c, q=q, k=k, v=v, do=do, sel=sel, cent=cent, o=o, lse=lse)
        if own:   # the lists as CSR, the pooled workspace and the buffers of the call
            from block_sparse_video_sol_b200 import sol
            kw = {} if c["routing"] == "tau" else dict(topk_ratio=c["ratio"], compressed=c["routing"] == "spark")
            p = sol.make_params(c["B"], c["N"], c["H"], c["D"], tau=c["tau"], prefix_len=c["prefix"],
                                log_mass_bias=c["mode"], **kw)
            buf = sol.alloc_buffers(p, DEV)
            sol.sol_pool(p, q, k, v, buf.ws)
            counts = sel.sum(-1).view(-1)
            st["row_ptr"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
            entries = sel.view(-1, sel.shape[-1]).nonzero()[:, 1].int()
            st["col_idx"] = torch.nn.functional.pad(entries, (0, 1))   # an address even where no block is listed
            st.update(p=p, ws=buf.ws, g=sol.alloc_grads(p, DEV))
        return st
    q, k, qw, kw, g = _rope_inputs(c, seed)
    cos, sin = _tables(c)
    st = dict(c=c, q=q, k=k, qw=qw, kw=kw, cos=cos, sin=sin)
    if c["op"] == "norm_rope_bwd":
        st["dqo"], st["dko"] = (_randn(g, c["B"], c["N"], c["H"], c["D"]).bfloat16() for _ in range(2))
    if own:
        from block_sparse_video_sol_b200 import sol
        st["p"] = sol.make_params(c["B"], c["N"], c["H"], c["D"], in_strides=q.stride()[:3])
        st["nr"] = sol.make_norm_rope(qw, kw, cos, sin, rot_dim=c["rot"], interleaved=c["interleaved"])
        if c["op"] == "norm_rope":
            st["out"] = tuple(torch.empty(q.shape, dtype=q.dtype, device=DEV) for _ in range(2))
        else:
            dqkv = torch.empty(c["B"], c["N"], 3, c["H"], c["D"], dtype=q.dtype, device=DEV)
            st["out"] = dqkv.unbind(2)[:2] if c["layout"] == "fused" else (torch.empty_like(q), torch.empty_like(k))
            st["dw"] = tuple(torch.empty(c["D"], device=DEV) for _ in range(2))
            st["ws"] = torch.empty(sol.sol_qk_norm_rope_bwd_workspace_bytes(st["p"]), dtype=torch.uint8, device=DEV)
    return st


# ---- plain forms --------------------------------------------------------------------------------
def _plain_attn_bwd(st):
    c = st["c"]
    N, D, s, mode = c["N"], c["D"], 1.0 / math.sqrt(c["D"]), c["mode"]
    sel, (kc, vc, off, a, w) = st["sel"], st["cent"]
    nb = sel.shape[-1]
    n = _counts(N).float()
    kc, vc = kc.float(), vc.float()
    Q, K, V, dO, O = (_blocks(st[x], nb) for x in ("q", "k", "v", "do", "o"))
    lse = torch.nn.functional.pad(st["lse"], (0, nb * BLOCK - N)).view(c["B"], c["H"], nb, BLOCK)
    delta = (dO * O).sum(-1)
    dead = torch.arange(nb * BLOCK, device=DEV).view(nb, 1, BLOCK) >= N
    out = tuple(torch.empty_like(st[x]) for x in ("q", "k", "v"))
    for b in range(c["B"]):
        for h in range(c["H"]):
            i, j = sel[b, h].nonzero(as_tuple=True)
            Qh, Kh, Vh, Oh = Q[b, h], K[b, h], V[b, h], dO[b, h]
            qi, kj, oi = Qh[i], Kh[j], Oh[i]
            pr = torch.exp((s * qi @ kj.transpose(-1, -2)).masked_fill(dead[j], -math.inf) - lse[b, h][i][..., None])
            dv = torch.zeros_like(Vh).index_add_(0, j, pr.transpose(-1, -2) @ oi)
            ds = s * pr * (oi @ Vh[j].transpose(-1, -2) - delta[b, h][i][..., None])
            dq = torch.zeros_like(Qh).index_add_(0, i, ds @ kj)
            dk = torch.zeros_like(Kh).index_add_(0, j, ds.transpose(-1, -2) @ qi)
            if c["routing"] != "drop":
                Sc = (s * Qh @ kc[b, h].T + off[b, h]).masked_fill(sel[b, h][:, None, :], -math.inf)
                Sc = Sc.view(-1, nb)
                live = (torch.arange(nb * BLOCK, device=DEV) < N)[:, None]
                pc = torch.exp(Sc - lse[b, h].view(-1, 1)) * live
                Qf, Of = Qh.reshape(-1, D), Oh.reshape(-1, D)
                dsc = pc * (Of @ vc[b, h].T - delta[b, h].view(-1, 1))
                dq += (s * dsc @ kc[b, h]).view_as(dq)
                gk, gv, gb = s * dsc.T @ Qf, pc.T @ Of, dsc.sum(0)
                ah = a[b, h]
                if mode == 2:
                    wt = w[b, h]
                    g2 = gk - s * gb[:, None] * ah
                    hh = torch.einsum("jd,jtd->jt", g2, Kh) + torch.einsum("jd,jtd->jt", gv, Vh)
                    beta = s * wt * (hh - (wt * hh).sum(-1, keepdim=True))
                    dk += wt[..., None] * gk[:, None] + beta[..., None] * ah
                    dv += wt[..., None] * gv[:, None]
                else:
                    dk += (gk / n[:, None])[:, None]
                    dv += (gv / n[:, None])[:, None]
                    beta = s * gb[:, None] * (w[b, h] - 1.0 / n[:, None]) * ~dead[:, 0]
                    if mode == 1:
                        dk += beta[..., None] * ah
                if mode:
                    lo = c["prefix"] if c["prefix"] < N else 0
                    dq.view(-1, D)[lo:N] += torch.einsum("jt,jtd->d", beta, Kh) / (N - lo)
            for g, x in zip(out, (dq, dk, dv)):
                g[b, :, h] = x.view(-1, D)[:N].bfloat16()
    return out


def _rotate(y, cos, sin, interleaved, sign):
    """The first 2 * cos.shape[-1] dims of y [B, N, H, D] turned by sign * angle."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sign * sin[:, None]
    r, rest = y[..., :2 * half], y[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _norm(x, w, eps=1e-6):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * w


def _norm_bwd(x, w, g, eps=1e-6):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    xh, u = x * r, g * w
    return r * (u - xh * (u * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1, 2))


def run(state):
    st, c = state, state["c"]
    if own:
        from block_sparse_video_sol_b200 import sol
        if c["op"] == "attn_bwd":
            g = st["g"]
            sol.sol_attn_bwd(st["p"], st["q"], st["k"], st["v"], st["ws"], st["row_ptr"], st["col_idx"], st["o"],
                             st["lse"], st["do"], g.dq, g.dk, g.dv, g.ws)
            return g.dq, g.dk, g.dv
        if c["op"] == "norm_rope":
            sol.sol_qk_norm_rope(st["p"], st["nr"], st["q"], st["k"], *st["out"])
            return st["out"]
        sol.sol_qk_norm_rope_bwd(st["p"], st["nr"], st["q"], st["k"], st["dqo"], st["dko"], *st["out"], *st["dw"],
                                 st["ws"])
        return (*st["out"], *st["dw"])
    if c["op"] == "attn_bwd":
        return _plain_attn_bwd(st)
    if c["op"] == "norm_rope":
        return tuple(_rotate(_norm(x.float(), w.float()), st["cos"], st["sin"], c["interleaved"], 1.0).bfloat16()
                     for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])))
    dq, dqw = _norm_bwd(st["q"].float(), st["qw"].float(),
                        _rotate(st["dqo"].float(), st["cos"], st["sin"], c["interleaved"], -1.0))
    dk, dkw = _norm_bwd(st["k"].float(), st["kw"].float(),
                        _rotate(st["dko"].float(), st["cos"], st["sin"], c["interleaved"], -1.0))
    return dq.bfloat16(), dk.bfloat16(), dqw, dkw


# ---- the definitions in 64 bits -------------------------------------------------------------------
def _exact_head(c, q, k, v, do, sel):
    """Gradients of one head by differentiating the forward's definition over dense masked rows."""
    N, D, s, mode, P = c["N"], c["D"], 1.0 / math.sqrt(c["D"]), c["mode"], c["prefix"]
    nb = -(-N // BLOCK)
    leaf = [x.double().requires_grad_() for x in (q, k, v)]
    grads = [torch.zeros_like(x) for x in leaf]
    blk = torch.arange(N, device=DEV) // BLOCK
    member = torch.nn.functional.one_hot(blk, nb).double()           # [N, nb]
    n = member.sum(0)
    for lo in range(0, N, 2048):
        Q, K, V = leaf
        rows = slice(lo, min(N, lo + 2048))
        seen = sel[blk[rows]]                                         # [rows, nb]
        logit = (s * Q[rows] @ K.T).masked_fill(~seen[:, blk], -math.inf)
        if c["routing"] != "drop":
            a = Q[P:].mean(0) if P < N else Q.mean(0)
            e = s * K @ a
            per = e[:, None].expand(-1, nb).masked_fill(member == 0, -math.inf)
            if mode == 2:
                wt = torch.softmax(per, 0)
                kc, vc = wt.T @ K, wt.T @ V
            else:
                kc, vc = member.T @ K / n[:, None], member.T @ V / n[:, None]
            off = n.log() if mode == 0 else torch.logsumexp(per, 0) - s * kc @ a
            kc, vc = (x + (x.float().bfloat16().double() - x).detach() for x in (kc, vc))
            lc = (s * Q[rows] @ kc.T + off).masked_fill(seen, -math.inf)
            o = torch.softmax(torch.cat([logit, lc], 1), 1) @ torch.cat([V, vc])
        else:
            o = torch.softmax(logit, 1) @ V
        for g, x in zip(grads, torch.autograd.grad((o * do[rows].double()).sum(), leaf)):
            g += x
    return grads


def exact(case, seed):
    c = case
    if c["op"] == "attn_bwd":
        if c["B"] * c["H"] * c["N"] ** 2 > 2.0e10:   # the largest would take over 20 seconds
            return None
        q, k, v, do = _topic_inputs(c, seed)
        sel = _route(c, q, k)
        out = tuple(torch.empty(q.shape, dtype=torch.float64, device=DEV) for _ in range(3))
        for b in range(c["B"]):
            for h in range(c["H"]):
                for g, x in zip(out, _exact_head(c, q[b, :, h], k[b, :, h], v[b, :, h], do[b, :, h], sel[b, h])):
                    g[b, :, h] = x
        return out
    q, k, qw, kw, g = _rope_inputs(c, seed)
    cos, sin = (t.double() for t in _tables(c))
    half = c["rot"] // 2
    pair = torch.arange(half, device=DEV)
    first, second = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + half)
    turn = torch.eye(c["D"], dtype=torch.float64, device=DEV).repeat(c["N"], 1, 1)   # [N, D, D] rotation
    turn[:, first, first], turn[:, second, second] = cos, cos
    turn[:, first, second], turn[:, second, first] = -sin, sin
    out, dw = [], []
    grads = [_randn(g, c["B"], c["N"], c["H"], c["D"]).bfloat16() for _ in range(2)] if c["op"] == "norm_rope_bwd" else [None, None]
    for x, w, dz in zip((q, k), (qw, kw), grads):
        y, gw = torch.empty(x.shape, dtype=torch.float64, device=DEV), torch.zeros(c["D"], dtype=torch.float64, device=DEV)
        for lo in range(0, c["N"], 8192):
            r = slice(lo, min(c["N"], lo + 8192))
            xd, wd, T = x[:, r].double(), w.double(), turn[r]
            inv = ((xd ** 2).sum(-1, keepdim=True) / c["D"] + 1e-6) ** -0.5
            if dz is None:
                y[:, r] = torch.einsum("nij,bnhj->bnhi", T, xd * inv * wd)
            else:
                gd = torch.einsum("nij,bnhi->bnhj", T, dz[:, r].double())
                dot = (gd * wd * xd).sum(-1, keepdim=True)
                y[:, r] = inv * gd * wd - xd * inv ** 3 * dot / c["D"]
                gw += (gd * xd * inv).sum((0, 1, 2))
        out.append(y)
        dw.append(gw)
    return tuple(out) if c["op"] == "norm_rope" else (*out, *dw)


# ---- what the path cannot do without ------------------------------------------------------------
def work(case):
    c = case
    rows = c["B"] * c["N"] * c["H"]
    if c["op"] != "attn_bwd":
        tensors = 4 if c["op"] == "norm_rope" else 6
        per = (12 if c["op"] == "norm_rope" else 24) * 2   # flops a dim of q and k
        return {"bytes": tensors * rows * c["D"] * 2 + c["N"] * c["rot"] * 4, "flops": rows * c["D"] * per}
    # five products over the selected keys and the other blocks' centroids; the share of selected blocks is
    # that of a normal distribution's tail above tau, or the ratio; prefix rows take all, prefix blocks are taken by all
    nb = -(-c["N"] // BLOCK)
    share = c["ratio"] if c["routing"] != "tau" else 0.5 * math.erfc(c["tau"] / math.sqrt(2.0))
    pre = min(1.0, -(-c["prefix"] // BLOCK) / nb)
    share = share * (1 - pre) ** 2 + (pre if c["routing"] == "drop" else 2 * pre - pre * pre)
    keys = share * c["N"] + (0 if c["routing"] == "drop" else (1 - share) * nb)
    return {"bytes": 8 * rows * c["D"] * 2 + rows * 4 + c["B"] * c["H"] * nb * nb * share * 4,
            "flops": 10 * rows * keys * c["D"]}
