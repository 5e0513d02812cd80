"""The balance-loss and 4-bit-expert operators on measurable cases.

Three families of calls, each with a plain form (elementary torch operations in
fp32, or fp64 where a decision needs it) and the library's own calls:

balance    the load-balancing loss and per-expert counts over sequences of a
           padded batch ("forward"), its gradient with respect to the router
           logits ("backward"), or both, as a training step makes them ("step")
quantize   4-bit weights with group scales, and the values they stand for
experts    the expert FFN on 4-bit weights, from single tokens to batches

4-bit layout (see include/moe.h): each row of K weights is cut into blocks of
128; a block is 64 bytes = 16 words of 32 bits; word 4 t + j holds the weights
k = 32 j + 8 t .. + 7 of the block: k + 2 i in bits 4 i .. 4 i + 3 and
k + 2 i + 1 in bits 16 + 4 i .. (i = 0..3), each as q + 8.  Weights past K are
0 (q + 8 = 8).  Scales are bf16, [matrix, group, row].
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # the fp32 test layer's router (512 tokens, 8 experts): a small call whose latency counts
        dict(name="balance_small_fwd", op="balance", way="forward", T=512, N=8, k=1, S=1, dtype="f32", mask=False, tail=0),
        # a top-1 layer of 64 experts on 65536 tokens in 128 sequences, padded positions masked
        dict(name="balance_64e_fwd", op="balance", way="forward", T=65536, N=64, k=1, S=128, dtype="f32", mask=True, tail=0),
        # the gradient for an 8-expert top-2 layer on 16384 tokens, one group
        dict(name="balance_8e_bwd", op="balance", way="backward", T=16384, N=8, k=2, S=1, dtype="f32", mask=False, tail=0),
        # a ragged batch with unused rows at its end, bf16 logits, an odd expert count
        dict(name="balance_ragged_bwd", op="balance", way="backward", T=10007, N=60, k=4, S=37, dtype="bf16", mask=True, tail=91),
        # loss and gradient of a large step with many experts
        dict(name="balance_256e_step", op="balance", way="step", T=262144, N=256, k=8, S=64, dtype="f32", mask=True, tail=0),
        # loading two d_model 4096, d_ff 14336 expert matrices as 4-bit weights
        dict(name="quantize_bf16", op="quantize", mats=2, rows=14336, K=4096, group=128, dtype="bf16"),
        # small fp32 master weights, a row length that ends inside a group
        dict(name="quantize_f32_odd", op="quantize", mats=5, rows=1008, K=1040, group=64, dtype="f32"),
        # one token of the d_model 4096 SwiGLU layer: a decoding step
        dict(name="experts_1tok", op="experts", T=1, d=4096, d_ff=14336, N=8, k=2, act="swiglu", group=128, bias=False),
        # sixteen tokens of the same layer: decoding a small batch
        dict(name="experts_16tok", op="experts", T=16, d=4096, d_ff=14336, N=8, k=2, act="swiglu", group=128, bias=False),
        # 64 tokens over 32 ReLU experts of the d_model 1024 layer
        dict(name="experts_relu", op="experts", T=64, d=1024, d_ff=4096, N=32, k=2, act="relu", group=64, bias=False),
        # odd sizes, biases, small groups
        dict(name="experts_odd", op="experts", T=37, d=528, d_ff=1360, N=12, k=1, act="swiglu", group=32, bias=True),
        # a prompt of 1024 tokens
        dict(name="experts_prompt", op="experts", T=1024, d=4096, d_ff=14336, N=8, k=2, act="swiglu", group=128, bias=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance", "quantize", "experts", "experts", "experts"])
    if op == "balance":
        N = _logint(rng, 4, 256)
        T = _logint(rng, 32, min(262144, 262144 * 256 // N))
        tail = rng.choice([0, rng.randint(1, max(1, T // 16))])
        return dict(op="balance", way=rng.choice(["forward", "backward", "step"]), T=T, N=N, k=rng.randint(1, min(8, N)),
                    S=_logint(rng, 1, 64), dtype=rng.choice(["f32", "bf16"]), mask=rng.random() < 0.5, tail=tail)
    if op == "quantize":
        mats, K = rng.randint(1, 8), 16 * _logint(rng, 4, 512)
        rows = 16 * _logint(rng, 4, max(5, min(1024, 117440512 // (mats * K * 16))))
        return dict(op="quantize", mats=mats, rows=rows, K=K, group=rng.choice([32, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
    act = rng.choice(["relu", "swiglu"])
    d = 16 * _logint(rng, 8, 256)
    d_ff = 16 * max(1, int(d * rng.uniform(1.0, 3.5)) // 16)
    N = _logint(rng, 2, max(2, min(64, 1409286144 // (d * d_ff * 3))))
    return dict(op="experts", T=_logint(rng, 1, 1024), d=d, d_ff=d_ff, N=N, k=rng.randint(1, 2), act=act,
                group=rng.choice([32, 64, 128]), bias=rng.random() < 0.5)


# ------------------------------------------------------------ preparation ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cuts(case, g):
    """Ragged sequence boundaries [S + 1]; `tail` rows lie behind the last one."""
    T, S = case["T"] - case["tail"], case["S"]
    inner = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values if S > 1 else \
        torch.zeros(0, dtype=torch.int64, device="cuda")
    ends = torch.tensor([0], device="cuda"), torch.tensor([T], device="cuda")
    return torch.cat([ends[0], inner, ends[1]]).to(torch.int32)


def _prepare_balance(case, seed):
    g = _gen(seed)
    T, N, k, S = case["T"], case["N"], case["k"], case["S"]
    popular = torch.randn(N, generator=g, device="cuda")   # some experts are liked by most tokens
    h = torch.randn(T, N, generator=g, device="cuda") * 1.5 + popular
    h = h.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    st = dict(case=case, h=h, idx=h.topk(k, dim=1).indices.to(torch.int32).contiguous(), seqs=_cuts(case, g),
              mask=(torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if case["mask"] else None,
              alpha=1e-2, z_coef=1e-3, dloss=torch.tensor([1.0, 0.75], device="cuda"))
    if case["way"] == "backward":   # what the forward left
        _, st["counts"], _, st["tokens"] = _balance_forward(st)
    st["dh"] = torch.zeros_like(h)
    if own:
        from mixture_experts_sparse_b200 import native as nat
        cfg = nat.balance_config(T, N, k, S, case["dtype"], st["alpha"], st["z_coef"])
        st.update(nat=nat, cfg=cfg, ws=nat.new_balance_workspace(cfg),
                  loss=torch.empty(2, device="cuda"), P=torch.empty(S, N, device="cuda"),
                  counts=st.get("counts", torch.empty(S, N, dtype=torch.int32, device="cuda")),
                  tokens=st.get("tokens", torch.empty(S + 2, dtype=torch.int32, device="cuda")))
    return st


def _prepare_quantize(case, seed):
    g = _gen(seed)
    M, R, K, G = case["mats"], case["rows"], case["K"], case["group"]
    w = torch.randn(M, R, K, generator=g, device="cuda") * math.sqrt(0.1 / K)
    w = w.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    st = dict(case=case, w=w)
    if own:
        from mixture_experts_sparse_b200 import native as nat
        st.update(nat=nat, q=torch.empty(M, R, nat.moe_w4_row_bytes(K), dtype=torch.uint8, device="cuda"),
                  scale=torch.empty(M, (K + G - 1) // G, R, dtype=torch.bfloat16, device="cuda"), out=torch.empty_like(w))
    return st


def _words(q):
    """[..., K] integers in -8..7 -> the packed rows [..., ceil(K / 128) * 64] uint8."""
    K = q.shape[-1]
    kb = (K + 127) // 128
    c = (q + 8).to(torch.uint8)
    if kb * 128 != K:
        c = torch.nn.functional.pad(c, (0, kb * 128 - K), value=8)
    # block, j, t, i, odd -> word (t, j), byte b = nibbles (2 b, 2 b + 1), nibble = i + 4 odd
    c = c.reshape(*q.shape[:-1], kb, 4, 4, 4, 2)
    n = c.permute(*range(c.dim() - 4), -3, -4, -1, -2).reshape(*q.shape[:-1], kb * 64, 2)
    return n[..., 0] | (n[..., 1] << 4)


def _values(q4, scale, K, group, dtype=torch.float32):
    """The weights that packed rows [R, bytes] and scales [groups, R] stand for: [R, K]."""
    R = q4.shape[0]
    n = torch.stack([q4 & 15, q4 >> 4], dim=-1).reshape(R, -1, 4, 4, 2, 4)   # block, t, j, odd, i
    q = n.permute(0, 1, 3, 2, 5, 4).reshape(R, -1)[:, :K].to(dtype) - 8
    return q * scale.to(dtype).t().repeat_interleave(group, dim=1)[:, :K]


def _prepare_experts(case, seed):
    g = _gen(seed)
    T, d, f, N, k, G = case["T"], case["d"], case["d_ff"], case["N"], case["k"], case["group"]

    def weight(rows, K):
        """Quantised normal weights of the layer's initialisation, one expert at a time."""
        ng = (K + G - 1) // G
        q4 = torch.empty(N, rows, (K + 127) // 128 * 64, dtype=torch.uint8, device="cuda")
        sc = torch.empty(N, ng, rows, dtype=torch.bfloat16, device="cuda")
        for e in range(N):
            w = torch.randn(rows, K, generator=g, device="cuda") * math.sqrt(0.1 / K)
            pad = torch.nn.functional.pad(w, (0, ng * G - K)).view(rows, ng, G)
            s = (pad.abs().amax(2) / 7).to(torch.bfloat16)
            q = (pad / s.float()[..., None]).round().clamp(-7, 7).view(rows, -1)[:, :K]
            q4[e], sc[e] = _words(q.to(torch.int8)), s.t()
        return q4, sc

    st = dict(case=case, w1=weight(f, d), w3=weight(f, d) if case["act"] == "swiglu" else None, w2=weight(d, f))

    def bias(n):
        return (torch.randn(N, n, generator=g, device="cuda") * 0.02).to(torch.bfloat16) if case["bias"] else None

    st.update(b1=bias(f), b3=bias(f) if case["act"] == "swiglu" else None, b2=bias(d))
    # each token's experts: some are more popular than others
    pick = (torch.rand(T, N, generator=g, device="cuda").log() / (torch.arange(N, device="cuda") + 4.0)).topk(min(k, N), dim=1).indices
    rows = torch.bincount(pick.flatten(), minlength=N)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), rows.cumsum(0)]).to(torch.int32)
    x = torch.randn(T * min(k, N), d, generator=g, device="cuda")
    st.update(x=(x / x.square().mean(1, keepdim=True).sqrt()).to(torch.bfloat16), offsets=offsets,
              rows=rows.tolist())
    if own:
        from mixture_experts_sparse_b200 import native as nat
        cfg = nat.config(T, d, f, N, k, T, "bf16", case["act"])
        st.update(nat=nat, cfg=cfg, ws=nat.new_w4_workspace(cfg), y=torch.empty_like(st["x"]))
    return st


def prepare(case, seed):
    return {"balance": _prepare_balance, "quantize": _prepare_quantize, "experts": _prepare_experts}[case["op"]](case, seed)


# ------------------------------------------------------------ plain forms ----

def _segments(st):
    """Each token's sequence (S for rows behind the last one), and whether it counts."""
    S, T = st["case"]["S"], st["case"]["T"]
    seg = torch.bucketize(torch.arange(T, device="cuda", dtype=torch.int32), st["seqs"], right=True) - 1
    m = seg < S
    if st["mask"] is not None:
        m = m & (st["mask"] != 0)
    return seg, m


def _softmax(h):
    top = h.amax(1, keepdim=True)
    e = (h - top).exp()
    s = e.sum(1, keepdim=True)
    return e / s, (top + s.log())[:, 0]


def _balance_forward(st):
    c = st["case"]
    N, S, k = c["N"], c["S"], c["k"]
    seg, m = _segments(st)
    p, lse = _softmax(st["h"].float())
    key = torch.where(m, seg, S)
    tokens = torch.bincount(key, minlength=S + 1)[:S]
    flat = (key[:, None] * N + st["idx"]).flatten()
    counts = torch.bincount(flat, minlength=(S + 1) * N)[:S * N].view(S, N)
    P = torch.zeros(S + 1, N, dtype=torch.float64, device="cuda").index_add_(0, key, p.double())[:S]
    P = P / tokens.clamp(min=1)[:, None]
    used = (tokens > 0).sum()
    f = counts / (k * tokens.clamp(min=1))[:, None].double()
    aux = st["alpha"] * N * (f * P).sum() / used.clamp(min=1)
    z = st["z_coef"] * (lse.double().square() * m).sum() / tokens.sum().clamp(min=1)
    loss = torch.stack([aux, z]).float()
    return loss, counts.int(), P.float(), torch.cat([tokens, tokens.sum()[None], used[None]]).int()


def _balance_backward(st, counts, tokens):
    c = st["case"]
    N, S, k = c["N"], c["S"], c["k"]
    seg, m = _segments(st)
    p, lse = _softmax(st["h"].float())
    n = tokens[:S].clamp(min=1).float()
    a = st["dloss"][0] * st["alpha"] * N / tokens[S + 1].clamp(min=1) * counts / (k * n * n)[:, None]
    a = a[seg.clamp(max=S - 1)]
    zg = st["dloss"][1] * 2 * st["z_coef"] / tokens[S].clamp(min=1) * lse
    d = p * (a - (p * a).sum(1, keepdim=True) + zg[:, None])
    return torch.where(m[:, None], d, 0.0).to(st["h"].dtype)


def _quantize(st):
    c = st["case"]
    K, G = c["K"], c["group"]
    w = st["w"].double()
    ng = (K + G - 1) // G
    w = torch.nn.functional.pad(w, (0, ng * G - K)).view(*w.shape[:-1], ng, G)
    mant, ex = torch.frexp(w.abs().amax(-1) / 7)
    scale = torch.ldexp((mant * 256).round() / 256, ex)   # eight significant bits, ties to even
    q = torch.where(scale[..., None] > 0, w / scale[..., None], 0.0).round().clamp(-7, 7)
    val = (q * scale[..., None]).reshape(*w.shape[:-2], ng * G)[..., :K]
    return val.to(st["w"].dtype), scale.transpose(-1, -2).to(torch.bfloat16)


def _ffn(st, dtype):
    c = st["case"]
    d, f, G = c["d"], c["d_ff"], c["group"]
    out, r0 = torch.empty(st["x"].shape, dtype=dtype, device="cuda"), 0
    for e, n in enumerate(st["rows"]):
        if n == 0:
            continue
        x = st["x"][r0:r0 + n].to(dtype)
        u = x @ _values(st["w1"][0][e], st["w1"][1][e], d, G, dtype).t()
        if st["b1"] is not None:
            u = u + st["b1"][e].to(dtype)
        if c["act"] == "swiglu":
            v = x @ _values(st["w3"][0][e], st["w3"][1][e], d, G, dtype).t()
            if st["b3"] is not None:
                v = v + st["b3"][e].to(dtype)
            u = u / (1 + (-u).exp()) * v
        else:
            u = u.clamp(min=0)
        y = u @ _values(st["w2"][0][e], st["w2"][1][e], f, G, dtype).t()
        out[r0:r0 + n] = y if st["b2"] is None else y + st["b2"][e].to(dtype)
        r0 += n
    return out


# -------------------------------------------------------------------- run ----

def run(st):
    c = st["case"]
    if own:
        nat = st["nat"]
        if c["op"] == "balance":
            outs = []
            if c["way"] != "backward":
                nat.check(nat.moe_balance_loss(st["cfg"], st["h"], st["idx"], st["mask"], st["seqs"], st["loss"], st["counts"],
                                               st["P"], st["tokens"], st["ws"]))
                outs = [st["loss"], st["counts"], st["P"], st["tokens"]]
            if c["way"] != "forward":
                nat.check(nat.moe_balance_loss_backward(st["cfg"], st["h"], st["mask"], st["seqs"], st["counts"], st["tokens"],
                                                        st["dloss"], st["dh"], False))
                outs.append(st["dh"])
            return outs
        if c["op"] == "quantize":
            a = (c["mats"], c["rows"], c["K"], c["group"], c["dtype"])
            nat.check(nat.moe_quantize_w4(*a, st["w"], st["q"], st["scale"]))
            nat.check(nat.moe_dequantize_w4(*a, st["q"], st["scale"], st["out"]))
            return [st["out"], st["scale"]]
        none = (None, None)
        nat.check(nat.moe_expert_ffn_w4(st["cfg"], c["group"], st["x"], st["offsets"], *st["w1"], st["b1"], *(st["w3"] or none),
                                        st["b3"], *st["w2"], st["b2"], st["y"], st["ws"]))
        return [st["y"]]
    if c["op"] == "balance":
        if c["way"] == "backward":
            return [_balance_backward(st, st["counts"], st["tokens"])]
        outs = list(_balance_forward(st))
        if c["way"] == "step":
            outs.append(_balance_backward(st, outs[1], outs[3]))
        return outs
    if c["op"] == "quantize":
        return list(_quantize(st))
    return [_ffn(st, torch.float32).to(torch.bfloat16)]


def work(case):
    if case["op"] == "balance":
        T, N, k, S = case["T"], case["N"], case["k"], case["S"]
        e = 2 if case["dtype"] == "bf16" else 4
        row = T * (1 if case["mask"] else 0) + 4 * (S + 1)
        fwd, bwd = T * N * e + 4 * T * k + row + 8 * S * N, 2 * T * N * e + row + 4 * S * N
        return {"forward": {"bytes": fwd, "flops": 8 * T * N}, "backward": {"bytes": bwd, "flops": 12 * T * N},
                # one call after the other reads the logits again: the loss of the whole batch comes before any gradient
                "step": {"bytes": fwd + bwd, "flops": 20 * T * N}}[case["way"]]
    if case["op"] == "quantize":
        n = case["mats"] * case["rows"] * case["K"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": int(n * (2 * e + 2 * (0.5 + 2 / case["group"]))), "flops": 4 * n}
    T, d, f, N, k = case["T"], case["d"], case["d_ff"], case["N"], min(case["k"], case["N"])
    mats = 3 if case["act"] == "swiglu" else 2
    hit = min(N, T * k) if T * k < 4 else min(N, max(1, round(N * (1 - (1 - 1 / N) ** (T * k)))))
    return {"bytes": int(hit * mats * d * f * (0.5 + 2 / case["group"])) + 4 * T * k * d, "flops": 2 * T * k * mats * d * f}


# ------------------------------------------------------ the definition, in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "experts":
        return [_ffn_exact(st)]
    if case["op"] == "quantize":
        return _quantize_exact(st)
    return _balance_exact(st)


def _balance_exact(st):
    """Sequence by sequence, through log-softmax and the derivative of the whole loss."""
    c = st["case"]
    N, S, k, T = c["N"], c["S"], c["k"], c["T"]
    cuts = st["seqs"].tolist()
    take = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
    h = st["h"].double()
    logp = h - torch.logsumexp(h, 1, keepdim=True)
    lse = torch.logsumexp(h, 1)
    sel = [torch.arange(a, b, device="cuda")[take[a:b]] for a, b in zip(cuts[:-1], cuts[1:])]
    n = [len(s) for s in sel]
    used, total = sum(x > 0 for x in n), sum(n)
    counts = torch.zeros(S, N, dtype=torch.int32, device="cuda")
    P = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    dh = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    aux, z = 0.0, 0.0
    g0, g1 = (float(v) for v in st["dloss"].double())
    for s, rows in enumerate(sel):
        if not len(rows):
            continue
        counts[s] = torch.bincount(st["idx"][rows].flatten(), minlength=N).int()
        p = logp[rows].exp()
        P[s] = p.sum(0) / n[s]
        f = counts[s].double() / (k * n[s])
        aux = aux + st["alpha"] * N * torch.dot(f, P[s]) / used
        z = z + st["z_coef"] * lse[rows].square().sum() / total
        centred = f - (p @ f)[:, None]
        dh[rows] = g0 * st["alpha"] * N / (used * n[s]) * p * centred + g1 * 2 * st["z_coef"] / total * lse[rows, None] * p
    loss = torch.stack([torch.as_tensor(v, dtype=torch.float64, device="cuda") for v in (aux, z)])
    tokens = torch.tensor(n + [total, used], dtype=torch.int32, device="cuda")
    if c["way"] == "backward":
        return [dh]
    return [loss, counts, P, tokens] + ([dh] if c["way"] == "step" else [])


def _quantize_exact(st):
    c = st["case"]
    K, G = c["K"], c["group"]
    out = torch.empty(st["w"].shape, dtype=torch.float64, device="cuda")
    scales = []
    for a in range(0, K, G):
        w = st["w"][..., a:a + G].double()
        top = w.abs().amax(-1) / 7
        step = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 7)   # one unit of the eighth bit
        s = (top / step).round() * step
        out[..., a:a + G] = torch.where(s[..., None] > 0, (w / s[..., None]).round(), 0.0).clamp(-7, 7) * s[..., None]
        scales.append(s)
    return [out, torch.stack(scales, dim=1)]


def _ffn_exact(st):
    """Group by group: a weight is an integer times its group's scale."""
    c = st["case"]
    G = c["group"]

    def unpack(q4, K):
        w = q4.view(torch.int32).to(torch.int64) & 0xFFFFFFFF                     # [R, blocks * 16]
        out = torch.empty(q4.shape[0], w.shape[1] // 16, 128, dtype=torch.float64, device="cuda")
        w = w.view(q4.shape[0], -1, 16)
        for t in range(4):
            for j in range(4):
                for i in range(4):
                    for odd in range(2):
                        out[:, :, 32 * j + 8 * t + 2 * i + odd] = ((w[:, :, 4 * t + j] >> (4 * i + 16 * odd)) & 15).double() - 8
        return out.view(q4.shape[0], -1)[:, :K]

    def product(x, w, e, b):
        q, y = unpack(w[0][e], x.shape[1]), 0.0
        for gi, a in enumerate(range(0, x.shape[1], G)):
            q[:, a:a + G] *= w[1][e, gi].double()[:, None]
        y = x @ q.t()
        return y if b is None else y + b[e].double()

    out, r0 = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda"), 0
    for e, n in enumerate(st["rows"]):
        if n:
            x = st["x"][r0:r0 + n].double()
            u = product(x, st["w1"], e, st["b1"])
            u = u * torch.sigmoid(u) * product(x, st["w3"], e, st["b3"]) if c["act"] == "swiglu" else torch.relu(u)
            out[r0:r0 + n] = product(u, st["w2"], e, st["b2"])
            r0 += n
    return out
