"""Cases of the operators with which the layer's router and weights learn.

  balance           balance_loss and its gradient: per-sequence balance loss of the router's
                    softmax with the per-expert counts, then the gradient of the logits
  route_backward    gradient of the gates and of the balance loss with respect to the logits
  combine_backward  gradient of the combine with respect to the gates and the experts' rows
  adamw             one AdamW step over many tensors, states in 32 or in 8 bits

``run`` computes each in elementary torch operations, or (``own``) through the framework's
calls.  All inputs are drawn on the GPU from the seed alone.
"""
import math

import torch

own = False

FP8_MAX = 448.0        # largest E4M3 value
BLOCK = 256            # elements per scale of an 8-bit state
FLOOR = 2.0 ** -100    # smallest block maximum a scale is made from
LR, BETAS, EPS, DECAY = 2e-5, (0.9, 0.95), 1e-8, 0.1


def listed():
    return [
        # the smallest layer of the workloads (256 tokens, 12 experts): launch latency
        dict(name="balance tiny", op="balance", T=256, E=12, K=2, S=1, mask=False, offset=False, tail=0),
        # a prefill-sized training batch as four sequences
        dict(name="balance 16k x 768", op="balance", T=16384, E=768, K=12, S=4, mask=False, offset=False, tail=0),
        # the skewed layer: ragged sequences (some empty), padding, rows behind the last, Zipf offset
        dict(name="balance ragged", op="balance", T=32767, E=384, K=8, S=29, mask=True, offset=True, tail=311),
        # gates only, fp32 gradient, the 4096-token layer
        dict(name="route_backward 4k x 96", op="route", T=4096, E=96, K=6, S=0, mask=False, offset=False, tail=0, out="fp32"),
        # gates and balance loss together at prefill, gradient in the type of the weight product
        dict(name="route_backward 16k x 768", op="route", T=16384, E=768, K=12, S=4, mask=False, offset=False, tail=0, out="bf16"),
        # odd counts: rows that are not 16-byte aligned, padding, ragged sequences
        dict(name="route_backward odd", op="route", T=1003, E=1021, K=9, S=5, mask=True, offset=True, tail=17, out="fp32"),
        # a decode-sized batch (64 tokens, 40% zero-expert picks)
        dict(name="combine_backward 64", op="combine", T=64, d=6144, K=12, zero=0.4, rows=True),
        # the prefill-sized batch, 30% zero-expert picks, rows' gradient for the experts
        dict(name="combine_backward 16k", op="combine", T=16384, d=6144, K=12, zero=0.3, rows=True),
        # frozen experts (only the router learns), odd token count
        dict(name="combine_backward frozen", op="combine", T=4093, d=2048, K=6, zero=0.33, rows=False),
        # the router's weight alone: bf16 weight with fp32 master and fp32 gradient
        dict(name="adamw router", op="adamw", n=768 * 6144, tensors=1, p="bf16", g="fp32", bits=32, master=True, clip=True),
        # many small ragged tensors, all fp32: launch latency
        dict(name="adamw 33 small", op="adamw", n=200_001, tensors=33, p="fp32", g="fp32", bits=32, master=False, clip=False),
        # the expert weights of the 4096-token layer, one tensor per expert and projection, 8-bit states
        dict(name="adamw experts 8 bits", op="adamw", n=192 * 2048 * 1024, tensors=192, p="bf16", g="bf16", bits=8, master=False, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "route", "combine", "adamw"])
    if op in ("balance", "route"):
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, min(32768, 16384 * 768 // E))
        c = dict(op=op, T=T, E=E, K=rng.randint(1, min(E, 16)), S=rng.choice([1, rng.randint(1, 64)]), mask=rng.random() < 0.5, offset=rng.random() < 0.5,
                 tail=rng.choice([0, T // rng.randint(2, 9)]))
        if op == "route":
            c["out"] = rng.choice(["fp32", "bf16"])
            c["S"] = rng.choice([0, c["S"]])
        return c
    if op == "combine":
        d = 8 * _log(rng, 8, 1024)
        K = rng.randint(1, 16)
        T = _log(rng, 1, min(32768, max(1, 16384 * 6144 * 12 // (d * K))))
        return dict(op=op, T=T, d=d, K=K, zero=round(rng.uniform(0, 0.6), 2), rows=rng.random() < 0.7)
    n = _log(rng, 1000, 192 * 2048 * 1024 // 2)
    p = rng.choice(["bf16", "fp32"])
    return dict(op=op, n=n, tensors=min(_log(rng, 1, 300), n), p=p, g=rng.choice(["bf16", "fp32"]), bits=rng.choice([8, 32]), master=p == "bf16" and rng.random() < 0.5,
                clip=rng.random() < 0.5)


def _dtype(name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def _bounds(T, S, tail):
    """S + 1 ragged offsets of sequences over the first T - tail tokens, every seventh sequence empty."""
    share = [0 if S > 6 and s % 7 == 3 else 1 + (s * 5) % 4 for s in range(S)]
    at, out = 0, [0]
    for s in share:
        at += s
        out.append((T - tail) * at // sum(share))
    return out


def _sizes(n, tensors):
    """Sizes of the tensors: even where the total divides, else ragged; n in all."""
    if n % tensors == 0:
        return [n // tensors] * tensors
    share = [1 + (7919 * i) % 29 for i in range(tensors)]
    ends = [0]
    for s in share:
        ends.append(ends[-1] + s)
    cut = [n * e // ends[-1] for e in ends]
    return [max(1, b - a) for a, b in zip(cut, cut[1:])]


def _quantise(x):
    """E4M3 values (as float8) and fp32 scales of x [blocks, BLOCK], one scale per block."""
    amax = x.abs().amax(1, keepdim=True).clamp(min=FLOOR)
    return (x * (FP8_MAX / amax)).to(torch.float8_e4m3fn), amax / FP8_MAX


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device=dev).normal_(0.0, std, generator=g)

    s = dict(case=case)
    op = case["op"]
    if op in ("balance", "route"):
        T, E, K, S = case["T"], case["E"], case["K"], case["S"]
        s["logits"] = normal(T, E, std=0.8)
        s["offset"] = -1.1 * torch.log(torch.randperm(E, generator=g, device=dev) + 1.0) if case["offset"] else None
        z = s["logits"] if s["offset"] is None else s["logits"] + s["offset"]
        p = torch.softmax(z, 1)
        bias = torch.empty(E, device=dev).uniform_(-1.0, 1.0, generator=g) / E
        s["idx"] = torch.topk(p + bias, K, dim=1).indices.to(torch.int32).contiguous()
        s["mask"] = torch.rand(T, generator=g, device=dev) < 0.9 if case["mask"] else None
        s["seq"] = torch.tensor(_bounds(T, S, case["tail"]), dtype=torch.int32, device=dev) if S else None
        s["dloss"] = torch.full((S,), 1e-2 / S, device=dev) if S else None
        if op == "route":
            s["dgate"] = normal(T, K, std=1e-3)
            s["dtype"] = _dtype(case["out"])
            s["coef"] = torch.rand(S, E, generator=g, device=dev) * (2.0 * S / T) if S else None
        return s
    if op == "combine":
        T, d, K = case["T"], case["d"], case["K"]
        P = max(1, round((1 - case["zero"]) * T * K))
        s["dout"] = normal(T, d, std=1e-2).to(torch.bfloat16)
        s["x"] = normal(T, d).to(torch.bfloat16)
        s["y"] = normal(P, d, std=0.1).to(torch.bfloat16)
        slot = torch.full((T * K,), -1, dtype=torch.int32, device=dev)
        slot[torch.randperm(T * K, generator=g, device=dev)[:P]] = torch.arange(P, dtype=torch.int32, device=dev)
        s["slot"] = slot.view(T, K)
        s["gate"] = torch.rand(T, K, generator=g, device=dev) * 0.1
        return s
    # adamw: every tensor starts a new block of the flat buffers; what pads them is zero
    sizes = _sizes(case["n"], case["tensors"])
    start, at = [], 0
    for n in sizes:
        start.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    s["p"] = normal(at, std=0.02)
    s["g"] = normal(at, std=1e-3)
    m, v = normal(at, std=3e-4), normal(at, std=1e-3)
    for o, n in zip(start, sizes):
        for t in (s["p"], s["g"], m, v):
            t[o + n:(o + n + BLOCK - 1) // BLOCK * BLOCK].zero_()
    s["master"] = s["p"] if case["master"] else None
    s["p"], s["g"] = s["p"].to(_dtype(case["p"])), s["g"].to(_dtype(case["g"]))
    if case["bits"] == 8:
        (mc, ms), (vc, vs) = _quantise(m.view(-1, BLOCK)), _quantise(v.abs_().view(-1, BLOCK))
        s["m"], s["ms"], s["v"], s["vs"] = mc.view(torch.uint8).view(-1), ms.view(-1), vc.view(torch.uint8).view(-1), vs.view(-1)
    else:
        s["m"], s["v"] = m, v.mul_(v)
    s["t"] = torch.tensor([1000], dtype=torch.int32, device=dev)
    s["clip"] = torch.tensor([0.37], device=dev) if case["clip"] else None
    if own:   # the optimiser object that a training program keeps, over its own tensors
        from mixture_experts_layer_28_b200 import moe_zc as mz

        def views(flat, per=1):
            return [flat[o // per:o // per + (n + per - 1) // per] for o, n in zip(start, sizes)]

        if case["bits"] == 8:
            states = [[mz.Moment8(c, f) for c, f in zip(views(s[k]), views(s[k + "s"], BLOCK))] for k in "mv"]
        else:
            states = [views(s["m"]), views(s["v"])]
        s["opt"] = mz.AdamW(views(s["p"]), LR, BETAS, EPS, DECAY, state_bits=case["bits"], exp_avg=states[0], exp_avg_sq=states[1],
                            master=views(s["master"]) if case["master"] else None, step=1000)
        s["grads"] = views(s["g"])
    return s


def _softmax(s):
    z = s["logits"] if s["offset"] is None else s["logits"] + s["offset"]
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _tokens(s):
    """Sequence of each token (S for the tokens of none) and which tokens count."""
    T, S = s["logits"].shape[0], s["case"]["S"]
    at = torch.arange(T, device=s["logits"].device, dtype=torch.int32)
    seq = torch.bucketize(at, s["seq"][1:].contiguous(), right=True)
    valid = seq < S
    return seq, valid if s["mask"] is None else valid & s["mask"]


def _plain_balance(s):
    S, E, K = s["case"]["S"], s["case"]["E"], s["case"]["K"]
    p = _softmax(s)
    seq, valid = _tokens(s)
    member = (seq[None, :] == torch.arange(S, device=p.device)[:, None]) & valid
    n = member.sum(1, dtype=torch.int32)[:, None].to(torch.float32)
    inv = torch.where(n > 0, 1.0 / n.clamp(min=1), 0.0)
    cell = (torch.where(valid, seq, S)[:, None] * E + s["idx"]).view(-1).long()
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=p.device).scatter_add_(0, cell, torch.ones_like(cell, dtype=torch.int32))[:S * E].view(S, E)
    prob = (member.to(torch.float32) @ p) * inv
    f = counts * (E / K) * inv
    c = _per_token(s, f * inv, seq, valid)
    return dict(loss=(f * prob).sum(1), counts=counts, prob=prob, coef=f * inv, dlogits=p * (c - (p * c).sum(1, keepdim=True)))


def _per_token(s, coef, seq, valid):
    """The loss's gradient by each probability: dloss coef of the token's sequence, 0 where the token does not count."""
    c = torch.cat([coef * s["dloss"][:, None], torch.zeros_like(coef[:1])])
    return c[torch.where(valid, seq, s["case"]["S"])]


def _plain_route(s):
    p = _softmax(s)
    a = torch.zeros_like(p).scatter_add_(1, s["idx"].long(), s["dgate"])
    if s["coef"] is not None:
        a = a + _per_token(s, s["coef"], *_tokens(s))
    out = p * (a - (p * a).sum(1, keepdim=True))
    if s["mask"] is not None:
        out = torch.where(s["mask"][:, None], out, 0.0)
    return dict(dlogits=out.to(s["dtype"]))


def _plain_combine(s):
    slot, d = s["slot"].long(), s["dout"].to(torch.float32)
    P = s["y"].shape[0]
    rows = torch.where((slot >= 0)[..., None], s["y"][slot.clamp(min=0)], s["x"][:, None, :])
    out = dict(dgate=(rows.to(torch.float32) * d[:, None, :]).sum(2))
    if s["case"]["rows"]:
        dy = torch.empty(P + 1, d.shape[1], dtype=torch.bfloat16, device=d.device)
        dy[torch.where(slot >= 0, slot, P)] = (s["gate"][..., None] * d[:, None, :]).to(torch.bfloat16)
        out["dy"] = dy[:P]
    return out


def _plain_adamw(s):
    b1, b2 = BETAS
    eight = s["case"]["bits"] == 8
    s["t"] += 1
    n = s["t"].to(torch.float64)
    g = s["g"].to(torch.float32)
    if s["clip"] is not None:
        g = g * s["clip"]
    if eight:
        m = s["m"].view(torch.float8_e4m3fn).view(-1, BLOCK).to(torch.float32) * s["ms"][:, None]
        v = s["v"].view(torch.float8_e4m3fn).view(-1, BLOCK).to(torch.float32) * s["vs"][:, None]
        v, g = v * v, g.view(-1, BLOCK)
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = torch.sqrt(v)
    p = s["master"] if s["master"] is not None else s["p"].to(torch.float32)
    p = p * (1 - LR * DECAY) - ((m / (r * torch.rsqrt(1 - b2 ** n) + EPS)) * (LR / (1 - b1 ** n))).view(-1)
    if s["master"] is not None:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if eight:
        (mc, ms), (vc, vs) = _quantise(m), _quantise(r)
        vc = vc.view(torch.uint8)
        vc = torch.where((r > 0) & (vc == 0), 1, vc)     # a positive root never gets the code of zero
        s["m"].copy_(mc.view(torch.uint8).view(-1)), s["v"].copy_(vc.view(-1))
        s["ms"].copy_(ms.view(-1)), s["vs"].copy_(vs.view(-1))
    else:
        s["m"].copy_(m), s["v"].copy_(v)


def _adamw_state(s):
    out = dict(p=s["p"], m=s["m"], v=s["v"])
    if s["case"]["bits"] == 8:     # the values that the codes stand for, in units of their block's scale
        out.update(m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), ms=s["ms"], vs=s["vs"])
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "adamw":
            _plain_adamw(s)
            return _adamw_state(s)
        return dict(balance=_plain_balance, route=_plain_route, combine=_plain_combine)[op](s)
    from mixture_experts_layer_28_b200 import moe_zc as mz
    if op == "balance":
        r = mz.balance_loss(s["logits"], s["idx"], logit_offset=s["offset"], mask=s["mask"], seq_start=s["seq"])
        dlogits = mz.route_backward(s["logits"], s["idx"], coef=r.coef, dloss=s["dloss"], logit_offset=s["offset"], mask=s["mask"], seq_start=s["seq"])
        return dict(loss=r.loss, counts=r.counts, prob=r.prob, coef=r.coef, dlogits=dlogits)
    if op == "route":
        return dict(dlogits=mz.route_backward(s["logits"], s["idx"], dgate=s["dgate"], coef=s["coef"], dloss=s["dloss"], logit_offset=s["offset"], mask=s["mask"],
                                              seq_start=s["seq"], dtype=s["dtype"]))
    if op == "combine":
        dgate, dy = mz.combine_backward(s["dout"], s["x"], s["y"], s["slot"], s["gate"], rows=s["case"]["rows"])
        return dict(dgate=dgate, dy=dy) if s["case"]["rows"] else dict(dgate=dgate)
    s["opt"].step(s["grads"], grad_scale=s["clip"])
    return _adamw_state(s)


def work(case):
    op = case["op"]
    if op == "combine":
        T, d, K = case["T"], case["d"], case["K"]
        P = max(1, round((1 - case["zero"]) * T * K))
        zero_rows = T if P < T * K else 0       # x is read only for zero-expert picks
        return dict(bytes=2 * d * (T + zero_rows + P * (2 if case["rows"] else 1)) + T * K * (12 if case["rows"] else 8),
                    flops=d * (2 * P + 2 * zero_rows + (P if case["rows"] else 0)))
    if op == "adamw":
        n = case["n"]
        size = {"fp32": 4, "bf16": 2}
        per = 2 * size[case["p"]] + size[case["g"]] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        if case["master"]:
            per += 8 - size[case["p"]]          # the weight itself is only written
        return dict(bytes=n * per, flops=16 * n)
    T, E, K, S = case["T"], case["E"], case["K"], case["S"]
    seen = T - case["tail"] if op == "balance" else T
    small = T * (1 if case["mask"] else 0) + 4 * (E if case["offset"] else 0) + 8 * S
    if op == "balance":     # both directions: the logits once, their gradient once
        return dict(bytes=4 * seen * (E + K) + 4 * T * E + small + S * (12 * E + 4), flops=10 * seen * E)
    return dict(bytes=T * E * (4 + (4 if case["out"] == "fp32" else 2)) + 8 * T * K + small + 4 * S * (E + 1), flops=8 * T * E)


# ---------------------------------------------------------------- in 64 bits, from the definitions


def _e4m3(x):
    """x >= 0 in units of the scale, rounded to the nearest E4M3 value (ties to even), in 64 bits."""
    _, e = torch.frexp(x)                                # x = f 2^e, f in [1/2, 1)
    step = torch.pow(2.0, (e.clamp(min=-5) - 4).to(torch.float64))
    return torch.round(x / step) * step


def _exact_sequences(case, s):
    """For each sequence the rows that count; and the rows of none."""
    on = torch.ones(case["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    edge = _bounds(case["T"], case["S"], case["tail"])
    return [a + torch.nonzero(on[a:b]).view(-1) for a, b in zip(edge, edge[1:])]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("balance", "route"):
        z = s["logits"].double()
        if s["offset"] is not None:
            z = z + s["offset"].double()
        p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    if op == "balance":
        E, K = case["E"], case["K"]
        loss, counts, prob, coef = [], [], [], []
        out = torch.zeros_like(p)
        for q, rows in enumerate(_exact_sequences(case, s)):
            n = rows.numel()
            c = torch.bincount(s["idx"][rows].long().view(-1), minlength=E).double()
            P = p[rows].sum(0) / max(n, 1)
            f = c * E / (K * max(n, 1))
            loss.append((f * P).sum()), counts.append(c.to(torch.int32)), prob.append(P), coef.append(f / max(n, 1))
            up = f * (s["dloss"][q].double() / max(n, 1))
            out[rows] = p[rows] * (up - (p[rows] @ up)[:, None])
        return dict(loss=torch.stack(loss), counts=torch.stack(counts), prob=torch.stack(prob), coef=torch.stack(coef), dlogits=out)
    if op == "route":
        # the derivative of sum_k dgate p[idx_k] + dloss sum_i coef_i p_i, term by term
        gate = torch.gather(p, 1, s["idx"].long()) * s["dgate"].double()
        out = -p * gate.sum(1, keepdim=True)
        for k in range(case["K"]):
            at = s["idx"][:, k:k + 1].long()
            out.scatter_add_(1, at, gate[:, k:k + 1])
        if case["S"]:
            for q, rows in enumerate(_exact_sequences(case, s)):
                c = s["coef"][q].double() * s["dloss"][q].double()
                out[rows] += p[rows] * (c - (p[rows] @ c)[:, None])
        if s["mask"] is not None:
            out[~s["mask"]] = 0.0
        return dict(dlogits=out)
    if op == "combine":
        d, x = s["dout"].double(), s["x"].double()
        dgate = torch.empty(s["slot"].shape, dtype=torch.float64, device="cuda")
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda") if case["rows"] else None
        for k in range(case["K"]):
            at = s["slot"][:, k].long()
            ffn = torch.nonzero(at >= 0).view(-1)
            dgate[:, k] = torch.einsum("td,td->t", d, x)
            dgate[ffn, k] = torch.einsum("td,td->t", d[ffn], s["y"][at[ffn]].double())
            if dy is not None:
                dy[at[ffn]] = d[ffn] * s["gate"][ffn, k].double()[:, None]
        return dict(dgate=dgate, dy=dy) if case["rows"] else dict(dgate=dgate)
    b1, b2 = BETAS
    eight = case["bits"] == 8
    g = s["g"].double() * (1.0 if s["clip"] is None else s["clip"].double())
    if eight:
        m = (s["m"].view(torch.float8_e4m3fn).double().view(-1, BLOCK) * s["ms"].double()[:, None]).view(-1)
        v = (s["v"].view(torch.float8_e4m3fn).double().view(-1, BLOCK) * s["vs"].double()[:, None]).view(-1).square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g.square()
    p = (s["master"] if s["master"] is not None else s["p"]).double()
    p = p - LR * DECAY * p - LR * (m / (1 - b1 ** 1001)) / ((v / (1 - b2 ** 1001)).sqrt() + EPS)
    out = dict(p=p, m=m, v=v)
    if s["master"] is not None:
        out["master"] = p
    if eight:
        for k, t in (("m", m.view(-1, BLOCK)), ("v", v.sqrt().view(-1, BLOCK))):
            scale = t.abs().amax(1, keepdim=True).clamp(min=FLOOR) / FP8_MAX
            q = _e4m3(t.abs() / scale)
            if k == "v":
                q = torch.where((t > 0) & (q == 0), 2.0 ** -9, q)
            out[k], out[k + "s"] = (torch.copysign(q, t)).view(-1), scale.view(-1)
    return out
