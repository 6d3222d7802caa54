"""The feed-forward, projection and distillation operators: cases, inputs and plain forms.

Three operators on the 4-bit group-symmetric weight
w[n, k] = (code[n, k] - 8) * scale[k / gs, n], each in its directions:

gated    the gated feed-forward block.  Forward: g = x Wg^T, u = x Wu^T,
         h = act(g) * u (fp16), with g and u saved in fp16 (column 2 j = g_j,
         2 j + 1 = u_j) where a backward pass will follow.  Backward:
         d_g = d_h u act'(g), d_u = d_h act(g), d_x = d_g Wg + d_u Wu.
linear   a projection with its epilogue.  Forward: z = x W^T + bias,
         y = act(z) + residual (fp16), z saved where a backward pass will
         follow.  Backward: d_z = d_y act'(z), d_x = d_z W,
         d_bias[n] = sum_m d_z[m, n].
distill  distillation from the teacher's top logits at temperature T.  With
         q = softmax over the k teacher logits / T and lse the log-sum-exp of
         the student's row / T:  loss = T^2 sum_j q_j (log q_j - z[i_j] / T + lse),
         d_z[i] = d_loss T (exp(z[i] / T - lse) - sum of q_j with i_j = i).
         An entry with index -1 is padding; a row of padding alone has loss 0
         and gradient 0.

The plain forms below use elementary torch operations in 32 bits, rounded once
at the end.
"""
import math

import torch

own = False

_ACTS = ("silu", "gelu_tanh")


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token through the gated block of the 1B-class layer (hidden 2048, MLP 8192): decode latency
        dict(name="gated_fwd_1", op="gated", dir="fwd", M=1, K=2048, F=8192, gs=32, f32s=False, act="silu", save=False),
        # a decode batch of 16 sequences through the 8B-class layer's gated block
        dict(name="gated_fwd_16", op="gated", dir="fwd", M=16, K=4096, F=14336, gs=128, f32s=False, act="silu", save=False),
        # the adapter-training step's 512 tokens, with g and u saved for the backward pass
        dict(name="gated_fwd_512", op="gated", dir="fwd", M=512, K=2048, F=8192, gs=32, f32s=False, act="gelu_tanh", save=True),
        # a long prompt through the 8B-class gated block
        dict(name="gated_fwd_4096", op="gated", dir="fwd", M=4096, K=4096, F=14336, gs=128, f32s=False, act="silu", save=False),
        # the input gradient of the same training step
        dict(name="gated_bwd_512", op="gated", dir="bwd", M=512, K=2048, F=8192, gs=32, f32s=False, act="gelu_tanh", save=True),
        # a ragged micro-batch of the 8B-class layer, fp32 scales
        dict(name="gated_bwd_1021", op="gated", dir="bwd", M=1021, K=4096, F=14336, gs=128, f32s=True, act="silu", save=True),
        # one token's down projection added to the residual stream: decode latency
        dict(name="linear_fwd_1", op="linear", dir="fwd", M=1, K=8192, N=2048, gs=32, f32s=False, act="none", bias=False, residual=True, save=False),
        # a 508-token prompt's down projection with bias and residual
        dict(name="linear_fwd_508", op="linear", dir="fwd", M=508, K=8192, N=2048, gs=32, f32s=False, act="none", bias=True, residual=True, save=False),
        # input and bias gradients of an up projection with bias and activation
        dict(name="linear_bwd_256", op="linear", dir="bwd", M=256, K=4096, N=14336, gs=128, f32s=False, act="gelu_tanh", bias=True, residual=False, save=True),
        # loss and gradient of the adapter-training step over a 32000-token vocabulary
        dict(name="distill_step_512", op="distill", dir="step", M=512, V=32000, k=64, T=2.0, logits="float32", teacher="float16", pad=True),
        # loss of a held-out sequence over the largest vocabulary
        dict(name="distill_fwd_37", op="distill", dir="fwd", M=37, V=262144, k=20, T=1.0, logits="float32", teacher="float32", pad=False),
        # gradient from a saved log-sum-exp, half-precision logits of a large batch
        dict(name="distill_bwd_2048", op="distill", dir="bwd", M=2048, V=32000, k=100, T=1.5, logits="float16", teacher="float16", pad=True),
    ]


_MOST_FLOPS = 2 * 4096 * 4096 * 2 * 14336
_MOST_WEIGHTS = 2 * 14336 * 4096
_MOST_LOGITS = 2048 * 32000


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "linear", "distill"))
    if op == "distill":
        V = 8 * _spread(rng, 8, 32768)
        M = max(1, min(_spread(rng, 1, 4096), _MOST_LOGITS // V))
        return dict(op=op, dir=rng.choice(("fwd", "bwd", "step")), M=M, V=V, k=min(V, _spread(rng, 1, 512)),
                    T=round(rng.uniform(0.5, 4.0), 3), logits=rng.choice(("float32", "float16")),
                    teacher=rng.choice(("float32", "float16")), pad=rng.random() < 0.5)
    K = 64 * _spread(rng, 1, 224)
    wide = 8 * _spread(rng, 1, 1792)
    groups = [g for g in (16, 32, 64, 128, 256, 512, 1024) if K % g == 0]
    rows = 2 * wide if op == "gated" else wide
    while rows * K > _MOST_WEIGHTS:
        K = max(64, K // 2 // 64 * 64)
        groups = [g for g in groups if K % g == 0]
    M = max(1, min(_spread(rng, 1, 4096), _MOST_FLOPS // (2 * rows * K)))
    c = dict(op=op, dir=rng.choice(("fwd", "bwd")), M=M, K=K)
    c["F" if op == "gated" else "N"] = wide
    c.update(gs=rng.choice(groups), f32s=rng.random() < 0.3)
    if op == "gated":
        c.update(act=rng.choice(_ACTS), save=rng.random() < 0.5)
    else:
        c.update(act=rng.choice(("none",) + _ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                 save=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _normal(g, shape, sigma, dtype=torch.float16):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, sigma, generator=g).to(dtype)


def _weight(g, N, K, gs, f32s):
    codes = torch.randint(0, 16, (N, K), device="cuda", dtype=torch.uint8, generator=g)
    s = torch.empty((K // gs, N), device="cuda").uniform_(0.005, 0.02, generator=g)
    return codes, s if f32s else s.half()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    M = case["M"]
    if case["op"] == "distill":
        V, k = case["V"], case["k"]
        ldt, tdt = getattr(torch, case["logits"]), getattr(torch, case["teacher"])
        z = _normal(g, (M, V), 3.0, torch.float32)
        # the teacher's top ids are distinct in a row, and the student leans towards them
        step = torch.randint(1, max(2, V // k), (M, 1), device="cuda", generator=g)
        first = torch.randint(0, V, (M, 1), device="cuda", generator=g)
        idx = (first + step * torch.arange(k, device="cuda")) % V
        t = _normal(g, (M, k), 2.0, torch.float32).sort(1, descending=True).values + 8.0
        z.scatter_(1, idx, t - 3.0 + _normal(g, (M, k), 1.0, torch.float32))
        idx = idx.int()
        if case["pad"]:   # shorter lists, padded with index -1 and whatever stands there; some rows are padding alone
            n = torch.randint(0, k + 1, (M, 1), device="cuda", generator=g)
            off = torch.arange(k, device="cuda") >= n
            idx = idx.masked_fill(off, -1)
            t = t.masked_fill(off, float("nan"))
        s.update(logits=z.to(ldt), idx=idx.contiguous(), teacher=t.to(tdt).contiguous())
        s["d_loss"] = torch.empty(M, device="cuda").uniform_(0.5, 1.5, generator=g) * (64.0 / M)
        if case["dir"] == "bwd":
            s["lse"] = torch.logsumexp(s["logits"].double() / case["T"], 1).float()
        return s
    K, gs = case["K"], case["gs"]
    if case["op"] == "gated":
        F = case["F"]
        s["gate"], s["up"] = _weight(g, F, K, gs, case["f32s"]), _weight(g, F, K, gs, case["f32s"])
        if case["dir"] == "fwd":
            s["x"] = _normal(g, (M, K), 1.0)
        else:
            s["gu"] = _normal(g, (M, 2 * F), 2.0)
            s["d_h"] = _normal(g, (M, F), 1e-2)
    else:
        N = case["N"]
        s["w"] = _weight(g, N, K, gs, case["f32s"])
        s["bias"] = _normal(g, (N,), 0.5) if case["bias"] else None
        if case["dir"] == "fwd":
            s["x"] = _normal(g, (M, K), 1.0)
            s["residual"] = _normal(g, (M, N), 1.0) if case["residual"] else None
        else:
            s["d_y"] = _normal(g, (M, N), 1e-2)
            s["z"] = _normal(g, (M, N), 2.0) if case["act"] != "none" else None
    if own:   # the packed weight: laid out once, kept by the program
        import bit_group_quantized_q4gsw_b200 as q
        if case["op"] == "gated":
            s["packed"] = q.q4gsw_prepack_gated(*s["gate"], *s["up"], gs)
        else:
            s["packed"] = q.q4gsw_prepack(*s["w"], gs)
    return s


# ---------------------------------------------------------------- plain forms
def _dequant(weight, gs):
    codes, scales = weight
    N, K = codes.shape
    w = (codes.float() - 8.0).view(N, K // gs, gs) * scales.float().t().unsqueeze(2)
    return w.view(N, K)


def _act(z, act):
    """(act(z), act'(z)) in fp32."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    v = c * (z + 0.044715 * z * z * z)
    s = 1.0 / (1.0 + torch.exp(-2.0 * v))     # 0.5 (1 + tanh v)
    return z * s, s + z * s * (1.0 - s) * 2.0 * c * (1.0 + 3.0 * 0.044715 * z * z)


def _gated_plain(s, c):
    wg, wu = _dequant(s["gate"], c["gs"]), _dequant(s["up"], c["gs"])
    if c["dir"] == "fwd":
        x = s["x"].float()
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(g, c["act"])[0] * u).half()
        return (h, torch.stack((g, u), 2).flatten(1).half()) if c["save"] else h
    gu, d_h = s["gu"].float(), s["d_h"].float()
    g, u = gu[:, 0::2], gu[:, 1::2]
    a, da = _act(g, c["act"])
    d_g, d_u = d_h * u * da, d_h * a
    return (d_g @ wg + d_u @ wu).half(), torch.stack((d_g, d_u), 2).flatten(1).half()


def _linear_plain(s, c):
    w = _dequant(s["w"], c["gs"])
    if c["dir"] == "fwd":
        z = s["x"].float() @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.half(), z.half()) if c["save"] else y.half()
    d_z = s["d_y"].float()
    if c["act"] != "none":
        d_z = d_z * _act(s["z"].float(), c["act"])[1]
    out = [(d_z @ w).half()]
    if c["act"] != "none":
        out.append(d_z.half())
    if c["bias"]:
        out.append(d_z.sum(0))
    return out


def _distill_plain(s, c):
    T = c["T"]
    z, t, idx = s["logits"].float() / T, s["teacher"].float() / T, s["idx"].long()
    valid = idx >= 0
    some = valid.any(1)
    at = idx.clamp_min(0)
    t = torch.where(valid, t, torch.full_like(t, float("-inf")))
    top = torch.where(some, t.max(1).values, torch.zeros_like(t[:, 0])).unsqueeze(1)
    e = torch.exp(t - top)
    total = e.sum(1, keepdim=True)
    q = torch.where(some.unsqueeze(1), e / total, torch.zeros_like(e))
    if c["dir"] == "bwd":
        lse = s["lse"].unsqueeze(1)
    else:
        m = z.max(1, keepdim=True).values
        lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
        log_q = t - top - torch.log(total)
        term = torch.where(q > 0, q * (log_q - z.gather(1, at) + lse), torch.zeros_like(q))
        loss = T * T * term.sum(1)
        if c["dir"] == "fwd":
            return loss, lse.squeeze(1)
    d = torch.exp(z - lse)
    d.scatter_add_(1, at, -q)
    d = torch.where(some.unsqueeze(1), d * (T * s["d_loss"]).unsqueeze(1), torch.zeros_like(d)).half()
    return d if c["dir"] == "bwd" else (loss, lse.squeeze(1), d)


def run(s):
    c = s["case"]
    if not own:
        return {"gated": _gated_plain, "linear": _linear_plain, "distill": _distill_plain}[c["op"]](s, c)
    import bit_group_quantized_q4gsw_b200 as q
    if c["op"] == "gated":
        if c["dir"] == "fwd":
            return q.q4gsw_gated_fwd(s["packed"], c["F"], c["K"], c["gs"], s["x"], act=c["act"], save_gu=c["save"],
                                     f32s=c["f32s"])
        return q.q4gsw_gated_bwd(s["packed"], c["F"], c["K"], c["gs"], s["gu"], s["d_h"], act=c["act"], f32s=c["f32s"])
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            return q.q4gsw_linear_act_fwd(s["packed"], c["N"], c["K"], c["gs"], s["x"], bias=s["bias"], act=c["act"],
                                          residual=s["residual"], save_z=c["save"], f32s=c["f32s"])
        out = q.q4gsw_linear_act_bwd(s["packed"], c["N"], c["K"], c["gs"], s["d_y"], z=s["z"], act=c["act"],
                                     want_bias=c["bias"], f32s=c["f32s"])
        return [v for v in out if v is not None]
    if c["dir"] == "fwd":
        return q.q4gsw_distill_fwd(s["logits"], s["idx"], s["teacher"], temperature=c["T"])
    if c["dir"] == "bwd":
        return q.q4gsw_distill_bwd(s["logits"], s["lse"], s["idx"], s["teacher"], s["d_loss"], temperature=c["T"])
    return q.q4gsw_distill_step(s["logits"], s["idx"], s["teacher"], s["d_loss"], temperature=c["T"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    M = case["M"]
    if case["op"] == "distill":
        V, k = case["V"], case["k"]
        z = 2 if case["logits"] == "float16" else 4
        t = 2 if case["teacher"] == "float16" else 4
        n = M * V * z + M * k * (4 + t)
        if case["dir"] != "bwd":
            n += 8 * M                       # loss and log-sum-exp
        else:
            n += 4 * M                       # the saved log-sum-exp
        if case["dir"] != "fwd":
            n += 4 * M + 2 * M * V           # d_loss, the fp16 gradient
        per = {"fwd": 4, "bwd": 4, "step": 8}[case["dir"]]
        return {"bytes": n, "flops": per * M * V}
    K = case["K"]
    rows = 2 * case["F"] if case["op"] == "gated" else case["N"]
    n = rows * K // 2 + (4 if case["f32s"] else 2) * rows * K // case["gs"]
    n += 2 * M * K                           # x, or d_x
    wide = case["F"] if case["op"] == "gated" else case["N"]
    if case["op"] == "gated":
        n += 2 * M * wide                    # h, or d_h
        if case["dir"] == "bwd":
            n += 2 * 2 * M * 2 * wide        # g and u read, their gradients written
        elif case["save"]:
            n += 2 * M * 2 * wide
    else:
        n += 2 * M * wide                    # y, or d_y
        if case["dir"] == "fwd":
            n += (2 * wide if case["bias"] else 0) + (2 * M * wide if case["residual"] else 0)
            n += 2 * M * wide if case["save"] else 0
        else:
            n += 2 * 2 * M * wide if case["act"] != "none" else 0
            n += 4 * wide if case["bias"] else 0
    return {"bytes": n, "flops": 2 * M * rows * K}


# ---------------------------------------------------------------- from the definition, in 64 bits
def _wide(weight, gs):
    codes, scales = weight
    s = torch.repeat_interleave(scales.double(), gs, dim=0)        # [K, N]
    return codes.double().sub_(8.0).mul_(s.t())


def _act64(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _slope64(z, act):
    if act == "silu":
        e = torch.exp(-z)
        return 1 / (1 + e) + z * e / (1 + e) ** 2
    if act == "gelu_tanh":
        b = math.sqrt(2 / math.pi)
        th = torch.tanh(b * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * b * (1 + 0.134145 * z * z)
    return torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    act = case.get("act")
    if case["op"] == "gated":
        wg, wu = _wide(s["gate"], case["gs"]), _wide(s["up"], case["gs"])
        if case["dir"] == "fwd":
            x = s["x"].double()
            g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            h = _act64(g, act) * u
            if not case["save"]:
                return h
            gu = torch.empty((g.shape[0], 2 * g.shape[1]), device=g.device, dtype=torch.float64)
            gu[:, 0::2], gu[:, 1::2] = g, u
            return h, gu
        g, u, d_h = s["gu"][:, 0::2].double(), s["gu"][:, 1::2].double(), s["d_h"].double()
        d_gu = torch.empty(s["gu"].shape, device=g.device, dtype=torch.float64)
        d_gu[:, 0::2] = d_h * u * _slope64(g, act)
        d_gu[:, 1::2] = d_h * _act64(g, act)
        return torch.mm(d_gu[:, 0::2], wg) + torch.mm(d_gu[:, 1::2], wu), d_gu
    if case["op"] == "linear":
        w = _wide(s["w"], case["gs"])
        if case["dir"] == "fwd":
            z = torch.mm(s["x"].double(), w.t())
            if s["bias"] is not None:
                z = z + s["bias"].double()
            y = _act64(z, act)
            if s["residual"] is not None:
                y = y + s["residual"].double()
            return (y, z) if case["save"] else y
        d_z = s["d_y"].double()
        if s["z"] is not None:
            d_z = d_z * _slope64(s["z"].double(), act)
        out = [torch.mm(d_z, w)]
        if s["z"] is not None:
            out.append(d_z)
        if case["bias"]:
            out.append(torch.mv(d_z.t(), torch.ones(d_z.shape[0], device=d_z.device, dtype=torch.float64)))
        return out
    T = case["T"]
    M = case["M"]
    loss, lse_all, grads = [], [], []
    for m in range(0, M, 128):      # rows in parts: 64-bit rows of a large vocabulary
        z = s["logits"][m:m + 128].double() / T
        idx = s["idx"][m:m + 128].long()
        keep = idx >= 0
        t = (s["teacher"][m:m + 128].double() / T).masked_fill(~keep, -math.inf)
        log_q = torch.log_softmax(t, 1)            # a row of padding alone: NaN, replaced below
        q = log_q.exp().masked_fill(~keep, 0.0)
        lse = torch.logsumexp(z, 1)
        has = keep.sum(1) > 0
        at = idx.masked_fill(~keep, 0)
        kl = (q * (log_q - (z.gather(1, at) - lse[:, None]))).masked_fill(q == 0, 0.0).masked_fill(~keep, 0.0)
        loss.append(torch.where(has, kl.sum(1) * T * T, torch.zeros_like(lse)))
        lse_all.append(lse)
        if case["dir"] != "fwd":
            d = torch.softmax(z, 1)
            if case["dir"] == "bwd":               # from the log-sum-exp as it was saved
                d = torch.exp(z - s["lse"][m:m + 128, None].double())
            d = d.scatter_add(1, at, -q)
            d = d * s["d_loss"][m:m + 128, None].double() * T
            grads.append(d.masked_fill(~has[:, None], 0.0))
    if case["dir"] == "fwd":
        return torch.cat(loss), torch.cat(lse_all)
    if case["dir"] == "bwd":
        return torch.cat(grads)
    return torch.cat(loss), torch.cat(lse_all), torch.cat(grads)
