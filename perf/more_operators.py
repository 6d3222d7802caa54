"""Adapters of many requests, the norms around a block and the gradients' clip: cases, inputs and plain forms.

Three operators around the 4-bit group-symmetric weight
w[n, k] = (code[n, k] - 8) * scale[k / gs, n], for serving many low-rank adapters on one frozen base and for
training them:

adapters  L low-rank adapters (A_a [r, K], B_a [N, r], factor s_a) beside one projection; token m has adapter
          a = ids[m], or none (-1).  Forward: u = x A_a^T, y = x W^T + bias + residual + s_a u B_a^T (fp16).
          Backward: v = s_a d_y B_a, d_x = d_y W + v A_a (fp16), and per adapter over its own tokens
          d_A_a = v^T x, d_B_a = s_a d_y^T u (fp32; zero for an adapter without tokens).
norms     what stands between two blocks: n = block * rsqrt(mean(block^2) + eps) * (o + w_post),
          h' = f h + gate * n (fp16), x = h' * rsqrt(mean(h'^2) + eps) * (o + w_pre) (fp16), with the post norm and
          the gate each left out where there is none.  Backward: the gradients of h, block and gate and, where they
          are trained, of the two weights (fp32 sums over the rows).
grads     the global norm over a list of gradients, and clipping: norm = |inv_scale g|, and
          out = inv_scale min(1, max_norm / (norm + 1e-6)) g (fp32).

The plain forms below use elementary torch operations in 32 bits (64 for the norm's long sum), rounded once at
the end.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request through the 1B-class up projection (hidden 2048, MLP 8192): decode latency
        dict(name="adapters_fwd_1", op="adapters", dir="fwd", M=1, K=2048, N=8192, gs=32, f32s=False, L=4, r=16,
             requests=1, scattered=False, none=False, bias=False, residual=False, save=False),
        # a decode batch of 16 requests, most with an adapter of their own, through the 8B-class down projection
        dict(name="adapters_fwd_16", op="adapters", dir="fwd", M=16, K=14336, N=4096, gs=128, f32s=False, L=32, r=16,
             requests=16, scattered=False, none=True, bias=False, residual=True, save=False),
        # the adapter-training step's 512 tokens, ragged sequences of 8 adapters, u saved for the backward pass
        dict(name="adapters_fwd_512", op="adapters", dir="fwd", M=512, K=2048, N=8192, gs=32, f32s=False, L=8, r=16,
             requests=8, scattered=False, none=False, bias=False, residual=False, save=True),
        # long prompts of 24 requests over 16 adapters of the largest rank, 8B-class
        dict(name="adapters_fwd_4096", op="adapters", dir="fwd", M=4096, K=4096, N=14336, gs=128, f32s=False, L=16, r=64,
             requests=24, scattered=False, none=True, bias=False, residual=False, save=False),
        # input, A and B gradients of the training step's down projection
        dict(name="adapters_bwd_512", op="adapters", dir="bwd", M=512, K=8192, N=2048, gs=32, f32s=False, L=8, r=16,
             requests=8, scattered=False, none=False, bias=False, residual=False, save=True),
        # a ragged micro-batch of the 8B-class layer whose tokens stand in no order, fp32 scales
        dict(name="adapters_bwd_1021", op="adapters", dir="bwd", M=1021, K=4096, N=14336, gs=128, f32s=True, L=4, r=64,
             requests=9, scattered=True, none=True, bias=False, residual=False, save=True),
        # one token between two blocks of the 1B-class layer: decode latency
        dict(name="norms_fwd_1", op="norms", dir="fwd", M=1, D=2048, post=True, gate="none", pre=True, weights=False),
        # a long prompt between two blocks of the 8B-class layer
        dict(name="norms_fwd_4096", op="norms", dir="fwd", M=4096, D=4096, post=True, gate="feature", pre=True,
             weights=False),
        # the training step's 512 tokens, norm weights and gate trained
        dict(name="norms_bwd_512", op="norms", dir="bwd", M=512, D=2048, post=True, gate="feature", pre=True,
             weights=True),
        # a ragged micro-batch with frozen norm weights and a gate of its own for every token
        dict(name="norms_bwd_1021", op="norms", dir="bwd", M=1021, D=4096, post=True, gate="token", pre=True,
             weights=False),
        # the gradients of rank-16 adapters on every projection of a 16-layer 1B-class model: 224 tensors
        dict(name="grads_clip_224", op="grads", dir="clip", count=224, total=11272192, half=0.0, packed=False,
             max_norm=1.0, scale=1.0),
        # the norm over a large unfrozen part, half of it fp16 under a loss scale, views without padding
        dict(name="grads_norm_61", op="grads", dir="norm", count=61, total=201326597, half=0.5, packed=True,
             max_norm=1.0, scale=1024.0),
    ]


_MOST_FLOPS = 2 * 4096 * 4096 * 14336
_MOST_WEIGHTS = 14336 * 4096
_MOST_RANKS = 4096 * 16 * 64      # tokens times ranks of all adapters
_MOST_NORMS = 4096 * 4096
_MOST_GRADS = 201326597


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adapters", "norms", "grads"))
    if op == "norms":
        D = 8 * _spread(rng, 8, 2048)
        M = max(1, min(_spread(rng, 1, 16384), _MOST_NORMS // D))
        kind = rng.choice(("whole", "whole", "pre", "add"))     # both norms, the pre norm alone, the sum alone
        return dict(op=op, dir=rng.choice(("fwd", "bwd")), M=M, D=D, post=kind == "whole" and rng.random() < 0.7,
                    gate="none" if kind == "pre" else rng.choice(("none", "feature", "token")), pre=kind != "add",
                    weights=rng.random() < 0.5, block=kind != "pre")
    if op == "grads":
        count = _spread(rng, 1, 512)
        return dict(op=op, dir=rng.choice(("norm", "clip")), count=count, total=max(count, _spread(rng, 1000, _MOST_GRADS // 4)),
                    half=rng.choice((0.0, 0.0, 0.5, 1.0)), packed=rng.random() < 0.4,
                    max_norm=rng.choice((0.5, 1.0, 1e6)), scale=rng.choice((1.0, 1024.0)))
    K = 64 * _spread(rng, 1, 224)
    N = 8 * _spread(rng, 1, 1792)
    groups = [g for g in (16, 32, 64, 128, 256, 512, 1024) if K % g == 0]
    while N * K > _MOST_WEIGHTS:
        K = max(64, K // 2 // 64 * 64)
        groups = [g for g in groups if K % g == 0]
    L, r = _spread(rng, 1, 64), 8 * rng.randint(1, 8)
    M = max(1, min(_spread(rng, 1, 4096), _MOST_FLOPS // (2 * N * K), _MOST_RANKS // (L * r)))
    return dict(op=op, dir=rng.choice(("fwd", "bwd")), M=M, K=K, N=N, gs=rng.choice(groups), f32s=rng.random() < 0.3,
                L=L, r=r, requests=min(M, _spread(rng, 1, 64)), scattered=rng.random() < 0.4, none=rng.random() < 0.5,
                bias=rng.random() < 0.4, residual=rng.random() < 0.4, save=rng.random() < 0.5)


def _sizes(case):
    """The sizes of a list of gradients: ragged, each at least one, their sum the case's total."""
    count, total = case["count"], case["total"]
    if (count, total) == (224, 11272192):      # A [16, K] and B [N, 16] of q, k, v, o, gate, up and down, 16 layers
        nk = ((2048, 2048), (512, 2048), (512, 2048), (2048, 2048), (8192, 2048), (8192, 2048), (2048, 8192))
        return [16 * v for n, k in nk for v in (k, n)] * 16
    w = np.random.RandomState(count * 7 + total % 9973).lognormal(0.0, 1.2, count)
    s = np.maximum(1, np.floor(w / w.sum() * (total - count))).astype(np.int64)
    s[int(np.argmax(s))] += total - int(s.sum())
    return [int(v) for v in s]


def _halves(case):
    """Which of the gradients are fp16."""
    n = int(round(case["half"] * case["count"]))
    return [i < n for i in range(case["count"])]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _normal(g, shape, sigma, dtype=torch.float16):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, sigma, generator=g).to(dtype)


def _owners(case):
    """The adapter of each request, -1 for none."""
    return [-1 if case["none"] and i % 4 == 3 else i * 5 % case["L"] if case["L"] % 5 else i % case["L"]
            for i in range(case["requests"])]


def _ids(case, seed):
    """The adapter of each token: ragged runs of the requests' tokens, or the same tokens in no order."""
    M, n = case["M"], case["requests"]
    rng = np.random.RandomState(seed % (1 << 31))
    cuts = np.sort(rng.choice(M - 1, n - 1, replace=False)) + 1 if n > 1 else np.zeros(0, np.int64)
    length = np.diff(np.concatenate([[0], cuts, [M]]))
    ids = np.repeat(np.array(_owners(case), np.int32), length)
    return rng.permutation(ids) if case["scattered"] else ids


def _prepare_adapters(s, case, g, seed):
    M, K, N, gs, L, r = (case[k] for k in ("M", "K", "N", "gs", "L", "r"))
    codes = torch.randint(0, 16, (N, K), device="cuda", dtype=torch.uint8, generator=g)
    scales = torch.empty((K // gs, N), device="cuda").uniform_(0.005, 0.02, generator=g)
    s["w"] = (codes, scales if case["f32s"] else scales.half())
    s["a"], s["b"] = _normal(g, (L, r, K), 0.05), _normal(g, (L, N, r), 0.05)
    s["scale"] = torch.empty(L, device="cuda").uniform_(0.5, 2.0, generator=g)
    s["ids"] = torch.from_numpy(_ids(case, seed)).cuda()
    s["x"] = _normal(g, (M, K), 1.0)
    if case["dir"] == "fwd":
        s["bias"] = _normal(g, (N,), 0.5) if case["bias"] else None
        s["residual"] = _normal(g, (M, N), 1.0) if case["residual"] else None
    else:
        s["d_y"] = _normal(g, (M, N), 1e-2)
        s["u"] = _normal(g, (M, r), 0.05 * math.sqrt(K), torch.float32) * (s["ids"] >= 0)[:, None]   # as the forward saves it
    if own:   # the packed weight, laid out once, and the batch's plan, made once for all projections of all layers
        import bit_group_quantized_q4gsw_b200 as q
        s["packed"] = q.q4gsw_prepack(*s["w"], gs)
        s["plan"] = q.q4gsw_adapters_plan(s["ids"], L)


def _prepare_norms(s, case, g):
    M, D = case["M"], case["D"]
    block = case.get("block", True)
    s["offset"], s["factor"], s["eps"] = 1.0, 0.75, 1e-6
    s["h"] = _normal(g, (M, D), 3.0)
    s["block"] = _normal(g, (M, D), 0.5) if block else None
    s["w_post"] = _normal(g, (D,), 0.3) if case["post"] else None
    s["w_pre"] = _normal(g, (D,), 0.3) if case["pre"] else None
    s["gate"] = {"none": None, "feature": _normal(g, (D,), 0.5), "token": _normal(g, (M, D), 0.5)}[case["gate"]]
    if case["dir"] == "bwd":
        s["h_out"] = _stream_plain(s)[0].half()      # as the forward leaves it
        s["d_x"] = _normal(g, (M, D), 1e-2) if case["pre"] else None
        s["d_h"] = _normal(g, (M, D), 1e-2)


def _prepare_grads(s, case, g):
    sizes, halves = _sizes(case), _halves(case)
    s["flat"], s["grads"], s["outs"], s["out"] = [], [], [], []
    for half in (False, True):
        dtype = torch.float16 if half else torch.float32
        mine = [n for n, f in zip(sizes, halves) if f == half]
        step = 1 if case["packed"] else 8
        starts = np.concatenate([[0], np.cumsum([-(-n // step) * step for n in mine])]).astype(np.int64)
        if not mine:
            continue
        flat = torch.zeros(int(starts[-1]), device="cuda", dtype=dtype)
        out = torch.zeros(int(starts[-1]) if case["dir"] == "clip" else 0, device="cuda", dtype=torch.float32)
        if case["packed"]:
            flat.copy_(_normal(g, flat.shape, 1e-2 * case["scale"], torch.float32))
        for a, n in zip(starts, mine):
            v = flat[int(a):int(a) + n]
            if not case["packed"]:
                v.normal_(0.0, 1e-2 * case["scale"], generator=g)
            s["grads"].append(v)
            s["outs"].append(out[int(a):int(a) + n])
        s["flat"].append(flat)
        s["out"].append(out)
    if own:   # the list's table on the device: made once for buffers that the program keeps
        import bit_group_quantized_q4gsw_b200 as q
        s["set"] = q.q4gsw_grad_set(s["grads"], s["outs"] if case["dir"] == "clip" else None)


def prepare(case, seed):
    s, g = dict(case=case), _gen(seed)
    if case["op"] == "adapters":
        _prepare_adapters(s, case, g, seed)
    elif case["op"] == "norms":
        _prepare_norms(s, case, g)
    else:
        _prepare_grads(s, case, g)
    return s


# ---------------------------------------------------------------- plain forms
def _dequant(weight, gs):
    codes, scales = weight
    N, K = codes.shape
    w = (codes.float() - 8.0).view(N, K // gs, gs) * scales.float().t().unsqueeze(2)
    return w.view(N, K)


def _adapters_plain(s, c):
    L, r, M = c["L"], c["r"], c["M"]
    w, x = _dequant(s["w"], c["gs"]), s["x"].float()
    a = s["a"].float().view(L * r, -1)                                   # all adapters' rows, one under another
    b = s["b"].float().permute(1, 0, 2).reshape(-1, L * r)
    # token m keeps the r of the L r columns that are its adapter's
    mine = (s["ids"].unsqueeze(1) == torch.arange(L, device="cuda")).float()     # [M, L]
    if c["dir"] == "fwd":
        u = ((x @ a.t()).view(M, L, r) * mine.unsqueeze(2))
        y = x @ w.t() + (u * s["scale"].view(1, L, 1)).view(M, L * r) @ b.t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.half(), u.sum(1)) if c["save"] else y.half()
    d_y = s["d_y"].float()
    factor = (mine * s["scale"]).unsqueeze(2)                            # [M, L, 1]
    v = ((d_y @ b).view(M, L, r) * factor).view(M, L * r)
    d_x = d_y @ w + v @ a
    d_a = (v.t() @ x).view(L, r, -1)
    d_b = ((s["u"].unsqueeze(1) * factor).view(M, L * r).t() @ d_y).view(L, r, -1).transpose(1, 2).contiguous()
    return d_x.half(), d_a, d_b


def _rms(v, eps):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + eps)


def _stream_plain(s):
    """(h', block's norm before its weight and gate) in fp32."""
    h = s["factor"] * s["h"].float()
    if s["block"] is None:
        return h, None
    n = s["block"].float()
    if s["w_post"] is not None:
        n = n * _rms(n, s["eps"]) * (s["offset"] + s["w_post"].float())
    return h + (n if s["gate"] is None else s["gate"].float() * n), n


def _norm_slope(v, w, d, eps):
    """Gradients of v and of the weight through v * rsqrt(mean(v^2) + eps) * w."""
    k = _rms(v, eps)
    e = d * w
    return k * e - v * (k * k * k) * (e * v).mean(1, keepdim=True), d * v * k


def _norms_plain(s, c):
    if c["dir"] == "fwd":
        h = _stream_plain(s)[0]
        if not c["pre"]:
            return h.half()
        x = h * _rms(h, s["eps"]) * (s["offset"] + s["w_pre"].float())
        return x.half(), h.half()
    d_h, out = s["d_h"].float(), []
    if c["pre"]:
        d, d_w = _norm_slope(s["h_out"].float(), s["offset"] + s["w_pre"].float(), s["d_x"].float(), s["eps"])
        d_h = d_h + d
        if c["weights"]:
            out.append(d_w.sum(0))
    if s["block"] is not None:
        d_n, n = d_h, _stream_plain(s)[1]
        if s["gate"] is not None:
            d_n = d_h * s["gate"].float()
            if c["gate"] == "token":
                out.append((d_h * n).half())
            elif c["weights"]:
                out.append((d_h * n).sum(0))
        if c["post"]:
            d_n, d_w = _norm_slope(s["block"].float(), s["offset"] + s["w_post"].float(), d_n, s["eps"])
            if c["weights"]:
                out.append(d_w.sum(0))
        out.append(d_n.half())
    return [(s["factor"] * d_h).half()] + out


def _grads_plain(s, c):
    inv = 1.0 / c["scale"]
    squares = torch.stack([(v.float() * inv).square().sum(dtype=torch.float64) for v in s["grads"]])
    norm = squares.sum().sqrt().float().view(1)
    if c["dir"] == "norm":
        return norm
    factor = (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(v.float() * inv * factor) for v, o in zip(s["grads"], s["outs"])]
    return [norm] + s["out"]


def run(s):
    c = s["case"]
    if not own:
        return {"adapters": _adapters_plain, "norms": _norms_plain, "grads": _grads_plain}[c["op"]](s, c)
    import bit_group_quantized_q4gsw_b200 as q
    if c["op"] == "adapters":
        if c["dir"] == "fwd":
            return q.q4gsw_adapters_fwd(s["packed"], c["N"], c["K"], c["gs"], s["plan"], s["a"], s["b"], s["x"],
                                        scale=s["scale"], bias=s["bias"], residual=s["residual"], save_u=c["save"],
                                        f32s=c["f32s"])
        return q.q4gsw_adapters_bwd(s["packed"], c["N"], c["K"], c["gs"], s["plan"], s["a"], s["b"], s["x"], s["u"],
                                    s["d_y"], scale=s["scale"], f32s=c["f32s"])
    if c["op"] == "norms":
        how = dict(block=s["block"], w_post=s["w_post"], gate=s["gate"], residual_scale=s["factor"], w_pre=s["w_pre"],
                   eps=s["eps"], weight_offset=s["offset"])
        if c["dir"] == "fwd":
            x, h = q.q4gsw_norms_fwd(s["h"], **how)
            return (x, h) if c["pre"] else h
        d = q.q4gsw_norms_bwd(s["h_out"], d_x=s["d_x"], d_h=s["d_h"], want_weights=c["weights"], **how)
        return [v for v in (d.residual, d.w_pre, d.gate, d.w_post, d.block) if v is not None]
    if c["dir"] == "norm":
        return q.q4gsw_grad_norm(s["set"], inv_scale=1.0 / c["scale"])
    return [q.q4gsw_grad_clip(s["set"], c["max_norm"], inv_scale=1.0 / c["scale"])] + s["out"]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "grads":
        sizes, halves = _sizes(case), _halves(case)
        n = sum(v * (2 if f else 4) for v, f in zip(sizes, halves)) + 4
        m = sum(sizes)
        return {"bytes": n + (4 * m if case["dir"] == "clip" else 0), "flops": (3 if case["dir"] == "clip" else 2) * m}
    if case["op"] == "norms":
        M, D = case["M"], case["D"]
        block = case.get("block", True)
        n = 2 * D * (case["post"] + case["pre"] + (case["gate"] == "feature"))
        n += 2 * M * D * (case["gate"] == "token")
        if case["dir"] == "fwd":
            return {"bytes": n + 2 * M * D * (2 + block + case["pre"]), "flops": M * D * (4 + 6 * block + 5 * case["pre"])}
        n += 2 * M * D * (3 + 2 * block) if case["pre"] else 2 * M * D * (2 + block + (block and (case["post"] or case["gate"] != "none")))
        n += 2 * M * D * (case["gate"] == "token") + 4 * D * case["weights"] * (case["post"] + case["pre"] + (case["gate"] == "feature"))
        return {"bytes": n, "flops": M * D * (4 + 14 * block + 10 * case["pre"])}
    M, K, N, r = case["M"], case["K"], case["N"], case["r"]
    owners = [a for a in _owners(case) if a >= 0]
    share = len(owners) / case["requests"]
    used = len(set(owners))
    n = N * K // 2 + (4 if case["f32s"] else 2) * N * K // case["gs"] + 2 * used * r * (N + K) + 4 * M
    n += 2 * M * (K + N)                     # x and y, or d_y and d_x
    low = 2 * M * r * (N + K) * share
    if case["dir"] == "fwd":
        n += (2 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0) + (4 * M * r if case["save"] else 0)
        return {"bytes": n, "flops": 2 * M * N * K + low}
    n += 2 * M * K + 4 * M * r + 4 * case["L"] * r * (N + K)     # x and u, the two gradients
    return {"bytes": n, "flops": 2 * M * N * K + 2 * low}


# ---------------------------------------------------------------- from the definition, in 64 bits
def _exact_adapters(s, c):
    codes, scales = s["w"]
    w = codes.double().sub_(8.0).mul_(torch.repeat_interleave(scales.double(), c["gs"], dim=0).t())
    ids, x = s["ids"].cpu(), s["x"].double()
    u = torch.zeros((c["M"], c["r"]), device="cuda", dtype=torch.float64)
    if c["dir"] == "fwd":
        y = torch.mm(x, w.t())
        for a in sorted(set(ids.tolist()) - {-1}):
            at = (ids == a).nonzero().flatten().cuda()
            u[at] = torch.mm(x[at], s["a"][a].double().t())
            y[at] += float(s["scale"][a]) * torch.mm(u[at], s["b"][a].double().t())
        for name in ("bias", "residual"):
            if s[name] is not None:
                y += s[name].double()
        return (y, u) if c["save"] else y
    d_y = s["d_y"].double()
    d_x = torch.mm(d_y, w)
    d_a = torch.zeros(s["a"].shape, device="cuda", dtype=torch.float64)
    d_b = torch.zeros(s["b"].shape, device="cuda", dtype=torch.float64)
    for a in sorted(set(ids.tolist()) - {-1}):
        at = (ids == a).nonzero().flatten().cuda()
        f = float(s["scale"][a])
        v = f * torch.mm(d_y[at], s["b"][a].double())
        d_x[at] += torch.mm(v, s["a"][a].double())
        d_a[a] = torch.mm(v.t(), x[at])
        d_b[a] = f * torch.mm(d_y[at].t(), s["u"][at].double())
    return d_x, d_a, d_b


def _exact_norms(s, c):
    with torch.enable_grad():
        leaf = lambda name: None if s[name] is None else s[name].double().requires_grad_()      # noqa: E731
        norm = lambda v, w: v / torch.sqrt(torch.mean(v ** 2, 1, keepdim=True) + s["eps"]) * (w + s["offset"])   # noqa: E731
        h, block, gate, w_post, w_pre = (leaf(k) for k in ("h", "block", "gate", "w_post", "w_pre"))
        stream = s["factor"] * h
        if block is not None:
            n = block if w_post is None else norm(block, w_post)
            stream = stream + (n if gate is None else gate * n)
        if c["dir"] == "fwd":
            return (norm(stream, w_pre).detach(), stream.detach()) if c["pre"] else stream.detach()
        # the pre norm's gradient is taken at the stream as it was saved, the rest at the inputs
        total = s["d_h"].double()
        d_pre = None
        if c["pre"]:
            saved = leaf("h_out")
            d_saved, d_pre = torch.autograd.grad(norm(saved, w_pre), (saved, w_pre), s["d_x"].double())
            total = total + d_saved
        names = [k for k, v in (("h", h), ("block", block), ("gate", gate), ("w_post", w_post)) if v is not None]
        leaves = dict(h=h, block=block, gate=gate, w_post=w_post)
        d = dict(zip(names, torch.autograd.grad(stream, [leaves[k] for k in names], total)))
    keep = [d["h"]]
    keep += [d_pre] if c["pre"] and c["weights"] else []
    keep += [d["gate"]] if c["gate"] == "token" or (c["gate"] == "feature" and c["weights"]) else []
    keep += [d["w_post"]] if c["post"] and c["weights"] else []
    return keep + ([d["block"]] if block is not None else [])


def _exact_grads(s, c):
    total = math.fsum(float(torch.dot(f, f)) for f in (v.double() for v in s["flat"]))      # padding is zero
    norm = math.sqrt(total) / c["scale"]
    n = torch.tensor([norm], device="cuda", dtype=torch.float64)
    if c["dir"] == "norm":
        return n
    k = min(1.0, c["max_norm"] / (norm + 1e-6)) / c["scale"]
    return [n] + [v.double() * k for v in s["flat"]]


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapters": _exact_adapters, "norms": _exact_norms, "grads": _exact_grads}[case["op"]](s, case)
