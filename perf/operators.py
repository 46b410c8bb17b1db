"""The expert operators of a mixture-of-experts layer as they are timed and compared.

Each case is one pass through one operator (or, where a case says so, through the forward and
the backward of one): the products grouped by expert, their weight gradient, the gated
up-projection with its 8-bit activation checkpoint, the backward pass that reads the
checkpoint, and the gradient of the combine.  `run` computes them plainly in torch, or, where
`own` is true, calls the library.  `exact` states the same results in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32  # columns that share a scale in an 8-bit checkpoint


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a 256-expert layer being decoded: eight rows, eight experts' weights
        dict(name="gemm one token", op="gemm", layout="nk", T=1, k=8, E=256, K=2048, N=1024, skew="even"),
        # a decode batch of 64 sequences: a few rows for nearly every expert, all weights read
        dict(name="gemm decode batch", op="gemm", layout="nk", T=64, k=8, E=128, K=1024, N=2048, skew="even"),
        # a short prompt or a small microbatch, skewed, with odd sizes: ragged row counts
        dict(name="gemm ragged", op="gemm", layout="nk", T=4093, k=6, E=64, K=2048, N=1416, skew="zipf"),
        # the input gradient of a training microbatch: weights read along their rows
        dict(name="gemm input gradient", op="gemm", layout="kn", T=16384, k=8, E=128, K=2048, N=1024, skew="zipf"),
        # weight gradient of a small, odd microbatch, many experts left empty, kept in bf16
        dict(name="wgrad small", op="wgrad", out="bf16", T=1021, k=2, E=64, K=1032, N=1416, skew="few"),
        # weight gradient of a training microbatch into the 32-bit gradient buffer
        dict(name="wgrad training", op="wgrad", out="f32", T=16384, k=8, E=128, K=1024, N=2048, skew="zipf"),
        # the up-projection of a decode batch of 16 sequences; nothing is kept
        dict(name="gated decode", op="gated", T=16, k=8, E=256, K=2048, F=512, skew="even"),
        # the up-projection of a training microbatch: forward with the checkpoint, then its backward
        dict(name="gated training", op="gated_train", T=8192, k=8, E=64, K=2048, F=1024, skew="zipf"),
        # the activation's backward pass from the checkpoint: one small microbatch, odd width
        dict(name="gated backward small", op="gated_backward", rows=771, F=1416),
        # and a training microbatch
        dict(name="gated backward", op="gated_backward", rows=131072, F=1024),
        # the combine's gradient: a small microbatch, and a training one at the widest rows
        dict(name="combine backward small", op="combine_backward", T=509, k=6, E=64, H=2048),
        dict(name="combine backward", op="combine_backward", T=32768, k=6, E=128, H=4096),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _one(rng):
    op = rng.choice(["gemm", "gemm", "wgrad", "gated", "gated_train", "gated_backward", "combine_backward"])
    if op == "gated_backward":
        return dict(op=op, rows=_log(rng, 1, 131072), F=_log(rng, 64, 2048, 8))
    k = rng.choice([1, 2, 4, 6, 8])
    if op == "combine_backward":
        return dict(op=op, T=_log(rng, 1, 32768), k=k, E=rng.choice([64, 128, 256]), H=_log(rng, 256, 4096, 8))
    c = dict(op=op, T=_log(rng, 1, 16384), k=k, E=rng.choice([8, 64, 128, 256]), K=_log(rng, 256, 4096, 8),
             skew=rng.choice(["even", "zipf", "few"]))
    if op in ("gemm", "wgrad"):
        c["N"] = _log(rng, 256, 4096, 8)
    if op == "gemm":
        c["layout"] = rng.choice(["nk", "kn"])
    elif op == "wgrad":
        c["out"] = rng.choice(["f32", "bf16"])
    else:
        c["F"] = _log(rng, 128, 2048, 8)
    return c


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.6e15)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _one(rng)
        if _cost(c) <= most:
            return c


def work(case):
    c = case
    if c["op"] == "gated_backward":
        n = c["rows"] * c["F"]
        # da and the two 8-bit halves with their scales in; both gradients and the activation out
        return {"bytes": n * 2 + 2 * n + 2 * c["rows"] * -(-c["F"] // BLOCK) + 4 * n + 2 * n, "flops": 20 * n}
    rows = c["T"] * c["k"]
    if c["op"] == "combine_backward":
        # dout once, the expert outputs in and their gradients out, rows and gates in, gate gradients out
        return {"bytes": 2 * c["T"] * c["H"] + 4 * rows * c["H"] + 12 * rows, "flops": 3 * rows * c["H"]}
    hit = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that some token chose
    if c["skew"] == "few":
        hit = min(hit, max(c["k"], c["E"] // 4))
    N = c["N"] if "N" in c else 2 * c["F"]
    flops = 2 * rows * N * c["K"]
    if c["op"] == "wgrad":
        out = 4 if c["out"] == "f32" else 2
        return {"bytes": 2 * rows * (N + c["K"]) + out * c["E"] * N * c["K"], "flops": flops}
    b = 2 * rows * c["K"] + 2 * hit * N * c["K"]
    if c["op"] == "gemm":
        return {"bytes": b + 2 * rows * N, "flops": flops}
    n = rows * c["F"]
    b += 2 * n
    if c["op"] == "gated_train":
        # the checkpoint written and read, da in, both gradients and the activation out
        b += 2 * (2 * n + 2 * rows * -(-c["F"] // BLOCK)) + 2 * n + 4 * n + 2 * n
    return {"bytes": b, "flops": flops}


# ------------------------------------------------------------------ inputs

def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000 + tag)
    return g


def _normal(seed, tag, *shape, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed, tag), device=DEV) * scale).to(torch.bfloat16)


def _routing(case, seed):
    """Top-k experts of every token and the expert-grouped rows: experts stand in the rows in the
    order of a placement, so their offsets do not rise with the expert's number."""
    T, k, E = case["T"], case["k"], case["E"]
    g = _gen(seed, 1)
    logits = torch.randn(T, E, generator=g, device=DEV)
    skew = case.get("skew", "zipf")
    if skew == "zipf":  # both experts of one pair stand out, the pair by a Zipf law
        pairs = torch.randperm(E, generator=g, device=DEV).view(-1, 2)
        p = 1.0 / torch.arange(1, E // 2 + 1, device=DEV, dtype=torch.float64) ** 1.1
        cdf = torch.cumsum(p / p.sum(), 0)
        u = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
        hit = torch.searchsorted(cdf, u).clamp_(max=E // 2 - 1)
        logits.scatter_add_(1, pairs[hit], torch.full((T, 2), 3.0, device=DEV))
    elif skew == "few":  # only a quarter of the experts are ever chosen
        some = torch.randperm(E, generator=g, device=DEV)[: max(k, E // 4)]
        keep = torch.zeros(E, dtype=torch.bool, device=DEV)
        keep[some] = True
        logits.masked_fill_(~keep, float("-inf"))
    top, idx = torch.topk(logits, k, dim=1)
    gates = torch.softmax(top, 1)
    place = torch.randperm(E, generator=g, device=DEV)  # position of expert e among the row blocks
    slots = torch.argsort(place[idx].flatten(), stable=True)
    assign_row = torch.empty(T * k, dtype=torch.int64, device=DEV)
    assign_row[slots] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(idx.flatten(), minlength=E)
    by_place = torch.argsort(place)
    starts = torch.cumsum(counts[by_place], 0) - counts[by_place]
    offsets = torch.full((E + 1,), T * k, dtype=torch.int64, device=DEV)
    offsets[by_place] = starts
    return dict(idx=idx.to(torch.int32), gates=gates, assign_row=assign_row.view(T, k).to(torch.int32),
                offsets=offsets.to(torch.int32), counts=counts.to(torch.int32),
                # the same on the host, for the plain form's split of the rows
                spans=[(e, o, c) for e, (o, c) in enumerate(zip(offsets.tolist(), counts.tolist())) if c])


def _pack(h):
    """8-bit checkpoint of h (float32, any columns): e4m3 codes and one power-of-two scale for
    each 32 columns, the smallest with which no value passes 448."""
    rows, cols = h.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(h, (0, pad)).view(rows, -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(-1))  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    s = torch.where(m > 0.875, e - 8, e - 9)
    s = torch.where(m == 0, torch.full_like(s, -127), s).clamp_(min=-127)
    codes = torch.ldexp(b, -s.unsqueeze(-1)).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return codes, (s + 127).to(torch.uint8)


def _unpack(codes, scales):
    rows, cols = codes.shape
    s = (scales.to(torch.int32) - 127).repeat_interleave(BLOCK, 1)[:, :cols]
    return torch.ldexp(codes.to(torch.float32), s)


def prepare(case, seed):
    c, op = case, case["op"]
    s = {"op": op}
    if op == "gated_backward":
        rows, F = c["rows"], c["F"]
        halves = [_pack(torch.randn(rows, F, generator=_gen(seed, 2 + i), device=DEV) * 1.5) for i in range(2)]
        s["codes"] = torch.cat([h[0].view(torch.uint8) for h in halves], 1).view(torch.float8_e4m3fn)
        s["scales"] = torch.cat([h[1] for h in halves], 1)
        s["da"] = _normal(seed, 4, rows, F, scale=0.1)
        return s
    s.update(_routing(c, seed))
    rows = c["T"] * c["k"]
    if op == "combine_backward":
        s["dout"] = _normal(seed, 2, c["T"], c["H"], scale=0.1)
        s["y"] = _normal(seed, 3, rows, c["H"])
        return s
    K = c["K"]
    s["x"] = _normal(seed, 2, rows, K)
    if op == "gemm":
        s["layout"] = c["layout"]
        shape = (c["E"], c["N"], K) if c["layout"] == "nk" else (c["E"], K, c["N"])
        s["w"] = _normal(seed, 3, *shape, scale=K ** -0.5)
    elif op == "wgrad":
        s["dy"] = _normal(seed, 3, rows, c["N"], scale=0.1)
        s["out"] = torch.float32 if c["out"] == "f32" else torch.bfloat16
    else:
        s["w"] = _normal(seed, 3, c["E"], 2 * c["F"], K, scale=1.5 * K ** -0.5)
        if op == "gated_train":
            s["da"] = _normal(seed, 4, rows, c["F"], scale=0.1)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import combine_warp_top_router_b200 as md
    op = s["op"]
    if op == "gated_backward":
        return md.md_expert_gated_backward(s["da"], s["codes"], s["scales"])
    if op == "combine_backward":
        return md.md_combine_backward(s["dout"], s["assign_row"], s["gates"], s["y"])
    if op == "gemm":
        return md.md_expert_gemm(s["x"], s["w"], s["offsets"], s["counts"],
                                 md.MD_W_NK if s["layout"] == "nk" else md.MD_W_KN)
    if op == "wgrad":
        return md.md_expert_wgrad(s["dy"], s["x"], s["offsets"], s["counts"], out_dtype=s["out"])
    if op == "gated":
        return md.md_expert_gated(s["x"], s["w"], s["offsets"], s["counts"])
    a, codes, scales = md.md_expert_gated(s["x"], s["w"], s["offsets"], s["counts"], keep=True)
    dh, again = md.md_expert_gated_backward(s["da"], codes, scales)
    return a, dh, again


def _products(x, w, spans, nk):
    """Float32 rows x[r] times their expert's matrix.  With few rows to an expert one padded batch
    takes all of them; with many, one product for each expert is the faster plain form."""
    out = torch.empty(x.shape[0], w.shape[1] if nk else w.shape[2], dtype=torch.float32, device=x.device)
    most = max(n for _, _, n in spans)
    if most <= 16:
        e = torch.tensor([e for e, _, _ in spans]).to(x.device, non_blocking=True)
        o = torch.tensor([o for _, o, _ in spans]).to(x.device, non_blocking=True)
        n = torch.tensor([n for _, _, n in spans]).to(x.device, non_blocking=True)
        j = torch.arange(most, device=x.device)
        r = o[:, None] + torch.minimum(j, n[:, None] - 1)  # short experts repeat their last row
        we = w[e].float()
        out[r] = torch.bmm(x[r].float(), we.transpose(1, 2) if nk else we)
        return out
    for e, o, n in spans:
        we = w[e].float()
        torch.matmul(x[o:o + n].float(), we.t() if nk else we, out=out[o:o + n])
    return out


def _act(g, u):
    return g * torch.sigmoid(g) * u


def _act_backward(da, g, u):
    s = torch.sigmoid(g)
    da = da.float()
    return torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1), g * s * u


def _plain(s):
    op, bf16 = s["op"], torch.bfloat16
    if op == "gated_backward":
        F = s["da"].shape[1]
        B = s["scales"].shape[1] // 2
        g, u = _unpack(s["codes"][:, :F], s["scales"][:, :B]), _unpack(s["codes"][:, F:], s["scales"][:, B:])
        dh, a = _act_backward(s["da"], g, u)
        return dh.to(bf16), a.to(bf16)
    if op == "combine_backward":
        T, k = s["gates"].shape
        rows = s["assign_row"].to(torch.int64)
        dout = s["dout"].float()
        dw = (s["y"][rows].float() * dout[:, None]).sum(-1)
        dy = torch.empty_like(s["y"])
        dy[rows.flatten()] = (s["gates"][:, :, None] * dout[:, None]).to(bf16).view(T * k, -1)
        return dy, dw
    if op == "gemm":
        return _products(s["x"], s["w"], s["spans"], s["layout"] == "nk").to(bf16)
    if op == "wgrad":
        dw = torch.zeros(s["counts"].shape[0], s["dy"].shape[1], s["x"].shape[1], device=s["x"].device)
        for e, o, n in s["spans"]:
            torch.matmul(s["dy"][o:o + n].float().t(), s["x"][o:o + n].float(), out=dw[e])
        return dw.to(s["out"])
    h = _products(s["x"], s["w"], s["spans"], True)
    F = h.shape[1] // 2
    a = _act(h[:, :F], h[:, F:]).to(bf16)
    if op == "gated":
        return a
    dh, again = _act_backward(s["da"], _unpack(*_pack(h[:, :F])), _unpack(*_pack(h[:, F:])))
    return a, dh.to(bf16), again.to(bf16)


# ------------------------------------------------------------------ 64 bits

def _stored64(h):
    """The values that an 8-bit checkpoint of h holds: three fraction bits above 2^-6 of the
    block's scale, a fixed step below it, ties to even."""
    out = torch.empty_like(h)
    for c in range(0, h.shape[1], BLOCK):
        b = h[:, c:c + BLOCK]
        top = b.abs().amax(1, keepdim=True)
        s = torch.ceil(torch.log2(torch.where(top > 0, top / 448, torch.full_like(top, 1e-300))))
        s = torch.where(448 * torch.exp2(s - 1) >= top, s - 1, s)  # the logarithm may be a hair off
        s = torch.where(448 * torch.exp2(s) < top, s + 1, s).clamp(min=-127)
        v = b / torch.exp2(s)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, c:c + BLOCK] = torch.round(v / step) * step * torch.exp2(s)
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = torch.float64

    def back(da, g, u):
        sig = 1 / (1 + torch.exp(-g))
        return torch.cat([da.to(d) * u * (sig + g * sig * (1 - sig)), da.to(d) * (g * sig)], 1), u * (g * sig)

    if op == "gated_backward":
        F = case["F"]
        h = []
        for half in (0, 1):
            codes = s["codes"][:, half * F:(half + 1) * F].to(d)
            sc = s["scales"].view(case["rows"], 2, -1)[:, half].to(d)
            at = torch.arange(F, device=DEV) // BLOCK
            h.append(codes * torch.exp2(sc - 127)[:, at])
        return back(s["da"], h[0], h[1])
    if op == "combine_backward":
        dy = torch.empty(s["y"].shape, dtype=d, device=DEV)
        dw = torch.empty(s["gates"].shape, dtype=d, device=DEV)
        dout = s["dout"].to(d)
        for j in range(case["k"]):
            r = s["assign_row"][:, j].long()
            dy[r] = dout * s["gates"][:, j:j + 1].to(d)
            dw[:, j] = (dout * s["y"][r].to(d)).sum(1)
        return dy, dw
    if op == "wgrad":
        dw = torch.zeros(case["E"], case["N"], case["K"], dtype=d, device=DEV)
        for e in range(case["E"]):
            o, n = int(s["offsets"][e]), int(s["counts"][e])
            dw[e] = s["dy"][o:o + n].to(d).t() @ s["x"][o:o + n].to(d)
        return dw
    w = s["w"] if op != "gemm" or s["layout"] == "nk" else s["w"].transpose(1, 2)
    h = torch.zeros(s["x"].shape[0], w.shape[1], dtype=d, device=DEV)
    for e in range(case["E"]):
        o, n = int(s["offsets"][e]), int(s["counts"][e])
        h[o:o + n] = s["x"][o:o + n].to(d) @ w[e].to(d).t()
    if op == "gemm":
        return h
    g, u = h.chunk(2, 1)
    a = u * (g / (1 + torch.exp(-g)))
    if op == "gated":
        return a
    dh, again = back(s["da"], _stored64(g), _stored64(u))
    return a, dh, again
