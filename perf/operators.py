"""The operators around the routed experts, as they are measured: plain forms and the library's calls.

  add_rmsnorm      afd_ffn_add_rmsnorm: residual addition and root-mean-square norm in front of the FFN, with bf16 rows
                   and e4m3 rows plus one scale each
  select_experts   afd_ffn_select_experts: scores, balance bias, expert groups, top-k and gate weights from router logits
  w4_rows          afd_ffn_w4_rows: rows grouped by expert times 4-bit weights with group scales
  w4_expert_rows   afd_ffn_w4_expert_rows: the whole expert (gate/up, SwiGLU, down) on such weights

`own` chooses the side: False runs elementary torch operations, True the library.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token in front of a W8A8 layer: a latency-bound call
        dict(name="norm_one_token", op="add_rmsnorm", T=1, H=7168, pad=0, residual="bf16", gamma="fp32", out=True, codes=True),
        # a large micro-batch in front of a W8A8 layer: the router reads the bf16 rows, the experts the e4m3 ones
        dict(name="norm_prompt", op="add_rmsnorm", T=8192, H=7168, pad=0, residual="bf16", gamma="bf16", out=True, codes=True),
        # rows that are slices of wider ones, an odd width, an fp32 residual stream
        dict(name="norm_odd_rows", op="add_rmsnorm", T=515, H=4097, pad=38, residual="fp32", gamma="fp32", out=True, codes=False),
        # a decode micro-batch with sigmoid scores, a balance bias and the best four of eight groups
        dict(name="select_decode", op="select_experts", T=256, E=256, k=8, score="sigmoid", groups=8, keep=4, best=2,
             renormalise=True, scale=2.5, bias=True, logits="fp32", masked=0.0),
        # one token, softmax scores that are not renormalised, groups ranked by their best expert
        dict(name="select_one_token", op="select_experts", T=1, E=160, k=6, score="softmax", groups=8, keep=3, best=1,
             renormalise=False, scale=16.0, bias=False, logits="fp32", masked=0.0),
        # a large micro-batch of bf16 logits (many equal ones), some experts out of service
        dict(name="select_prompt", op="select_experts", T=8192, E=256, k=8, score="softmax", groups=1, keep=1, best=1,
             renormalise=True, scale=1.0, bias=False, logits="bf16", masked=0.05),
        # one token through a dense gate/up projection: a matrix-vector product
        dict(name="w4_one_row", op="w4_rows", E=1, K=7168, N=4096, rows=1, group=128, zeros=False, scales="bf16", y="bf16", skew=0.0),
        # a small group of rows over a few experts, small groups with zero points, fp32 results
        dict(name="w4_few_rows", op="w4_rows", E=6, K=2048, N=7168, rows=21, group=32, zeros=True, scales="fp32", y="fp32", skew=0.5),
        # the smallest layer: every expert gets many rows
        dict(name="w4_experts_tiny", op="w4_expert_rows", E=8, H=256, I=512, rows=128, group=64, zeros=False, scales="bf16", skew=0.0),
        # one token's eight experts out of sixteen
        dict(name="w4_experts_one_token", op="w4_expert_rows", E=16, H=7168, I=2048, rows=8, group=128, zeros=False, scales="bf16", skew=-1.0),
        # a decode micro-batch, about two rows an expert, zero points
        dict(name="w4_experts_decode", op="w4_expert_rows", E=64, H=4096, I=1024, rows=128, group=128, zeros=True, scales="bf16", skew=0.5),
        # a larger micro-batch with hot experts and empty ones
        dict(name="w4_experts_hot", op="w4_expert_rows", E=24, H=7168, I=2048, rows=512, group=64, zeros=False, scales="bf16", skew=1.2),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["add_rmsnorm", "select_experts", "w4_rows", "w4_expert_rows"])
    if op == "add_rmsnorm":
        out, codes = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, T=_spread(rng, 1, 8192), H=_spread(rng, 128, 7168) if rng.random() < 0.5 else 8 * _spread(rng, 16, 896),
                    pad=rng.choice([0, 0, 8, 24, 3]), residual=rng.choice(["bf16", "fp32", "none"]), gamma=rng.choice(["bf16", "fp32"]),
                    out=out, codes=codes)
    if op == "select_experts":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(4, 256 // groups)
        best = rng.choice([1, 2])
        keep = rng.randint(1, groups)
        score = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, T=_spread(rng, 1, 8192), E=E, k=rng.randint(1, min(16, keep * (E // groups))), score=score, groups=groups,
                    keep=keep, best=best, renormalise=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    # two sums of two coarse scores can be equal but for their rounding: no order of theirs is right
                    bias=rng.random() < 0.6, logits="fp32" if groups > 1 and best == 2 else rng.choice(["fp32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.05]))
    group = rng.choice([32, 64, 128])
    if op == "w4_rows":
        E = _spread(rng, 1, 32)
        K = group * _spread(rng, 1, 7168 // group)
        N = _spread(rng, 16, min(8192, max(16, 500_000_000 // (E * K))))
        return dict(op=op, E=E, K=K, N=N, rows=_spread(rng, 1, 256), group=group, zeros=rng.random() < 0.5,
                    scales=rng.choice(["bf16", "fp32"]), y=rng.choice(["bf16", "bf16", "fp32"]), skew=rng.choice([0.0, 0.5, 1.2]))
    E = _spread(rng, 1, 64)
    H = group * _spread(rng, 2, 7168 // group)
    I = group * _spread(rng, 1, max(1, min(2048, 1_000_000_000 // (3 * E * H)) // group))
    return dict(op=op, E=E, H=H, I=I, rows=_spread(rng, 1, 512), group=group, zeros=rng.random() < 0.5,
                scales=rng.choice(["bf16", "fp32"]), skew=rng.choice([0.0, 0.5, 1.2]))


def _counts(case, seed):
    """Rows of each expert: spread by popularity r^-skew over a shuffled ranking; skew -1: one row each for `rows` of the experts."""
    import random
    rng = random.Random(seed * 7919 + 13)
    E, rows = case["E"], case["rows"]
    order = rng.sample(range(E), E)
    got = [0] * E
    if case["skew"] < 0:
        for e in order[:rows]:
            got[e] = 1
        return got
    for e in rng.choices(order, weights=[(r + 1.0) ** -case["skew"] for r in range(E)], k=rows):
        got[e] += 1
    return got


# ------------------------------------------------------------------ inputs
def _w4(gen, E, N, K, case):
    G = case["group"]
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scale = (torch.rand((E, N, K // G), device="cuda", generator=gen) * 0.6 + 0.7) * (0.22 / math.sqrt(K))
    zero = torch.randint(5, 12, (E, N, K // G), dtype=torch.uint8, device="cuda", generator=gen) if case["zeros"] else None
    return dict(codes=codes, scale=scale.to(BF16) if case["scales"] == "bf16" else scale, zero=zero, group=G)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _plan(s)
    return s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "add_rmsnorm":
        T, H, ld = case["T"], case["H"], case["H"] + case["pad"]
        s["x"] = torch.randn((T, ld), device="cuda", generator=gen).to(BF16)[:, :H]
        kind = case["residual"]
        r = None if kind == "none" else 3.0 * torch.randn((T, ld), device="cuda", generator=gen)
        s["r"] = None if r is None else (r.to(BF16) if kind == "bf16" else r)[:, :H]
        g = 1.0 + 0.2 * torch.randn((H,), device="cuda", generator=gen)
        s["g"], s["eps"] = g.to(BF16) if case["gamma"] == "bf16" else g, 1e-6
        # what the call writes: the new residual, the rows, and the e4m3 rows with their scales
        s["sum"] = None if r is None else torch.empty((T, H), dtype=s["r"].dtype, device="cuda")
        s["y"] = torch.empty((T, H), dtype=BF16, device="cuda") if case["out"] else None
        s["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda") if case["codes"] else None
        s["qs"] = torch.empty((T,), device="cuda") if case["codes"] else None
    elif case["op"] == "select_experts":
        T, E, k = case["T"], case["E"], case["k"]
        l = torch.randn((T, E), device="cuda", generator=gen) * 1.2
        if case["masked"]:  # experts out of service, the same for every token; k of each kept set of groups stay
            off = torch.rand((E,), device="cuda", generator=gen) < case["masked"]
            off[(torch.arange(E, device="cuda") % (E // case["groups"])) < -(-k // case["keep"])] = False
            l = l.masked_fill(off, -math.inf)
        s["l"] = l.to(BF16) if case["logits"] == "bf16" else l
        s["b"] = 0.05 * torch.randn((E,), device="cuda", generator=gen) if case["bias"] else None
        s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, k), device="cuda")
    else:
        counts = _counts(case, seed)
        E, rows = case["E"], case["rows"]
        s["most"] = max(counts)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        if case["op"] == "w4_rows":
            s["x"] = torch.randn((rows, case["K"]), device="cuda", generator=gen).to(BF16)
            s["w"] = _w4(gen, E, case["N"], case["K"], case)
            s["y_out"] = torch.empty((rows, case["N"]), dtype=BF16 if case["y"] == "bf16" else F32, device="cuda")
        else:
            H, I = case["H"], case["I"]
            s["x"] = torch.randn((rows, H), device="cuda", generator=gen).to(BF16)
            s["w13"], s["w2"] = _w4(gen, E, 2 * I, H, case), _w4(gen, E, H, I, case)
            s["y_out"] = torch.empty((rows, H), dtype=BF16, device="cuda")
    return s


def _plan(s):
    """What a user of the library keeps between calls: its description structs and the scratch."""
    import ffn_side_expert_b200 as afd
    s["afd"] = afd
    if s["op"] == "add_rmsnorm":
        f32 = {"bf16": afd.AFD_DT_BF16, "fp32": afd.AFD_DT_F32, "none": afd.AFD_DT_BF16}
        r = s["r"]
        s["cfg"] = afd.afd_ffn_norm_cfg(T=s["T"], H=s["H"], residual_dtype=f32[s["residual"]], gamma_dtype=f32[s["gamma"]],
                                        x_stride=s["x"].stride(0), residual_stride=r.stride(0) if r is not None else 0,
                                        sum_stride=0, out_stride=0, eps=s["eps"])
    elif s["op"] == "select_experts":
        s["routing"] = afd.afd_ffn_routing(score=afd.AFD_SCORE_SIGMOID if s["score"] == "sigmoid" else afd.AFD_SCORE_SOFTMAX,
                                           n_groups=s["groups"], topk_groups=s["keep"], group_best=s["best"],
                                           renormalise=int(s["renormalise"]), weight_scale=s["scale"])
    elif s["op"] == "w4_rows":
        s["plan"] = afd.w4_weights(**s["w"])
    else:
        s["plan"] = afd.w4_weights(**s["w13"]), afd.w4_weights(**s["w2"])
        s["scratch"] = torch.empty((afd.afd_ffn_w4_scratch_bytes(s["rows"], s["I"]),), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass
def run(s):
    return {"add_rmsnorm": _norm, "select_experts": _select, "w4_rows": _rows, "w4_expert_rows": _experts}[s["op"]](s)


def _ok(s, status):
    if status != 0:
        raise s["afd"].AfdError(status, s["op"])


def _norm(s):
    if own:
        _ok(s, s["afd"].afd_ffn_add_rmsnorm(s["cfg"], s["x"], s["r"], s["g"], s["sum"], s["y"], s["q"], s["qs"]))
        return {"sum": s["sum"], "out": s["y"], "codes": s["q"], "scale": s["qs"]}
    v = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + s["eps"]) * s["g"].float()
    got = {"sum": None if s["r"] is None else v.to(s["r"].dtype), "out": y.to(BF16) if s["out"] else None, "codes": None, "scale": None}
    if s["codes"]:
        top = y.abs().amax(1, keepdim=True)
        scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        got["codes"], got["scale"] = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale[:, 0]
    return got


def _select(s):
    if own:
        _ok(s, s["afd"].afd_ffn_select_experts(s["l"], s["b"], s["T"], s["E"], s["k"], s["routing"], s["idx"], s["w"]))
        return {"idx": s["idx"], "w": s["w"]}
    # 64 bits: an expert next to the border of the selection has to fall on the right side of it
    T, E, G, k = s["T"], s["E"], s["groups"], s["k"]
    l = s["l"].double()
    out = l == -math.inf
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    choice = (score if s["b"] is None else score + s["b"].double()).masked_fill(out, -math.inf)
    if s["keep"] < G:
        per = choice.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, : s["best"]]
        rank = per.masked_fill(per == -math.inf, 0.0).sum(2).masked_fill(per[:, :, 0] == -math.inf, -math.inf)
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device)
        kept.scatter_(1, rank.sort(dim=1, descending=True, stable=True)[1][:, : s["keep"]], True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    best, idx = choice.sort(dim=1, descending=True, stable=True)
    best, idx = best[:, :k], idx[:, :k]
    w = torch.gather(score, 1, idx)
    if s["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    none = best == -math.inf
    return {"idx": idx.masked_fill(none, -1).int(), "w": (w * s["scale"]).masked_fill(none, 0.0).float()}


def _unpack(w):
    """[E][N][K/2] codes -> fp32 weights [E][N][K]."""
    c = w["codes"]
    q = torch.stack((c & 15, c >> 4), 3).view(*c.shape[:2], -1, w["group"]).float()
    q = q - (8.0 if w["zero"] is None else w["zero"].float().unsqueeze(3))
    return (q * w["scale"].float().unsqueeze(3)).view(*c.shape[:2], -1)


def _places(s):
    """Expert of each row and its place among that expert's rows."""
    ends = s["counts"].long().cumsum(0)
    r = torch.arange(s["rows"], device=ends.device)
    e = torch.searchsorted(ends, r, right=True)
    return e, r - (ends - s["counts"])[e]


def _product(x, w, e, at, most):
    """x [rows][K] fp32 times its expert's weights: rows of an expert side by side, one batched product."""
    wide = torch.zeros((w["codes"].shape[0], most, x.shape[1]), device=x.device)
    wide[e, at] = x
    return torch.bmm(wide, _unpack(w).transpose(1, 2))[e, at]


def _rows(s):
    if own:
        _ok(s, s["afd"].afd_ffn_w4_rows(s["plan"], s["E"], s["x"], s["counts"], s["rows"], s["y_out"]))
        return s["y_out"]
    e, at = _places(s)
    return _product(s["x"].float(), s["w"], e, at, s["most"]).to(s["y_out"].dtype)


def _experts(s):
    if own:
        _ok(s, s["afd"].afd_ffn_w4_expert_rows(*s["plan"], s["E"], s["x"], s["counts"], s["rows"], s["y_out"], s["scratch"]))
        return s["y_out"]
    e, at = _places(s)
    gate, up = _product(s["x"].float(), s["w13"], e, at, s["most"]).chunk(2, 1)
    act = gate / (1.0 + torch.exp(-gate)) * up
    return _product(act, s["w2"], e, at, s["most"]).to(BF16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b = {"bf16": 2, "fp32": 4, "none": 0}
    if case["op"] == "add_rmsnorm":
        T, H, r = case["T"], case["H"], b[case["residual"]]
        per = 2 + 2 * r + 2 * case["out"] + case["codes"]
        return {"bytes": T * H * per + 4 * T * case["codes"] + H * b[case["gamma"]], "flops": T * H * (5 + 3 * case["codes"])}
    if case["op"] == "select_experts":
        T, E = case["T"], case["E"]
        return {"bytes": T * E * b[case["logits"]] + T * case["k"] * 8 + 4 * E * case["bias"], "flops": 10 * T * E}
    rows, G, E = case["rows"], case["group"], case["E"]
    # experts that rows reach, on average over seeds
    if case["skew"] < 0:
        touched = min(E, rows)
    else:
        p = [(r + 1.0) ** -case["skew"] for r in range(E)]
        touched = sum(1.0 - (1.0 - v / sum(p)) ** rows for v in p)
    per = 0.5 + (b[case["scales"]] + case["zeros"]) / G  # bytes of a weight
    if case["op"] == "w4_rows":
        K, N = case["K"], case["N"]
        return {"bytes": touched * N * K * per + rows * (2 * K + b[case["y"]] * N), "flops": 2 * rows * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": touched * 3 * H * I * per + rows * 4 * H, "flops": 6 * rows * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "add_rmsnorm":
        v = s["x"].double()
        if s["r"] is not None:
            v = v + s["r"].double()
        y = v * s["g"].double() / torch.sqrt((v * v).sum(1) / case["H"] + s["eps"])[:, None]
        scale = y.abs().max(1)[0] / 448.0
        return {"sum": None if s["r"] is None else v, "out": y if case["out"] else None,
                "codes": y / scale[:, None] if case["codes"] else None, "scale": scale if case["codes"] else None}
    if case["op"] == "select_experts":
        if case["T"] > 1024:
            return None
        rows = s["l"].double().cpu().tolist()
        bias = s["b"].double().cpu().tolist() if s["b"] is not None else [0.0] * case["E"]
        return {"idx": None, "w": torch.tensor([_weights_of(l, bias, case) for l in rows], dtype=torch.float64)}
    counts = s["counts"].tolist()
    out, first = [], 0
    for e, m in enumerate(counts):
        if m == 0:
            continue
        x = s["x"][first:first + m].double()
        first += m
        if case["op"] == "w4_rows":
            out.append(x @ _dense(s["w"], e).T)
        else:
            w13 = _dense(s["w13"], e)
            g, u = x @ w13[: case["I"]].T, x @ w13[case["I"]:].T
            out.append((torch.sigmoid(g) * g * u) @ _dense(s["w2"], e).T)
    return torch.cat(out)


def _dense(w, e):
    c = w["codes"][e]
    q = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.float64, device=c.device)
    q[:, 0::2] = (c % 16).double()
    q[:, 1::2] = (c // 16).double()
    G = w["group"]
    z = 8.0 if w["zero"] is None else w["zero"][e].double().repeat_interleave(G, 1)
    return (q - z) * w["scale"][e].double().repeat_interleave(G, 1)


def _weights_of(l, bias, case):
    E, per = case["E"], case["E"] // case["groups"]
    live = [e for e in range(E) if l[e] != -math.inf]
    if case["score"] == "sigmoid":
        p = {e: 1.0 / (1.0 + math.exp(-l[e])) for e in live}
    else:
        top = max(l[e] for e in live)
        total = math.fsum(math.exp(l[e] - top) for e in live)
        p = {e: math.exp(l[e] - top) / total for e in live}
    c = {e: p[e] + bias[e] for e in live}
    ranks = []
    for g in range(case["groups"]):
        mine = sorted((c[e] for e in live if e // per == g), reverse=True)[: case["best"]]
        if mine:
            ranks.append((-sum(mine), g))
    kept = {g for _, g in sorted(ranks)[: case["keep"]]}
    chosen = sorted((-c[e], e) for e in live if e // per in kept)[: case["k"]]
    p = [p[e] for _, e in chosen]
    total = math.fsum(p) if case["renormalise"] else 1.0
    return [v / total * case["scale"] for v in p] + [0.0] * (case["k"] - len(p))
