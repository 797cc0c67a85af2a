"""The operators around the routed experts, as one call each: the residual's
addition with the root-mean-square norm and its MXFP8 output, the norm's
gradient, expert routing with groups, the routing weights' gradient down to the
router's logits, and the combine's gradient with respect to those weights.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU,
`run()` one pass: with `own` the library's entry points, without it the same
operators in elementary torch operations.  `exact()` evaluates the definitions
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
EXPERTS = 896
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    H = 7168
    return [
        # ---- residual + norm + MXFP8: rows entering the expert layer
        # one token of a decode step: latency only
        {"name": "norm decode T1", "op": "norm", "T": 1, "H": H, "stream": "bf16", "weight": "bf16", "mx": True},
        # a prefill chunk of the layer's size: memory bound
        {"name": "norm prefill T8192", "op": "norm", "T": 8192, "H": H, "stream": "bf16", "weight": "bf16", "mx": True},
        # an fp32 residual stream with fp32 weights, a ragged batch and a width that is no multiple of a scale group
        {"name": "norm f32 stream T1023", "op": "norm", "T": 1023, "H": 5000, "stream": "f32", "weight": "f32",
         "mx": False},
        # ---- the norm's gradient
        # one training step's rows at the layer's width
        {"name": "norm grad T8192", "op": "norm_grad", "T": 8192, "H": H, "stream": "bf16", "weight": "bf16"},
        # a short ragged sequence, fp32 stream, the narrower checkpoint's width
        {"name": "norm grad f32 T333", "op": "norm_grad", "T": 333, "H": 3584, "stream": "f32", "weight": "f32"},
        # ---- routing
        # a decode batch: 8 groups of 112 experts, the best 4 kept
        {"name": "route decode T16", "op": "route", "T": 16, "E": 896, "k": 16, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "renorm": True, "scale": 2.5, "down": 0, "pad": 0},
        # a prefill chunk of the same router, a few experts out of service and padded rows at the end
        {"name": "route prefill T8192", "op": "route", "T": 8192, "E": 896, "k": 16, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "renorm": True, "scale": 2.5, "down": 5, "pad": 100},
        # softmax routing without groups or bias, an odd number of tokens
        {"name": "route softmax T2049", "op": "route", "T": 2049, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "renorm": True, "scale": 1.0, "down": 0, "pad": 0},
        # ---- the routing weights' gradient
        {"name": "route grad T8192", "op": "route_grad", "T": 8192, "E": 896, "k": 16, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "pad": 100},
        # softmax weights that are not renormalised: every expert's logit has a gradient
        {"name": "route grad softmax T500", "op": "route_grad", "T": 500, "E": 160, "k": 6, "score": "softmax",
         "renorm": False, "scale": 1.0, "pad": 3},
        # ---- the combine's gradient
        # a training step of the full layer: the experts' outputs are read once
        {"name": "combine grad T8192", "op": "combine_grad", "T": 8192, "H": H, "k": 16, "pad": 0},
        # a short ragged batch, some slots masked
        {"name": "combine grad T129", "op": "combine_grad", "T": 129, "H": 3584, "k": 8, "pad": 9},
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], even over the logarithm; 3072 is not drawn."""
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9))))
    return n if n != 3072 else n + 1


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "route_grad", "combine_grad"])
    if op in ("norm", "norm_grad"):
        c = {"op": op}
        mx = op == "norm" and rng.random() < 0.6
        H = 32 * _size(rng, 4, 256) if mx else _size(rng, 128, 8192)
        c["T"] = _size(rng, 1, min(16384, 8192 * 7168 // H))
        c["H"] = H if H != 3072 else H + 32
        c["stream"] = rng.choice(["bf16", "f32"])
        c["weight"] = rng.choice(["bf16", "f32"])
        # an fp32 stream moves about 1.6 times the bytes of a row
        if c["stream"] == "f32":
            c["T"] = max(1, c["T"] * 5 // 8)
        if op == "norm":
            c["mx"] = mx
        if c["T"] == 3072:
            c["T"] += 1
        return c
    if op == "combine_grad":
        H, k = 4 * _size(rng, 32, 2048), rng.randint(1, 32)
        H = H if H != 3072 else H + 4
        T = _size(rng, 1, min(16384, 8192 * 16 * 7168 // (k * H)))
        return {"op": op, "T": T, "H": H, "k": k, "pad": rng.choice([0, T // 10])}
    groups = rng.choice([1, 1, 4, 8, 16])
    per = _size(rng, 1 + 31 // groups, 896 // groups)
    E = groups * per
    E = E if E != 3072 else E + groups
    keep = rng.randint(max(1, groups // 2), groups)
    k = rng.randint(1, min(32, keep * per))
    T = _size(rng, 1, 8192)
    c = {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]), "renorm": rng.random() < 0.7,
         "scale": rng.choice([1.0, 2.5]), "pad": rng.choice([0, T // 10])}
    if op == "route":
        # a bias goes with sigmoid scores here; softmax scores choose by the logits
        c.update(bias=c["score"] == "sigmoid" and rng.random() < 0.8, groups=groups, keep=keep,
                 down=rng.choice([0, E // 20]))
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if op in ("norm", "norm_grad"):
        H, st = case["H"], DT[case["stream"]]
        # a residual stream whose channels differ in size, norm weights near one
        chan = torch.exp(0.5 * randn(H))
        s["weight"] = (1.0 + 0.1 * randn(H)).to(DT[case["weight"]])
        if op == "norm":
            s["x"] = randn(T, H).to(torch.bfloat16)
            s["residual"] = (3.0 * randn(T, H) * chan).to(st)
            s["h"] = torch.empty(T, H, dtype=st, device="cuda")
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
            if case["mx"]:
                s["codes"] = torch.empty(T, H, dtype=torch.uint8, device="cuda")
                s["scales"] = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
        else:
            s["dy"] = (1e-2 * randn(T, H)).to(torch.bfloat16)
            s["h"] = (3.0 * randn(T, H) * chan).to(st)
            s["dh_in"] = (1e-2 * randn(T, H)).to(st)
            s["dh"] = torch.empty(T, H, dtype=st, device="cuda")
            s["dweight"] = torch.empty(H, dtype=torch.float32, device="cuda")
        return s
    pad = case["pad"]
    if op in ("route", "route_grad"):
        E, k = case["E"], case["k"]
        logits = 1.7 * randn(T, E)  # bf16 N(0, 1) rows on a gate of N(0, 0.02) at the layer's width
        if op == "route":
            if case["down"]:  # experts out of service
                logits[:, torch.randperm(E, generator=g, device="cuda")[: case["down"]]] = -math.inf
            if pad:  # rows that no token stands on
                logits[T - pad:] = -math.inf
            s["logits"] = logits
            s["bias"] = 0.1 * randn(E) if case["bias"] else None
            s["topk_ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["topk_w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        else:
            ids = logits.topk(k, dim=1).indices.to(torch.int32)
            if pad:
                ids[T - pad:] = -1
            s.update(logits=logits, topk_ids=ids, d_w=randn(T, k),
                     d_logits=torch.empty(T, E, dtype=torch.float32, device="cuda"))
        return s
    H, k = case["H"], case["k"]
    ids = torch.randint(0, EXPERTS, (T, k), generator=g, device="cuda", dtype=torch.int32)
    if pad:
        ids[torch.rand(T, k, generator=g, device="cuda") < 0.1] = -1
    s.update(topk_ids=ids, y=randn(T * k, H), d_out=(1e-2 * randn(T, H)).to(torch.bfloat16),
             d_w=torch.empty(T, k, dtype=torch.float32, device="cuda"))
    return s


def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)[c["op"]](s, c)


# ---------------------------------------------------------------- the library's entry points


def _own_norm(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    h, y, codes, scales = K.kmoe_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, mx=c["mx"], h=s["h"],
                                         y=s["y"], codes=s.get("codes"), scales=s.get("scales"))
    if not c["mx"]:
        return {"h": h, "y": y}
    return {"h": h, "y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _own_norm_grad(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    dh, dweight = K.kmoe_rmsnorm_backward(s["dy"], s["h"], s["weight"], dh_in=s["dh_in"], eps=EPS, dh=s["dh"],
                                          dweight=s["dweight"])
    return {"dh": dh, "dweight": dweight}


def _own_route(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    ids, w = K.kmoe_route_grouped(s["logits"], s["bias"], c["k"], score=c["score"], n_group=c["groups"],
                                  topk_group=c["keep"], renormalize=c["renorm"], scale=c["scale"],
                                  topk_ids=s["topk_ids"], topk_w=s["topk_w"])
    return {"ids": ids, "w": w}


def _own_route_grad(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    return {"d_logits": K.kmoe_route_backward(s["d_w"], s["logits"], s["topk_ids"], score=c["score"],
                                              renormalize=c["renorm"], scale=c["scale"], d_logits=s["d_logits"])}


def _own_combine_grad(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    return {"d_w": K.kmoe_combine_backward(s["d_out"], s["y"], s["topk_ids"], EXPERTS, d_w=s["d_w"])}


_run_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "route": _own_route, "route_grad": _own_route_grad,
            "combine_grad": _own_combine_grad}


# ---------------------------------------------------------------- plain forms


def _plain_norm(s, c):
    h = s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    y = (h * rstd * s["weight"].float()).to(torch.bfloat16)
    out = {"h": h.to(s["residual"].dtype), "y": y}
    if c["mx"]:
        # the codes are the bf16 row's, as the layer quantises it: per 32 columns the
        # smallest e with amax <= 448 * 2^e, where 448 = 0.875 * 2^9
        grp = y.float().view(c["T"], -1, 32)
        m, q = torch.frexp(grp.abs().amax(-1, keepdim=True))
        e = torch.where(m > 0, q - 9 + (m > 0.875), -127).clamp(-127, 127)
        codes = torch.ldexp(grp, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["codes"] = codes.view(c["T"], c["H"])
        out["scales"] = (e + 127).to(torch.uint8).view(c["T"], -1).view(torch.float8_e8m0fnu)
    return out


def _plain_norm_grad(s, c):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * rstd
    g = dy * s["weight"].float()
    dh = s["dh_in"].float() + rstd * (g - n * (g * n).mean(-1, keepdim=True))
    return {"dh": dh.to(s["h"].dtype), "dweight": (dy * n).sum(0)}


def _softmax(logits):
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
    return e / e.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_route(s, c):
    logits, T, E = s["logits"], c["T"], c["E"]
    lowest = -math.inf
    scores = None
    if c["score"] == "softmax":
        scores = _softmax(logits)
    elif c["bias"]:
        # the key is defined by the sigmoid rounded once to 32 bits, as in the layer's routing:
        # the ids have to be equal, so it is evaluated wider here and rounded
        scores = (1.0 / (1.0 + torch.exp(-logits.double()))).float()
    else:
        scores = 1.0 / (1.0 + torch.exp(-logits))
    # without a bias the scores are in the logits' order
    key = torch.where(logits > lowest, scores + s["bias"], lowest) if c["bias"] else logits
    if c["groups"] > 1:
        per = key.view(T, c["groups"], E // c["groups"])
        if c["bias"]:  # a group's two best keys (one, where it has one)
            best = per.topk(min(2, per.shape[2]), dim=-1).values
            of_group = best[..., 0] + torch.where(best[..., 1:] > lowest, best[..., 1:], 0.0).sum(-1)
        else:
            of_group = per.amax(-1)
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        ok = torch.zeros(T, c["groups"], dtype=torch.bool, device=key.device).scatter_(1, kept, True)
        key = torch.where(ok[..., None], per, lowest).view(T, E)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, : c["k"]], ids[:, : c["k"]]
    w = torch.where(key > lowest, scores.gather(1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
    return {"ids": torch.where(key > lowest, ids, -1).to(torch.int32), "w": w * c["scale"]}


def _plain_route_grad(s, c):
    logits, ids = s["logits"], s["topk_ids"].long()
    ok = ids >= 0
    at = ids.clamp_min(0)
    d_w = torch.where(ok, s["d_w"] * c["scale"], 0.0)
    soft = c["score"] == "softmax"
    scores = _softmax(logits) if soft else 1.0 / (1.0 + torch.exp(-logits))
    chosen = torch.where(ok, scores.gather(1, at), 0.0)
    if c["renorm"]:
        total = chosen.sum(-1, keepdim=True).clamp_min(1e-30)
        d_s = torch.where(ok, (d_w - (d_w * chosen).sum(-1, keepdim=True) / total) / total, 0.0)
    else:
        d_s = d_w
    d_scores = torch.zeros_like(logits).scatter_add_(1, at, d_s)
    if soft:
        return {"d_logits": scores * (d_scores - (d_scores * scores).sum(-1, keepdim=True))}
    return {"d_logits": d_scores * scores * (1.0 - scores)}


def _plain_combine_grad(s, c):
    d_w = (s["y"].view(c["T"], c["k"], c["H"]) * s["d_out"].float()[:, None, :]).sum(-1)
    return {"d_w": torch.where(s["topk_ids"] >= 0, d_w, 0.0)}


_run_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "route": _plain_route,
              "route_grad": _plain_route_grad, "combine_grad": _plain_combine_grad}


# ---------------------------------------------------------------- bytes and operations


def work(case):
    op, T = case["op"], case["T"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm":
        H, st = case["H"], size[case["stream"]]
        row = H * (2 + st + st + 2) + (H + H // 32 if case["mx"] else 0)
        return {"bytes": T * row + H * size[case["weight"]], "flops": T * H * (8 if case["mx"] else 5)}
    if op == "norm_grad":
        H, st = case["H"], size[case["stream"]]
        return {"bytes": T * H * (2 + 3 * st) + H * (size[case["weight"]] + 4), "flops": T * H * 12}
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * (4 * E + 8 * k) + (4 * E if case["bias"] else 0), "flops": T * E * 4}
    if op == "route_grad":
        E, k = case["E"], case["k"]
        # the chosen logits alone, except where every logit has a gradient of its own
        read = 4 * E if case["score"] == "softmax" and not case["renorm"] else 4 * k
        return {"bytes": T * (4 * E + read + 8 * k), "flops": T * (k * 10 + read)}
    H, k = case["H"], case["k"]
    return {"bytes": T * (k * (4 * H + 8) + 2 * H), "flops": 2 * T * k * H}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_weights(case, s, score):
    """The chosen scores in choosing order, and their sum (1 where it is 0), on the host."""
    logits, score = s["logits"].cpu().numpy(), score.cpu().numpy()
    key = logits
    if case["bias"]:
        key = score.astype(np.float32) + s["bias"].cpu().numpy()
        key[np.isneginf(logits)] = -np.inf
    per = key.reshape(len(key), case["groups"], -1)
    if case["groups"] > 1:
        two = -np.sort(-per, axis=2)[:, :, : 2 if case["bias"] else 1]
        best = two[:, :, 0] + np.where(np.isneginf(two), np.float32(0), two)[:, :, 1:].sum(axis=2, dtype=np.float32)
        order = np.argsort(-best, axis=1, kind="stable")
        per = per.copy()
        np.put_along_axis(per, order[:, case["keep"]:, None], -np.inf, axis=1)
    key = per.reshape(key.shape)
    ids = np.argsort(-key, axis=1, kind="stable")[:, : case["k"]]
    w = np.where(np.isneginf(np.take_along_axis(key, ids, 1)), 0.0, np.take_along_axis(score, ids, 1))
    total = w.sum(axis=1, keepdims=True)
    return torch.from_numpy(w).cuda(), torch.from_numpy(np.where(total > 0, total, 1.0)).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    d = torch.float64
    if op == "norm":
        h = torch.add(s["x"].to(d), s["residual"].to(d))
        y = torch.einsum("th,t,h->th", h, (torch.linalg.vector_norm(h, dim=1) ** 2 / case["H"] + EPS) ** -0.5,
                         s["weight"].to(d))
        out = {"h": h, "y": y}
        if case["mx"]:
            blocks = y.reshape(T, case["H"] // 32, 32)
            e = torch.ceil(torch.log2(torch.linalg.vector_norm(blocks, ord=math.inf, dim=2) / 448.0))
            out["scales"] = torch.pow(torch.tensor(2.0, dtype=d, device=e.device), e)
            out["codes"] = (blocks / out["scales"][..., None]).reshape(T, case["H"])
        return out
    if op == "norm_grad":
        h, dy, w = s["h"].to(d), s["dy"].to(d), s["weight"].to(d)
        var = torch.linalg.vector_norm(h, dim=1) ** 2 / case["H"] + EPS
        dot = torch.einsum("th,th,h->t", dy, h, w) / case["H"]
        dh = s["dh_in"].to(d) + (dy * w - h * (dot / var)[:, None]) / var.sqrt()[:, None]
        return {"dh": dh, "dweight": torch.einsum("th,th,t->h", dy, h, var ** -0.5)}
    if op == "combine_grad":
        y = s["y"].view(T, case["k"], case["H"])
        d_w = torch.stack([torch.mv(y[t].to(d), s["d_out"][t].to(d)) for t in range(T)])
        return {"d_w": d_w * (s["topk_ids"] >= 0)}
    l64 = s["logits"].to(d)
    if case["score"] == "softmax":
        score = torch.nan_to_num(torch.softmax(l64, dim=1), nan=0.0)
    else:
        score = torch.sigmoid(l64)
    if op == "route":
        w, total = _exact_weights(case, s, score)
        return {"ids": None, "w": w * case["scale"] / (total if case["renorm"] else 1.0)}
    ids = s["topk_ids"].long()
    mask = ids >= 0
    index = torch.where(mask, ids, 0)
    picked = torch.take_along_dim(score, index, 1) * mask
    # gradient of sum(d_w * w) by the chain rule, logit by logit
    g = s["d_w"].to(d) * case["scale"] * mask
    if case["score"] == "sigmoid":
        slope = torch.take_along_dim(torch.sigmoid(-l64), index, 1) * mask  # d log(score) / d logit
        if case["renorm"]:
            share = picked / torch.where(mask.any(1, keepdim=True), picked.sum(1, keepdim=True), 1.0)
            val = share * (g - (g * share).sum(1, keepdim=True)) * slope
        else:
            val = g * picked * slope
        return {"d_logits": torch.zeros_like(l64).scatter_add(1, index, val * mask)}
    if case["renorm"]:
        share = picked / torch.where(mask.any(1, keepdim=True), picked.sum(1, keepdim=True), 1.0)
        val = share * (g - (g * share).sum(1, keepdim=True))
        return {"d_logits": torch.zeros_like(l64).scatter_add(1, index, val * mask)}
    out = torch.zeros_like(l64).scatter_add(1, index, g * picked) - score * (g * picked).sum(1, keepdim=True)
    return {"d_logits": out}
