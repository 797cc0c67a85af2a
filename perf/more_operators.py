"""Expert products in 8 bits with a scale for each block of 128, the sort of the
tokens' rows by expert in front of them, the weighted way back behind them, and
the gradients of all three, as calls of their own.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU,
`run()` one pass: with `own` the library's entry points, without it the same
operators in elementary torch operations.  `exact()` evaluates the definitions
in 64 bits.
"""
import math

import torch

own = False

B = 128  # values a scale, along the sum (and, for weights, across it)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


def listed():
    H, I = 7168, 3584
    return [
        # ---- tokens sorted by expert
        # a decode step's 16 tokens, bf16 rows: launches and latency
        {"name": "permute decode T16", "op": "permute", "T": 16, "H": H, "E": 896, "k": 16, "fp8": False, "pad": 0},
        # a prefill chunk of the layer's size, padded rows at the end, quantised on the way
        {"name": "permute fp8 prefill T8192", "op": "permute", "T": 8192, "H": H, "E": 896, "k": 16, "fp8": True,
         "pad": 100},
        # ---- and back
        # the combine of a prefill chunk: memory bound
        {"name": "unpermute T8192", "op": "unpermute", "T": 8192, "H": H, "E": 896, "k": 16, "rows": "bf16",
         "weights": True, "pad": 100},
        # the gradient of the permutation for a short ragged batch, fp32 rows
        {"name": "unpermute sum T1023 f32", "op": "unpermute", "T": 1023, "H": 5000, "E": 64, "k": 8, "rows": "f32",
         "weights": False, "pad": 0},
        # ---- the gradient of the way back: the rows' and the weights'
        # one training step's tokens at the layer's width
        {"name": "unpermute grad T4096", "op": "unpermute_grad", "T": 4096, "H": H, "E": 896, "k": 16, "rows": "bf16",
         "pad": 0},
        # a short ragged batch, some slots masked
        {"name": "unpermute grad T129", "op": "unpermute_grad", "T": 129, "H": I, "E": 64, "k": 8, "rows": "bf16",
         "pad": 9},
        # ---- products, from bf16 rows: quantised and multiplied
        # one token through a dense projection (a shared expert): reads the weights once
        {"name": "product decode M1", "op": "product", "M": 1, "N": H, "K": H, "E": 1, "back": False, "out": "bf16",
         "pad": 0},
        # a decode batch over 64 experts: every expert's weights for a few rows
        {"name": "product experts M128", "op": "product", "M": 128, "N": H, "K": H, "E": 64, "back": False,
         "out": "bf16", "pad": 0},
        # a prefill chunk, 64 experts, some hundred rows each: bound by the tensor cores
        {"name": "product experts M32768", "op": "product", "M": 32768, "N": H, "K": H, "E": 64, "back": False,
         "out": "bf16", "pad": 0},
        # the rows' gradient of a down projection's training step, ragged, rows behind the last expert's
        {"name": "product grad M16001", "op": "product", "M": 16001, "N": H, "K": I, "E": 64, "back": True,
         "out": "bf16", "pad": 33},
        # ---- the weights' gradient
        # a dense projection's, an odd number of tokens
        {"name": "weight grad M4095", "op": "weight_grad", "M": 4095, "N": 2048, "K": H, "E": 1, "pad": 0},
        # experts' of a training step, ragged
        {"name": "weight grad experts M16384", "op": "weight_grad", "M": 16384, "N": H, "K": I, "E": 16, "pad": 0},
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], even over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "unpermute_grad", "product", "product", "weight_grad"])
    if op in ("product", "weight_grad"):
        back = op == "product" and rng.random() < 0.4
        E = rng.choice([1, _size(rng, 2, 64)])
        N, K = 16 * _size(rng, 8, 448), 16 * _size(rng, 8, 448)
        if op == "weight_grad":
            E = min(E, max(1, 16 * 7168 * 3584 // (N * K)))
            M = _size(rng, 1, 16384)
            return {"op": op, "M": M, "N": N, "K": K, "E": E, "pad": rng.choice([0, M // 20])}
        M = _size(rng, 1, 32768)
        return {"op": op, "M": M, "N": N, "K": K, "E": E, "back": back, "out": rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, M // 20]) if E > 1 else 0}
    H, k = 8 * _size(rng, 16, 1024), rng.randint(1, 32)
    E = _size(rng, k, 1024)
    T = _size(rng, 1, min(16384, 4096 * 16 * 7168 // (k * H)))
    c = {"op": op, "T": T, "H": H, "E": E, "k": k, "pad": rng.choice([0, T // 10])}
    if op == "permute":
        c["fp8"] = rng.random() < 0.5
        if c["fp8"]:
            c["H"] = H = max(128, H // 16 * 16)
    else:
        c["rows"] = rng.choice(["bf16", "f32"])
        if op == "unpermute":
            c["weights"] = rng.random() < 0.6
    return c


# ---------------------------------------------------------------- inputs


def _popular(E, randn):
    """How likely a token is to choose each expert: some are chosen several times as often as others."""
    return torch.exp(0.5 * randn(E))


def _quantised_weights(E, N, K, randn):
    """E4M3 codes and fp32 scales of 128x128 blocks, largest magnitude on 448, as a checkpoint holds them."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-N // B), -(-K // B), device="cuda")
    for e in range(E):
        w = torch.nn.functional.pad(0.02 * randn(N, K), (0, -K % B, 0, -N % B))
        w = w.view(w.shape[0] // B, B, w.shape[1] // B, B)
        scales[e] = w.abs().amax((1, 3)) / 448.0
        w = (w / scales[e][:, None, :, None]).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
        codes[e] = w.view(scales.shape[1] * B, scales.shape[2] * B)[:N, :K]
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, E, pad = case["op"], case["E"], case["pad"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def zeros(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    s = {"case": case}
    if op in ("product", "weight_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        s["seg"], s["cap"] = None, M
        if E > 1:
            chosen = torch.multinomial(_popular(E, randn), M - pad, replacement=True, generator=g)
            count = torch.bincount(chosen, minlength=E)
            s["seg"] = torch.cat([zeros(1, dtype=torch.int64), count.cumsum(0)]).to(torch.int32)
            s["cap"] = max(1, int(count.max()))

        def rows(cols, scale):  # channels and rows of different sizes
            return (scale * randn(M, cols) * torch.exp(0.5 * randn(cols)) * torch.exp(0.3 * randn(M, 1))).to(
                torch.bfloat16)

        if op == "product":
            wide, s["width"] = (N, K) if case["back"] else (K, N)
            s["x"] = rows(wide, 1e-2 if case["back"] else 1.0)
            s["w"], s["w_scales"] = _quantised_weights(E, N, K, randn)
            s["codes"], s["scales"] = zeros(M, wide, dtype=torch.uint8), zeros(-(-wide // B), M, dtype=torch.float32)
            s["out"] = zeros(M, s["width"], dtype=DT[case["out"]])
        else:
            s["dy"], s["x"] = rows(N, 1e-2), rows(K, 1.0)
            s["dw"] = zeros(E, N, K, dtype=torch.float32)
        s["workspace"] = zeros(256, dtype=torch.uint8)
        return s
    T, H, k = case["T"], case["H"], case["k"]
    # k experts a token, none twice
    ids = (_popular(E, randn).log() - torch.empty(T, E, device="cuda").exponential_(generator=g).log()).topk(k).indices
    ids = ids.to(torch.int32)
    if pad:
        ids[T - pad:] = -1  # rows that no token stands on
        ids[torch.rand(T, k, generator=g, device="cuda") < 0.05] = -1  # and experts of another machine
    s["ids"] = ids
    R = T * k
    if op == "permute":
        s["x"] = (randn(T, H) * torch.exp(0.5 * randn(H))).to(torch.bfloat16)
        s["row_of_slot"], s["slot_of_row"] = zeros(T, k, dtype=torch.int32), zeros(R, dtype=torch.int32)
        s["seg_start"] = zeros(E + 1, dtype=torch.int32)
        if case["fp8"]:
            s["codes"], s["scales"] = zeros(R, H, dtype=torch.uint8), zeros(-(-H // B), R, dtype=torch.float32)
        else:
            s["xp"] = zeros(R, H, dtype=torch.bfloat16)
        s["workspace"] = zeros(4 * R + 4 * E * (R // 1024 + 2) + 4096, dtype=torch.uint8)
        return s
    flat = ids.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(R, device="cuda")
    s["row_of_slot"] = torch.where(flat < 0, -1, row).to(torch.int32).view(T, k)
    s["y"] = randn(R, H).to(DT[case["rows"]])
    if op == "unpermute_grad" or case["weights"]:
        w = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
    else:
        s["w"] = None
    if op == "unpermute":
        s["out"] = zeros(T, H, dtype=torch.bfloat16)
    else:
        s["d_out"] = (1e-2 * randn(T, H)).to(torch.bfloat16)
        s["d_y"], s["d_w"] = zeros(R, H, dtype=DT[case["rows"]]), zeros(T, k, dtype=torch.float32)
    return s


def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)[c["op"]](s, c)


# ---------------------------------------------------------------- the library's entry points


def _own_permute(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    row_of_slot, slot_of_row, seg_start = K.kmoe_sort_tokens(
        s["ids"], c["E"], row_of_slot=s["row_of_slot"], slot_of_row=s["slot_of_row"], seg_start=s["seg_start"],
        workspace=s["workspace"])
    out = {"row_of_slot": row_of_slot, "slot_of_row": slot_of_row, "seg_start": seg_start}
    if c["fp8"]:
        codes, out["scales"] = K.kmoe_quantize_fp8(s["x"], row_of_slot=row_of_slot, codes=s["codes"],
                                                   scales=s["scales"])
        out["codes"] = codes.view(F8)
    else:
        out["xp"] = K.kmoe_permute(s["x"], row_of_slot, out=s["xp"])
    return out


def _own_unpermute(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    return {"out": K.kmoe_unpermute(s["y"], s["row_of_slot"], s["w"], out=s["out"])}


def _own_unpermute_grad(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    d_y, d_w = K.kmoe_unpermute_backward(s["d_out"], s["y"], s["row_of_slot"], s["w"], d_y=s["d_y"], d_w=s["d_w"])
    return {"d_y": d_y, "d_w": d_w}


def _own_product(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    codes, scales = K.kmoe_quantize_fp8(s["x"], codes=s["codes"], scales=s["scales"])
    out, _ = K.kmoe_gemm_fp8(codes, scales, s["w"], s["w_scales"], seg_start=s["seg"], transpose=c["back"],
                             out=s["out"], workspace=s["workspace"])
    return {"out": out}


def _own_weight_grad(s, c):
    import mxfp8_mxfp4_moe_gb300 as K
    dy, dy_scales = K.kmoe_quantize_fp8_cols(s["dy"], seg_start=s["seg"])
    x, x_scales = K.kmoe_quantize_fp8_cols(s["x"], seg_start=s["seg"])
    dw, _ = K.kmoe_gemm_fp8_wgrad(dy, dy_scales, x, x_scales, seg_start=s["seg"], dw=s["dw"],
                                  workspace=s["workspace"])
    return {"dw": dw}


_run_own = {"permute": _own_permute, "unpermute": _own_unpermute, "unpermute_grad": _own_unpermute_grad,
            "product": _own_product, "weight_grad": _own_weight_grad}


# ---------------------------------------------------------------- plain forms


def _quantise(x, dim):
    """Codes (as fp32 values) and power-of-two scales of groups of values along `dim`, which holds whole groups."""
    m, q = torch.frexp(x.abs().amax(dim, keepdim=True))
    # the smallest e with amax <= 448 * 2^e, where 448 = 0.875 * 2^9
    e = torch.where(m > 0, q - 9 + (m > 0.875), -126).clamp(-126, 127)
    # 2^e and 2^-e by their exponent fields: a power function is not exact everywhere
    scale, inverse = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    return (x * inverse).clamp(-448.0, 448.0).to(F8), scale


def _quantise_rows(x):
    """[rows, cols] -> E4M3 codes [rows, cols], scales [ceil(cols / 128), rows]."""
    rows, cols = x.shape
    grp = torch.nn.functional.pad(x.float(), (0, -cols % B)).view(rows, -1, B)
    codes, scales = _quantise(grp, 2)
    return codes.view(rows, -1)[:, :cols], scales.view(rows, -1).t().contiguous()


def _plain_permute(s, c):
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    ids = s["ids"].view(-1)
    order = torch.sort(torch.where(ids < 0, E, ids), stable=True)
    seg_start = torch.searchsorted(order.values, torch.arange(E + 1, device=ids.device, dtype=torch.int32))
    live = torch.arange(T * k, device=ids.device) < seg_start[E]
    row = torch.empty_like(order.indices)
    row[order.indices] = torch.arange(T * k, device=ids.device)
    out = {"row_of_slot": torch.where(ids < 0, -1, row).to(torch.int32).view(T, k),
           "slot_of_row": torch.where(live, order.indices, -1).to(torch.int32), "seg_start": seg_start.to(torch.int32)}
    token = order.indices // k
    if c["fp8"]:
        codes, scales = _quantise_rows(s["x"])
        out["scales"] = torch.where(live, scales[:, token], 0.0)
        out["codes"] = torch.where(live[:, None], codes.view(torch.uint8)[token], 0).view(F8)
    else:
        out["xp"] = torch.where(live[:, None], s["x"][token], 0.0)
    return out


def _rows_of_slots(s):
    """The slots' rows [T, k], 0 for masked ones, and which are not."""
    row = s["row_of_slot"].long()
    return row.clamp_min(0), row >= 0


def _plain_unpermute(s, c):
    row, ok = _rows_of_slots(s)
    y = torch.where(ok[..., None], s["y"][row].float(), 0.0)
    if s["w"] is not None:
        y = y * s["w"][..., None]
    return {"out": y.sum(1).to(torch.bfloat16)}


def _plain_unpermute_grad(s, c):
    row, ok = _rows_of_slots(s)
    d_out = s["d_out"].float()[:, None, :]
    d_w = torch.where(ok, (d_out * s["y"][row].float()).sum(-1), 0.0)
    # one row more for the slots that have none
    R = row.numel()
    d_y = torch.zeros(R + 1, c["H"], dtype=s["y"].dtype, device=row.device)
    d_y[torch.where(ok, row, R).view(-1)] = (d_out * s["w"][..., None]).view(R, -1).to(d_y.dtype)
    return {"d_y": d_y[:R], "d_w": d_w}


def _segments(s, c, whole=1):
    """Each expert's rows, [E, cap] as indices of rows, and which of them are its own; cap a multiple of `whole`."""
    cap = -(-s["cap"] // whole) * whole
    at = torch.arange(cap, device="cuda")[None, :]
    if s["seg"] is None:
        return at.clamp_max(c["M"] - 1), at < c["M"]
    seg = s["seg"].long()
    at = at + seg[:-1, None]
    return at.clamp_max(c["M"] - 1), at < seg[1:, None]


def _plain_product(s, c):
    codes, scales = _quantise_rows(s["x"])
    x = codes.float() * scales.t().repeat_interleave(B, 1)[:, : codes.shape[1]]
    w = s["w"].view(F8).float()
    w *= s["w_scales"].repeat_interleave(B, 2)[:, :, : c["K"]].repeat_interleave(B, 1)[:, : c["N"]]
    w = w if c["back"] else w.mT
    if s["seg"] is None:
        return {"out": (x @ w[0]).to(DT[c["out"]])}
    at, ok = _segments(s, c)
    y = torch.bmm(torch.where(ok[..., None], x[at], 0.0), w).to(DT[c["out"]])
    row, seg = torch.arange(c["M"], device=x.device), s["seg"].long()
    e = torch.searchsorted(seg[1:], row, right=True).clamp_max(c["E"] - 1)
    y = y[e, (row - seg[e]).clamp_max(s["cap"] - 1)]
    return {"out": torch.where((row < seg[-1])[:, None], y, 0.0)}


def _plain_weight_grad(s, c):
    at, ok = _segments(s, c, B)

    def blocks(t):
        t = torch.where(ok[..., None], t[at].float(), 0.0).view(c["E"], -1, B, t.shape[1])
        codes, scales = _quantise(t, 2)
        return (codes.float() * scales).view(c["E"], -1, t.shape[3])

    return {"dw": torch.bmm(blocks(s["dy"]).mT, blocks(s["x"]))}


_run_plain = {"permute": _plain_permute, "unpermute": _plain_unpermute, "unpermute_grad": _plain_unpermute_grad,
              "product": _plain_product, "weight_grad": _plain_weight_grad}


# ---------------------------------------------------------------- bytes and operations


def work(case):
    op, E = case["op"], case["E"]
    if op in ("product", "weight_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        live = M - case["pad"]
        if op == "weight_grad":
            return {"bytes": 2 * live * (N + K) + 4 * E * N * K, "flops": 2 * live * N * K}
        used = min(E, live)  # experts that can have rows
        rows = 2 * live * (N if case["back"] else K)
        out = live * (K if case["back"] else N) * (2 if case["out"] == "bf16" else 4)
        return {"bytes": rows + used * (N * K + 4 * -(-N // B) * -(-K // B)) + out, "flops": 2 * live * N * K}
    T, H, k = case["T"], case["H"], case["k"]
    live = T - case["pad"]
    R = live * k
    if op == "permute":
        row = H + 4 * -(-H // B) if case["fp8"] else 2 * H
        return {"bytes": 2 * live * H + R * row + 4 * (3 * T * k + E + 1),
                "flops": T * k + (2 * live * H if case["fp8"] else 0)}
    size = 2 if case["rows"] == "bf16" else 4
    if op == "unpermute":
        return {"bytes": R * size * H + 2 * T * H + T * k * (8 if case["weights"] else 4), "flops": 2 * R * H}
    return {"bytes": 2 * R * size * H + 2 * live * H + 12 * T * k, "flops": 3 * R * H}


# ---------------------------------------------------------------- the definitions in 64 bits


def _two_to(e):
    """2^e in 64 bits, by its exponent field (a power function is not exact everywhere)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_groups(v):
    """Values that 8 bits hold of each row of `v` [groups, up to 128], its scale's exponent apart."""
    top = torch.linalg.vector_norm(v, ord=math.inf, dim=-1, keepdim=True)
    # (a bf16 magnitude is on a bound, or further than 1e-9 from it)
    e = torch.ceil(torch.log2(top / 448.0) - 1e-9).clamp(-126.0, 127.0)
    e = torch.where(top > 0, e, -126.0)
    scaled = v * _two_to(-e)
    # four significant bits, or multiples of 2^-9, halves to even
    step = torch.floor(torch.log2(scaled.abs().clamp_min(2.0 ** -6)) + 1e-9) - 3
    return torch.round(scaled * _two_to(-step)) * _two_to(step), e


def _exact_rows(x):
    """What the quantised rows [rows, cols] stand for, the values alone, and the scales [rows, groups]."""
    parts = [_exact_groups(p) for p in x.split(B, dim=1)]
    return (torch.cat([c * _two_to(e) for c, e in parts], 1), torch.cat([c for c, _ in parts], 1),
            _two_to(torch.cat([e for _, e in parts], 1)))


def exact(case, seed):
    s = prepare(case, seed)
    op, E, d = case["op"], case["E"], torch.float64
    if op == "permute":
        T, H, k = case["T"], case["H"], case["k"]
        flat = s["ids"].view(-1).tolist()
        order = sorted((e, i) for i, e in enumerate(flat) if e >= 0)
        token = torch.tensor([i // k for _, i in order], dtype=torch.long, device="cuda")
        none = {"row_of_slot": None, "slot_of_row": None, "seg_start": None}
        rest = T * k - len(order)

        def whole(t):
            return torch.nn.functional.pad(t, (0, 0, 0, rest))

        if not case["fp8"]:
            return {**none, "xp": whole(s["x"].to(d)[token])}
        _, codes, scales = _exact_rows(s["x"].to(d))
        return {**none, "codes": whole(codes[token]), "scales": whole(scales[token]).T}
    if op in ("unpermute", "unpermute_grad"):
        T, H, k = case["T"], case["H"], case["k"]
        out, d_w, d_y = torch.zeros(T, H, dtype=d, device="cuda"), torch.zeros(T, k, dtype=d, device="cuda"), None
        weights = torch.ones(T, k, dtype=d, device="cuda") if s["w"] is None else s["w"].to(d)
        if op == "unpermute_grad":
            d_y = torch.zeros(T * k, H, dtype=d, device="cuda")
        for j in range(k):
            t = torch.nonzero(s["row_of_slot"][:, j] >= 0).view(-1)
            r = s["row_of_slot"][t, j].long()
            if op == "unpermute":
                out[t] += torch.einsum("t,th->th", weights[t, j], s["y"][r].to(d))
            else:
                d_w[t, j] = torch.einsum("th,th->t", s["d_out"][t].to(d), s["y"][r].to(d))
                d_y[r] = torch.einsum("t,th->th", weights[t, j], s["d_out"][t].to(d))
        return {"out": out} if op == "unpermute" else {"d_y": d_y, "d_w": d_w}
    M, N, K = case["M"], case["N"], case["K"]
    bounds = [0, M] if s["seg"] is None else s["seg"].tolist()
    if op == "weight_grad":
        dw = torch.zeros(E, N, K, dtype=d, device="cuda")
        for e in range(E):
            for at in range(bounds[e], bounds[e + 1], 8 * B):
                end = min(at + 8 * B, bounds[e + 1])
                dy, x = (torch.cat([_exact_rows(p.T)[0].T for p in s[name][at:end].to(d).split(B)])
                         for name in ("dy", "x"))
                dw[e].addmm_(dy.T, x)
        return {"dw": dw}
    out = torch.zeros(M, s["width"], dtype=d, device="cuda")
    for e in range(E):
        at, end = bounds[e], bounds[e + 1]
        if at == end:
            continue
        w = torch.kron(s["w_scales"][e].to(d), torch.ones(B, B, dtype=d, device="cuda"))[:N, :K]
        w = w * s["w"][e].view(F8).to(d)
        out[at:end] = _exact_rows(s["x"][at:end].to(d))[0] @ (w if case["back"] else w.T)
    return {"out": out}
