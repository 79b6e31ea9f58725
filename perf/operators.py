"""Cases of three operators of an int8 mixture-of-experts model: routing tokens to experts, the int8
matrix product with one scale per token and one per output channel (dense and grouped over experts),
and the int8 quantization of 16-bit rows that feeds it (alone, and joined with SwiGLU).

`own` False: the operators in plain torch; True: the calls a user makes of quantized_gemm_amd.

The formulas, for a row of logits l, expert scores s, int8 codes x and w:

* routing: s = softmax(l) or sigmoid(l); the choice value of an expert is s + bias, or s itself; experts
  lie in equal runs (groups), a group's value is its best choice value or the sum of its two best; the
  topk best experts of the topk_groups best groups are chosen in descending order of choice value, ties
  to the lowest index; the weights are the chosen scores, divided by their sum where renormalized, times
  a constant.  Scores are compared in 64 bits: neighbouring float32 scores would decide which is chosen.
* product: y[m, n] = (sum_k x[m, k] w[n, k]) * sw[n] * sx[m].
* quantization: scale = max|row| / 127 in float32, code = round(row / scale), half to even.
"""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decoding step: the time of the call itself
        route("route_softmax_t1", 1, 128, 8, "bf16"),
        # a prefill chunk, softmax scores of a 128-expert layer in the router's float32
        route("route_softmax_t4096", 4096, 128, 8, "f32", renorm=True),
        # the largest batch: sigmoid scores, balance bias, 8 groups of which 4 are kept
        route("route_sigmoid_groups_t8192", 8192, 256, 8, "f32", scoring="sigmoid", bias=True, groups=8,
              topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # an odd batch and expert count, logits as columns of a wider product
        route("route_f16_ragged", 1021, 60, 4, "f16", bias=True, pad=4),
        # a dense layer for one token: the weights are read once
        gemm("int8_dense_m1", 1, 7168, 7168),
        # the same layer for a decoding batch
        gemm("int8_dense_m64", 64, 7168, 7168),
        # and for a prefill: bound by the matrix cores
        gemm("int8_dense_m4096", 4096, 7168, 7168),
        # ragged rows, a reduction that is an odd multiple of 128, columns that end inside a tile
        gemm("int8_dense_ragged", 777, 1856, 1408, out="f16"),
        # gate and up projections of an expert layer, decoding batch: each expert has few rows
        moe("int8_moe_t64", 64, 64, 6, 2816, 4096),
        # the same for a prefill
        moe("int8_moe_t8192", 8192, 64, 6, 2816, 4096),
        # activations of a dense prefill on their way into the product
        quant("quant_rows_m4096", 4096, 7168),
        # SwiGLU of every routed row of a prefill, quantized for the down projection
        quant("swiglu_rows_49152", 49152, 1408, swiglu=True),
    ]


def route(name, tokens, experts, topk, dtype, scoring="softmax", bias=False, groups=1, topk_groups=1, group_top=1,
          renorm=False, scale=1.0, pad=0):
    return dict(name=name, op="route", tokens=tokens, experts=experts, topk=topk, dtype=dtype, scoring=scoring, bias=bias,
                groups=groups, topk_groups=topk_groups, group_top=group_top, renorm=renorm, scale=scale, pad=pad)


def gemm(name, m, n, k, out="bf16"):
    return dict(name=name, op="gemm", m=m, n=n, k=k, out=out)


def moe(name, tokens, experts, topk, n, k, out="bf16"):
    return dict(name=name, op="moe", tokens=tokens, experts=experts, topk=topk, n=n, k=k, out=out)


def quant(name, rows, k, dtype="bf16", swiglu=False):
    return dict(name=name, op="quant", rows=rows, k=k, dtype=dtype, swiglu=swiglu)


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["route", "route", "gemm", "gemm", "moe", "quant", "quant"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(2, 256 // groups)
        topk_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(16, topk_groups * (experts // groups)))
        c = route("", log(1, 8192), experts, topk, rng.choice(["f16", "bf16", "f32"]), rng.choice(["softmax", "sigmoid"]),
                  rng.random() < 0.5, groups, topk_groups, rng.choice([1, 2]), rng.random() < 0.5,
                  rng.choice([1.0, 2.5]), rng.choice([0, 0, 3]))
    elif kind == "gemm":
        c = gemm("", log(1, 4096), 64 * log(1, 112), 128 * log(1, 56), rng.choice(["bf16", "f16"]))
    elif kind == "moe":
        experts = log(2, 64)
        c = moe("", log(1, 4096), experts, rng.randint(1, min(8, experts)), 64 * log(1, 44), 128 * log(1, 32),
                rng.choice(["bf16", "f16"]))
    else:
        swiglu = rng.random() < 0.5
        k = 8 * log(1, 1024)
        c = quant("", log(1, max(1, min(16384, (1 << 26) // k))), k, rng.choice(["bf16", "f16"]), swiglu)
    del c["name"]
    return c


def rows_of_codes(gen, rows, k, sigma):
    """Normal rows, quantized to int8 by their largest magnitude: codes and scales."""
    v = torch.randn((rows, k), generator=gen, device="cuda") * sigma
    s = v.abs().amax(1).clamp_min(1e-20) / 127
    return torch.round(v / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        wide = torch.randn((case["tokens"], case["experts"] + case["pad"]), generator=gen, device="cuda") * 1.5
        s["logits"] = wide.to(DT[case["dtype"]])
        s["bias_row"] = None
        if case["bias"]:
            s["bias_row"] = torch.randn(case["experts"], generator=gen, device="cuda") * 0.05
        if own:
            import quantized_gemm_amd as qg
            s["desc"] = qg.make_route_desc(qg.R_SOFTMAX if case["scoring"] == "softmax" else qg.R_SIGMOID,
                                           case["experts"], case["topk"], case["groups"], case["topk_groups"],
                                           case["group_top"], case["renorm"], case["scale"])
            s["type"] = {"f16": qg.L_F16, "bf16": qg.L_BF16, "f32": qg.L_F32}[case["dtype"]]
    elif case["op"] == "gemm":
        s["x"], s["sx"] = rows_of_codes(gen, case["m"], case["k"], 1.0)
        w, sw = rows_of_codes(gen, case["n"], case["k"], 0.02)
        keep_weights(s, w, sw, 1)
    elif case["op"] == "moe":
        t, e, topk = case["tokens"], case["experts"], case["topk"]
        s["x"], s["sx"] = rows_of_codes(gen, t, case["k"], 1.0)
        ids = torch.topk(torch.randn((t, e), generator=gen, device="cuda"), topk, dim=1).indices
        s["ids"] = ids.to(torch.int32).contiguous()
        s["most"] = int(torch.bincount(ids.flatten(), minlength=e).max())   # rows of the busiest expert
        w, sw = rows_of_codes(gen, e * case["n"], case["k"], 0.02)
        keep_weights(s, w, sw, e)
        if own:
            import quantized_gemm_amd as qg
            s["block"] = qg.moe_block_m(s["handle"], t, topk)
            cap_rows, cap_blocks = qg.moe_capacity(t, topk, e, s["block"])
            s["map"] = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (cap_rows, cap_blocks, 1)]
    else:
        width = case["k"] * (2 if case["swiglu"] else 1)
        s["x"] = (torch.randn((case["rows"], width), generator=gen, device="cuda") * 2).to(DT[case["dtype"]])
    return s


def keep_weights(s, w, sw, experts):
    """The layer's weights: as they are, or in the image the framework's products read."""
    if own:
        import quantized_gemm_amd as qg
        desc = qg.make_desc(qg.W_INT8, qg.S_F32, 0, 0, qg.A_INT8, qg.C_NATIVE, qg.O_F16 if s["out"] == "f16" else qg.O_BF16,
                            experts, s["n"], s["k"])
        s["image"] = torch.empty(qg.prepared_bytes(desc), dtype=torch.uint8, device="cuda")
        s["handle"] = qg.prepare(desc, w, sw, None, s["image"])
        need = qg.workspace_bytes(s["handle"], s["m"]) if "m" in s else 0
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    else:
        s["w"], s["sw"] = w, sw


def run(s):
    if own:
        return run_own(s)
    if s["op"] == "route":
        return plain_route(s)
    if s["op"] == "gemm":
        y = s["x"].float() @ s["w"].float().t()
        return (y * s["sw"] * s["sx"][:, None]).to(DT[s["out"]])
    if s["op"] == "moe":
        return plain_moe(s)
    return plain_quant(s)


def run_own(s):
    import quantized_gemm_amd as qg
    if s["op"] == "route":
        ids = torch.empty((s["tokens"], s["topk"]), dtype=torch.int32, device="cuda")
        weights = torch.empty((s["tokens"], s["topk"]), dtype=torch.float32, device="cuda")
        qg.moe_route(s["desc"], s["logits"], s["type"], s["tokens"], ids, weights, s["bias_row"],
                     row_stride=s["experts"] + s["pad"])
        return {"ids": ids, "weights": weights}
    if s["op"] == "gemm":
        y = torch.empty((s["m"], s["n"]), dtype=DT[s["out"]], device="cuda")
        qg.gemm(s["handle"], s["x"], s["sx"], y, s["m"], s["ws"])
        return y
    if s["op"] == "moe":
        t, topk = s["tokens"], s["topk"]
        y = torch.empty((t, topk, s["n"]), dtype=DT[s["out"]], device="cuda")
        qg.moe_align(s["ids"], t, topk, s["experts"], s["block"], *s["map"])
        qg.moe_gemm(s["handle"], s["x"], s["sx"], *s["map"], t, topk, s["block"], y)
        return y
    codes = torch.empty((s["rows"], s["k"]), dtype=torch.int8, device="cuda")
    scale = torch.empty(s["rows"], dtype=torch.float32, device="cuda")
    if s["swiglu"]:
        qg.moe_swiglu(s["x"], s["rows"], s["k"], qg.O_F16 if s["dtype"] == "f16" else qg.O_BF16, qg.A_INT8, codes, scale)
    else:
        qg.quantize_int8_rows(s["x"], s["rows"], s["k"], qg.A_F16 if s["dtype"] == "f16" else qg.A_BF16, codes, scale)
    return values_of(codes, scale)


def values_of(codes, scale):
    """int8 codes as the values they stand for (16 bits are enough to tell codes apart)."""
    values = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    torch.mul(codes, scale[:, None], out=values)
    return {"values": values, "scale": scale}


def plain_route(s):
    e, g = s["experts"], s["groups"]
    l = s["logits"][:, :e].double()
    if s["scoring"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    choice = score if s["bias_row"] is None else score + s["bias_row"].double()
    if g > 1:
        by_group = choice.reshape(-1, g, e // g)
        value = torch.sort(by_group, dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], by_group, -math.inf).reshape(-1, e)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    weights = torch.gather(score, 1, ids)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (weights * s["scale"]).float()}


def plain_moe(s):
    t, topk, e, n, k = s["tokens"], s["topk"], s["experts"], s["n"], s["k"]
    flat = s["ids"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    expert = flat[order]
    counts = (flat[:, None] == torch.arange(e, device=flat.device)).sum(0)
    start = torch.cumsum(counts, 0) - counts
    slot = expert * s["most"] + torch.arange(t * topk, device=flat.device) - start[expert]
    rows = torch.zeros((e * s["most"], k), device=flat.device)
    rows[slot] = s["x"].float()[order // topk]
    products = torch.bmm(rows.reshape(e, s["most"], k), s["w"].float().reshape(e, n, k).transpose(1, 2))
    y = products.reshape(-1, n)[slot] * s["sw"].reshape(e, n)[expert] * s["sx"][order // topk][:, None]
    out = torch.empty((t * topk, n), dtype=DT[s["out"]], device=flat.device)
    out[order] = y.to(out.dtype)
    return out.reshape(t, topk, n)


def plain_quant(s):
    x = s["x"].float()
    if s["swiglu"]:
        gate, up = x[:, :s["k"]], x[:, s["k"]:]
        x = gate / (1 + torch.exp(-gate)) * up
    largest = x.abs().amax(1)
    scale = torch.where(largest == 0, 1.0, largest / 127)
    codes = torch.clamp(torch.round(x / scale[:, None]), -127, 127)
    return {"values": (codes * scale[:, None]).to(torch.bfloat16), "scale": scale}


def work(case):
    if case["op"] == "route":
        size = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
        t, e = case["tokens"], case["experts"]
        # an exponential, a sum and a comparison for each logit
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * case["topk"], "flops": 3 * t * e}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "moe":
        t, topk, n, k = case["tokens"], case["topk"], case["n"], case["k"]
        e = case["experts"]
        used = e * (1 - (1 - topk / e) ** t)   # experts that some token goes to, on average
        return {"bytes": used * n * (k + 4) + t * (k + 4) + t * topk * (4 + 2 * n), "flops": 2 * t * topk * n * k}
    read = case["rows"] * case["k"] * (4 if case["swiglu"] else 2)
    return {"bytes": read + case["rows"] * (case["k"] + 4), "flops": (8 if case["swiglu"] else 4) * case["rows"] * case["k"]}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits, on the inputs of prepare()."""
    s = prepare(case, seed)
    if case["op"] == "route":
        return exact_route(s)
    if case["op"] == "gemm":
        acc = torch.matmul(s["x"].double(), s["w"].double().t())
        return acc * (s["sw"].double()[None, :] * s["sx"].double()[:, None])
    if case["op"] == "moe":
        t, topk, n, k = s["tokens"], s["topk"], s["n"], s["k"]
        out = torch.zeros((t, topk, n), dtype=torch.float64, device="cuda")
        w, sw = s["w"].reshape(-1, n, k), s["sw"].reshape(-1, n)
        for e in range(s["experts"]):
            tok, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            if tok.numel():
                out[tok, slot] = (s["x"][tok].double() @ w[e].double().t()) * sw[e].double() * s["sx"][tok].double()[:, None]
        return out
    x = s["x"].double()
    if s["swiglu"]:
        x = torch.sigmoid(x[:, :s["k"]]) * x[:, :s["k"]] * x[:, s["k"]:]
    # the scale is a float32 and the quotient is rounded to one before it is rounded to a code
    scale = (x.abs().amax(1) / 127).float().double()
    scale[scale == 0] = 1
    codes = (x / scale[:, None]).float().double().round().clamp(-127, 127)
    return {"values": codes * scale[:, None], "scale": scale}


def exact_route(s):
    e, g = s["experts"], s["groups"]
    l = s["logits"].double().cpu().numpy()[:, :e]
    if s["scoring"] == "softmax":
        score = np.exp(l - np.logaddexp.reduce(l, axis=1)[:, None])
    else:
        score = np.exp(-np.logaddexp(0, -l))
    choice = score + (0 if s["bias_row"] is None else s["bias_row"].double().cpu().numpy())
    # numbers that go up with the choice value and, among equal ones, down with the index
    size = e // g
    best = -np.sort(-choice.reshape(-1, g, size), axis=2)[:, :, :s["group_top"]].sum(2)
    group_rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
    open_ = np.repeat(group_rank < s["topk_groups"], size, axis=1)
    ids = np.argsort(np.where(open_ if g > 1 else True, -choice, np.inf), axis=1, kind="stable")[:, :s["topk"]]
    weights = np.take_along_axis(score, ids, 1)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdims=True)
    return {"ids": None, "weights": weights * s["scale"]}
