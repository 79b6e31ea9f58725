"""Cases of operators around the quantized projections of a decoder layer: the norms before and after a
block, with its gate, its residual and the quantization of what the next projection reads; the low-rank
adapters of many requests beside a projection that they share; a paged cache of keys and values in 4 bits;
and the attention that reads it.

`own` False: the operators in plain torch; True: the calls a user makes of quantized_gemm_amd.

The formulas, with N(v) = (v - c) / sqrt(mean((v - c)^2) + eps) * (offset + weight) + bias, c = 0 (RMS) or
mean(v) (layer norm):

* norm rows: h = y or N_post(y), the block's output; u = residual + res_scale * gate * h, the new residual;
  z = N(u), in 16 bits and/or as codes: e4m3 (scale = max|row| / 448), int8 (max|row| / 127) or MXFP4
  (one power of two per 32: exponent of their largest magnitude less 2; e2m1 codes).  Codes are taken
  from z before any rounding to 16 bits.
* adapters: a token with adapter a, t = x A[a, s]^T over the first rank[a] rows for each slice s of the
  projection's columns, out[n] = base[n] + scale[a] * sum_r t[slice of n, r] B[a, n, r].  A token without
  an adapter keeps its row.
* cache: the key and value rows of a token are held as MXFP4 along the head's dimension, at the token's slot
  (page * page's tokens + place in the page).
* attention: query i of a sequence's n_q newest tokens stands at position len - n_q + i and sees the tokens up
  to that; out = softmax(scale q K^T) V per query head, consecutive query heads sharing a key head.
"""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]   # between neighbouring magnitudes


def listed():
    return [
        # one token of a decoding step, in front of an e4m3 projection with adapters: codes and 16-bit rows
        norm("norm_t1_e4m3", 1, 7168, code="e4m3", out=True),
        # the largest batch: norms on both sides of a block, one gate for all tokens, e4m3 codes
        norm("norm_both_t16384", 16384, 4096, post="rms", gate="one", res_scale=1.4, offset=1.0, code="e4m3"),
        # odd sizes, layer norm with a bias, int8 codes, a residual kept in float32, rows of wider tensors
        norm("norm_layer_ragged", 1021, 1416, dtype="f16", kind="layer", bias=True, res="f32", pad=8, code="int8"),
        # one token of a decoding step
        lora("lora_t1", 1, 8, 16, 7168, 7168),
        # a decoding batch on the joint q, k, v projection, every token of another request, mixed ranks
        lora("lora_qkv_t256", 256, 32, 64, 4096, 6144, slices=3, mixed=True),
        # the prefill of several requests, gate and up projections, high rank
        lora("lora_gate_up_t8192", 8192, 4, 128, 4096, 5632, slices=2, dtype="f16", runs=True),
        # the new tokens of a decoding batch on their way into the cache, and back
        kv("kv_t64", 64, 8, 128, 16),
        # those of a prefill
        kv("kv_t8192", 8192, 8, 128, 64),
        # one token of one long sequence
        attn("attn_b1_l32768", 1, 32, 8, 128, 64, 32768),
        # a decoding batch with sequences of all lengths
        attn("attn_b64_l8192", 64, 64, 8, 128, 16, 8192),
        # a chunk of a prefill behind what is cached
        attn("attn_b4_q512_l4608", 4, 32, 8, 128, 64, 4608, nq=512),
        # odd counts, three tokens of each sequence (a guess to be checked)
        attn("attn_f16_ragged", 13, 15, 5, 64, 32, 1009, nq=3, dtype="f16"),
    ]


def norm(name, rows, k, dtype="bf16", kind="rms", post="", gate="", res="", res_scale=1.0, offset=0.0, bias=False,
         code="", out=False, pad=0):
    return dict(name=name, op="norm", rows=rows, k=k, dtype=dtype, kind=kind, post=post, gate=gate, res=res or dtype,
                res_scale=res_scale, offset=offset, bias=bias, code=code, out=out, pad=pad)


def lora(name, tokens, adapters, rank, k, n, slices=1, mixed=False, dtype="bf16", runs=False, pad=0):
    return dict(name=name, op="lora", tokens=tokens, adapters=adapters, rank=rank, k=k, n=n, slices=slices, mixed=mixed,
                dtype=dtype, runs=runs, pad=pad)


def kv(name, tokens, kv_heads, dim, page, dtype="bf16", pad=0):
    return dict(name=name, op="kv", tokens=tokens, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, pad=pad)


def attn(name, batch, heads, kv_heads, dim, page, length, nq=1, dtype="bf16"):
    """`length`: of the longest sequence; nq: new tokens of each sequence, the newest."""
    return dict(name=name, op="attn", batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page, length=length, nq=nq,
                dtype=dtype)


def lengths(case):
    """The sequences' lengths, spread evenly up to the longest."""
    return [max(case["nq"], case["length"] * (i + 1) // case["batch"]) for i in range(case["batch"])]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["norm", "norm", "lora", "lora", "kv", "attn", "attn"])
    if kind == "norm":
        code = rng.choice(["", "", "e4m3", "e4m3", "int8", "e2m1"])
        k = 32 * log(1, 1024) if code == "e2m1" else 8 * log(4, 4096)
        dtype = rng.choice(["bf16", "bf16", "f16"])
        c = norm("", log(1, max(1, min(16384, (1 << 25) // k))), k, dtype, rng.choice(["rms", "rms", "layer"]),
                 rng.choice(["", "rms", "layer"]), rng.choice(["", "one", "rows"]), rng.choice([dtype, "f32"]),
                 rng.choice([1.0, 0.5, 1.4]), rng.choice([0.0, 1.0]), rng.random() < 0.3, code,
                 not code or rng.random() < 0.3, rng.choice([0, 0, 8, 24]))
    elif kind == "lora":
        rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
        slices = rng.choice([1, 1, 2, 3])
        k, n = 8 * log(16, 896), slices * 32 * log(2, 224 // slices) + rng.choice([0, 8, 24])
        # no more operations and bytes than the largest listed case
        most = min(8192, (1 << 20) * 13824 // (rank * (slices * k + n)), (1 << 28) // (2 * k + 4 * n))
        tokens = log(1, most)
        adapters = log(1, min(32, max(1, 80_000_000_000 // (tokens * rank * slices * (k + n)))))
        c = lora("", tokens, adapters, rank, k, n, slices, rng.random() < 0.5, rng.choice(["bf16", "bf16", "f16"]),
                 tokens > 256 or rng.random() < 0.3, rng.choice([0, 0, 8]))
    elif kind == "kv":
        dim, heads = rng.choice([64, 128, 128, 256]), rng.randint(1, 16)
        c = kv("", log(1, min(8192, (1 << 23) // (dim * heads))), heads, dim, rng.choice([16, 32, 64, 128]),
               rng.choice(["bf16", "f16"]), rng.choice([0, 8]))
    else:
        dim, kv_heads, group = rng.choice([64, 128, 128, 256]), rng.randint(1, 8), rng.choice([1, 2, 3, 4, 6, 8, 16])
        nq = rng.choice([1, 1, 1, 1, log(2, 8), log(2, 512)])
        length = log(max(nq, 2), 32768)
        # no more operations and bytes than the largest listed cases
        wide = length * group * kv_heads * dim
        nq = min(nq, max(1, 20_000_000_000 // wide))
        c = attn("", log(1, max(1, min(64, (1 << 28) // (length * kv_heads * dim), 20_000_000_000 // (nq * wide)))), group * kv_heads, kv_heads, dim, rng.choice([16, 32, 64, 128]), length, nq,
                 rng.choice(["bf16", "bf16", "f16"]))
    del c["name"]
    return c


def slice_ends(case):
    """Ends of the slices: multiples of 32, the first half of the columns or more where there are several."""
    n, s = case["n"], case["slices"]
    if s == 1:
        return [n]
    if s == 2:
        return [n // 64 * 32, n]
    first = n * 2 // 3 // 32 * 32
    return [first, first + (n - first) // 64 * 32, n]


def strided(gen, rows, width, pad, dtype, sigma=1.0):
    """Normal rows; with `pad` the first columns of wider rows."""
    return (torch.randn((rows, width + pad), generator=gen, device="cuda") * sigma).to(dtype)[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    t = DT[case["dtype"]]
    if case["op"] == "norm":
        rows, k, pad = case["rows"], case["k"], case["pad"]
        s["y"] = strided(gen, rows, k, pad, t)
        s["residual"] = strided(gen, rows, k, pad, DT[case["res"]], 3.0)
        s["w"] = (torch.randn(k, generator=gen, device="cuda") * 0.2 + 1 - case["offset"]).to(t)
        s["wp"] = (torch.randn(k, generator=gen, device="cuda") * 0.2 + 1 - case["offset"]).to(t) if case["post"] else None
        s["b"] = (torch.randn(k, generator=gen, device="cuda") * 0.1).to(t) if case["bias"] else None
        gates = {"": 0, "one": 1, "rows": rows}[case["gate"]]
        s["g"] = torch.sigmoid(torch.randn((gates, k), generator=gen, device="cuda")).to(t) if gates else None
        if own:
            prepare_norm(s)
    elif case["op"] == "kv":
        m, h, d = case["tokens"], case["kv_heads"], case["dim"]
        s["k"], s["v"] = (strided(gen, m, h * d, case["pad"], t) for _ in range(2))
        s["pages"] = 2 * (m // case["page"] + 1)
        s["slots"] = torch.randperm(s["pages"] * case["page"], generator=gen, device="cuda")[:m].to(torch.int32)
        if own:
            prepare_kv(s)
            s["k_back"], s["v_back"] = (torch.empty((m, h * d), dtype=t, device="cuda") for _ in range(2))
    elif case["op"] == "attn":
        prepare_attn(s, gen)
    else:
        m, e, r, k, n, pad = (case[i] for i in ("tokens", "adapters", "rank", "k", "n", "pad"))
        s["ends"] = slice_ends(case)
        s["x"] = strided(gen, m, k, pad, t)
        s["base"] = strided(gen, m, n, pad, t)
        s["a"] = (torch.randn((e, case["slices"], r, k), generator=gen, device="cuda") / k ** 0.5).to(t)
        s["b"] = (torch.randn((e, n, r), generator=gen, device="cuda") / r ** 0.5).to(t)
        s["ranks"] = torch.full((e,), r, dtype=torch.int32, device="cuda")
        if case["mixed"]:
            s["ranks"] = torch.randint(1, r // 8 + 1, (e,), generator=gen, device="cuda").to(torch.int32) * 8
        s["scales"] = 0.25 + torch.rand(e, generator=gen, device="cuda")
        if case["runs"]:   # requests of neighbouring tokens
            starts = torch.randint(0, m, (2 * e,), generator=gen, device="cuda").sort().values
            run_of = torch.searchsorted(starts, torch.arange(m, device="cuda"), right=True)
            s["ids"] = torch.randint(0, e, (2 * e + 1,), generator=gen, device="cuda")[run_of].to(torch.int32)
        else:
            s["ids"] = torch.randint(-1 if m > 1 else 0, e, (m,), generator=gen, device="cuda").to(torch.int32)
        if own:
            prepare_lora(s)
    return s


def prepare_norm(s):
    """What a program keeps: the description and the tensors that the outputs go to."""
    import quantized_gemm_amd as qg
    kinds = {"": 0, "rms": qg.N_RMS, "layer": qg.N_LAYER}
    rows, k, width = s["rows"], s["k"], s["k"] + s["pad"]
    s["desc"] = qg.make_norm_desc(
        kinds[s["kind"]], qg.O_F16 if s["dtype"] == "f16" else qg.O_BF16, k, EPS, post_norm=kinds[s["post"]],
        res_type={"f16": qg.L_F16, "bf16": qg.L_BF16, "f32": qg.L_F32}[s["res"]],
        code_type={"": 0, "e4m3": qg.A_FP8_E4M3, "int8": qg.A_INT8, "e2m1": qg.A_FP4_E2M1}[s["code"]],
        weight_offset=s["offset"], res_scale=s["res_scale"], y_stride=width, res_stride=width,
        gate_stride=k if s["gate"] == "rows" else 0)
    s["res_out"] = torch.empty((rows, width), dtype=DT[s["res"]], device="cuda")[:, :k]
    s["z"] = torch.empty((rows, k), dtype=DT[s["dtype"]], device="cuda") if s["out"] else None
    s["codes"] = s["scale"] = None
    if s["code"]:
        s["codes"] = torch.empty((rows, k // 2 if s["code"] == "e2m1" else k), device="cuda",
                                 dtype=torch.int8 if s["code"] == "int8" else torch.uint8)
        s["scale"] = torch.empty((rows, k // 32) if s["code"] == "e2m1" else (rows,), device="cuda",
                                 dtype=torch.uint8 if s["code"] == "e2m1" else torch.float32)
    if s["code"] == "e2m1":
        byte = torch.arange(256, device="cuda")
        value = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
        s["pairs"] = torch.stack([value[byte % 16], value[byte // 16]], 1).to(torch.bfloat16)


def prepare_lora(s):
    """What a program keeps for a batch: which tokens use which adapter, in blocks, for all its projections."""
    import quantized_gemm_amd as qg
    m, e, width = s["tokens"], s["adapters"], s["n"] + s["pad"]
    s["desc"] = qg.make_lora_desc(qg.O_F16 if s["dtype"] == "f16" else qg.O_BF16, e, s["rank"], s["k"], s["ends"],
                                  x_stride=s["k"] + s["pad"], base_stride=width, y_stride=width)
    s["block"] = qg.lora_block_m(m, e)
    cap_rows, cap_blocks = qg.moe_capacity(m, 1, e, s["block"])
    s["map"] = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (cap_rows, cap_blocks, 1)]
    qg.moe_align(s["ids"], m, 1, e, s["block"], *s["map"])
    s["ws"] = torch.empty(qg.lora_workspace_bytes(s["desc"], m, s["block"]), dtype=torch.uint8, device="cuda")
    s["y"] = torch.empty((m, width), dtype=DT[s["dtype"]], device="cuda")[:, :s["n"]]
    s["some_without"] = bool((s["ids"] < 0).any())


def prepare_kv(s):
    """What a program keeps: the description and the cache's pages."""
    import quantized_gemm_amd as qg
    s["desc"] = qg.make_kv_desc(qg.O_F16 if s["dtype"] == "f16" else qg.O_BF16, s["kv_heads"], s["dim"], s["page"], s["pages"])
    s["cache"] = torch.zeros(qg.kv_cache_bytes(s["desc"]), dtype=torch.uint8, device="cuda")


def prepare_attn(s, gen):
    """The queries, and keys and values of all cached tokens in 4 bits, pages in any order."""
    b, h, d, p, t = s["batch"], s["kv_heads"], s["dim"], s["page"], DT[s["dtype"]]
    lens = lengths(s)
    order = torch.randperm(b, generator=gen, device="cuda").tolist()
    lens = [lens[i] for i in order]
    most = -(-max(lens) // p)
    held = torch.tensor([-(-n // p) for n in lens], device="cuda")
    s["pages"] = int(held.sum())
    table = torch.zeros((b, most), dtype=torch.int64, device="cuda")
    places = torch.arange(most, device="cuda") < held[:, None]
    table[places] = torch.randperm(s["pages"], generator=gen, device="cuda")
    s["table"], s["lens"] = table.to(torch.int32), torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["offsets"] = torch.arange(b + 1, dtype=torch.int32, device="cuda") * s["nq"]
    s["q"] = (torch.randn((b * s["nq"], s["heads"] * d), generator=gen, device="cuda") * 1.5).to(t)
    s["scale"] = d ** -0.5
    if own:
        import quantized_gemm_amd as qg
        prepare_kv(s)
        s["ws"] = torch.empty(max(1, qg.attention_workspace_bytes(s["desc"], s["heads"], b, s["nq"], b * s["nq"], max(lens))),
                              dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["q"])
    else:
        rows = s["pages"] * p
        s["held"] = [[torch.empty((rows, h, w), dtype=torch.uint8, device="cuda") for w in (d // 2, d // 32)] for _ in "kv"]
    step = max(p, (1 << 24) // (h * d) // p * p)
    for first in range(0, s["pages"] * p, step):   # rows in parts, so that little memory is needed
        rows = min(step, s["pages"] * p - first)
        new = [torch.randn((rows, h * d), generator=gen, device="cuda").to(t) for _ in "kv"]
        if own:
            qg.kv_append(s["desc"], *new, torch.arange(first, first + rows, dtype=torch.int32, device="cuda"), rows, s["cache"])
        else:
            for held, x in zip(s["held"], new):
                codes, power = e2m1_codes(x.float().reshape(rows, h, d // 32, 32))
                codes = codes.reshape(rows, h, d // 2, 2)
                held[0][first:first + rows] = codes[..., 0] + 16 * codes[..., 1]
                held[1][first:first + rows] = (power + 127).to(torch.uint8)


def run(s):
    return globals()[("own_" if own else "plain_") + s["op"]](s)


def own_norm(s):
    import quantized_gemm_amd as qg
    qg.norm_rows(s["desc"], s["rows"], s["y"], s["residual"], s["res_out"], s["z"], s["codes"], s["scale"], weight=s["w"],
                 bias=s["b"], gate=s["g"], post_weight=s["wp"])
    got = {"residual": s["res_out"]}
    if s["out"]:
        got["out"] = s["z"]
    if s["code"] == "e4m3":
        got["codes"], got["scale"] = s["codes"].view(torch.float8_e4m3fn), s["scale"]
    elif s["code"] == "int8":
        got["codes"], got["scale"] = s["codes"].to(torch.bfloat16), s["scale"]   # whole numbers up to 127
    elif s["code"] == "e2m1":
        power = torch.exp2(s["scale"].float() - 127)
        values = s["pairs"][s["codes"].int()].reshape(s["rows"], -1, 32) * power[:, :, None]
        got["values"] = values.reshape(s["rows"], -1).to(torch.bfloat16)
    return got


def own_lora(s):
    import quantized_gemm_amd as qg
    base = s["base"]
    if s["some_without"]:   # the rows of tokens without an adapter are not written: y in base's place
        base = s["y"].copy_(base)
    qg.lora(s["desc"], s["x"], s["a"], s["b"], *s["map"], s["tokens"], s["block"], base, s["y"], s["ws"],
            ranks=s["ranks"], scales=s["scales"])
    return s["y"]


def own_kv(s):
    import quantized_gemm_amd as qg
    width = s["kv_heads"] * s["dim"] + s["pad"]
    qg.kv_append(s["desc"], s["k"], s["v"], s["slots"], s["tokens"], s["cache"], k_stride=width, v_stride=width)
    qg.kv_read(s["desc"], s["cache"], s["slots"], s["tokens"], s["k_back"], s["v_back"])
    return {"k": s["k_back"], "v": s["v_back"]}


def own_attn(s):
    import quantized_gemm_amd as qg
    qg.attention(s["desc"], s["q"], s["heads"], s["cache"], s["table"], s["lens"], s["batch"], s["length"], s["scale"],
                 s["out"], s["ws"], q_offsets=s["offsets"] if s["nq"] > 1 else None, max_q=s["nq"])
    return s["out"]


def plain_norm_of(v, kind, weight, offset, bias):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * (weight.float() + offset)
    return v if bias is None else v + bias.float()


def plain_norm(s):
    h = s["y"].float()
    if s["post"]:
        h = plain_norm_of(h, s["post"], s["wp"], s["offset"], None)
    if s["g"] is not None:
        h = h * s["g"].float()
    u = s["residual"].float() + s["res_scale"] * h
    z = plain_norm_of(u, s["kind"], s["w"], s["offset"], s["b"])
    got = {"residual": u.to(DT[s["res"]])}
    if s["out"]:
        got["out"] = z.to(DT[s["dtype"]])
    if s["code"] == "e2m1":
        got["values"] = e2m1_values(z.reshape(s["rows"], -1, 32)).reshape(s["rows"], -1).to(torch.bfloat16)
    elif s["code"]:
        scale = z.abs().amax(1) / (448 if s["code"] == "e4m3" else 127)
        scale = torch.where(scale == 0, 1.0, scale)
        q = z / scale[:, None]
        got["codes"] = q.to(torch.float8_e4m3fn) if s["code"] == "e4m3" else torch.round(q).to(torch.bfloat16)
        got["scale"] = scale
    return got


def e2m1_codes(blocks):
    """e2m1 codes of blocks [..., 32] and their powers of two.  A code is the place of a value's magnitude, over
    the power, among the borders, a border itself going to the even code."""
    power = torch.floor(torch.log2(blocks.abs().amax(-1).double())) - 2
    borders = torch.tensor(E2M1_BORDERS, device=blocks.device)
    up = torch.tensor([False, True, False, True, False, True, False], device=blocks.device)
    q = blocks * torch.exp2(-power).float()[..., None]
    m = q.abs()[..., None]
    code = torch.where(up, m >= borders, m > borders).sum(-1)
    return torch.where((q < 0) & (code > 0), code + 8, code).to(torch.uint8), power


def e2m1_values(blocks):
    codes, power = e2m1_codes(blocks)
    value = torch.tensor(E2M1 + [-v for v in E2M1], device=blocks.device)
    return value[codes.int()] * torch.exp2(power).float()[..., None]


def plain_kv(s):
    m, t = s["tokens"], DT[s["dtype"]]
    back = e2m1_values(torch.stack([s["k"], s["v"]]).float().reshape(2, m, -1, 32)).reshape(2, m, -1).to(t)
    return {"k": back[0], "v": back[1]}


def plain_attn(s):
    b, h, d, p, nq = s["batch"], s["kv_heads"], s["dim"], s["page"], s["nq"]
    group = s["heads"] // h
    place = torch.arange(s["length"], device="cuda")
    slots = (s["table"][:, place // p] * p + place % p).long()          # [b, length]
    byte = torch.arange(256, device="cuda")
    value = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    pairs = torch.stack([value[byte % 16], value[byte // 16]], 1)

    def rows(held):
        codes, power = held[0][slots], held[1][slots]
        x = pairs[codes.int()].reshape(b, s["length"], h, d // 32, 32) * torch.exp2(power.float() - 127)[..., None]
        return x.reshape(b, s["length"], h, d).transpose(1, 2).contiguous()

    # query rows of a key head together: [b * h, nq * group, d]
    q = s["q"].float().reshape(b, nq, h, group, d).permute(0, 2, 1, 3, 4).reshape(b * h, nq * group, d).contiguous()
    keys = rows(s["held"][0]).reshape(b * h, -1, d)
    score = torch.bmm(q, keys.transpose(1, 2).contiguous()).reshape(b, h, nq, group, -1) * s["scale"]
    last = s["lens"][:, None] - nq + torch.arange(nq, device="cuda")    # [b, nq]
    seen = place <= last[:, :, None]
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    weight = (e / e.sum(-1, keepdim=True)).reshape(b * h, nq * group, -1)
    # what no query sees holds no finite numbers for sure
    inside = (place < s["lens"][:, None])[:, None, :, None]
    values = torch.where(inside, rows(s["held"][1]), 0.0).reshape(b * h, -1, d)
    out = torch.bmm(weight, values).reshape(b, h, nq, group, d).permute(0, 2, 1, 3, 4)
    return out.reshape(b * nq, -1).to(DT[s["dtype"]])


def plain_lora(s):
    m, e, r, n, parts = s["tokens"], s["adapters"], s["rank"], s["n"], s["slices"]
    t = s["x"].float() @ s["a"].float().reshape(-1, s["k"]).t()
    inside = torch.arange(r, device="cuda") < s["ranks"][:, None]
    used = torch.arange(e, device="cuda") == s["ids"][:, None]
    t = torch.where(used[:, :, None, None], t.reshape(m, e, parts, r), 0.0)
    t = t * torch.where(inside, s["scales"][:, None], 0.0)[:, None]
    ends = torch.tensor(s["ends"], device="cuda")
    slice_of = (torch.arange(n, device="cuda")[:, None] >= ends).sum(1)
    mine = slice_of == torch.arange(parts, device="cuda")[:, None]
    b = torch.where(mine[None, :, None], s["b"].float().transpose(1, 2)[:, None], 0.0)   # [e, slice, r, n]
    delta = t.reshape(m, -1) @ b.reshape(-1, n)
    return (s["base"].float() + delta).to(DT[s["dtype"]])


def work(case):
    if case["op"] == "norm":
        rows, k = case["rows"], case["k"]
        res = 4 if case["res"] == "f32" else 2
        per = 2 + 2 * res + (2 if case["out"] else 0) + (2 if case["gate"] == "rows" else 0)
        per += {"": 0, "e4m3": 1, "int8": 1, "e2m1": 0.5 + 1 / 32}[case["code"]]
        vectors = 1 + (case["post"] != "") + (case["gate"] == "one") + case["bias"]
        scales = 4 * rows if case["code"] in ("e4m3", "int8") else 0
        return {"bytes": rows * k * per + 2 * k * vectors + scales, "flops": rows * k * (12 if case["post"] else 8)}
    if case["op"] == "kv":   # rows in, codes and scales out and in again, rows out
        width = case["kv_heads"] * case["dim"]
        return {"bytes": case["tokens"] * (8 * width + 4 * (width // 2 + width // 32)), "flops": 20 * case["tokens"] * width}
    if case["op"] == "attn":
        b, nq, hd = case["batch"], case["nq"], case["heads"] * case["dim"]
        tokens = sum(lengths(case))
        seen = nq * tokens - b * nq * (nq - 1) // 2
        cached = tokens * case["kv_heads"] * (case["dim"] + case["dim"] // 16)
        return {"bytes": cached + 4 * b * nq * hd, "flops": 4 * seen * hd}
    m, e, r, k, n, parts = (case[i] for i in ("tokens", "adapters", "rank", "k", "n", "slices"))
    mean = r * (0.5 + 4 / r) if case["mixed"] else r   # ranks are even multiples of 8 up to the largest
    used = e * (1 - (1 - 1 / e) ** min(m, 2 * e + 1 if case["runs"] else m))
    return {"bytes": m * (2 * k + 4 * n) + used * mean * 2 * (parts * k + n), "flops": 2 * m * mean * (parts * k + n)}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits, on the inputs of prepare()."""
    if case["op"] == "attn":
        return exact_attn(case, seed)
    s = prepare(case, seed)
    if case["op"] == "kv":
        return {i: exact_e2m1(s[i].double().reshape(s["tokens"], -1, 32)).reshape(s["tokens"], -1) for i in "kv"}
    return exact_norm(s) if case["op"] == "norm" else exact_lora(s)


def exact_e2m1(blocks):
    exponent = torch.frexp(blocks.abs().amax(-1, keepdim=True)).exponent - 3
    q = torch.ldexp(blocks, -exponent)
    # the steps between e2m1 magnitudes: 1/2 below 2, 1 below 4, 2 above; halves go to even multiples
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0)).double()
    return torch.ldexp((torch.round(q / step) * step).clamp(-6, 6), exponent)


def exact_attn(case, seed):
    global own
    mine, own = own, False   # the codes, in the plain form's order
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    h, d, p, nq = s["kv_heads"], s["dim"], s["page"], s["nq"]
    group = s["heads"] // h
    value = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda", dtype=torch.float64)
    out = torch.empty((s["batch"], nq, h, group, d), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(s["batch"], nq, h, group, d)
    for b, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[at // p] * p + at % p
        rows = []
        for codes, power in s["held"]:
            c = codes[slots].int()
            x = torch.stack([value[c & 15], value[c >> 4]], -1).reshape(n, h, d // 32, 32)
            rows.append(torch.ldexp(x, (power[slots].int() - 127)[..., None]).reshape(n, h, d))
        hidden = at[None, :] > n - nq + torch.arange(nq, device="cuda")[:, None]
        for head in range(h):
            score = q[b, :, head].reshape(nq * group, d) @ rows[0][:, head].t().contiguous() * s["scale"]
            score = score.reshape(nq, group, n).masked_fill(hidden[:, None], -math.inf)
            out[b, :, head] = torch.softmax(score, -1) @ rows[1][:, head].contiguous()
    return out.reshape(s["batch"] * nq, -1)


def exact_norm(s):
    def normed(v, kind, w, b):
        c = torch.mean(v, 1, keepdim=True) if kind == "layer" else 0.0
        spread = torch.rsqrt(torch.var(v, 1, correction=0, keepdim=True) + EPS) if kind == "layer" else \
            torch.rsqrt(torch.mean(torch.square(v), 1, keepdim=True) + EPS)
        add = torch.zeros_like(w, dtype=torch.float64) if b is None else b.double()
        return torch.addcmul(add.expand_as(v), (v - c) * spread, w.double() + s["offset"])

    h = s["y"].double()
    if s["post"]:
        h = normed(h, s["post"], s["wp"], None)
    u = s["residual"].double() + h * (1.0 if s["g"] is None else s["g"].double()) * s["res_scale"]
    z = normed(u, s["kind"], s["w"], s["b"])
    got = {"residual": u}
    if s["out"]:
        got["out"] = z
    if s["code"] == "e2m1":
        got["values"] = exact_e2m1(z.reshape(s["rows"], -1, 32)).reshape(s["rows"], -1)
    elif s["code"]:
        most = 448 if s["code"] == "e4m3" else 127
        scale = (z.abs().amax(1) / most).float().double()
        scale[scale == 0] = 1
        q = (z / scale[:, None]).clamp(-most, most)
        if s["code"] == "int8":
            got["codes"] = q.round()
        else:   # e4m3: four significant bits, and multiples of 2^-9 below 2^-6
            step = torch.exp2(torch.frexp(q).exponent.clamp_min(-5).double() - 4)
            got["codes"] = torch.round(q / step) * step
        got["scale"] = z.abs().amax(1) / most
    return got


def exact_lora(s):
    out = s["base"].double()
    ids, ranks, scales = s["ids"].cpu().numpy(), s["ranks"].cpu().numpy(), s["scales"].double().cpu().numpy()
    for e in np.unique(ids[ids >= 0]):
        rows = torch.from_numpy(np.nonzero(ids == e)[0]).to("cuda")
        x = s["x"][rows].double()
        begin = 0
        for part, end in enumerate(s["ends"]):
            t = x @ s["a"][e, part, :ranks[e]].double().t().contiguous()
            out[rows, begin:end] += (t @ s["b"][e, begin:end, :ranks[e]].double().t().contiguous()) * scales[e]
            begin = end
    return out
