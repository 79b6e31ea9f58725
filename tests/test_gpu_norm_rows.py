"""GPU parity of the norms around a block (qg_norm_rows).

Bars, from the arithmetic: a float32 sum of a row's squares here takes at most 32 values per thread, 6 exchanges and 16
waves in turn, so it is off by at most 54 * 2^-24 of itself, a factor of the norm (half of that for the root, a reciprocal,
a weight) by less than 2^-18; u and z are a few operations on such values, each rounded to 2^-24 of its
magnitude.  So u is off by 2^-18 of the sum of its terms' magnitudes, z by 2^-17 of its own (it takes u's error
times the factor, and the norm's), before the output's rounding of half a step: bf16 2^-8, f16 2^-11, float32 2^-24 of the
value, and 2^-25 where an f16 is subnormal.  Codes: within half a step of z / scale, and that noise.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import formats as F
from oracle import layer_ops as LO

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
O = {"bf16": qg.O_BF16, "f16": qg.O_F16}
L = {"bf16": qg.L_BF16, "f16": qg.L_F16, "f32": qg.L_F32}
N = {"": 0, "rms": qg.N_RMS, "layer": qg.N_LAYER}
CODE = {"": 0, "e4m3": qg.A_FP8_E4M3, "int8": qg.A_INT8, "e2m1": qg.A_FP4_E2M1}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _d(t):
    return None if t is None else t.double().cpu().numpy()


def _wide(rng, rows, k, pad, dtype, sigma=1.0, mean=0.0):
    v = torch.from_numpy(rng.standard_normal((rows, k + pad)).astype(np.float32) * sigma + mean).to(DT[dtype]).cuda()
    return v, v[:, :k]


class Case:
    """Inputs of one call, its outputs (filled with a pattern first) and the reference."""

    def __init__(self, rows, k, dtype="bf16", kind="rms", post="", res="", code="", out=True, gate="", pad=0, offset=0.0,
                 res_scale=1.0, weight=True, bias=False, y=True, residual=True, res_out=True, eps=1e-6, mean=0.0, seed=0, inplace=False):
        rng = np.random.default_rng(seed + 1000 * rows + k)
        self.rows, self.k, self.dtype, self.res, self.code, self.pad = rows, k, dtype, res or dtype, code, pad
        self.wide_y, self.y = _wide(rng, rows, k, pad, dtype, 1.0, mean) if y else (None, None)
        self.wide_r, self.r = _wide(rng, rows, k, pad, self.res, 3.0, mean) if residual else (None, None)
        vec = lambda s, m: torch.from_numpy(rng.standard_normal(k).astype(np.float32) * s + m).to(DT[dtype]).cuda()  # noqa: E731
        self.w = vec(0.2, 1 - offset) if weight and kind else None
        self.wp = vec(0.2, 1 - offset) if weight and post else None
        self.b = vec(0.3, 0.1) if bias else None
        self.g = None
        if gate:
            self.g = torch.from_numpy(rng.random((1 if gate == "one" else rows, k)).astype(np.float32)).to(DT[dtype]).cuda()
        self.args = dict(kind=kind, post=post, eps=eps, offset=offset, res_scale=res_scale)
        self.desc = qg.make_norm_desc(N[kind], O[dtype], k, eps, post_norm=N[post], res_type=L[self.res], code_type=CODE[code],
                                      weight_offset=offset, res_scale=res_scale, y_stride=k + pad, res_stride=k + pad,
                                      out_stride=k + pad, gate_stride=k if gate == "rows" else 0)
        nan = float("nan")
        self.res_wide = self.out_wide = self.codes = self.scale = None
        if res_out:
            self.res_wide = torch.full((rows, k + pad), nan, dtype=DT[self.res], device="cuda")
        if out and kind:
            self.out_wide = torch.full((rows, k + pad), nan, dtype=DT[dtype], device="cuda")
        if code:
            self.codes = torch.full((rows, k // 2 if code == "e2m1" else k), 0xA5, dtype=torch.uint8, device="cuda")
            self.scale = torch.full((rows, k // 32), 7, dtype=torch.uint8, device="cuda") if code == "e2m1" else \
                torch.full((rows,), nan, device="cuda")
        if inplace:
            self.res_wide, self.out_wide = self.wide_r, self.wide_y
        f = lambda t: _d(t)  # noqa: E731
        self.want = LO.norm_rows(y=f(self.y), res=f(self.r), weight=f(self.w), bias=f(self.b), gate=f(self.g),
                                 post_weight=f(self.wp), **self.args)

    def run(self, stream=None):
        qg.norm_rows(self.desc, self.rows, self.wide_y, self.wide_r, self.res_wide, self.out_wide, self.codes, self.scale,
                     weight=self.w, bias=self.b, gate=self.g, post_weight=self.wp, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        u, z, umag, zmag = self.want
        k = self.k
        if self.res_wide is not None:
            got = _d(self.res_wide[:, :k])
            assert (np.abs(got - u) <= U[self.res] * np.abs(u) + 2.0 ** -18 * umag + 2.0 ** -25).all()
        if self.out_wide is not None:
            got = _d(self.out_wide[:, :k])
            assert (np.abs(got - z) <= U[self.dtype] * np.abs(z) + 2.0 ** -17 * zmag + 2.0 ** -25).all()
        if self.code:
            check_codes(self.code, self.codes, self.scale, z, 2.0 ** -17 * zmag)


def check_codes(code, codes, scale, z, noise):
    rows, k = z.shape
    if code == "e2m1":
        blocks, nb = z.reshape(rows, -1, 32), noise.reshape(rows, -1, 32)
        e = scale.cpu().numpy().astype(int) - 127
        amax, slack = np.abs(blocks).max(axis=2), nb.max(axis=2)
        low, high = np.frexp(amax - slack)[1] - 3, np.frexp(amax + slack)[1] - 3     # where noise can put the exponent
        assert (((e >= low) & (e <= high)) | (amax <= slack)).all()
        power = np.exp2(e.astype(float))[:, :, None]
        got = F.decode_e2m1(F.unpack_u8_nibbles(codes.cpu().numpy())).reshape(blocks.shape)
        q = np.abs(blocks) / power
        half = np.where(q <= 2, 0.25, np.where(q <= 4, 0.5, np.maximum(1.0, q - 6)))
        assert (np.abs(got * power - blocks) <= half * power * (1 + 1e-12) + nb).all()
        return
    most = 448.0 if code == "e4m3" else 127.0
    sc = scale.double().cpu().numpy()
    want = np.abs(z).max(axis=1) / most
    zero = want == 0
    assert (sc[zero] == 1.0).all()
    assert (np.abs(sc - want)[~zero] <= (noise.max(axis=1) / most + 2.0 ** -23 * want)[~zero]).all()
    q = z / sc[:, None]
    slack = noise / sc[:, None] + 2.0 ** -22 * np.abs(q)
    if code == "int8":
        got = codes.view(torch.int8).cpu().numpy().astype(float)
        assert (np.abs(got) <= 127).all() and (np.abs(got - q) <= 0.5 + slack).all()
    else:
        got = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
        # half a step: 2^-4 of the value, 2^-10 where it is subnormal
        assert (np.abs(got - q) <= np.maximum(2.0 ** -4 * np.abs(got), 2.0 ** -10) * (1 + 1e-9) + slack).all()


@pytest.mark.parametrize("k", [8, 128, 512, 520, 1024, 1416, 2048, 2056, 4096, 5120, 8192, 8200, 16384, 16392, 32768])
@pytest.mark.parametrize("rows", [1, 3, 260])
def test_row_lengths(rows, k):
    Case(rows, k, code="e4m3", res="f32" if k % 16 else "").run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", ["", "rms", "layer"])
@pytest.mark.parametrize("gate", ["", "one", "rows"])
def test_variants(dtype, kind, post, gate):
    Case(5, 1416, dtype, kind, post, gate=gate, bias=kind == "layer", offset=1.0 if post else 0.0, res_scale=0.5, pad=8).run().check()
    Case(5, 672, dtype, kind, post, res="f32", code="int8", gate=gate, bias=True, pad=24).run().check()


@pytest.mark.parametrize("code", ["", "e4m3", "int8", "e2m1"])
@pytest.mark.parametrize("k", [32, 672, 2048, 4128, 9248])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_codes(code, k, dtype):
    Case(7, k, dtype, code=code, out=not code).run().check()
    Case(7, k, dtype, "layer", "rms", code=code, out=True, bias=True).run().check()


def test_parts_left_out():
    Case(4, 256, y=False).run().check()                                     # norm of the residual
    Case(4, 256, residual=False, res_scale=0.25).run().check()              # no residual yet
    Case(4, 256, res_out=False).run().check()
    Case(4, 256, kind="", post="rms", gate="one").run().check()             # the residual alone
    Case(4, 256, weight=False, post="layer").run().check()
    Case(4, 256, out=False, res_out=False, code="int8").run().check()
    Case(4, 256, inplace=True, code="e4m3").run().check()                   # res_out = res, out = y
    Case(4, 264, inplace=True, pad=8, res="f32", post="layer").run().check()


def test_rows_beside_the_outputs_are_left_alone():
    c = Case(5, 672, pad=16, code="int8").run()
    c.check()
    assert torch.isnan(c.res_wide[:, 672:]).all() and torch.isnan(c.out_wide[:, 672:]).all()
    # fewer rows than the tensors have
    c = Case(5, 672, code="int8")
    c.rows = 3
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.res_wide[3:]).all() and torch.isnan(c.out_wide[3:]).all() and (c.codes[3:] == 0xA5).all()
    assert torch.isnan(c.scale[3:]).all() and not torch.isnan(c.out_wide[:3]).any()


def test_mean_far_from_zero():
    # the mean is 200 times the spread: a sum of squares less the squared mean would lose it
    Case(6, 4096, "bf16", "layer", y=False, res="f32", mean=600.0).run().check()
    Case(6, 1000, "f16", "layer", "layer", res="f32", mean=600.0).run().check()


def test_rows_of_zeros_and_extremes():
    for code in ("e4m3", "int8", "e2m1"):
        c = Case(3, 256, residual=False, code=code)
        c.wide_y.zero_()
        c.run()
        torch.cuda.synchronize()
        assert not c.out_wide.any() and not c.codes.any()
        assert (c.scale == (0 if code == "e2m1" else 1.0)).all()
    # squares beyond float32, finite values: the largest bf16 rows
    for kind in ("rms", "layer"):
        for post in ("", kind):
            c = Case(4, 1024, kind=kind, post=post, y=bool(post), residual=not post)
            big = c.wide_y if post else c.wide_r
            big.copy_((torch.randn(4, 1024, device="cuda") * 1e38).clamp(-3e38, 3e38).to(torch.bfloat16))
            c.run()
            torch.cuda.synchronize()
            v = _d(big)
            w = c.wp if post else c.w
            z = LO.normed(v, kind, 1e-6, _d(w))[0]
            got = _d(c.res_wide if post else c.out_wide)
            # the scaling by a power of two adds no error
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -16 * (1 + np.abs(z))).all()
    # the smallest eps with the smallest rows
    c = Case(3, 512, y=False, res="f32", eps=1e-30)
    c.wide_r.mul_(1e-18)
    c.want = LO.norm_rows(res=_d(c.r), weight=_d(c.w), **c.args)
    c.run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8", "e2m1"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("k", [256, 4096])
def test_rows_that_are_not_finite(code, value, k):
    c = Case(4, k, code=code, weight=False)
    c.wide_y[2, 77] = value
    c.run()
    torch.cuda.synchronize()
    if code == "e2m1":
        # NaN: everything; an infinity: its own value is NaN (inf * 0), the others are divided by infinity
        if np.isnan(value):
            assert (c.scale[2] == 255).all()
        else:
            assert c.scale[2, 77 // 32] == 255 and (c.scale[2] != 255).sum() == k // 32 - 1
        assert not c.codes[2].any()
    else:
        assert torch.isnan(c.scale[2]) and not c.codes[2].any() and not torch.isnan(c.scale[[0, 1, 3]]).any()
    u = _d(c.res_wide)
    assert np.isnan(u[2, 77]) if np.isnan(value) else u[2, 77] == value
    assert np.isfinite(u[[0, 1, 3]]).all() and np.isfinite(_d(c.out_wide)[[0, 1, 3]]).all()


def test_codes_are_those_of_the_row_quantizers():
    # z exact in 16 bits: rows of one magnitude, a power of two, have a root mean square that is exact
    k = 512
    sign = torch.randint(0, 2, (9, k), device="cuda").to(torch.bfloat16) * 2 - 1
    w = (torch.randn(k, device="cuda")).to(torch.bfloat16)
    r = sign * torch.exp2(torch.arange(9, device="cuda").float() - 4).to(torch.bfloat16)[:, None]
    for code, quant, shape in (("e4m3", qg.quantize_e4m3_rows, (9, k)), ("int8", qg.quantize_int8_rows, (9, k)),
                               ("e2m1", qg.quantize_e2m1_rows, (9, k // 2))):
        out = torch.empty((9, k), dtype=torch.bfloat16, device="cuda")
        mk = lambda: (torch.zeros(shape, dtype=torch.uint8, device="cuda"),   # noqa: E731
                      torch.zeros((9, k // 32), dtype=torch.uint8, device="cuda") if code == "e2m1" else torch.zeros(9, device="cuda"))
        (c0, s0), (c1, s1) = mk(), mk()
        # eps below half a step of the mean squares: 2^-8 and more
        qg.norm_rows(qg.make_norm_desc(qg.N_RMS, qg.O_BF16, k, 1e-12, code_type=CODE[code]), 9, None, r, None, out, c0, s0, weight=w)
        assert torch.equal(out.float(), sign.float() * w.float())
        quant(out, 9, k, qg.A_BF16, c1, s1)
        torch.cuda.synchronize()
        assert torch.equal(c0, c1) and torch.equal(s0, s1)


def test_many_short_rows():
    # more rows than one launch takes (2^21), and a second launch with a part of one
    rows = (1 << 21) + 5
    c = Case(3, 8)
    x = torch.randn((rows, 8), device="cuda").to(torch.bfloat16)
    out = torch.full((rows, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.norm_rows(qg.make_norm_desc(qg.N_RMS, qg.O_BF16, 8, 1e-6), rows, None, x, None, out, weight=c.w)
    torch.cuda.synchronize()
    z = LO.normed(_d(x[-2000:]), "rms", 1e-6, _d(c.w))[0]
    assert (np.abs(_d(out[-2000:]) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -16 * (1 + np.abs(z))).all()
    assert not torch.isnan(out).any()


def test_other_stream_and_graph():
    c = Case(65, 1416, post="rms", gate="rows", code="e4m3")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    c.check()
    first = [t.clone() for t in (c.res_wide, c.out_wide, c.codes, c.scale)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        for t in (c.res_wide, c.out_wide, c.codes, c.scale):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (c.res_wide, c.out_wide, c.codes, c.scale)):
            assert torch.equal(a, b)
