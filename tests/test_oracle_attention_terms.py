"""Pins of the attention reference that keeps the magnitudes of its roundings apart (no GPU)."""
import numpy as np
import pytest

from oracle import layer_ops as LO


def _case(lens, counts, heads, kv, dim, seed=0):
    rng = np.random.default_rng(seed)
    k, v = ([rng.standard_normal((n, kv, dim)) for n in lens] for _ in "kv")
    return rng.standard_normal((sum(counts), heads, dim)), k, v, rng


@pytest.mark.parametrize("lens,counts", [([5, 1, 70, 0], [1, 1, 1, 1]), ([40, 3, 9], [40, 5, 0])])
def test_outputs_are_those_of_the_plain_reference(lens, counts):
    q, k, v, rng = _case(lens, counts, 6, 2, 8)
    seen = [rng.random(n) < 0.8 for n in lens]
    for s in (None, seen):
        got = LO.attention_terms(q, k, v, lens, counts, -0.7, s)
        want, _ = LO.attention(q, k, v, lens, counts, -0.7, s)
        assert np.allclose(got["out"], want, rtol=0, atol=1e-13)


def test_worked_example():
    k = [np.zeros((2, 1, 1))]
    v = [np.array([[[1.0]], [[3.0]]])]
    r = LO.attention_terms(np.ones((1, 1, 1)), k, v, [2], [1], 1.0)
    assert r["out"].item() == 2 and r["dev"].item() == 1 and r["dev2"].item() == 0.5 and r["wv"].item() == 2 and r["terms"].item() == 0


def test_errors_of_weights_stay_inside():
    # weights changed by errors of at most e, the same in the numerator and in the sum, move the outputs by e * dev
    q, k, v, rng = _case([60], [7], 2, 1, 8, 3)
    r = LO.attention_terms(q, k, v, [60], [7], 1.0)
    e = 2.0 ** -8
    moved = np.zeros_like(q)
    for i in range(7):
        n = 54 + i
        for h in range(2):
            w = np.exp(k[0][:n, 0] @ q[i, h]) * (1 + rng.uniform(-e, e, n))
            moved[i, h] = w @ v[0][:n, 0] / w.sum()
    d = np.abs(moved - r["out"])
    assert (d <= e * (1 + 4 * e) * r["dev"]).all()
    assert np.sqrt(np.mean(d ** 2)) <= 1.3 * e / 3 ** 0.5 * np.sqrt(np.mean(r["dev2"]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,tokens", [(64, 3000), (128, 3000), (256, 700), (128, 40)])
def test_the_bars_do_not_pass_a_lost_token(dtype, dim, tokens):
    # outputs with the roundings that the kernels make are inside; those that lack a token, or see one too many, are not
    import torch
    from test_gpu_attention_paths import inside
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    rounded = lambda x: torch.from_numpy(x).to(t).double().numpy()  # noqa: E731
    rng = np.random.default_rng(dim + tokens)
    q = rounded(1.5 * rng.standard_normal((4, 2, dim)))
    k, v = (LO.mxfp4_values(rounded(rng.standard_normal((tokens + 1, dim)))) for _ in "kv")
    r = LO.attention_terms(q, [k[:tokens, None]], [v[:tokens, None]], [tokens], [4], dim ** -0.5)

    def out(skip=(), ahead=0):
        o = np.zeros_like(q)
        for i in range(4):
            at = np.setdiff1d(np.arange(tokens - 3 + i + ahead), skip)
            for h in range(2):
                s = dim ** -0.5 * (k[at] @ q[i, h])
                w = np.exp(s - s.max())
                w = torch.from_numpy(w).to(torch.bfloat16).double().numpy() if dtype == "bf16" else w
                o[i, h] = w @ v[at] / w.sum()
        return rounded(o)

    inside(out(), r, dim, dtype)
    for wrong in (out(skip=[tokens // 2]), out(ahead=1), out(skip=range(tokens - 35, tokens - 3))):
        with pytest.raises(AssertionError):
            inside(wrong, r, dim, dtype)
