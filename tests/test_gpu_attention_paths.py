"""Attention over every way its work is divided, under bars that a lost token does not pass.

Bars, from the arithmetic (test_gpu_attention has the roundings): with w the weights of a row, which add up to one,
|out - ref| <= u |ref| + wb dev + 2^-20 dev + (D / 4 + 2) 2^-24 terms + 2^-13 (sum w |V| + |ref|), where dev bounds
sum w |V - ref|: an error that a weight has in both sums moves the output by its distance from it.  wb is 2^-8
for bf16 (the rounding of the weights) and 2^-16 for f16 (two bf16 parts; not in the sum of weights: of sum w |V|).

Roundings are independent of each other, so a row's root mean square over its D values is far smaller than that: those of
the output and of the weights are at most u / sqrt(3) |ref| and wb / sqrt(3) sqrt(sum (w (V - ref))^2).  Three times
that (a row that two or three tokens share may have their roundings the wrong way round: 2.5), and 2^-18 of sum w |V| for the sums
and scores, is the bar of each row: a token that is left out of 3000 is eight times the rounding.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO
from test_gpu_attention import U, Case, _d

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def inside(got, r, dim, dtype):
    """Outputs [rows][heads][D] against attention_terms' reference, by element and by row."""
    u, out = U[dtype], r["out"]
    weights = 2.0 ** -8 * r["dev"] if dtype == "bf16" else 2.0 ** -16 * r["wv"]
    tol = u * np.abs(out) + weights + 2.0 ** -20 * r["dev"] + (dim / 4 + 2) * 2.0 ** -24 * r["terms"] + \
        2.0 ** -13 * (r["wv"] + np.abs(out)) + 2.0 ** -25
    err = np.abs(got - out)
    assert (err <= tol).all(), np.max(err / tol)
    rms = lambda x: np.sqrt(np.mean(x, axis=-1))  # noqa: E731
    bar = 3 * rms((u * u * out * out + (2.0 ** -16 * r["dev2"] if dtype == "bf16" else 0.0)) / 3) + \
        rms(((2.0 ** -18 + (2.0 ** -16 if dtype == "f16" else 0.0)) * r["wv"] + (dim / 4 + 2) * 2.0 ** -24 * r["terms"]) ** 2) + 2.0 ** -25
    assert (rms(err ** 2) <= bar).all(), np.max(rms(err ** 2) / bar)


def check(c):
    torch.cuda.synchronize()
    w = c.heads * c.dim
    got = _d(c.out)
    assert np.isnan(got[c.used:]).all() and np.isnan(got[:, w:]).all()          # left as they were
    q = _d(c.q)[:c.used, :w].reshape(c.used, c.heads, c.dim)
    r = LO.attention_terms(q, c.k, c.v, c.lens, c.counts, c.scale, c.seen)
    inside(got[:c.used, :w].reshape(r["out"].shape), r, c.dim, c.dtype)
    return r


def parts(c):
    """How many parts the tokens are split in, as the workspace shows."""
    return 1 if c.ws is None else c.ws.numel() // (c.tokens * c.heads * (c.dim + 2) * 4)


def longest_part(c):
    """Steps of 32 tokens that some part has at least."""
    return -(-(-(-c.max_len // 32)) // parts(c))


TYPES = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 64), ("f16", 128), ("f16", 256)]


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_few_tokens_to_many(dtype, dim):
    check(Case([1, 15, 33, 257, 0, 700, 3000], 6, 3, dim, 16, dtype=dtype, pad=8).run())
    check(Case([40, 7, 300, 64, 90, 3, 0], 4, 1, dim, 32, counts=[3, 7, 1, 64, 0, 5, 2], dtype=dtype, extra_rows=2).run())
    check(Case([200, 333, 1300], 4, 2, dim, 64, counts=[200, 150, 90], dtype=dtype, pad=8).run())


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_joins_of_many_rows(dtype, dim):
    # more rows than a workgroup each: several to a workgroup, also where the heads do not fill one
    c = Case([2500, 1700, 90], 10, 2, dim, 32, counts=[300, 280, 1], dtype=dtype, pad=8).run()
    assert parts(c) > 1 and c.batch * c.max_q * c.heads > 4096
    check(c)
    c = Case([2100, 3], 3, 3, dim, 16, counts=[700, 2], dtype=dtype).run()
    assert parts(c) > 1 and c.batch * c.max_q * c.heads > 4096 and c.heads % (1024 // dim) != 0
    check(c)


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_long_parts_of_single_tokens(dtype, dim):
    # a wave's turns beyond those whose pages it holds at a time (32 of every fourth step): pages in any order
    lens = [8100, 8192] + [i % 4 for i in range(510)]
    order = np.random.default_rng(dim).permutation(512)
    c = Case([lens[i] for i in order], 4, 2, dim, 16, dtype=dtype).run()
    assert parts(c) > 1 and longest_part(c) > 4 * 30
    check(c)


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_long_parts_of_many_rows(dtype, dim):
    # a part's steps beyond those whose pages are held at a time (32)
    lens = [7000, 6900] + [3 * i for i in range(30)]
    counts = [300, 40] + [i % 3 for i in range(30)]
    c = Case(lens, 4, 2, dim, 16, counts=counts, dtype=dtype).run()
    assert longest_part(c) > 32 and (dim == 256 or parts(c) > 1)
    check(c)


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_prompts_in_one_part(dtype, dim):
    # so many tiles that none is split, and more steps than pages are held for at a time
    lens = [1500, 1311] + [5 * i for i in range(62)]
    counts = [200, 17] + [min(5 * i, 3) for i in range(62)]
    c = Case(lens, 16, 4, dim, 32, counts=counts, max_q=2000, dtype=dtype).run()
    assert parts(c) == 1 and longest_part(c) > 32
    check(c)


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_a_few_queries_of_many_heads(dtype, dim):
    # three tokens to verify, eight query heads per key head: 24 rows, in the kernel of many rows
    check(Case([3000, 40, 700, 2500, 3, 2], 16, 2, dim, 16, counts=[3] * 6, dtype=dtype).run())
    check(Case([3000, 40, 700], 34, 2, dim, 64, dtype=dtype).run())             # 17 rows of one token


@pytest.mark.parametrize("dtype,dim", TYPES)
def test_prompts_and_single_tokens_together(dtype, dim):
    rng = np.random.default_rng(3)
    lens = [900] + list(rng.integers(1, 4000, 11))
    c = Case([int(n) for n in lens], 16, 2, dim, 32, counts=[500] + [1] * 11, dtype=dtype, extra_rows=1).run()
    check(c)
    c = Case([int(n) for n in lens], 16, 2, dim, 32, counts=[1] * 6 + [40] + [1] * 5, dtype=dtype, max_len=8192).run()
    assert parts(c) > 1
    check(c)


def test_bad_pages_in_long_parts():
    bad = [(0, 0), (0, 200), (0, 511), (1, 7), (1, 260)]
    for counts in (None, [60, 9] + [1] * 510):
        c = Case([8192, 8111] + [i % 4 for i in range(510)], 4, 2, 128, 16, counts=counts, bad_pages=bad).run()
        check(c)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
def test_a_query_alone_and_in_its_chunk(dtype, dim):
    # the same rows against the same tokens: as a chunk, and each as its sequence's only query
    n = 33
    c = Case([200], 4, 1, dim, 16, counts=[n], dtype=dtype).run()
    r = check(c)
    lens = torch.arange(200 - n + 1, 201, dtype=torch.int32, device="cuda")
    alone = torch.full_like(c.out, float("nan"))
    need = qg.attention_workspace_bytes(c.desc, 4, n, 1, n, 200)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    qg.attention(c.desc, c.q, 4, c.cache, c.table.expand(n, -1).contiguous(), lens, n, 200, c.scale, alone, ws)
    torch.cuda.synchronize()
    inside(_d(alone).reshape(r["out"].shape), r, dim, dtype)
    # and among other sequences' queries
    twice = torch.cat([c.q, c.q.flip(0)])
    out = torch.full_like(twice, float("nan"))
    ws = torch.empty(max(16, qg.attention_workspace_bytes(c.desc, 4, 2, n, 2 * n, 200)), dtype=torch.uint8, device="cuda")
    qg.attention(c.desc, twice, 4, c.cache, c.table.repeat(2, 1), torch.tensor([200, 150], dtype=torch.int32, device="cuda"), 2, 200,
                 c.scale, out, ws, q_offsets=torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda"), max_q=n)
    torch.cuda.synchronize()
    inside(_d(out[:n]).reshape(r["out"].shape), r, dim, dtype)
