"""The paged 4-bit cache's attention over long caches, where every CTA goes
round its stages many times, with checks that every single token can be seen
in (an ordinary bound in the largest value cannot: over 30000 random tokens the
outputs are a hundred times smaller, and a tile that is left out stays inside
it).

Queries of zeros weigh all tokens alike, so an output is the plain mean of the
values that its query sees.  The values are whole numbers of at most 8, the
weights powers of two: all sums are exact in float32 (below 2^24 units), and an
output is off by its own rounding (half a step) and a few float32 roundings (the
reciprocal of the sum, the products with it and, where parts are joined, with
their factors: under 16 half steps, 2^-20).  A tile of 64 tokens left out, or
taken twice, changes the sum by some 35, where the tolerance is 2^-11 (binary16)
or 2^-8 (bfloat16) of some 700.

Queries that equal one token's key, among keys of signs, find that token: its
score is 64, all others' 64 r with r the correlation of two sign
vectors.  At d = 64, r is below 0.75 but for one in 10^10 pairs (56 of 64 signs
or more alike), and the rest weighs 32000 E[exp(64 r)] exp(-64), below
32000 exp(32 - 64) = 4e-10 of it, plus exp(-16) for a pair at 0.75: the output
is the token's value, up to 16 * 2 * 1.2e-7 < 2^-17, and a value of at most
four bits is rounded from there to itself or to something no farther from it
than twice that."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DEV, _gen, tq

pytestmark = pytest.mark.gpu


def _fill(lens, H, d, page, seed):
    """A pool with the sequences in it, pages in random order: the cache, its
    table and lengths, and each sequence's stored keys and values."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    counts = [(n + page - 1) // page for n in lens]
    cache = tq.PagedCache(sum(counts), H, d, page_size=page)
    order = torch.randperm(sum(counts), generator=_gen(seed)).int().to(DEV)
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device=DEV)
    rows, at = [], 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        table[b, :c] = order[at:at + c]
        at += c
        t = torch.arange(n, device=DEV)
        k = torch.randint(0, 2, (n, H, d), generator=g, device=DEV, dtype=torch.int8).half() * 2 - 1
        v = torch.randint(-7, 8, (n, H, d), generator=g, device=DEV, dtype=torch.int8).half()
        v[..., ::32] = 7.5                           # scale 1: whole numbers are kept as they are
        rows.append(cache.write(k, v, table[b, t // page].long() * page + t % page, stored=True))
        assert torch.equal(rows[-1][1][..., 1:32], v[..., 1:32])
    return cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), rows, g


def _means(v, pos, window, sinks):
    """The mean of the values [n, H, d] that queries at `pos` see, in 64 bits."""
    sums = torch.cat((torch.zeros_like(v[:1], dtype=torch.float64), v.double().cumsum(0)))
    hi = (pos + 1).clamp(min=0)
    lo = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
    s = lo.clamp(max=sinks) if window else torch.zeros_like(pos)
    n = (hi - lo + s).clamp(min=1)
    return (sums[hi] - sums[lo] + sums[s]) / n[:, None, None]


def _run(lens, new, H, G, d, page, window, sinks, dtype, most):
    cache, table, lens_t, rows, g = _fill(lens, H, d, page, seed=d + G + window)
    starts = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device=DEV)
    pos = [torch.arange(n - m, n, device=DEV) for n, m in zip(lens, new)]
    kw = dict(q_starts=starts, max_q_len=most, window=window, sinks=sinks)

    q = torch.zeros(sum(new), H * G, d, dtype=dtype, device=DEV)
    ref = torch.cat([_means(v, p, window, sinks) for (_, v), p in zip(rows, pos)]).repeat_interleave(G, 1)
    out = cache.attention(q, table, lens_t, **kw).double()
    err, tol = (out - ref).abs(), ref.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -20) + 2.0 ** -25
    assert (err <= tol).all(), (float((err / tol).max()), (err > tol).nonzero()[:4].tolist())

    # each row its own token, anywhere in what it sees
    want = torch.empty(sum(new), H * G, d, dtype=torch.float64, device=DEV)
    at = 0
    for (k, v), p in zip(rows, pos):
        lo = (p - window + 1).clamp(min=0) if window else torch.zeros_like(p)
        s = lo.clamp(max=sinks) if window else torch.zeros_like(p)
        pick = (torch.rand(len(p), H * G, generator=g, device=DEV) * (p + 1 - lo + s)[:, None]).long()
        pick = torch.minimum(pick, (p - lo + s)[:, None])
        t = torch.where(pick < s[:, None], pick, pick - s[:, None] + lo[:, None])
        head = torch.arange(H * G, device=DEV) // G
        kt = k[t, head].float()
        q[at:at + len(p)] = (kt * (64 * d ** 0.5 / (kt * kt).sum(-1, keepdim=True))).to(dtype)
        want[at:at + len(p)] = v[t, head].double()
        at += len(p)
    out = cache.attention(q, table, lens_t, **kw).double()
    assert (out - want).abs().max() <= 2.0 ** -16, float((out - want).abs().max())
    assert torch.equal(out, cache.attention(q, table, lens_t, **kw).double())
    assert cache.status() == (0, 0)


LONG = [32000, 32001, 17, 31007]     # ten rounds and more a CTA, at the heads below
RAGGED = [1 + (517 * i) % 4099 for i in range(130)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,H,G,page", [(64, 16, 1, 16), (64, 12, 12, 256), (128, 8, 4, 16), (128, 8, 12, 64), (256, 4, 2, 32)])
@pytest.mark.parametrize("lens,window,sinks", [(LONG, 0, 0), (LONG, 20011, 77), (RAGGED, 0, 0), (RAGGED, 700, 5)])
def test_one_query(dtype, d, H, G, page, lens, window, sinks):
    _run(lens, [1] * len(lens), H, G, d, page, window, sinks, dtype, 1)


@pytest.mark.parametrize("d,H,G,page", [(64, 12, 4, 32), (128, 8, 3, 16), (256, 4, 2, 64)])
@pytest.mark.parametrize("lens,window,sinks", [(LONG, 0, 0), (RAGGED, 130, 70)])
def test_a_few_queries(d, H, G, page, lens, window, sinks):
    _run(lens, [min(n, 1 + i % 5) for i, n in enumerate(lens)], H, G, d, page, window, sinks, torch.float16, 5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,H,G,page,lens,new", [
    # more than 128 rows of a kv head: dozens of tiles a CTA, several items
    (64, 8, 2, 16, [4000], [4000]), (128, 4, 4, 16, [4000], [4000]), (256, 2, 4, 32, [4000], [4000]),
    (128, 2, 4, 64, [9000, 3001, 77], [1500, 3001, 20]),
    # at most 128 rows
    (64, 8, 4, 16, [5000] * 7 + [5011], [25] * 8), (128, 8, 4, 16, [5000] * 7 + [5011], [30] * 8), (256, 8, 4, 16, [2500] * 8, [30] * 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 70)])
def test_many_queries(dtype, d, H, G, page, lens, new, window, sinks):
    _run(lens, new, H, G, d, page, window, sinks, dtype, max(new))
