"""The paged 4-bit cache on the GPU: calls at the edges of what its
documentation allows, and calls that it refuses."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DEV, _check, _gen, _pool, _randn, tq

pytestmark = pytest.mark.gpu


# ------------------------------------------------ queries that are not finite

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 60])
def test_queries_that_are_not_finite_where_sequences_are_split(dtype, d, most):
    """A NaN in a query, or an infinity (some score is then NaN or +inf), makes
    its row NaN whether the sequence is split or not, and no other row; a row
    that sees nothing is zeros whatever its query."""
    lens, new = [5000, 20, 300], [most, min(most, 59), 1]
    if most > 1:
        new[1] = 33                              # 13 queries before the first token
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, 2, d, 16, seed=d + most, dtype=dtype)
    assert cache.workspace_bytes(8, 3, table.shape[1], most) > 0
    q = _randn(g, int(starts[-1]), 8, d, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    good = cache.attention(q, table, lens_t, q_starts=st, max_q_len=most)
    bad = q.clone()
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for i, (row, head) in enumerate([(0, 0), (0, 3), (0, 5), (new[0] - 1, 6), (int(starts[2]), 1), (int(starts[2]) - 1, 2)]):
        bad[row, head, (7 * i) % d] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        hit[row, head] = True
    if most > 1:
        bad[new[0], 4, 3] = bad[new[0] + 5, 4, 9] = float("nan")     # these see nothing
    out = cache.attention(bad, table, lens_t, q_starts=st, max_q_len=most)
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], good[~hit])
    if most > 1:
        assert not out[new[0]:new[0] + 13].any()


# -------------------------------------------------- what no query sees

def _visible(lens, new, width, page, window, sinks):
    """Of each sequence: which of `width` pages hold a token that some query
    sees, and which tokens are seen."""
    pages, tokens = torch.zeros(len(lens), width, dtype=torch.bool), []
    for b, (n, m) in enumerate(zip(lens, new)):
        t = torch.arange(n)
        see = ((t > n - m - window) | (t < sinks)) if m else torch.zeros(n, dtype=torch.bool)
        pages[b, (t[see] // page).unique()] = True
        tokens.append(see)
    return pages, tokens


WINDOWS = [(1, 0), (100, 4), (64, 0), (130, 70), (17, 1000)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("most", [1, 5, 70])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_pages_that_no_query_sees_may_be_freed(d, page, most, window, sinks):
    """A serving loop gives back the pages behind the window: their entries
    are not looked up and nothing is flagged."""
    lens = [900, 40, 513, 0, 300, 2600]
    new = [min(n, most) for n in lens]
    starts = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device=DEV)
    cache, table, lens_t, g = _pool(lens, 2, d, page, seed=d + page + most)
    q = _randn(g, sum(new), 4, d, dtype=torch.float16)
    kw = dict(q_starts=starts, max_q_len=most, window=window, sinks=sinks)
    good = cache.attention(q, table, lens_t, **kw)
    _check(cache, q, table, lens_t, starts.cpu().numpy(), good, window=window, sinks=sinks)
    keep, _ = _visible(lens, new, table.shape[1], page, window, sinks)
    for entry in (-1, 1 << 30):
        out = cache.attention(q, torch.where(keep.to(DEV), table, entry), lens_t, **kw)
        assert torch.equal(out, good)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("most", [1, 5, 70])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_rows_that_no_query_sees_may_hold_anything(d, page, most, window, sinks):
    """Rows outside every query's window and sinks, in pages that are partly
    seen too: their scale bytes may stand for NaN or infinity."""
    lens = [900, 40, 513, 0, 300, 2600]
    new = [min(n, most) for n in lens]
    starts = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device=DEV)
    cache, table, lens_t, g = _pool(lens, 2, d, page, seed=d + page + most)
    q = _randn(g, sum(new), 4, d, dtype=torch.float16)
    kw = dict(q_starts=starts, max_q_len=most, window=window, sinks=sinks)
    good = cache.attention(q, table, lens_t, **kw)
    seen = torch.zeros(cache.n_pages * page, dtype=torch.bool)
    for b, see in enumerate(_visible(lens, new, table.shape[1], page, window, sinks)[1]):
        t = torch.arange(lens[b])[see]
        seen[table[b].cpu()[t // page].long() * page + t % page] = True
    hide = ~seen.view(cache.n_pages, page).to(DEV)
    for byte in (0xFF, 0xF8):                        # scales of NaN and of infinity
        for pool in (cache.k, cache.v):
            scales = pool[..., page * d // 2:].view(cache.n_pages, 2, page, d // 32)
            scales.copy_(torch.where(hide[:, None, :, None], byte, scales))
        assert torch.equal(cache.attention(q, table, lens_t, **kw), good)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_padding_rows_are_not_counted(dtype):
    """Rows without a place in the cache (padding, slots past the pool) may
    hold anything; only rows that are kept are counted as not finite."""
    cache = tq.PagedCache(2, 2, 64, page_size=16)
    x = _randn(_gen(1), 6, 2, 64, dtype=dtype)
    x[1] = float("nan")
    x[2, 0, 3] = float("inf")
    x[4] = -float("inf")
    x[5, 1, 0] = float("nan")
    slots = torch.tensor([0, -1, -7, 3, 32, 5], device=DEV)
    ks, vs = cache.write(x, x, slots, stored=True)
    assert cache.status() == (2, 2)                  # the row (5, 1) of keys and of values; a slot past the pool
    assert not ks[1].any() and not ks[2, 0].any() and ks[2, 1].any() and not vs[4].any() and not ks[5, 1].any()
    assert not cache.read(torch.tensor([5], device=DEV))[0][0, 1].any()


# ------------------------------------------------------- arguments

@pytest.mark.parametrize("scale", [0.0, -0.0, 0, 1e-60, -1e-60, float("inf"), 1e60, float("nan")])
def test_scales_that_are_not_positive_float32_are_refused(scale):
    """Zero among them: it is not the default."""
    cache, table, lens_t, g = _pool([40, 30], 2, 64, 16, seed=1)
    q = _randn(g, 2, 4, 64, dtype=torch.float16)
    with pytest.raises(tq.TQError, match="DIM_MISMATCH"):
        cache.attention(q, table, lens_t, scale=scale)
    assert torch.equal(cache.attention(q, table, lens_t, scale=64 ** -0.5), cache.attention(q, table, lens_t))


@pytest.mark.parametrize("kw", [dict(window=(1 << 32) + 5), dict(window=1 << 32), dict(sinks=1 << 31, window=4),
                                dict(sinks=(1 << 32) + 2, window=4), dict(max_q_len=(1 << 32) + 1), dict(max_q_len=1 << 31),
                                dict(window=-(1 << 32) + 4), dict(sinks=-(1 << 32) + 4, window=4), dict(max_q_len=-(1 << 32) + 1)])
def test_numbers_beyond_32_bits_are_refused(kw):
    """They are not taken modulo 2^32."""
    cache, table, lens_t, g = _pool([40, 30], 2, 64, 16, seed=1)
    with pytest.raises(tq.TQError, match="LIMIT"):
        cache.attention(_randn(g, 2, 4, 64, dtype=torch.float16), table, lens_t, **kw)
    for args in [(1 << 32, 1, 1, 1), (4, (1 << 32) + 1, 100, 1), (4, 1, 1 << 31, 1), (4, 1, 100, (1 << 32) + 1)]:
        with pytest.raises(tq.TQError, match="LIMIT"):
            cache.workspace_bytes(*args)
    for args in [(4, 8, 64, (1 << 32) + 64), (4, 8, (1 << 32) + 64, 64), (4, (1 << 32) + 8, 64, 64)]:
        with pytest.raises(tq.TQError, match="LIMIT"):
            tq.PagedCache(*args)


def test_workspaces_that_are_not_contiguous_are_refused():
    """An expanded tensor has fewer bytes than elements, a strided one has
    others between them."""
    cache, table, lens_t, g = _pool([4000], 1, 64, 16, seed=2)
    q = _randn(g, 1, 2, 64, dtype=torch.float16)
    need = cache.workspace_bytes(2, 1, table.shape[1])
    assert need > 0
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(need), torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2],
               torch.empty(64, dtype=torch.float32, device=DEV).expand(need, 64)):
        with pytest.raises(tq.TQError, match="WORKSPACE"):
            cache.attention(q, table, lens_t, workspace=ws)
    ws = torch.empty(need // 4 + 1, dtype=torch.float32, device=DEV)         # any type will do
    assert torch.equal(cache.attention(q, table, lens_t, workspace=ws), cache.attention(q, table, lens_t))


def test_a_new_cache_may_be_used_on_any_stream_at_once():
    """The constructor's zeros are in place when it returns: a row written on
    another stream right away stays."""
    x, s = _randn(_gen(1), 1, 8, 128), torch.cuda.Stream()
    warm = tq.PagedCache(1, 8, 128, page_size=64)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    warm.write(x, x, slots, stored=True, stream=s)
    room = torch.empty(3 << 30, dtype=torch.uint8, device=DEV)       # two pools of 1 GB come from what this leaves
    del room
    last = slots + 30000 * 64 - 1
    torch.cuda.synchronize()
    cache = tq.PagedCache(30000, 8, 128, page_size=64)
    ks, vs = cache.write(x, x, last, stored=True, stream=s)
    torch.cuda.synchronize()
    kr, vr = cache.read(last, dtype=torch.float32)
    assert torch.equal(kr, ks) and torch.equal(vr, vs)


# ------------------------------------------------------- division of the work

@pytest.mark.parametrize("d,B,H", [(64, 290, 2), (64, 592, 1), (128, 290, 1), (128, 37, 8), (256, 296, 1), (64, 593, 1)])
@pytest.mark.parametrize("most", [1, 4])
def test_short_sequences_with_a_cta_each(d, B, H, most):
    """No more sequences and kv heads than CTAs, of unlike lengths, some empty
    or without queries; too few queries announced (more items than CTAs then)."""
    lens = [(37 * i) % 480 for i in range(B)]
    new = [min(lens[i], (i % 7 == 0) * 30 + i % 5) for i in range(B)]
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, H, d, 16, seed=d + B)
    assert cache.workspace_bytes(4 * H, B, table.shape[1], most) == 0
    q = _randn(g, int(starts[-1]) + 2, 4 * H, d, dtype=torch.float16)
    out = torch.full_like(q, 7.0)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    cache.attention(q, table, lens_t, q_starts=st, max_q_len=most, out=out, window=300, sinks=3)
    _check(cache, q, table, lens_t, starts, out, window=300, sinks=3)
    assert (out[int(starts[-1]):] == 7.0).all() and cache.status() == (0, 0)


@pytest.mark.parametrize("d,B,H", [(64, 18, 8), (128, 36, 4), (256, 70, 2)])
def test_short_prompts_with_a_cta_each(d, B, H):
    lens = [(37 * i) % 62 for i in range(B)]
    starts = np.concatenate(([0], np.cumsum(lens)))
    cache, table, lens_t, g = _pool(lens, H, d, 32, seed=d + B)
    q = _randn(g, int(starts[-1]), 2 * H, d, dtype=torch.bfloat16)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    for most in (62, 30):
        out = cache.attention(q, table, lens_t, q_starts=st, max_q_len=most)
        _check(cache, q, table, lens_t, starts, out)
    assert cache.status() == (0, 0)
