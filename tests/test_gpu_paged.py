"""The paged 4-bit cache on the GPU against its plain 64-bit forms
(paged_util): rows written and read back bit for bit, attention at the sizes,
masks and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

import paged_util as pu

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("kv_cache_vector_10_b200")
DEV = "cuda"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


# ------------------------------------------------------------ write and read

@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,H,page,n", [(64, 1, 16, 1), (64, 3, 256, 77), (128, 8, 64, 33), (128, 1, 16, 130), (256, 2, 32, 19),
                                        (128, 8, 64, 9000), (64, 32, 16, 5000)])
def test_write_then_read_bit_for_bit(dtype, d, H, page, n):
    g = _gen(n + d)
    n_pages = (n + page - 1) // page + 2
    cache = tq.PagedCache(n_pages, H, d, page_size=page)
    before = torch.randint(0, 256, cache.k.shape, generator=g, dtype=torch.int32).to(torch.uint8)
    cache.k.copy_(before)
    cache.v.copy_(before)
    # magnitudes over many powers of two, exact half-way points, zeros
    k = torch.randn(n, H, d, generator=g) * torch.exp2(torch.randint(-18, 9, (n, H, 1), generator=g).float())
    v = torch.randn(n, H, d, generator=g)
    v[::3] = torch.randint(-15, 16, v[::3].shape, generator=g).float() / 2
    v[1::5, :, :32] = 0
    k, v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
    slots = torch.randperm(n_pages * page, generator=g)[:n]
    slots[1::7] = -1
    ks, vs = cache.write(k, v, slots.to(DEV), stored=True)
    for x, xs, pool in ((k, ks, cache.k), (v, vs, cache.v)):
        c, byte = pu.quantise(x)
        assert xs.dtype == dtype and np.array_equal(xs.cpu().double().numpy(), pu.values(c, byte))
        codes, _ = pu.pack_page_rows(c, byte)
        want = before.numpy().copy()
        for i in np.nonzero(slots.numpy() >= 0)[0]:
            wc, ws = pu.page_row(want, page, d, slots[i])
            wc[...] = codes[i]
            ws[...] = byte[i]
        assert np.array_equal(pool.cpu().numpy(), want)          # everything else as it was
    kr, vr = cache.read(slots.to(DEV), dtype=dtype)
    keep = (slots >= 0).to(DEV)
    assert torch.equal(kr[keep], ks[keep]) and torch.equal(vr[keep], vs[keep])
    assert not kr[~keep].any() and not vr[~keep].any()
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_borders_between_codes_and_scales(dtype):
    """Values next to every border of the format: scales where max|x| is just
    on or beside 7.5 s, values on and beside (n + 1/2) s."""
    cache = tq.PagedCache(200, 1, 64, page_size=16)
    step = torch.finfo(dtype).eps
    rows = []
    for b in range(1, 224, 3):
        s = float(pu.SCALES[b])
        for m in (7.5 * s * (1 - 2 * step), 7.5 * s, 7.5 * s * (1 + 2 * step)):
            x = torch.zeros(64, dtype=torch.float64)
            x[0] = m
            for i in range(15):
                x[1 + 4 * i: 5 + 4 * i] = torch.tensor([(i - 7.5) * s, (i - 7.5) * s * (1 - step), (i - 7.5) * s * (1 + step), (i - 7) * s])
            x[61:] = torch.tensor([s / 2, -s / 2, 0.0])
            rows.append(x)
    x = torch.stack(rows)[:, None].clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype).to(DEV)
    slots = torch.arange(x.shape[0], device=DEV)
    ks, vs = cache.write(x, -x, slots, stored=True)
    for y, ys in ((x, ks), (-x, vs)):
        assert np.array_equal(ys.cpu().double().numpy(), pu.values(*pu.quantise(y)))
    assert torch.equal(cache.read(slots, dtype=dtype)[0], ks)


def test_error_bound_saturation_and_rows_that_are_not_finite():
    cache = tq.PagedCache(4, 2, 128, page_size=16)
    g = _gen(1)
    x = torch.randn(20, 2, 128, generator=g) * 30
    x[3, 1, 77] = float("nan")
    x[4, 0, 0] = float("inf")
    x[5, 0, 127] = -float("inf")
    x[6] = 1e30                   # beyond the largest scale: held to 7 * 7680
    x[7] = 1e-30                  # below half the smallest: zero
    xk = x.to(DEV)
    ks, vs = cache.write(xk, -xk, torch.arange(20, device=DEV), stored=True)
    ks = ks.cpu()
    assert not ks[3, 1].any() and not ks[4, 0].any() and not ks[5, 0].any()
    assert ks[3, 0].any() and ks[4, 1].any()
    assert (ks[6] == 7 * 7680).all() and (vs[6] == -8 * 7680).all() and not ks[7].any()
    fine = torch.tensor([i for i in range(20) if i not in (3, 4, 5, 6)])
    s = torch.from_numpy(pu.SCALES[pu.quantise(x[fine])[1]]).repeat_interleave(32, -1)
    assert ((x[fine].double() - ks[fine].double()).abs() <= s / 2).all()
    assert cache.status() == (6, 0)          # three rows of keys, the same three of values
    cache.reset_status()
    assert cache.status() == (0, 0)


def test_strided_rows_one_side_only_and_other_streams():
    g = _gen(2)
    cache = tq.PagedCache(8, 4, 128, page_size=32)
    qkv = _randn(g, 50, 3 * 4, 128, dtype=torch.bfloat16)
    slots = torch.randperm(256, generator=g)[:50].to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ks, none = cache.write(qkv[:, 4:8], None, slots, stored=True, stream=s)
    _, vs = cache.write(None, qkv[:, 8:], slots, stored=True, stream=s)
    kr, vr = cache.read(slots, stream=s)
    k_only, v_none = cache.read(slots, values=False, stream=s)
    s.synchronize()
    assert none is None and v_none is None
    assert np.array_equal(ks.cpu().double().numpy(), pu.values(*pu.quantise(qkv[:, 4:8])))
    assert torch.equal(kr, ks) and torch.equal(vr, vs) and torch.equal(k_only, ks)
    # odd strides and a misaligned base are copied first
    odd = torch.randn(50 * 4 * 129 + 3, generator=g).half().to(DEV)
    x = odd[3:].as_strided((50, 4, 128), (4 * 129, 129, 1))
    xs, _ = cache.write(x, None, slots, stored=True)
    assert np.array_equal(xs.cpu().double().numpy(), pu.values(*pu.quantise(x)))
    y = qkv[:, 4:8].transpose(1, 2).contiguous().transpose(1, 2)       # channels not contiguous
    ys, _ = cache.write(y, None, slots, stored=True)
    assert torch.equal(ys, ks)


def test_no_rows_and_slots_out_of_range():
    cache = tq.PagedCache(2, 2, 64, page_size=16)
    none = torch.empty(0, 2, 64, device=DEV)
    ks, vs = cache.write(none, none, torch.empty(0, dtype=torch.int64, device=DEV), stored=True)
    assert ks.shape == (0, 2, 64)
    assert cache.read(torch.empty(0, dtype=torch.int64, device=DEV))[0].shape == (0, 2, 64)
    x = _randn(_gen(3), 4, 2, 64)
    before = cache.k.clone()
    cache.write(x, x, torch.tensor([-1, 32, 1 << 40, -(1 << 62)], device=DEV))
    assert torch.equal(cache.k, before) and cache.status() == (0, 2)
    cache.reset_status()
    k, _ = cache.read(torch.tensor([-5, 33, 0, (1 << 62)], device=DEV))
    assert not k.any() and cache.status() == (0, 2)


def test_calls_that_are_refused():
    cache = tq.PagedCache(2, 2, 64, page_size=16)
    x, slots = _randn(_gen(3), 4, 2, 64), torch.arange(4, device=DEV)
    for bad in [(None, None, slots), (x, x.half(), slots), (x[:, :1], x[:, :1], slots), (x, x[:3], slots), (x, x, slots[:3]),
                (x, x, slots.int()), (x.double(), x.double(), slots), (x, x, slots.cpu()), (x.cpu(), x.cpu(), slots)]:
        with pytest.raises(tq.TQError):
            cache.write(*bad)
    for bad in [slots.int(), slots[None], slots.cpu()]:
        with pytest.raises(tq.TQError):
            cache.read(bad)
    with pytest.raises(tq.TQError):
        cache.read(slots, dtype=torch.float64)
    q, table, lens = _randn(_gen(4), 2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    cache.attention(q, table, lens)
    for kw in [dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :3]), dict(q=q[:1]), dict(q=q.cpu()), dict(page_table=table.long()),
               dict(page_table=table[:1]), dict(seq_lens=lens.long()), dict(seq_lens=lens[:1]), dict(q_starts=lens), dict(window=-1),
               dict(sinks=-1), dict(scale=-1.0), dict(out=torch.empty_like(q).float()), dict(max_q_len=-3)]:
        with pytest.raises(tq.TQError):
            cache.attention(**(dict(q=q, page_table=table, seq_lens=lens) | kw))
    for args in [(0, 2, 64), (2, 0, 64), (2, 2, 96), (2, 2, 0)]:
        with pytest.raises(tq.TQError):
            tq.PagedCache(*args)
    with pytest.raises(tq.TQError):
        tq.PagedCache(2, 2, 64, page_size=24)


# ---------------------------------------------------------------- attention

def _pool(lens, H, d, page, seed, dtype=torch.float16, garbage=True):
    """A pool with the sequences' rows in it (pages in random order, one page
    spare at each end of the order), everything else random bytes."""
    g = _gen(seed)
    counts = [(int(n) + page - 1) // page for n in lens]
    n_pages = sum(counts) + 2
    cache = tq.PagedCache(n_pages, H, d, page_size=page)
    if garbage:
        for pool in (cache.k, cache.v):
            pool.copy_(torch.randint(0, 256, pool.shape, generator=g, dtype=torch.int32).to(torch.uint8))
    order = torch.randperm(n_pages, generator=g).int()
    table = torch.full((len(lens), max(max(counts), 1) + 1), -7, dtype=torch.int32)
    at, slots = 0, []
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
        t = torch.arange(int(lens[b]))
        slots.append(table[b, t // page].long() * page + t % page)
    slots = torch.cat(slots).to(DEV)
    if len(slots):
        cache.write(_randn(g, len(slots), H, d, dtype=dtype), _randn(g, len(slots), H, d, dtype=dtype), slots)
    return cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), g


def _check(cache, q, table, lens, starts, out, **kw):
    kp, vp = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    ref = pu.attention(kp, vp, cache.page_size, q, table.cpu().numpy(), lens.cpu().numpy(), starts, **kw)
    vmax = 0.0
    for b in range(len(lens)):
        n = int(lens[b])
        if n:
            t = np.arange(n)
            tab = table[b].cpu().numpy()
            vmax = max(vmax, np.abs(pu.row_values(vp, cache.page_size, cache.head_dim, tab[t // cache.page_size].astype(np.int64) * cache.page_size + t % cache.page_size)).max())
    got = out.cpu().double().numpy()
    rows = ~np.isnan(ref).any((1, 2))
    assert np.isfinite(got[rows]).all()
    err = np.abs(got[rows] - ref[rows])
    tol = pu.bound(ref[rows], q.dtype, vmax)
    assert (err <= tol).all(), float((err / tol).max())
    return ref


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,G,page,lens", [(1, 1, 64, [1]), (1, 4, 16, [64]), (2, 1, 32, [65, 1, 63]), (1, 8, 256, [1000]),
                                           (3, 3, 16, [17, 0, 511, 33]), (2, 12, 64, [300, 129]), (8, 1, 64, [2500])])
def test_decode(dtype, d, H, G, page, lens):
    cache, table, lens_t, g = _pool(lens, H, d, page, seed=d + H * G, dtype=dtype)
    q = _randn(g, len(lens), H * G, d, dtype=dtype)
    out = cache.attention(q, table, lens_t)
    _check(cache, q, table, lens_t, np.arange(len(lens) + 1), out)
    assert cache.status() == (0, 0)
    assert torch.equal(out, cache.attention(q, table, lens_t))       # the same bits again


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 2), (64, 0), (100, 4), (128, 70), (1000, 1), (3, 1 << 30), (1 << 29, 5)])
def test_window_and_sinks(d, window, sinks):
    lens = [1, 5, 64, 200, 777]
    cache, table, lens_t, g = _pool(lens, 2, d, 16, seed=window + sinks % 97, dtype=torch.bfloat16)
    q = _randn(g, len(lens), 6, d, dtype=torch.bfloat16)
    out = cache.attention(q, table, lens_t, window=window, sinks=sinks)
    _check(cache, q, table, lens_t, np.arange(len(lens) + 1), out, window=window, sinks=sinks)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,H,G,page", [(64, 2, 4, 32), (128, 2, 4, 64), (128, 1, 5, 16), (128, 3, 1, 128), (256, 1, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 3)])
def test_several_queries(dtype, d, H, G, page, window, sinks):
    """Ragged numbers of queries: none, one, some, all of a sequence's tokens,
    more than it has (queries before its first token see nothing)."""
    lens, new = [130, 40, 64, 3, 200, 0, 90], [1, 0, 64, 5, 37, 2, 3]
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, H, d, page, seed=d + G, dtype=dtype)
    total = int(starts[-1])
    q = _randn(g, total + 3, H * G, d, dtype=dtype)
    out = torch.full_like(q, 7.0)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    for most in (64, 1, None):                   # right, too few, unknown
        out.fill_(7.0)
        cache.attention(q, table, lens_t, q_starts=st, max_q_len=most, window=window, sinks=sinks, out=out)
        _check(cache, q, table, lens_t, starts, out, window=window, sinks=sinks)
        assert (out[total:] == 7.0).all()        # rows behind the last sequence stay
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("d,H,G,n", [(128, 1, 4, 20000), (64, 2, 1, 30001), (256, 1, 8, 9000), (128, 1, 16, 7000)])
def test_long_sequence_split_over_the_gpu(d, H, G, n):
    cache, table, lens_t, g = _pool([n], H, d, 64, seed=n)
    q = _randn(g, 1, H * G, d, dtype=torch.float16)
    out = cache.attention(q, table, lens_t)
    _check(cache, q, table, lens_t, np.arange(2), out)
    assert torch.equal(out, cache.attention(q, table, lens_t))


def test_many_short_sequences_and_a_long_one():
    lens = [(7 * i) % 90 for i in range(300)] + [5000] + [3] * 20
    cache, table, lens_t, g = _pool(lens, 2, 64, 16, seed=9)
    q = _randn(g, len(lens), 4, 64, dtype=torch.float16)
    _check(cache, q, table, lens_t, np.arange(len(lens) + 1), cache.attention(q, table, lens_t))


def test_scores_far_apart():
    """Scores that span hundreds of powers of two (the running maximum moves,
    weights vanish) and a query of large and small channels."""
    cache, table, lens_t, g = _pool([900, 400], 1, 128, 64, seed=4, dtype=torch.bfloat16)
    q = _randn(g, 2, 4, 128, dtype=torch.bfloat16) * 100
    q[0, 1] *= 1e4
    q[1, 2] *= 1e-30
    q[1, 3] = 0
    _check(cache, q, table, lens_t, np.arange(3), cache.attention(q, table, lens_t, scale=0.5), scale=0.5)


def test_strides_of_queries_output_and_table():
    cache, table, lens_t, g = _pool([100, 333], 2, 64, 32, seed=6)
    qkv = _randn(g, 2, 4 * 64 + 256, dtype=torch.float16)
    q = qkv[:, :256].unflatten(1, (4, 64))
    big = torch.full((2, 6, 64), 3.0, dtype=torch.float16, device=DEV)
    wide = torch.full((2, table.shape[1] + 9), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    out = cache.attention(q, wide[:, :table.shape[1]], lens_t, out=big[:, 1:5])
    _check(cache, q, table, lens_t, np.arange(3), out)
    assert (big[:, 0] == 3).all() and (big[:, 5] == 3).all()
    odd = torch.empty(2 * 4 * 65 + 1, dtype=torch.float16, device=DEV)[1:].as_strided((2, 4, 64), (260, 65, 1))
    odd.copy_(q)
    assert torch.equal(cache.attention(odd, table, lens_t), out)
    with pytest.raises(tq.TQError, match="ALIGN"):
        cache.attention(q, table, lens_t, out=odd)


def test_pages_lengths_and_starts_out_of_range():
    """Bad indices are held to the buffers, flagged, and harm no other sequence."""
    cache, table, lens_t, g = _pool([200, 150, 100], 2, 128, 32, seed=8)
    q = _randn(g, 3, 4, 128, dtype=torch.float16)
    good = cache.attention(q, table, lens_t)
    assert cache.status() == (0, 0)
    bad = table.clone()
    bad[1, 0], bad[1, 3], bad[1, 4] = -1, cache.n_pages, 1 << 30
    out = cache.attention(q, bad, lens_t)
    assert cache.status() == (0, 2)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    kp, vp = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    t = np.array([i for i in range(150) if i // 32 in (1, 2)])
    slots = table[1].cpu().numpy()[t // 32].astype(np.int64) * 32 + t % 32
    k, v = pu.row_values(kp, 32, 128, slots), pu.row_values(vp, 32, 128, slots)
    for h in range(4):
        s = k[:, h // 2] @ q[1, h].cpu().double().numpy() / np.sqrt(128)
        w = np.exp(s - s.max())
        ref = w @ v[:, h // 2] / w.sum()
        assert (np.abs(out[1, h].cpu().double().numpy() - ref) <= pu.bound(ref, q.dtype, np.abs(v).max())).all()
    # other lengths and starts: the work is split otherwise, so float32 sums
    # come in another order and the rows are compared with the 64-bit form
    cache.reset_status()
    lens = lens_t.clone()
    lens[1] = -5                                     # as if 0
    _check(cache, q, table, lens.clamp(min=0), np.arange(4), cache.attention(q, table, lens))
    assert cache.status() == (0, 2)
    cache.reset_status()
    starts = torch.tensor([0, 1, 9, 3], dtype=torch.int32, device=DEV)      # as if 0 1 3 3
    _check(cache, q, table, lens_t, np.array([0, 1, 3, 3]), cache.attention(q, table, lens_t, q_starts=starts, max_q_len=2))
    assert cache.status() == (0, 2)
    cache.reset_status()
    lens[1] = 1 << 30                                # as if the whole row of the table
    out = cache.attention(q, table, lens)
    out[1] = good[1]
    _check(cache, q, table, lens_t, np.arange(4), out)
    assert cache.status() == (0, 2)


def test_queries_that_are_not_finite_stay_in_their_rows():
    cache, table, lens_t, g = _pool([70, 90], 1, 64, 16, seed=3, dtype=torch.bfloat16)
    q = _randn(g, 2, 4, 64, dtype=torch.bfloat16)
    good = cache.attention(q, table, lens_t)
    p = q.clone()
    p[0, 1, 5] = float("nan")
    p[1, 2, 0] = float("inf")
    out = cache.attention(p, table, lens_t)
    same = torch.ones(2, 4, dtype=torch.bool)
    same[0, 1] = same[1, 2] = False
    assert torch.equal(out[same.to(DEV)], good[same.to(DEV)])
    assert out[0, 1].isnan().all()


# ------------------------------------------------- together, graphs, streams

def _run_steps(cache, table, steps, lens, k, v, q, window, sinks):
    outs = []
    B = len(lens)
    for i in range(steps):
        lens = lens + 1
        pos = (lens - 1).long()
        slots = torch.gather(table.long(), 1, (pos // cache.page_size)[:, None])[:, 0] * cache.page_size + pos % cache.page_size
        cache.write(k[i], v[i], slots)
        outs.append(cache.attention(q[i], table, lens, window=window, sinks=sinks))
    return outs, lens


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 2)])
def test_prompt_then_decode_steps(window, sinks):
    """A prompt written and attended to in one go, then tokens one by one:
    each step equals the plain form over what the cache then holds, and the
    prompt's rows equal those of the same tokens fed one by one."""
    B, H, G, d, page, prompt, steps = 3, 2, 4, 128, 16, 37, 12
    g = _gen(12)
    cache = tq.PagedCache(B * 4 + 1, H, d, page_size=page)
    table = torch.randperm(B * 4 + 1, generator=g)[:B * 4].view(B, 4).int().to(DEV)
    t = torch.arange(prompt, device=DEV)
    slots = (table.long()[:, t // page] * page + t % page).flatten()
    k0, v0 = (_randn(g, B * prompt, H, d, dtype=torch.bfloat16) for _ in range(2))
    q0 = _randn(g, B * prompt, H * G, d, dtype=torch.bfloat16)
    cache.write(k0, v0, slots)
    lens = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    starts = np.arange(B + 1) * prompt
    out0 = cache.attention(q0, table, lens, q_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), max_q_len=prompt, window=window, sinks=sinks)
    ref0 = _check(cache, q0, table, lens, starts, out0, window=window, sinks=sinks)
    # the prompt's last token alone: one query a sequence
    last = torch.arange(1, B + 1, device=DEV) * prompt - 1
    one = cache.attention(q0[last], table, lens, window=window, sinks=sinks)
    _check(cache, q0[last], table, lens, np.arange(B + 1), one, window=window, sinks=sinks)
    assert np.array_equal(ref0[last.cpu().numpy()], pu.attention(cache.k.cpu().numpy(), cache.v.cpu().numpy(), page, q0[last], table.cpu().numpy(), lens.cpu().numpy(), np.arange(B + 1), window=window, sinks=sinks))
    k, v = (_randn(g, steps, B, H, d, dtype=torch.bfloat16) for _ in range(2))
    q = _randn(g, steps, B, H * G, d, dtype=torch.bfloat16)
    for i in range(steps):
        (out,), lens = _run_steps(cache, table, 1, lens, k[i:i + 1], v[i:i + 1], q[i:i + 1], window, sinks)
        _check(cache, q[i], table, lens, np.arange(B + 1), out, window=window, sinks=sinks)
    assert cache.status() == (0, 0)


def test_a_captured_step_replays():
    """A step (write, attention with its split) captured once and replayed as
    lengths, slots, rows and queries change in place, two graphs in turn."""
    B, H, G, d, page = 2, 2, 4, 128, 32
    lens = [700, 90]
    cache, table, lens_t, g = _pool(lens, H, d, page, seed=21)
    twin = tq.PagedCache(cache.n_pages, H, d, page_size=page)
    table = torch.cat((table[:, :-1], torch.full((B, 1), cache.n_pages - 1, dtype=torch.int32, device=DEV)), 1)
    table[1, 3:] = table[1, 2]
    k, v = _randn(g, B, H, d, dtype=torch.float16), _randn(g, B, H, d, dtype=torch.float16)
    q = _randn(g, B, H * G, d, dtype=torch.float16)
    slots = torch.zeros(B, dtype=torch.int64, device=DEV)
    outs = [torch.empty_like(q) for _ in range(2)]
    ws = [torch.empty(cache.workspace_bytes(H * G, B, table.shape[1]), dtype=torch.uint8, device=DEV) for _ in range(2)]
    graphs = []
    cache.attention(q, table, lens_t, out=outs[0], workspace=ws[0])
    torch.cuda.synchronize()
    saved = cache.k.clone(), cache.v.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                cache.write(k, v, slots)
                cache.attention(q, table, lens_t, out=outs[i], workspace=ws[i])
        graphs.append(graph)
    torch.cuda.current_stream().wait_stream(s)
    cache.k.copy_(saved[0])
    cache.v.copy_(saved[1])
    twin.k.copy_(saved[0])
    twin.v.copy_(saved[1])
    for i in range(6):
        for x in (k, v, q):
            x.copy_(_randn(g, *x.shape, dtype=torch.float16))
        pos = lens_t.long()
        slots.copy_(torch.gather(table.long(), 1, (pos // page)[:, None])[:, 0] * page + pos % page)
        lens_t += 1
        graphs[i % 2].replay()
        twin.write(k, v, slots)
        ref = twin.attention(q, table, lens_t)
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], ref) and torch.equal(cache.k, twin.k) and torch.equal(cache.v, twin.v)


def test_two_streams_at_once():
    cache, table, lens_t, g = _pool([3000, 100, 2000], 2, 128, 64, seed=5)
    qs = [_randn(g, 3, 8, 128, dtype=torch.float16) for _ in range(2)]
    want = [cache.attention(q, table, lens_t) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(cache.attention(qs[i], table, lens_t, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,H,G,page,lens,new", [(64, 1, 1, 64, [64], [64]), (128, 2, 4, 64, [200], [33]), (128, 1, 8, 16, [300, 17], [40, 17]),
                                                 (64, 2, 3, 128, [500, 20, 129], [500, 20, 1]), (256, 1, 4, 32, [333, 90], [90, 77]),
                                                 (128, 1, 1, 256, [700], [699])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_prompts(dtype, d, H, G, page, lens, new, window, sinks):
    """Many queries a sequence: chunks and whole prompts on the tensor cores."""
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, H, d, page, seed=d + G + page, dtype=dtype)
    q = _randn(g, int(starts[-1]), H * G, d, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    out = cache.attention(q, table, lens_t, q_starts=st, max_q_len=max(new), window=window, sinks=sinks)
    _check(cache, q, table, lens_t, starts, out, window=window, sinks=sinks)
    assert torch.equal(out, cache.attention(q, table, lens_t, q_starts=st, max_q_len=max(new), window=window, sinks=sinks))
    assert cache.status() == (0, 0)


def test_long_prompt_chunk_split_over_the_gpu():
    cache, table, lens_t, g = _pool([6000], 1, 128, 64, seed=77)
    q = _randn(g, 90, 4, 128, dtype=torch.bfloat16)
    st = torch.tensor([0, 90], dtype=torch.int32, device=DEV)
    out = cache.attention(q, table, lens_t, q_starts=st, max_q_len=90)
    _check(cache, q, table, lens_t, np.array([0, 90]), out)
    assert torch.equal(out, cache.attention(q, table, lens_t, q_starts=st, max_q_len=90))


def test_prompt_scores_far_apart():
    """The running maximum moves late and by much: the outputs so far are
    scaled down, rows of one warp by unlike factors."""
    cache, table, lens_t, g = _pool([800], 1, 128, 64, seed=78)
    q = _randn(g, 200, 1, 128, dtype=torch.float16) * torch.linspace(0.01, 60, 200, device=DEV)[:, None, None].half()
    st = torch.tensor([0, 200], dtype=torch.int32, device=DEV)
    out = cache.attention(q, table, lens_t, q_starts=st, max_q_len=200)
    _check(cache, q, table, lens_t, np.array([0, 200]), out)


def test_no_tokens_no_pages_no_queries():
    cache = tq.PagedCache(2, 1, 64, page_size=16)
    q = _randn(_gen(1), 3, 2, 64, dtype=torch.float16)
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    out = cache.attention(q, torch.empty(3, 0, dtype=torch.int32, device=DEV), zero)
    assert not out.any() and cache.status() == (0, 0)
    none = cache.attention(q[:0], torch.empty(3, 0, dtype=torch.int32, device=DEV), zero, q_starts=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert none.shape == (0, 2, 64)
    with pytest.raises(tq.TQError, match="EMPTY"):
        cache.attention(q[:0], torch.empty(0, 0, dtype=torch.int32, device=DEV), zero[:0])


def test_many_sequences_of_several_queries():
    """More sequences than a CTA has threads, on both kernels, sequences without queries among them."""
    B = 700
    lens = [(11 * i) % 75 for i in range(B)]
    new = [min(lens[i], i % 4) for i in range(B)]
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, 1, 64, 16, seed=10)
    q = _randn(g, int(starts[-1]), 2, 64, dtype=torch.float16)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    for most in (4, 40):
        _check(cache, q, table, lens_t, starts, cache.attention(q, table, lens_t, q_starts=st, max_q_len=most))


@pytest.mark.parametrize("rows", [1, 40])
def test_pool_past_four_gigabytes(rows):
    """Pages whose byte offsets pass 32 bits, written, read and attended to."""
    H, d, page = 32, 128, 64
    n_pages = (1 << 32) // (H * page * 68) + 40
    cache = tq.PagedCache(n_pages, H, d, page_size=page)
    g = _gen(5)
    pages = torch.tensor([n_pages - 1, 3, n_pages - 20, n_pages - 7])
    t = torch.arange(230)
    slots = (pages[t // page] * page + t % page).to(DEV)
    k, v = _randn(g, 230, H, d, dtype=torch.float16), _randn(g, 230, H, d, dtype=torch.float16)
    ks, vs = cache.write(k, v, slots, stored=True)
    kr, vr = cache.read(slots, dtype=torch.float16)
    assert torch.equal(kr, ks) and torch.equal(vr, vs)
    q = _randn(g, rows, H, d, dtype=torch.float16)
    out = cache.attention(q, pages.int()[None].to(DEV), torch.tensor([230], dtype=torch.int32, device=DEV),
                          q_starts=torch.tensor([0, rows], dtype=torch.int32, device=DEV), max_q_len=rows)
    # the same rows in a small pool give the same bits
    small = tq.PagedCache(4, H, d, page_size=page)
    small.write(k, v, t.to(DEV))
    same = small.attention(q, torch.arange(4, dtype=torch.int32, device=DEV)[None], torch.tensor([230], dtype=torch.int32, device=DEV),
                           q_starts=torch.tensor([0, rows], dtype=torch.int32, device=DEV), max_q_len=rows)
    assert torch.equal(out, same)
    assert cache.status() == (0, 0)


def test_a_captured_prompt_replays():
    """Chunks on the tensor cores, captured and replayed with other lengths,
    pages and queries; a stream of its own."""
    cache, table, lens_t, g = _pool([500, 300], 1, 128, 32, seed=31)
    q = _randn(g, 120, 4, 128, dtype=torch.float16)
    st = torch.tensor([0, 80, 120], dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    cache.attention(q, table, lens_t, q_starts=st, max_q_len=80, window=200, sinks=3, out=out)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            cache.attention(q, table, lens_t, q_starts=st, max_q_len=80, window=200, sinks=3, out=out)
    torch.cuda.current_stream().wait_stream(s)
    for lens, starts in (([500, 300], [0, 80, 120]), ([77, 300], [0, 5, 120]), ([490, 1], [0, 119, 120])):
        lens_t.copy_(torch.tensor(lens))
        st.copy_(torch.tensor(starts))
        q.copy_(_randn(g, *q.shape, dtype=torch.float16))
        out.zero_()
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        _check(cache, q, table, lens_t, np.array(starts), got, window=200, sinks=3)
        assert torch.equal(got, cache.attention(q, table, lens_t, q_starts=st, max_q_len=80, window=200, sinks=3))


def test_workspace_is_checked():
    cache, table, lens_t, g = _pool([4000], 1, 64, 16, seed=2)
    q = _randn(g, 1, 2, 64, dtype=torch.float16)
    need = cache.workspace_bytes(2, 1, table.shape[1])
    ws = torch.empty(need + 32, dtype=torch.uint8, device=DEV)
    want = cache.attention(q, table, lens_t)
    ws.fill_(255)                                    # contents on entry are ignored
    assert torch.equal(cache.attention(q, table, lens_t, workspace=ws[:need]), want)
    with pytest.raises(tq.TQError, match="WORKSPACE"):
        cache.attention(q, table, lens_t, workspace=ws[:need - 1])
    with pytest.raises(tq.TQError, match="ALIGN"):
        cache.attention(q, table, lens_t, workspace=ws[16:])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 50])
def test_short_sequences_whole_or_split(d, most):
    """Where the page table allows only short sequences none is split and no
    workspace is needed; a wider table, the same sequences: split and joined."""
    lens, new = [500, 3, 256, 0, 77, 130], [min(n, most) for n in (50, 3, 17, 1, 1, 40)]
    starts = np.concatenate(([0], np.cumsum(new)))
    cache, table, lens_t, g = _pool(lens, 2, d, 16, seed=d + most, dtype=torch.bfloat16)
    table = table[:, :32].contiguous()
    wide = torch.cat((table, torch.full((len(lens), 4096 // 16), -1, dtype=torch.int32, device=DEV)), 1)
    assert cache.workspace_bytes(8, len(lens), 32, most) == 0 < cache.workspace_bytes(8, len(lens), wide.shape[1], most)
    q = _randn(g, int(starts[-1]), 8, d, dtype=torch.bfloat16)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    for t in (table, wide):
        for window, sinks in ((0, 0), (100, 2)):
            out = cache.attention(q, t, lens_t, q_starts=st, max_q_len=most, window=window, sinks=sinks)
            _check(cache, q, table, lens_t, starts, out, window=window, sinks=sinks)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 60])
@pytest.mark.parametrize("page_ids", [0, 300])
def test_equal_values_are_given_back(d, most, page_ids):
    """Weights are divided by the sum of what they are rounded to, so that
    values which are the same for every token come back as they are stored:
    the float32 sums of at most 500 products are off by less than 500 * 2^-22,
    under half a step of binary16 (2^-11 relative), and a stored value has
    seven significant bits.  A wider page table: split and joined."""
    lens, new = [500, 2, 5, 257, 33], [min(n, most) for n in (60, 2, 5, 50, 1)]
    starts = np.concatenate(([0], np.cumsum(new)))
    n = sum(lens)
    g = _gen(d + most)
    cache = tq.PagedCache(sum((x + 31) // 32 for x in lens), 2, d, page_size=32)
    table = torch.full((len(lens), max(16, page_ids)), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, x in enumerate(lens):
        pages = (x + 31) // 32
        table[b, :pages] = torch.arange(at, at + pages)
        slots.append(at * 32 + torch.arange(x))
        at += pages
    k = _randn(g, n, 2, d, dtype=torch.float16) * 2
    row = _randn(g, 1, 2, d, dtype=torch.float16)
    stored = cache.write(k, row.expand(n, 2, d).contiguous(), torch.cat(slots).to(DEV), stored=True)[1][0]
    q = _randn(g, int(starts[-1]), 8, d, dtype=torch.float16)
    out = cache.attention(q, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                          q_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), max_q_len=most)
    assert torch.equal(out, stored.repeat_interleave(4, 0).expand_as(out))
