"""The 8-bit paged cache on the GPU against plain 64-bit forms: writing,
reading back, the attention of a chunk over it, and a run of them together."""
import numpy as np
import pytest

import _kv8 as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dfl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__ as g
    g.build()
    import block_diffusion_speculative_layer_gb300 as m
    return m


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf(x):
    return gpu(np.asarray(x, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def on_gpu(dfl, c, cache):
    return (dfl.KV8Cache(gpu(cache.codes), gpu(cache.exps), torch.zeros(1, dtype=torch.int32, device="cuda")),
            gpu(c.table), gpu(c.row_start), gpu(c.kv_len))


def filled(c, fill=None):
    """A cache holding every sequence's positions 0 .. kv_len - 1; other bytes zero, or random."""
    cache = R.Cache(c, fill)
    for s, n in enumerate(c.kv_len):
        if n:
            cache.put_many(s, 0, c.vectors(n), c.vectors(n))
    return cache


def attend(dfl, c, cache, q, causal=True, window=0, scale=None, **kw):
    h, table, start, lens = on_gpu(dfl, c, cache)
    x = bf(q).view(c.rows, -1)
    out, lse = dfl.attention_kv8(x, h, table, start, lens, int(c.n.max()), int(c.kv_len.max()), causal=causal,
                                 window=window, scale=scale, lse=True, **kw)
    dfl.kv8_check(h)
    return f64(out).reshape(c.rows, c.q_heads, c.hd), f64(lse), x


def compare(c, cache, got, lse, x, **kw):
    q = f64(x).reshape(c.rows, c.q_heads, c.hd)
    out, ref, dout, dlse = R.attention(c, cache, q, **kw)
    mine = ~np.isnan(ref) | np.isnan(lse)
    rows = slice(int(c.row_start[0]), int(c.row_start[-1]))
    assert mine[rows].all()
    empty = np.isneginf(ref[rows])
    assert np.array_equal(np.isneginf(lse[rows]), empty) and (got[rows][empty] == 0).all()
    far = np.abs(got - out)[rows]
    assert (far <= dout[rows]).all(), (far / np.maximum(dout[rows], 1e-300)).max()
    with np.errstate(invalid="ignore"):
        off = np.where(empty, 0.0, np.abs(lse - ref)[rows])
    assert (off <= dlse[rows]).all(), (off / dlse[rows])[~empty].max()


# ------------------------------------------------------------------ write, read
SHAPES = [  # sequences as (rows, positions before them), heads, head dim, page
    ([(1, 0)], 1, 128, 16),
    ([(1, 37), (1, 0), (1, 15), (1, 16), (1, 500)], 8, 128, 16),
    ([(16, 5), (0, 40), (3, 0), (40, 120), (0, 0), (17, 15)], 2, 64, 32),
    ([(300, 1)], 5, 64, 48),
    ([(129, 127), (64, 64)], 4, 128, 64),
    ([(5, -3), (4, -4), (20, -2), (33, -17)], 3, 128, 16),   # left padding
    ([(1, 3 + i) for i in range(70)], 1, 64, 1024),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("seqs,heads,hd,page", SHAPES)
def test_write_and_read(dfl, seqs, heads, hd, page, dtype):
    c = R.Case(seqs, heads, hd, page, seed=3, first_row=2, extra_rows=3)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    # rows cut out of a fused projection: a row is 2 heads of something else, then keys, then values
    x = gpu(c.vectors(c.rows * 3).reshape(c.rows, 3 * heads, hd).astype(np.float32))
    x = torch.cat([torch.zeros((c.rows, 2, hd), device="cuda"), x], 1).to(dt)
    k, v = x[:, 2:2 + heads], x[:, 2 + heads:2 + 2 * heads]
    cache = R.Cache(c, np.random.default_rng(1))   # bytes that are not the call's stay
    h, table, start, lens = on_gpu(dfl, c, cache)
    dfl.kv8_write(h, k, v, table, start, lens)
    for s in range(len(seqs)):
        r0, pos = c.row_start[s], c.positions(s)
        keep = pos >= 0
        if keep.any():
            rows = slice(int(r0 + np.argmax(keep)), int(c.row_start[s + 1]))
            cache.put_many(s, int(pos[keep][0]), f64(k)[rows], f64(v)[rows])
    np.testing.assert_array_equal(h.codes.cpu().numpy(), cache.codes)
    np.testing.assert_array_equal(h.exps.cpu().numpy(), cache.exps)
    for rt in (torch.bfloat16, torch.float32):
        kr, vr = (torch.full((c.rows, heads, hd), -7.0, dtype=rt, device="cuda") for _ in range(2))
        dfl.kv8_read(h, table, start, lens, c.rows, k=kr, v=vr)
        dfl.kv8_check(h)
        want_k, want_v = np.full((2, c.rows, heads, hd), -7.0)
        for s, n in enumerate(c.kv_len):
            kk, vv = cache.get(s, int(n))
            for j, p in enumerate(c.positions(s)):
                row = c.row_start[s] + j
                want_k[row], want_v[row] = (kk[p], vv[p]) if p >= 0 else (0.0, 0.0)
        np.testing.assert_array_equal(f64(kr), want_k)
        np.testing.assert_array_equal(f64(vr), want_v)


def test_write_of_unusual_values(dfl):
    # zeros, subnormals, ties, infinities, NaN, the largest numbers: codes and bytes as the format says
    c = R.Case([(24, 0)], 2, 64, 16)
    x = c.vectors(24).astype(np.float32)
    x[0], x[1, 0] = 0.0, -0.0
    x[2] *= np.float32(1e-38)
    x[3, 0, 5], x[3, 1, 6], x[4, 0, 0] = np.inf, -np.inf, np.nan
    x[5] = (np.arange(64) - 32) * np.float32(448 / 32)      # ties between codes
    x[6, 0] = np.float32(3.3e38)
    x[7, 0, 1:], x[7, 0, 0] = np.float32(2.0 ** -140), 1.0   # far below the vector's largest
    x[8, 0], x[8, 1] = 448.0, np.nextafter(np.float32(448), np.float32(449))
    x[9] = np.float32(2.0 ** -130)
    cache = R.Cache(c)
    h, table, start, lens = on_gpu(dfl, c, cache)
    dfl.kv8_write(h, gpu(x), gpu(x[::-1].copy()), table, start, lens)
    cache.put_many(0, 0, x.astype(np.float64), x[::-1].astype(np.float64))
    np.testing.assert_array_equal(h.exps.cpu().numpy(), cache.exps)
    np.testing.assert_array_equal(h.codes.cpu().numpy(), cache.codes)
    k, v = dfl.kv8_read(h, table, start, lens, 24, dtype=torch.float32)
    bad = ~np.isfinite(x).all(-1)
    assert np.isnan(f64(k)[bad]).all() and np.isfinite(f64(k)[~bad]).all()
    # half a step of 3 mantissa bits, or of the smallest code, of the vector's power of two
    good = x[~bad].astype(np.float64)
    top = np.abs(good).max(-1, keepdims=True)
    assert (np.abs(f64(k)[~bad] - np.clip(good, -448 * 2.0 ** 119, 448 * 2.0 ** 119)) <=
            np.abs(good) * 2.0 ** -4 + np.maximum(top * 2.0 ** -17, 2.0 ** -110)).all()


# -------------------------------------------------------------------- attention
ATTENTION = {  # sequences, query heads, KV heads, head dim, page
    "one-token": ([(1, 0)], 4, 1, 128, 16),
    "decode": ([(1, 511), (1, 0), (1, 1300), (1, 127), (1, 128)], 32, 8, 128, 16),
    "decode-g1-hd64": ([(1, 77), (1, 640)], 3, 3, 64, 32),
    "block": ([(16, 1024)], 32, 8, 128, 16),
    "block-ragged": ([(16, 130), (0, 9), (3, 0), (16, 0), (7, 1000)], 10, 2, 128, 64),
    "group-16": ([(5, 300)], 32, 2, 64, 16),
    "group-40": ([(2, 200), (1, 3)], 40, 1, 128, 48),
    "chunk": ([(200, 333), (65, 0)], 8, 2, 128, 16),
    "chunk-hd64-g7": ([(131, 70), (1, 5)], 14, 2, 64, 32),
    "padding": ([(6, -2), (4, -4), (40, -33), (3, 10)], 8, 2, 128, 16),
}


@pytest.mark.parametrize("mask", ["causal", "all", "window1", "window100"])
@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention(dfl, name, mask):
    seqs, hq, hkv, hd, page = ATTENTION[name]
    c = R.Case(seqs, hkv, hd, page, seed=len(name), first_row=1, extra_rows=2, q_heads=hq)
    cache = filled(c, np.random.default_rng(9))   # bytes behind a sequence's end: anything, NaN codes among them
    q = c.g.standard_normal((c.rows, hq, hd)) * 2
    causal, window = mask != "all", int(mask[6:]) if mask.startswith("window") else 0
    got, lse, x = attend(dfl, c, cache, q, causal, window)
    compare(c, cache, got, lse, x, causal=causal, window=window)


@pytest.mark.parametrize("cluster", [1, 2, 4, 8, 16])
def test_every_split(dfl, cluster):
    c = R.Case([(16, 900), (1, 3), (2, 4000)], 2, 128, 16, seed=5, q_heads=8)
    cache = filled(c)
    got, lse, x = attend(dfl, c, cache, c.g.standard_normal((c.rows, 8, 128)), cluster_ctas=cluster)
    compare(c, cache, got, lse, x)


def test_long_context(dfl):
    c = R.Case([(1, 32767), (16, 20000)], 1, 128, 16, seed=6, q_heads=4)
    cache = filled(c)
    got, lse, x = attend(dfl, c, cache, c.g.standard_normal((c.rows, 4, 128)))
    compare(c, cache, got, lse, x)


def test_rising_falling_and_sharp_scores(dfl):
    # scores that grow along the keys (the running maximum moves all the time), fall, or pick one key
    c = R.Case([(4, 1500)] * 3, 1, 64, 16, seed=8, q_heads=2)
    cache = R.Cache(c)
    n = 1504
    for s in range(3):
        k = 0.05 * c.vectors(n)
        k[:, 0, 0] = np.linspace(0, 60, n) if s == 0 else np.linspace(60, 0, n) if s == 1 else 0.0
        if s == 2:
            k[777, 0, 0] = 60.0
        cache.put_many(s, 0, k, c.vectors(n))
    q = np.ones((c.rows, 2, 64))
    q[:, :, 0] = 30.0
    got, lse, x = attend(dfl, c, cache, q)
    compare(c, cache, got, lse, x)


def test_values_of_very_different_size(dfl):
    # one token's values are 2^40 times another's; a token of large values far behind the others in score
    c = R.Case([(2, 600)], 2, 128, 16, seed=12)
    cache = R.Cache(c)
    k, v = c.vectors(602), c.vectors(602)
    v[::7] *= 2.0 ** 40
    v[5::7] *= 2.0 ** -40
    k[300], v[300] = -8 * np.sign(c.vectors(1)[0]), 2.0 ** 60
    cache.put_many(0, 0, k, v)
    got, lse, x = attend(dfl, c, cache, c.g.standard_normal((2, 2, 128)))
    compare(c, cache, got, lse, x)


def test_large_and_tiny_queries(dfl):
    c = R.Case([(6, 200)], 1, 128, 16, seed=13, q_heads=2)
    cache = R.Cache(c)
    cache.put_many(0, 0, c.vectors(206) * 1e-3, c.vectors(206))
    q = c.g.standard_normal((6, 2, 128))
    q[0] *= 3e4
    q[1] *= 1e6
    q[2] *= 1e-6
    q[3, 0, 0], q[4] = 1e5, 0.0
    got, lse, x = attend(dfl, c, cache, q, scale=1e-3)
    compare(c, cache, got, lse, x, scale=1e-3)
    got, lse, x = attend(dfl, c, cache, q[::-1].copy() * 1e-3, scale=-2.0)
    compare(c, cache, got, lse, x, scale=-2.0)


def test_vectors_without_numbers_reach_only_the_rows_that_see_them(dfl):
    c = R.Case([(20, 100)], 1, 128, 16, seed=14, q_heads=2)
    cache = R.Cache(c)
    k, v = c.vectors(120), c.vectors(120)
    k[110, 0, 3], v[115, 0, 9] = np.nan, np.inf
    cache.put_many(0, 0, k, v)
    q = c.g.standard_normal((20, 2, 128))
    got, lse, x = attend(dfl, c, cache, q)
    clean = R.Cache(c)
    clean.put_many(0, 0, np.nan_to_num(k), np.nan_to_num(v, posinf=0.0))
    want, wlse, _ = attend(dfl, c, clean, q)
    np.testing.assert_array_equal(got[:10], want[:10])
    np.testing.assert_array_equal(lse[:10], wlse[:10])
    assert np.isnan(got[10:]).all() and np.isnan(lse[10:]).all()
    # a window that has passed both sees numbers again
    got, lse, x = attend(dfl, c, cache, q, window=3)
    bad = np.array([j in (10, 11, 12, 15, 16, 17) for j in range(20)])
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_rows_of_no_sequence_stay(dfl):
    c = R.Case([(3, 40), (2, 0)], 2, 64, 16, seed=15, first_row=4, extra_rows=5, q_heads=4)
    cache = filled(c)
    q = c.g.standard_normal((c.rows, 4, 64))
    wide = torch.full((c.rows, 512), 3.5, dtype=torch.bfloat16, device="cuda")   # rows of a wider buffer
    x = torch.zeros((c.rows, 384), dtype=torch.bfloat16, device="cuda")
    x[:, 64:320] = bf(q).view(c.rows, 256)
    lse = torch.full((c.rows, 4), 9.0, device="cuda")
    h, table, start, lens = on_gpu(dfl, c, cache)
    dfl.attention_kv8(x[:, 64:320], h, table, start, lens, 3, 43, out=wide[:, 128:384], lse=lse)
    dfl.kv8_check(h)
    got, want_lse, y = attend(dfl, c, cache, q)
    w = f64(wide)
    assert (w[:, :128] == 3.5).all() and (w[:, 384:] == 3.5).all()
    assert (w[:4] == 3.5).all() and (w[9:] == 3.5).all() and (f64(lse)[:4] == 9).all() and (f64(lse)[9:] == 9).all()
    np.testing.assert_array_equal(w[4:9, 128:384], got[4:9].reshape(5, 256))
    np.testing.assert_array_equal(f64(lse)[4:9], want_lse[4:9])
    compare(c, cache, got, want_lse, y)


@pytest.mark.parametrize("cluster", [1, 4])
def test_a_row_alone_equals_the_row_in_its_chunk(dfl, cluster):
    c = R.Case([(70, 700), (70, 30)], 2, 128, 16, seed=16, q_heads=8)
    cache = filled(c)
    q = c.g.standard_normal((c.rows, 8, 128)) * 3
    full, lse, _ = attend(dfl, c, cache, q, cluster_ctas=cluster)
    for j in (0, 13, 69):
        one = R.Case([(1, 700 + j), (1, 30 + j)], 2, 128, 16, q_heads=8)
        one.table, one.n_pages = c.table, c.n_pages
        got, l1, _ = attend(dfl, one, cache, q[[j, 70 + j]], cluster_ctas=cluster)
        np.testing.assert_array_equal(got, full[[j, 70 + j]])
        np.testing.assert_array_equal(l1, lse[[j, 70 + j]])


@pytest.mark.parametrize("cluster", [1, 4])
def test_a_row_of_sharp_scores_leaves_its_neighbours_alone(dfl, cluster):
    # some rows' scores jump by far more than 2^14 over their first chunk's: those come out right, and the
    # other rows of their tile keep their bits
    c = R.Case([(24, 1400)], 1, 128, 16, seed=19, q_heads=4)
    cache = R.Cache(c)
    k, v = 0.3 * c.vectors(1424), c.vectors(1424)
    k[900, 0, 0], k[1300, 0, 0], k[200, 0, 1] = 40.0, 60.0, 50.0
    cache.put_many(0, 0, k, v)
    q = c.g.standard_normal((24, 4, 128))
    q[:, :, :2] = 0.0
    calm, calm_lse, _ = attend(dfl, c, cache, q, cluster_ctas=cluster)
    q[5, 1, 0], q[11, 2, 0], q[17, 0, 1] = 30.0, 9.0, 20.0
    got, lse, x = attend(dfl, c, cache, q, cluster_ctas=cluster)
    compare(c, cache, got, lse, x)
    same = np.ones((24, 4), bool)
    same[5, 1] = same[11, 2] = same[17, 0] = False
    np.testing.assert_array_equal(got[same], calm[same])
    np.testing.assert_array_equal(lse[same], calm_lse[same])


def test_joining_two_parts_by_lse(dfl):
    # attention over all keys = the parts' outputs weighted by their lse
    c = R.Case([(8, 500)], 1, 128, 16, seed=17, q_heads=4)
    cache = filled(c)
    q = c.g.standard_normal((8, 4, 128))
    whole, lse, x = attend(dfl, c, cache, q, causal=False)
    parts = []
    for lo, hi in ((0, 256), (256, 508)):
        p = R.Case([(8, hi - lo - 8)], 1, 128, 16, q_heads=4)
        p.table, p.n_pages = c.table[:, lo // 16:], c.n_pages
        sub = R.Cache(p)
        sub.codes, sub.exps = cache.codes, cache.exps
        parts.append(attend(dfl, p, sub, q, causal=False)[:2])
    w = np.exp(np.stack([l for _, l in parts]) - lse)
    both = sum(o * wi[..., None] for (o, _), wi in zip(parts, w))
    # each side within its own bound: three bf16 roundings and the parts' sums
    A = np.abs(whole) + sum(np.abs(o) * wi[..., None] for (o, _), wi in zip(parts, w))
    assert (np.abs(both - whole) <= 2.0 ** -8 * A + 2.0 ** -9 * np.abs(whole).max()).all()
    np.testing.assert_allclose(w.sum(0), 1.0, atol=2.0 ** -14)


# ----------------------------------------------------------- misuse and the run
def test_out_of_range_pages_and_lengths_are_flagged_and_skipped(dfl):
    c = R.Case([(4, 60), (4, 60), (4, 60)], 2, 64, 16, seed=18)
    cache = filled(c)
    q = c.g.standard_normal((c.rows, 2, 64))
    want, wlse, _ = attend(dfl, c, cache, q)
    c.table[1, 2] = c.n_pages               # positions 32..47 of sequence 1
    c.table[2, 3] = -1                      # the page the rows of sequence 2 go to
    h, table, start, lens = on_gpu(dfl, c, cache)
    x = bf(q).view(c.rows, -1)
    out, lse = dfl.attention_kv8(x, h, table, start, lens, 4, 64, lse=True)
    with pytest.raises(dfl.DfError):
        dfl.kv8_check(h)
    dfl.kv8_check(h)                        # cleared
    got, lse = f64(out).reshape(c.rows, 2, 64), f64(lse)
    np.testing.assert_array_equal(got[:4], want[:4])
    c2 = cache.c = R.Case([(4, 60), (4, 60), (4, 60)], 2, 64, 16, seed=18)   # the table before
    hide = lambda s, t: ((t // 16 == 2) & (s == 1)) | ((t // 16 == 3) & (s == 2))
    ref, rlse, dout, dlse = R.attention(c2, cache, f64(x).reshape(c.rows, 2, 64), hidden=hide)
    assert (np.abs(got - ref) <= dout).all() and (np.abs(lse - rlse) <= dlse).all()
    kv = torch.ones((c.rows, 2, 64), device="cuda")
    before = h.codes.clone()
    dfl.kv8_write(h, kv, kv, table, start, lens)
    with pytest.raises(dfl.DfError):
        dfl.kv8_check(h)
    changed = (h.codes != before).flatten(1).any(1).cpu().numpy()
    assert set(np.flatnonzero(changed)) == {c.table[0, 3], c.table[1, 3]}
    k, v = dfl.kv8_read(h, table, start, lens, c.rows)
    with pytest.raises(dfl.DfError):
        dfl.kv8_check(h)
    assert (f64(k)[8:] == 0).all() and (f64(v)[8:] == 0).all() and (f64(k)[:8] == 1).all()
    # a sequence whose length passes its page table, or whose rows pass the buffer, is left out
    for bad_start, bad_len, left_out in ((c.row_start, [64, 64, 16 * c.table.shape[1] + 1], 2),
                                         ([0, 4, 8, 13], c.kv_len, 2), ([0, 4, 3, 12], c.kv_len, 1),
                                         ([0, 4, 8, 12], [64, 64, -1], 2)):
        h, table, _, _ = on_gpu(dfl, c2, cache)
        start, lens = gpu(np.asarray(bad_start, np.int32)), gpu(np.asarray(bad_len, np.int32))
        out = torch.full_like(x, 5.0)
        dfl.attention_kv8(x, h, table, start, lens, 4, 64, out=out)
        with pytest.raises(dfl.DfError):
            dfl.kv8_check(h)
        assert (f64(out)[:4] == want[:4].reshape(4, -1)).all()
        before = h.codes.clone()
        dfl.kv8_write(h, kv, kv, table, start, lens)
        with pytest.raises(dfl.DfError):
            dfl.kv8_check(h)
        assert not bool((h.codes != before)[c2.table[left_out, 3]].any())
    h, table, start, lens = on_gpu(dfl, c2, cache)
    out = torch.full_like(x, 5.0)
    dfl.attention_kv8(x, h, table, start, lens, 3, 64, out=out)   # more rows than max_rows
    with pytest.raises(dfl.DfError):
        dfl.kv8_check(h)
    assert (f64(out) == 5.0).all()


def test_binding_refuses(dfl):
    c = R.Case([(4, 60)], 2, 64, 16, q_heads=4)
    h, table, start, lens = on_gpu(dfl, c, R.Cache(c))
    q = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((4, 2, 64), device="cuda")
    ok = dict(cache=h, page_table=table, row_start=start, kv_len=lens)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :200]), dict(q=q.t()), dict(q=q[:, :192]),
                dict(out=torch.zeros_like(q).float()), dict(out=q[:2].clone()), dict(lse=torch.zeros((4, 3), device="cuda")),
                dict(lse=torch.zeros((4, 4), device="cuda").half()), dict(window=3, causal=False),
                dict(scale=float("nan")), dict(cluster_ctas=5), dict(page_table=table.long()),
                dict(kv_len=lens.cpu()), dict(row_start=start[:1]), dict(page_table=table[:, ::2]),
                dict(q=torch.zeros((4, 260), dtype=torch.bfloat16, device="cuda")[:, :256])):
        with pytest.raises(dfl.DfError):
            dfl.attention_kv8(**dict(dict(ok, q=q, max_rows=4, max_len=64), **bad))
    for bad in (dict(k=kv.double()), dict(k=kv.bfloat16()), dict(v=kv[:3]), dict(k=kv[..., :32]), dict(v=kv.cpu()),
                dict(k=torch.zeros((4, 64, 2), device="cuda").transpose(1, 2)), dict(k=kv[:1].expand(4, -1, -1)),
                dict(cache=h._replace(codes=h.codes[:, :, :1])), dict(cache=h._replace(exps=h.exps[:1]))):
        with pytest.raises(dfl.DfError):
            dfl.kv8_write(**dict(dict(ok, k=kv, v=kv), **bad))
    for bad in (dict(dtype=torch.float16), dict(k=kv[:3]), dict(rows=-1), dict(k=kv, dtype=torch.bfloat16)):
        with pytest.raises(dfl.DfError):
            dfl.kv8_read(**dict(dict(ok, rows=4), **bad))
    dfl.kv8_check(h)
    e = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    out, lse = dfl.attention_kv8(e, h, table, start, lens, 0, 64, lse=True)   # no rows: nothing to do
    assert out.shape == (0, 256) and lse.shape == (0, 4)
    dfl.kv8_write(h, kv[:0], kv[:0], table, start, lens)


def test_cache_beyond_four_gigabytes(dfl):
    # page ids at the end of a pool of 5.4 GB: byte offsets pass 32 bits
    c = R.Case([(3, 50), (16, 1000)], 2, 128, 16, seed=20, n_pages=700000, q_heads=8)
    assert c.n_pages * 2 * 2 * 16 * 128 > 5 * 2 ** 30
    h = dfl.kv8_cache(c.n_pages, 2, 128, 16)
    table, lens = gpu(c.table), gpu(c.kv_len)
    k, v = bf(c.vectors(int(c.kv_len.sum()))), bf(c.vectors(int(c.kv_len.sum())))
    start = gpu(np.concatenate([[0], np.cumsum(c.kv_len)]).astype(np.int32))
    dfl.kv8_write(h, k, v, table, start, lens)
    kr, vr = dfl.kv8_read(h, table, start, lens, k.shape[0], dtype=torch.float32)
    small = R.Case([(3, 50), (16, 1000)], 2, 128, 16, seed=20, q_heads=8)
    cache = R.Cache(small)
    for s in range(2):
        rows = slice(int(start[s]), int(start[s + 1]))
        cache.put_many(s, 0, f64(k)[rows], f64(v)[rows])
        np.testing.assert_array_equal(f64(kr)[rows], cache.get(s, int(c.kv_len[s]))[0])
        np.testing.assert_array_equal(f64(vr)[rows], cache.get(s, int(c.kv_len[s]))[1])
    q = c.g.standard_normal((c.rows, 8, 128))
    x = bf(q).view(c.rows, -1)
    out, lse = dfl.attention_kv8(x, h, table, gpu(c.row_start), lens, 16, 1016, lse=True)
    dfl.kv8_check(h)
    compare(small, cache, f64(out).reshape(c.rows, 8, 128), f64(lse), x)


def test_serving_run(dfl):
    # a prompt in two chunks, then single tokens, then a rejected block written over: after each step the
    # attention equals the plain one over the plain cache
    g = np.random.default_rng(21)
    hq, hkv, hd, page = 8, 2, 128, 16
    plan = [[(130, 0), (40, 0)], [(70, 130), (1, 40)], [(1, 200), (1, 41)], [(16, 201), (16, 42)],
            [(16, 205), (16, 42)], [(1, 221), (1, 58)]]
    pages = R.Case([(260, 0), (100, 0)], hkv, hd, page)
    h = dfl.kv8_cache(pages.n_pages, hkv, hd, page)
    table, cache = gpu(pages.table), R.Cache(pages)
    for step in plan:
        c = R.Case(step, hkv, hd, page, q_heads=hq)
        c.table, c.n_pages = pages.table, pages.n_pages
        k, v = bf(g.standard_normal((c.rows, hkv, hd))), bf(g.standard_normal((c.rows, hkv, hd)))
        q = bf(g.standard_normal((c.rows, hq * hd)))
        start, lens = gpu(c.row_start), gpu(c.kv_len)
        dfl.kv8_write(h, k, v, table, start, lens)
        out, lse = dfl.attention_kv8(q, h, table, start, lens, int(c.n.max()), int(c.kv_len.max()), lse=True)
        cache.c = c
        for s in range(2):
            rows = slice(int(c.row_start[s]), int(c.row_start[s + 1]))
            cache.put_many(s, int(c.positions(s)[0]), f64(k)[rows], f64(v)[rows])
        compare(c, cache, f64(out).reshape(c.rows, hq, hd), f64(lse), q)
    np.testing.assert_array_equal(h.codes.cpu().numpy(), cache.codes)
    np.testing.assert_array_equal(h.exps.cpu().numpy()[:, :, :, 0], cache.exps[:, :, :, 0])
    dfl.kv8_check(h)


def test_captured_step_replays_with_other_lengths(dfl):
    # one graph of write + attention, replayed as the sequences grow, next to eager calls on another stream
    g = np.random.default_rng(22)
    hq, hkv, hd, page = 8, 2, 128, 16
    pages = R.Case([(300, 0), (300, 0)], hkv, hd, page)
    table = gpu(pages.table)
    h, h2 = dfl.kv8_cache(pages.n_pages, hkv, hd, page), dfl.kv8_cache(pages.n_pages, hkv, hd, page)
    start = gpu(np.array([0, 1, 2], np.int32))
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    k, v = bf(np.zeros((2, hkv, hd))), bf(np.zeros((2, hkv, hd)))
    q, out = bf(np.zeros((2, hq * hd))), bf(np.zeros((2, hq * hd)))
    lse = torch.zeros((2, hq), device="cuda")

    def step(cache, stream=None):
        dfl.kv8_write(cache, k, v, table, start, lens, stream=stream)
        return dfl.attention_kv8(q, cache, table, start, lens, 1, 300, out=out if cache is h else None,
                                 lse=lse if cache is h else True, stream=stream)

    step(h)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(h)
    for i in range(40):
        k.copy_(bf(g.standard_normal((2, hkv, hd))))
        v.copy_(bf(g.standard_normal((2, hkv, hd))))
        q.copy_(bf(g.standard_normal((2, hq * hd))))
        lens.copy_(torch.tensor([i + 1, 7 * i + 1], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        o2, l2 = step(h2, side)       # runs beside the replay, on its own cache
        torch.cuda.synchronize()
        if i % 13 == 0 or i == 39:
            assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert torch.equal(h.codes, h2.codes) and torch.equal(h.exps, h2.exps)
    dfl.kv8_check(h)
    dfl.kv8_check(h2)


@pytest.mark.parametrize("rows,seqs,heads,group,hd", [(1, 39, 8, 2, 64), (640, 1, 8, 4, 64), (16, 20, 16, 4, 128)])
def test_more_tiles_than_run_at_once(dfl, rows, seqs, heads, group, hd):
    # the tiles behind the last full round are shared by two CTAs each; sequences share their pages
    n = 4200
    c = R.Case([(rows, n - rows - s) for s in range(seqs)], heads, hd, 64, seed=23, q_heads=heads * group)
    c.table, c.n_pages = np.tile(np.arange(66, dtype=np.int32), (seqs, 1)), 66
    cache = R.Cache(c)
    cache.put_many(0, 0, c.vectors(n), c.vectors(n))
    q = c.g.standard_normal((c.rows, heads * group, hd))
    got, lse, x = attend(dfl, c, cache, q)
    for j in np.unique(np.linspace(0, c.rows - 1, 24).astype(int)):   # these rows, every head
        s = j // rows
        one = R.Case([(1, int(c.positions(s)[j - s * rows]))], heads, hd, 64, q_heads=heads * group)
        one.table, one.n_pages, cache.c = c.table, c.n_pages, one
        compare(one, cache, got[[j]], lse[[j]], x[[j]])
    assert np.isfinite(got).all() and np.isfinite(lse).all()


def test_no_length_given_and_bounds_too_large(dfl):
    # max_rows and max_len are bounds: far too large ones change nothing but the split
    c = R.Case([(7, 300), (1, 0)], 2, 64, 32, seed=24, q_heads=6)
    cache = filled(c)
    h, table, start, lens = on_gpu(dfl, c, cache)
    x = bf(c.g.standard_normal((c.rows, 6, 64))).view(c.rows, -1)
    for max_rows, max_len in ((7, 0), (8, 307), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 40, 2 ** 40)):
        for window in (0, 50, 2 ** 31 - 1):
            out, lse = dfl.attention_kv8(x, h, table, start, lens, max_rows, max_len, window=window, lse=True)
            dfl.kv8_check(h)
            compare(c, cache, f64(out).reshape(c.rows, 6, 64), f64(lse), x, window=window)


@pytest.mark.parametrize("hd,page,rows", [(128, 16, 1), (128, 16, 5), (64, 32, 40), (128, 64, 70)])
def test_pages_that_a_window_has_left(dfl, hd, page, rows):
    # no page id, or bytes that are no numbers, at every position that no row sees
    window, n = 77, 900
    c = R.Case([(rows, n - rows), (1, 30)], 2, hd, page, seed=25, q_heads=8)
    cache = R.Cache(c)
    cache.codes[:] = 0x7F                                   # NaN codes
    cache.exps[:] = 255
    first = n - rows - window + 1                           # the first position that a row sees
    k, v = c.vectors(n), c.vectors(n)
    cache.put_many(0, first, k[first:], v[first:])
    cache.put_many(1, 0, c.vectors(31), c.vectors(31))
    q = c.g.standard_normal((c.rows, 8, hd))
    whole = c.table.copy()
    c.table[0, :first // page] = -1
    got, lse, x = attend(dfl, c, cache, q, window=window)   # kv8_check: nothing was flagged
    c.table = whole
    cache.put_many(0, 0, k, v)
    compare(c, cache, got, lse, x, window=window)
    want, wlse, _ = attend(dfl, c, cache, q, window=window)
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(lse, wlse)


def test_check_waits_for_other_streams(dfl):
    c = R.Case([(4, 60)], 2, 64, 16, seed=26)
    c.table[0, 0] = c.n_pages
    h, table, start, lens = on_gpu(dfl, c, R.Cache(c))
    q = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # about 10 ms
        dfl.attention_kv8(q, h, table, start, lens, 4, 64, out=torch.empty_like(q))
    with pytest.raises(dfl.DfError):
        dfl.kv8_check(h)
    dfl.kv8_check(h)


@pytest.mark.parametrize("cluster", [3, 6, 12])
def test_splits_that_are_no_power_of_two(dfl, cluster):
    c = R.Case([(16, 900), (1, 3), (2, 4000), (40, 130)], 2, 128, 16, seed=27, q_heads=8)
    cache = filled(c)
    q = c.g.standard_normal((c.rows, 8, 128))
    for window in (0, 700):
        got, lse, x = attend(dfl, c, cache, q, window=window, cluster_ctas=cluster)
        compare(c, cache, got, lse, x, window=window)
