"""Rotary positions, the paged cache's append and decode over it, on the GPU against fp64.

Tolerances, from the arithmetic (a rounding is off by at most u = eps / 2 of the value):
  * rotation: c a - n b in fp32 from an angle off by at most 2^-25 half turns (pi 2^-25 < 1e-7 rad)
    and cos, sin off by 2 units of 2^-24: the pair's result is off by at most 4e-7 of its length,
    times scale; then one rounding to the result's type, u |y| (fp32's own is in the 4e-7).
  * attention: softmax weights are rounded to bf16 (2^-8 of each) before they weigh the values, their
    sum is not: off by 2^-8 W, W = sum of weight * |v|; logits in fp32 from bf16 products, at most 128
    terms of a few units each: off by less than 1e-4, another 1e-4 W; then the output's rounding, 2^-8 |o|.
Selections are exact: index inputs are small integers.
"""
import numpy as np
import pytest
import torch

import serving_reference as ref
from block_sparse_long_tcgen05_b200 import msa

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}


def _np(t):
    return t.detach().cpu().double().numpy()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def _ints(gen, *shape, a=4):
    return torch.randint(-a, a + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)


def _close_rotated(y, x, want, dtype, scale, what):
    """Every element within its rounding and 4e-7 of the longest pair of its head."""
    x = _np(x)
    length = abs(scale) * np.sqrt(2.0) * np.abs(x).max(axis=-1, keepdims=True)
    err = np.abs(_np(y) - want)
    bad = err > U[dtype] * np.abs(want) * (1 + 1e-6) + 4e-7 * length + (6e-8 if dtype == torch.float16 else 0.0)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, max err {err.max():.3e}"


# ------------------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,D,rot", [
    (1, 1, 2, 2), (1, 8, 128, 128), (7, 3, 64, 64), (33, 5, 128, 64), (20, 2, 96, 32), (13, 4, 64, 20),
    (5, 7, 118, 118), (9, 2, 30, 14), (300, 64, 128, 128), (17, 1, 256, 16),
])
def test_rope_matches_fp64(cuda_ok, dtype, interleaved, N, H, D, rot):
    gen = _gen(N * 1000 + D + rot)
    x = _randn(gen, N, H, D, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (N,), generator=gen, device="cuda")
    f, s = msa.rope_frequencies(rot, scaling="yarn", factor=4.0)
    for backward in (False, True):
        y = msa.rope(x, pos, f, interleaved=interleaved, scale=s, backward=backward)
        want = ref.rotate(_np(x), pos.cpu().numpy(), _np(f), interleaved, s, backward)
        _close_rotated(y, x, want, dtype, s, f"backward={backward}")


@pytest.mark.parametrize("positions", [
    [0, 1, -1, -100000, 2 ** 31 - 1, -2 ** 31, 123456789, 5], [0] * 8,
])
@pytest.mark.parametrize("int64", [False, True])
def test_rope_positions_far_and_negative(cuda_ok, positions, int64):
    """The turns stay exact: fp64's own product p * f is off by |p| 2^-53 of a radian, which at 2^31
    is 2.4e-7, added to the tolerance on the reference's account."""
    gen = _gen(3)
    x = _randn(gen, 8, 3, 64, dtype=torch.float32)
    pos = torch.tensor(positions, dtype=torch.int64 if int64 else torch.int32, device="cuda")
    f, s = msa.rope_frequencies(64)
    y = msa.rope(x, pos, f)
    want = ref.rotate(_np(x), positions, _np(f))
    err = np.abs(_np(y) - want)
    assert err.max() <= (4e-7 + 5e-7) * np.sqrt(2.0) * np.abs(_np(x)).max()


def test_rope_frequencies_outside_one_turn(cuda_ok):
    """Frequencies are taken modulo whole turns a position: negative ones and ones above 2 pi too."""
    gen = _gen(4)
    x = _randn(gen, 50, 2, 8, dtype=torch.float32)
    pos = torch.arange(50, device="cuda")
    f = torch.tensor([-1.0, 7.5, 0.0, 100.25], dtype=torch.float64, device="cuda")
    y = msa.rope(x, pos, f)
    err = np.abs(_np(y) - ref.rotate(_np(x), np.arange(50), _np(f)))
    assert err.max() <= 1e-6 * np.sqrt(2.0) * np.abs(_np(x)).max()


def test_rope_slices_in_place_and_several_tensors(cuda_ok):
    """Heads as slices of one projection, other head counts and dims in a call, odd offsets, in place;
    what lies between the slices stays."""
    gen = _gen(5)
    N = 37
    fused = _randn(gen, N, 64 * 8 + 64 * 2 + 32 * 2 + 3)
    before = fused.clone()
    q = fused[:, :512].unflatten(1, (8, 64))
    k = fused[:, 512:640].unflatten(1, (2, 64))
    ki = fused[:, 641:705].unflatten(1, (2, 32))      # an odd offset
    pos = torch.randint(0, 5000, (N,), generator=gen, device="cuda", dtype=torch.int32)
    f, _ = msa.rope_frequencies(32)
    want = [ref.rotate(_np(t), pos.cpu().numpy(), _np(f)) for t in (q, k, ki)]
    old = [t.clone() for t in (q, k, ki)]
    got = msa.rope((q, k, ki), pos, f, out=(q, k, ki))
    assert got[0] is q
    for t, x, w in zip((q, k, ki), old, want):
        _close_rotated(t, x, w, torch.bfloat16, 1.0, "slice")
    assert torch.equal(fused[:, 640], before[:, 640]) and torch.equal(fused[:, 705:], before[:, 705:])
    # heads before tokens, out of place
    x = _randn(gen, 4, N, 64).transpose(0, 1)
    y = torch.empty(4, N, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    msa.rope(x, pos, f, out=y)
    _close_rotated(y, x, ref.rotate(_np(x), pos.cpu().numpy(), _np(f)), torch.bfloat16, 1.0, "transposed")


def test_rope_gradient_against_differences(cuda_ok):
    """The map is linear, so <g, rope(x + h e) - rope(x)> / h for h = 1 is the gradient's element: both
    sides in fp32, 64 terms off by 1e-6 each."""
    gen = _gen(6)
    x, g = _randn(gen, 3, 2, 32, dtype=torch.float32), _randn(gen, 3, 2, 32, dtype=torch.float32)
    pos = torch.tensor([3, 70, 9999], device="cuda")
    for inter in (False, True):
        f, s = msa.rope_frequencies(24, scaling="yarn", factor=8.0)
        got = msa.rope(g, pos, f, interleaved=inter, scale=s, backward=True)
        base = msa.rope(x, pos, f, interleaved=inter, scale=s)
        for t, h, e in ((0, 0, 0), (1, 1, 5), (2, 0, 23), (2, 1, 31)):
            step = x.clone()
            step[t, h, e] += 1.0
            diff = (msa.rope(step, pos, f, interleaved=inter, scale=s).double() - base.double())
            assert abs(float((diff * g.double()).sum()) - float(got[t, h, e])) < 64e-6


def test_rope_of_no_tokens(cuda_ok):
    f, _ = msa.rope_frequencies(64)
    y = msa.rope(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), f)
    assert y.shape == (0, 4, 64)


# ------------------------------------------------------------------------------------ paged cache
def _cache(gen, pages, ps, G, d, di, poison=True, shared=False):
    """A pool; K and V alternate in one allocation if shared. Unwritten rows hold NaN."""
    if shared:
        kv = torch.empty(pages, 2, ps, G, d, dtype=torch.bfloat16, device="cuda")
        kp, vp = kv[:, 0], kv[:, 1]
    else:
        kp, vp = (torch.empty(pages, ps, G, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ip = torch.empty(pages, ps, G, di, dtype=torch.bfloat16, device="cuda")
    for t in (kp, vp, ip):
        t.fill_(float("nan") if poison else 0.0)
    return msa.PagedCache(kp, vp, ip)


def _deal(gen, lengths, ps, max_pages, pages, shared=0):
    """A page table [B, max_pages] dealt from a shuffled pool; unused entries are out of range."""
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    common = [order.pop() for _ in range(shared)]
    table = torch.full((len(lengths), max_pages), -7, dtype=torch.int32)
    for b, L in enumerate(lengths):
        for p in range(-(-L // ps)):
            table[b, p] = common[p] if p < shared else order.pop()
    return table.cuda(), torch.tensor(common, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("counts,before,ps,G,Hq,d,di,rot,irot,interleaved,shared", [
    ([1, 1, 1], [0, 15, 16], 16, 2, 8, 64, 32, 32, 32, True, False),
    ([5, 0, 40, 1], [3, 9, 30, 0], 32, 4, 16, 128, 64, 128, 64, False, True),
    ([0, 0, 17], [5, 0, 100], 64, 1, 3, 64, 128, 20, 14, False, False),
    ([2] * 300, [7] * 300, 16, 1, 1, 64, 32, 64, 32, True, False),
    ([1], [200], 256, 8, 64, 128, 128, 0, 0, False, False),
])
def test_append_matches_fp64(cuda_ok, dtype, counts, before, ps, G, Hq, d, di, rot, irot, interleaved, shared):
    gen = _gen(sum(counts) + ps)
    lengths = [a + b for a, b in zip(before, counts)]
    pad = 3
    N = sum(counts) + pad
    max_pages = max(-(-L // ps) for L in lengths) + 1
    pages = sum(-(-L // ps) for L in lengths) + 2
    cache = _cache(gen, pages, ps, G, d, di, shared=shared)
    table, _ = _deal(gen, lengths, ps, max_pages, pages)
    x = {n: _randn(gen, N, h, w, dtype=dtype) for n, h, w in
         (("k", G, d), ("v", G, d), ("k_idx", G, di), ("q", Hq, d), ("q_idx", G, di))}
    f = msa.rope_frequencies(rot)[0] if rot else None
    fi = msa.rope_frequencies(irot, base=500.0)[0] if irot else None
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    q_out = torch.full((N, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    qi_out = torch.full((N, G, di), 9.0, dtype=torch.bfloat16, device="cuda")
    msa.paged_append(cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), **{n: x[n] for n in ("k", "v", "k_idx")},
                     cu_seqlens=cu, freqs=f, idx_freqs=fi, rotate_index=False, interleaved=interleaved, rope_scale=1.25,
                     q=x["q"], q_idx=x["q_idx"], q_out=q_out, q_idx_out=qi_out)
    msa.check_device_error()
    rows = ref.new_rows(lengths, counts)
    pos = np.zeros(N, dtype=np.int64)
    for r, _, p in rows:
        pos[r] = p
    live = [r for r, _, _ in rows]
    turned = {n: (ref.rotate(_np(t), pos, _np(w), interleaved, 1.25) if w is not None else _np(t))
              for n, t, w in (("k", x["k"], f), ("k_idx", x["k_idx"], fi), ("q", x["q"], f), ("q_idx", x["q_idx"], fi))}
    turned["v"] = _np(x["v"])
    tab = table.cpu().numpy()
    for name, pool in (("k", cache.k_pages), ("v", cache.v_pages), ("k_idx", cache.k_idx_pages)):
        got = _np(pool)
        at = [(tab[b, p // ps], p % ps) for _, b, p in rows]
        mine = torch.from_numpy(np.stack([got[i, j] for i, j in at]))
        _close_rotated(mine, x[name][live], turned[name][live], torch.bfloat16, 1.25, name)
        for i, j in at:
            got[i, j] = np.nan
        assert np.isnan(got).all(), f"{name}: rows of other tokens were written"
    for name, out in (("q", q_out), ("q_idx", qi_out)):
        _close_rotated(out[live], x[name][live], turned[name][live], torch.bfloat16, 1.25, name)
        assert (out[N - pad:] == 9.0).all()   # rows behind the last sequence


def test_append_uniform_counts_and_queries_left_out(cuda_ok):
    gen = _gen(8)
    B, S, ps, G, d, di = 5, 3, 16, 2, 64, 32
    cache = _cache(gen, 20, ps, G, d, di)
    lengths = [3, 4, 16, 17, 40]
    table, _ = _deal(gen, lengths, ps, 3, 20)
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k, v, ki = _randn(gen, B * S, G, d), _randn(gen, B * S, G, d), _randn(gen, B * S, G, di)
    assert msa.paged_append(cache, table, seq, k, v, ki) == (None, None)
    tab = table.cpu().numpy()
    for r, b, p in ref.new_rows(lengths, [S] * B):
        assert torch.equal(cache.k_pages[int(tab[b, p // ps]), p % ps], k[r])
        assert torch.equal(cache.k_idx_pages[int(tab[b, p // ps]), p % ps], ki[r])


def test_append_reports_bad_pages_and_lengths(cuda_ok):
    """A page outside the cache and a length above the table's: recorded, left out, the rest written."""
    gen = _gen(9)
    for bad_page, bad_len in ((10 ** 6, 0), (-1, 0), (None, 1000), (None, -5)):
        cache = _cache(gen, 4, 16, 1, 64, 32)
        table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
        seq = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
        if bad_page is not None:
            table[1, 1] = bad_page
        else:
            seq[1] = bad_len
        k, v, ki = _randn(gen, 2, 1, 64), _randn(gen, 2, 1, 64), _randn(gen, 2, 1, 32)
        msa.paged_append(cache, table, seq, k, v, ki)
        assert msa.msa_get_device_error() == 6
        assert msa.msa_get_device_error() == 0
        assert torch.equal(cache.k_pages[1, 3], k[0])
        rest = cache.k_pages.clone()
        rest[1, 3] = float("nan")
        assert rest.isnan().all()


# ------------------------------------------------------------------------------------ decode
def _filled(gen, lengths, ps, G, d, di, S, Hq, max_pages, shared=0, spare=2, hot=True):
    """A cache holding the sequences, NaN in every row that belongs to none."""
    pages = sum(-(-L // ps) for L in lengths) + shared + spare
    cache = _cache(gen, pages, ps, G, d, di)
    table, common = _deal(gen, lengths, ps, max_pages, pages, shared)
    tab = table.cpu().numpy()
    hot_dir = torch.randint(-2, 3, (G, di), generator=gen, device="cuda").to(torch.bfloat16)
    for b, L in enumerate(lengths):
        for p in range(-(-L // ps)):
            n = min(ps, L - p * ps)
            pg = int(tab[b, p])
            fresh = _ints(gen, n, G, di)
            if hot and p % 7 == 3:
                fresh = fresh + hot_dir
            cache.k_pages[pg, :n] = _randn(gen, n, G, d)
            cache.v_pages[pg, :n] = _randn(gen, n, G, d)
            cache.k_idx_pages[pg, :n] = fresh
    B = len(lengths)
    q, qi = _randn(gen, B, S, Hq, d), _ints(gen, B, S, G, di)
    return cache, table, common, torch.tensor(lengths, dtype=torch.int32, device="cuda"), q, qi


def _check_decode(cache, table, seq, q, qi, k, bk, scale, o, ids, full_table=None):
    tab = (table if full_table is None else full_table).cpu().numpy()
    want, want_ids, weight = ref.decode(_np(q), _np(qi), _np(cache.k_pages), _np(cache.v_pages), _np(cache.k_idx_pages),
                                        tab, seq.cpu().numpy(), k, bk, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    err = np.abs(_np(o) - want)
    bad = ~(err <= (2.0 ** -8 + 1e-4) * weight + 2.0 ** -8 * (np.abs(want) + 2.0 ** -8 * weight))
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, max err {err.max():.3e}"


DECODE = [
    # lengths, S, Hq, G, d, di, k, bk, ps
    ([1], 1, 8, 2, 64, 32, 4, 128, 16),
    ([700, 0, 129, 128, 127, 1], 1, 8, 2, 64, 32, 4, 128, 16),
    ([2500, 3, 0, 1111], 1, 16, 1, 128, 128, 5, 128, 64),          # R = 16
    ([1300, 96, 33, 32, 31, 0], 1, 8, 8, 64, 64, 8, 32, 128),       # R = 1, blocks smaller than pages
    ([1900, 640, 65, 64], 1, 12, 3, 128, 32, 13, 64, 32),           # three groups, odd k
    ([3000, 2177], 1, 64, 8, 128, 128, 16, 128, 256),
    ([900, 400], 1, 5, 1, 64, 64, 1, 64, 16),                       # R = 5; the local block alone
    ([4100, 200], 1, 2, 2, 64, 32, 32, 64, 1024),
    ([5, 2, 0, 260, 129, 1025], 4, 8, 2, 64, 32, 4, 128, 16),       # several new tokens; fewer tokens than that
    ([1537, 513, 7], 8, 16, 4, 128, 64, 8, 32, 64),
    ([1290, 3], 2, 64, 8, 128, 128, 4, 128, 32),
    ([40000], 1, 4, 1, 64, 32, 16, 32, 64),                         # 1250 blocks: two chunks of Top-k
]


def _wider(table, ps):
    """The same table with room for 20000 tokens: calls of that capacity take the kernels for long sequences."""
    wide = torch.full((table.shape[0], max(table.shape[1], 20000 // ps + 1)), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lengths,S,Hq,G,d,di,k,bk,ps", DECODE)
def test_decode_matches_fp64(cuda_ok, lengths, S, Hq, G, d, di, k, bk, ps, wide):
    gen = _gen(sum(lengths) + k)
    max_pages = -(-max(lengths) // ps) + 2
    cache, table, _, seq, q, qi = _filled(gen, lengths, ps, G, d, di, S, Hq, max_pages)
    if wide:
        table = _wider(table, ps)
    ids = torch.full((len(lengths), S, G, k), -9, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, k, bk=bk, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, k, bk, None, o, ids)
    again = msa.paged_decode(cache, table, seq, q, qi, k, bk=bk)
    assert torch.equal(o, again)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("shared,own,S,Hq,G,d,di,k,bk,ps", [
    (8, [700, 1, 0, 130], 1, 8, 2, 64, 32, 4, 128, 16),      # a prefix of one block
    (5, [300, 20, 900], 1, 16, 4, 128, 64, 5, 128, 16),      # shorter than a block
    (13, [300, 20, 0], 2, 16, 4, 128, 64, 4, 32, 16),        # ends inside a tile of 128 tokens
    (21, [1, 64, 511, 4], 1, 64, 8, 128, 128, 16, 128, 64),  # ends inside a block
    (9, [40, 1000], 4, 12, 3, 128, 32, 8, 64, 128),
    (3, [100] * 70, 2, 4, 2, 64, 64, 4, 32, 256),            # 140 rows: two row tiles
    (40, [17] * 150, 2, 1, 1, 64, 128, 8, 32, 32),           # 300 rows: three
    (24, [300, 20, 900], 2, 16, 1, 128, 128, 5, 64, 16),     # R = 16
    (30, [9, 8, 7, 100], 1, 10, 2, 64, 64, 13, 32, 32),      # R = 5
    (12, [260] * 9, 4, 9, 1, 64, 32, 6, 128, 64),            # R = 9, 36 rows
    # prefixes worth a scan of their own (16 MB of keys spared)
    (21, [1, 64, 511, 4] * 10, 1, 4, 2, 64, 128, 5, 128, 64),        # ends inside a block; one row tile
    (5, [100, 0, -1270] * 24, 2, 4, 2, 64, 64, 4, 32, 256),          # 144 rows: two row tiles; sequences that end inside
    (70, [33, 1, 200] * 30, 1, 12, 3, 128, 32, 8, 32, 16),           # 35 blocks: the last tile of 128 tokens is not full
    (2, [5, 900] * 15, 1, 8, 4, 128, 128, 3, 128, 1024),             # pages of more than a tile
    (3, [9, 40] * 300, 1, 64, 64, 64, 32, 2, 32, 32),                # 192 pairs of row tiles and groups: more than SMs
    (17, [-200, -1, 0, -272, 33], 1, 8, 2, 64, 32, 4, 32, 16),   # sequences that end inside the prefix, or are empty
])
def test_decode_behind_a_shared_prefix(cuda_ok, shared, own, S, Hq, G, d, di, k, bk, ps, wide):
    gen = _gen(shared * 31 + k)
    lengths = [max(0, shared * ps + n) for n in own]
    max_pages = -(-max(lengths) // ps) + 1
    cache, table, common, seq, q, qi = _filled(gen, lengths, ps, G, d, di, S, Hq, max_pages, shared=shared)
    if wide:
        table = _wider(table, ps)
    full = table.clone()
    table[:, :shared] = -1   # the prefix's columns are not read
    ids = torch.full((len(lengths), S, G, k), -9, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, k, bk=bk, prefix_pages=common, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, k, bk, None, o, ids, full)
    assert torch.equal(o, msa.paged_decode(cache, table, seq, q, qi, k, bk=bk, prefix_pages=common))
    # the same pages through the table alone: the same selection; weights are rounded to bf16 against
    # other maxima (a slot's, not the running one), so the outputs agree with fp64 and not in every bit
    plain_ids = torch.empty_like(ids)
    plain = msa.paged_decode(cache, full, seq, q, qi, k, bk=bk, block_ids=plain_ids)
    assert torch.equal(ids, plain_ids)
    _check_decode(cache, full, seq, q, qi, k, bk, None, plain, plain_ids)


def test_decode_scale_single_token_form_and_strided_pages(cuda_ok):
    gen = _gen(12)
    lengths, ps, G, d, di, Hq, k = [600, 90], 16, 2, 64, 32, 8, 4
    cache, table, _, seq, q, qi = _filled(gen, lengths, ps, G, d, di, 1, Hq, 40)
    kv = torch.full((cache.num_pages, 2, ps, G, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kv[:, 0], kv[:, 1] = cache.k_pages, cache.v_pages
    wide = torch.zeros(cache.num_pages, 3, ps, G, di, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = cache.k_idx_pages
    other = msa.PagedCache(kv[:, 0], kv[:, 1], wide[:, 1])
    wide_table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    wide_table[:, :40] = table
    ids = torch.empty(2, G, k, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(other, wide_table[:, :40], seq, q[:, 0].contiguous(), qi[:, 0].contiguous(), k, scale=0.5, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, k, 128, 0.5, o[:, None], ids[:, None])


@pytest.mark.parametrize("wide", [False, True])
def test_decode_selects_the_lower_of_equal_blocks(cuda_ok, wide):
    """All index keys alike: the first k - 1 blocks and the local one; -0 and +0 are equal."""
    gen = _gen(13)
    cache, table, _, seq, q, qi = _filled(gen, [2000], 16, 2, 64, 32, 1, 4, 130, hot=False)
    if wide:
        table = _wider(table, 16)
    cache.k_idx_pages.zero_()
    cache.k_idx_pages[::2] = -0.0
    ids = torch.empty(1, 1, 2, 5, dtype=torch.int32, device="cuda")
    msa.paged_decode(cache, table, seq, q, qi, 5, bk=32, block_ids=ids)
    assert ids.flatten(0, 2).tolist() == [[0, 1, 2, 3, 62]] * 2


def test_decode_of_thousands_of_short_sequences(cuda_ok):
    gen = _gen(19)
    lengths = [int(x) for x in torch.randint(0, 300, (2100,), generator=torch.Generator().manual_seed(3))]
    cache, table, _, seq, q, qi = _filled(gen, lengths, 64, 1, 64, 32, 1, 2, 5)
    ids = torch.empty(2100, 1, 1, 4, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, 4, bk=32, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, 4, 32, None, o, ids)


@pytest.mark.parametrize("wide", [False, True])
def test_pages_beyond_2_31_elements(cuda_ok, wide):
    """A pool of 2^31 elements and more: append to and decode from its last pages gives what a small pool
    gives, bit for bit."""
    gen = _gen(20)
    ps, G, d, di, k = 128, 8, 128, 128, 4
    pages = (1 << 31) // (ps * G * d) + 16
    far, near = (msa.PagedCache(*(torch.empty(n, ps, G, w, dtype=torch.bfloat16, device="cuda") for w in (d, d, di)))
                 for n in (pages, 16))
    lengths = [900, 300, 500]
    B, seq = 3, torch.tensor([900, 300, 500], dtype=torch.int32, device="cuda")
    table, common = _deal(gen, lengths, ps, 9, 16, shared=1)
    if wide:
        table = _wider(table, ps)
    cu = torch.tensor([0, 900, 1200, 1700], dtype=torch.int32, device="cuda")
    f, s = msa.rope_frequencies(128)
    new = [_randn(gen, 1700, G, d), _randn(gen, 1700, G, d), _ints(gen, 1700, G, di)]
    q, qi = _randn(gen, B, 16, d), _ints(gen, B, G, di)
    out = []
    for cache, shift in ((far, pages - 16), (near, 0)):
        at = torch.where(table >= 0, table + shift, table).to(torch.int32)
        # the first page is every sequence's: the last writer's keys would depend on the order, so one writes
        msa.paged_append(cache, at[:1].contiguous(), seq[:1], *(x[:900] for x in new), freqs=f, rotate_index=False)
        for b in (1, 2):
            at_b = at[b:b + 1].clone()
            lo = int(cu[b])
            at_b[0, 0] = int(at_b[0, 1])   # its first page's tokens go where its second's come after them
            msa.paged_append(cache, at_b, torch.tensor([128], dtype=torch.int32, device="cuda"), *(x[lo:lo + 128] for x in new),
                             freqs=f, rotate_index=False)
            msa.paged_append(cache, at[b:b + 1].contiguous(), seq[b:b + 1], *(x[lo + 128:lo + lengths[b]] for x in new), freqs=f,
                             rotate_index=False)
        ids = torch.empty(B, G, k, dtype=torch.int32, device="cuda")
        o = msa.paged_decode(cache, at, seq, q, qi, k, prefix_pages=(common + shift).to(torch.int32), block_ids=ids)
        msa.check_device_error()
        out.append((o, ids))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert out[0][0].isfinite().all()


def test_decode_matches_the_contiguous_forward(cuda_ok):
    """The same cache through msa.decode: equal selections, outputs within both's tolerance."""
    gen = _gen(14)
    lengths, G, d, di, Hq, k, ps = [1, 300, 1500, 2048], 2, 128, 64, 16, 8, 64
    cache, table, _, seq, q, qi = _filled(gen, lengths, ps, G, d, di, 1, Hq, 32)
    flat = {}
    for name, pool in (("k", cache.k_pages), ("v", cache.v_pages), ("ki", cache.k_idx_pages)):
        flat[name] = pool[table.long().clamp(min=0)].flatten(1, 2).nan_to_num(0.0).contiguous()
    a, b = (torch.empty(4, G, k, dtype=torch.int32, device="cuda") for _ in range(2))
    want = msa.decode(q[:, 0].contiguous(), flat["k"], flat["v"], qi[:, 0].contiguous(), flat["ki"], seq, k, block_ids=a)
    got = msa.paged_decode(cache, table, seq, q[:, 0].contiguous(), qi[:, 0].contiguous(), k, block_ids=b)
    msa.check_device_error()
    assert torch.equal(a, b)
    assert (want.float() - got.float()).abs().max() <= 2e-2


@pytest.mark.parametrize("wide", [False, True])
def test_decode_reports_bad_pages_and_lengths(cuda_ok, wide):
    gen = _gen(15)
    lengths = [1000, 1000, 1000]
    cache, table, common, seq, q, qi = _filled(gen, lengths, 16, 2, 64, 32, 1, 8, 64, shared=16)
    if wide:
        table = _wider(table, 16)
    good = msa.paged_decode(cache, table, seq, q, qi, 4, bk=32)
    msa.check_device_error()
    for what in ("page", "long", "negative", "prefix"):
        t, n, pre = table.clone(), seq.clone(), None
        if what == "page":
            t[1, :60] = cache.num_pages
        elif what == "long":
            n[1] = table.shape[1] * 16 + 1
        elif what == "negative":
            n[1] = -3
        else:
            pre = common.clone()
            pre[5] = -1
        o = msa.paged_decode(cache, t, n, q, qi, 4, bk=32, prefix_pages=pre)
        assert msa.msa_get_device_error() == 6, what
        if what != "prefix":
            assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])


def test_decode_reports_bad_pages_of_a_scanned_prefix(cuda_ok):
    gen = _gen(21)
    lengths = [2100] * 30
    cache, table, common, seq, q, qi = _filled(gen, lengths, 64, 4, 64, 128, 1, 8, 34, shared=32)
    table = _wider(table, 64)
    good = msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=common)
    msa.check_device_error()
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        pre = common.clone()
        pre[7] = bad
        msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=pre)
        assert msa.msa_get_device_error() == 6
    assert torch.equal(good, msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=common))
    msa.check_device_error()


def test_prefix_scan_waits_end(cuda_ok):
    """The prefix scan's gating waits are bounded: with a limit that every wait exceeds, the call ends
    with a timeout status and the next one, at the default, is right again."""
    gen = _gen(22)
    cache, table, common, seq, q, qi = _filled(gen, [2100] * 30, 64, 4, 64, 128, 1, 8, 34, shared=32)
    table = _wider(table, 64)
    good = msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=common)
    msa.check_device_error()
    msa.set_wait_limit_ns(1)
    try:
        msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=common)
        assert msa.msa_get_device_error() == 5
    finally:
        msa.set_wait_limit_ns(0)
    assert torch.equal(good, msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=common))
    msa.check_device_error()


# ------------------------------------------------------------------------------------ together
def _step(cache, table, seq, x, f, s, k, common, out, ws):
    q, qi = msa.paged_append(cache, table, seq, x["k"], x["v"], x["k_idx"], freqs=f, rope_scale=s, rotate_index=False,
                             q=x["q"], q_idx=x["q_idx"], q_out=out["q"], q_idx_out=out["q_idx"])
    return msa.paged_decode(cache, table, seq, q, qi, k, prefix_pages=common, o=out["o"], block_ids=out["ids"], workspace=ws)


def _fresh_step(gen, B, G, Hq, d, di):
    x = {n: _randn(gen, B, h, d) for n, h in (("k", G), ("v", G), ("q", Hq))}
    x.update({n: _ints(gen, B, G, di) for n in ("k_idx", "q_idx")})
    return x


@pytest.mark.parametrize("wide", [False, True])
def test_prompt_and_steps_as_a_server_makes_them(cuda_ok, wide):
    """Prompts appended in ragged chunks behind a shared prefix, then steps of one token: rotation,
    append and decode, each step checked against fp64 on the cache; then a captured step replayed on
    new tokens and lengths gives what the eager one does, bit for bit."""
    gen = _gen(16)
    B, ps, G, Hq, d, di, k, max_pages = 4, 16, 2, 8, 64, 32, 4, 48
    shared = 20
    f, s = msa.rope_frequencies(64, scaling="ntk", factor=4.0)
    cache = _cache(gen, 1 + shared + B * (max_pages - shared), ps, G, d, di)
    order = torch.randperm(cache.num_pages, generator=gen, device="cuda").to(torch.int32)
    common = order[:shared].contiguous()
    table = torch.cat([common.expand(B, shared), order[shared:shared + B * (max_pages - shared)].view(B, -1)], 1).contiguous()
    if wide:
        table = _wider(table, ps)
    # the prefix, once, as a sequence of its own
    P = shared * ps
    x = _fresh_step(gen, P, G, Hq, d, di)
    msa.paged_append(cache, common[None], torch.tensor([P], dtype=torch.int32, device="cuda"), x["k"], x["v"], x["k_idx"],
                     freqs=f, rope_scale=s, rotate_index=False)
    counts = [37, 0, 200, 5]
    lengths = [P + c for c in counts]
    x = _fresh_step(gen, sum(counts), G, Hq, d, di)
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    msa.paged_append(cache, table, seq, x["k"], x["v"], x["k_idx"], cu_seqlens=cu, freqs=f, rope_scale=s, rotate_index=False)
    out = {"q": torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"),
           "q_idx": torch.empty(B, G, di, dtype=torch.bfloat16, device="cuda"),
           "o": torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"),
           "ids": torch.empty(B, G, k, dtype=torch.int32, device="cuda")}
    ws = torch.empty(msa.paged_decode_workspace(cache, B, table.shape[1], Hq, k), dtype=torch.uint8, device="cuda")
    x = _fresh_step(gen, B, G, Hq, d, di)
    for _ in range(3):
        seq += 1
        for n, t in _fresh_step(gen, B, G, Hq, d, di).items():
            x[n].copy_(t)
        _step(cache, table, seq, x, f, s, k, common, out, ws)
        msa.check_device_error()
        _check_decode(cache, table, seq, out["q"][:, None], out["q_idx"][:, None], k, 128, None, out["o"][:, None],
                      out["ids"][:, None])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(cache, table, seq, x, f, s, k, common, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(cache, table, seq, x, f, s, k, common, out, ws)
    for step in (1, 90):
        seq += step
        if step > 1:   # tokens that were never appended: give the rows between something finite
            for t in (cache.k_pages, cache.v_pages, cache.k_idx_pages):
                t.nan_to_num_(0.0)
        for n, t in _fresh_step(gen, B, G, Hq, d, di).items():
            x[n].copy_(t)
        out["o"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        msa.check_device_error()
        got = {n: t.clone() for n, t in out.items()}
        _step(cache, table, seq, x, f, s, k, common, out, ws)
        msa.check_device_error()
        for n in out:
            assert torch.equal(got[n], out[n]), n
        _check_decode(cache, table, seq, out["q"][:, None], out["q_idx"][:, None], k, 128, None, out["o"][:, None],
                      out["ids"][:, None])


@pytest.mark.parametrize("wide", [False, True])
def test_calls_on_two_streams(cuda_ok, wide):
    """Two decodes at once, each with a workspace of its own, give what they give alone."""
    gen = _gen(17)
    a = list(_filled(gen, [3000, 500], 64, 2, 128, 64, 1, 16, 50))
    b = list(_filled(gen, [100, 2900, 1], 16, 2, 64, 32, 2, 8, 200, shared=10))
    if wide:
        a[1], b[1] = _wider(a[1], 64), _wider(b[1], 16)
    run = lambda c, pre: msa.paged_decode(c[0], c[1], c[3], c[4], c[5], 8, prefix_pages=c[2] if pre else None)  # noqa: E731
    want = run(a, False), run(b, False)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = run(a, False)
        with torch.cuda.stream(s2):
            y = run(b, False)
        got.append((x, y))
    torch.cuda.synchronize()
    msa.check_device_error()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


# ------------------------------------------------------------------------------------ refusals
def test_python_refusals(cuda_ok):
    gen = _gen(18)
    x = _randn(gen, 4, 2, 64)
    pos = torch.arange(4, device="cuda")
    f, _ = msa.rope_frequencies(64)
    for args in ((x.double(), pos, f), (x, pos.float(), f), (x, pos[:3], f), (x, pos, f.float()), (x.cpu(), pos, f),
                 ([x] * 5, pos, f), (x[0], pos, f), (x.transpose(1, 2), pos, f), (x, pos.cpu(), f)):
        with pytest.raises(ValueError):
            msa.rope(*args)
    with pytest.raises(ValueError):
        msa.rope(x, pos, f, out=torch.empty(4, 2, 62, dtype=x.dtype, device="cuda"))
    with pytest.raises(msa.MsaError):
        msa.rope(x, pos, msa.rope_frequencies(128)[0])           # more than the head has
    with pytest.raises(msa.MsaError):
        msa.rope(x, pos, f, scale=float("nan"))
    with pytest.raises(ValueError, match="gradient"):
        msa.rope(x.float().requires_grad_(), pos, f)
    with pytest.raises(ValueError):
        msa.rope_frequencies(7)
    with pytest.raises(ValueError):
        msa.rope_frequencies(8, scaling="other")
    cache, table, common, seq, q, qi = _filled(gen, [200, 100], 16, 2, 64, 32, 1, 8, 13)
    k, v, ki = _randn(gen, 2, 2, 64), _randn(gen, 2, 2, 64), _randn(gen, 2, 2, 32)
    with pytest.raises(msa.MsaError):
        msa.paged_append(cache, table, seq, k[:1], v[:1], ki[:1])      # one row for two sequences
    with pytest.raises(ValueError):
        msa.paged_append(cache, table.long(), seq, k, v, ki)
    with pytest.raises(ValueError):
        msa.paged_append(cache, table, seq, k, v.float(), ki)
    with pytest.raises(msa.MsaError):
        msa.paged_append(cache, table, seq, ki, v, ki)
    with pytest.raises(ValueError):
        msa.paged_decode(cache, table, seq, q, qi[:, :, :1], 4)
    with pytest.raises(ValueError):
        msa.paged_decode(cache, table, seq, q.transpose(2, 3).contiguous(), qi, 4)
    with pytest.raises(ValueError):
        msa.paged_decode(cache, table, seq.cpu(), q, qi, 4)
    with pytest.raises(msa.MsaError):
        msa.paged_decode(cache, table, seq, q, qi, 33)
    with pytest.raises(msa.MsaError):
        msa.paged_decode(cache, table, seq, q, qi, 4, bk=48)
    with pytest.raises(msa.MsaError):
        msa.paged_decode(cache, table, seq, q, qi, 4, prefix_pages=torch.zeros(14, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        msa.PagedCache(cache.k_pages, cache.v_pages[:1], cache.k_idx_pages)
    with pytest.raises(ValueError):
        msa.PagedCache(cache.k_pages.float(), cache.v_pages, cache.k_idx_pages)
    bad = torch.zeros(4, 24, 2, 64, dtype=torch.bfloat16, device="cuda")   # 24 tokens a page
    badi = torch.zeros(4, 24, 2, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(msa.MsaError):
        msa.paged_decode(msa.PagedCache(bad, bad, badi), table, seq, q, qi, 4)
