"""Serving calls where they can go wrong: padded batches, equal and nearly equal scores, long runs. On the GPU,
against fp64; tolerances as in test_gpu_serving.py unless a test derives its own."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from block_sparse_long_tcgen05_b200 import msa
from test_gpu_serving import (_cache, _check_decode, _close_rotated, _deal, _filled, _fresh_step, _gen, _ints, _np, _randn, _step,
                              _wider)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ padded batches
@pytest.mark.parametrize("each,lengths", [(1, [0, 1, 17, 0]), (4, [0, 2, 4, 33, 1])])
def test_append_of_equal_counts_passes_over_rows_without_a_token(cuda_ok, each, lengths):
    """Rows of positions below 0 (empty sequences, sequences of fewer tokens than rows): neither read nor
    written, and no error."""
    gen = _gen(40 + each)
    B, ps, G, Hq, d, di = len(lengths), 16, 2, 8, 64, 32
    cache = _cache(gen, 12, ps, G, d, di)
    table, _ = _deal(gen, lengths, ps, 3, 12)
    x = {n: _randn(gen, B * each, h, w) for n, h, w in (("k", G, d), ("v", G, d), ("k_idx", G, di), ("q", Hq, d))}
    rows = [(r, b, p) for r, b, p in ref.new_rows(lengths, [each] * B) if p >= 0]
    live = [r for r, _, _ in rows]
    dead = [r for r in range(B * each) if r not in live]
    for t in x.values():
        t[dead] = float("nan")
    f, _ = msa.rope_frequencies(64)
    q_out = torch.full((B * each, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    msa.paged_append(cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), x["k"], x["v"], x["k_idx"], freqs=f,
                     rotate_index=False, q=x["q"], q_out=q_out)
    assert msa.msa_get_device_error() == 0
    pos = np.zeros(B * each, dtype=np.int64)
    for r, _, p in rows:
        pos[r] = p
    tab = table.cpu().numpy()
    got = _np(cache.k_pages)
    mine = torch.from_numpy(np.stack([got[tab[b, p // ps], p % ps] for _, b, p in rows]))
    _close_rotated(mine, x["k"][live], ref.rotate(_np(x["k"]), pos, _np(f))[live], torch.bfloat16, 1.0, "k")
    for _, b, p in rows:
        got[tab[b, p // ps], p % ps] = np.nan
    assert np.isnan(got).all()
    _close_rotated(q_out[live], x["q"][live], ref.rotate(_np(x["q"]), pos, _np(f))[live], torch.bfloat16, 1.0, "q")
    assert (q_out[dead] == 9.0).all()


@pytest.mark.parametrize("wide", [False, True])
def test_captured_step_of_a_padded_batch(cuda_ok, wide):
    """Append and decode captured at a padded batch size: no error on any replay, zeros and ids of -1 for the
    empty sequences, the others as eager calls on them give them; then a sequence takes an empty place."""
    gen = _gen(43)
    B, ps, G, Hq, d, di, k, max_pages = 5, 16, 2, 8, 64, 32, 4, 40
    cache = _cache(gen, B * max_pages, ps, G, d, di, poison=False)
    table = torch.randperm(B * max_pages, generator=gen, device="cuda").to(torch.int32).view(B, max_pages)
    if wide:
        table = _wider(table, ps)
    for t in (cache.k_pages, cache.v_pages):
        t.copy_(_randn(gen, *t.shape))
    cache.k_idx_pages.copy_(_ints(gen, *cache.k_idx_pages.shape))
    f, s = msa.rope_frequencies(64)
    seq = torch.tensor([600, 0, 17, 0, 1], dtype=torch.int32, device="cuda")
    x = _fresh_step(gen, B, G, Hq, d, di)
    out = {"q": torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda"),
           "q_idx": torch.zeros(B, G, di, dtype=torch.bfloat16, device="cuda"),
           "o": torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"),
           "ids": torch.empty(B, G, k, dtype=torch.int32, device="cuda")}
    ws = torch.empty(msa.paged_decode_workspace(cache, B, table.shape[1], Hq, k), dtype=torch.uint8, device="cuda")
    _step(cache, table, seq, x, f, s, k, None, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(cache, table, seq, x, f, s, k, None, out, ws)
    for lengths in ([600, 0, 17, 0, 1], [601, 0, 18, 0, 2], [0, 500, 0, 3, 0]):
        seq.copy_(torch.tensor(lengths, dtype=torch.int32))
        for n, t in _fresh_step(gen, B, G, Hq, d, di).items():
            x[n].copy_(t)
        out["o"].fill_(5.0)
        graph.replay()
        assert msa.msa_get_device_error() == 0, lengths
        for b, L in enumerate(lengths):
            if L == 0:
                assert (out["o"][b] == 0).all() and (out["ids"][b] == -1).all()
        _check_decode(cache, table, seq, out["q"][:, None], out["q_idx"][:, None], k, 128, None, out["o"][:, None],
                      out["ids"][:, None])


# ------------------------------------------------------------------------------------ in place
def test_queries_rotated_in_place(cuda_ok):
    """q_out = q where both have two bytes an element (fp16 becomes bf16 where it lies); fp32 queries into a
    bf16 view of themselves are refused."""
    gen = _gen(44)
    N, ps, G, Hq, d, di = 9, 16, 2, 8, 64, 32
    f, _ = msa.rope_frequencies(64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([N], dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        cache = _cache(gen, 1, ps, G, d, di)
        k, v, ki, q = (_randn(gen, N, h, w, dtype=dtype) for h, w in ((G, d), (G, d), (G, di), (Hq, d)))
        old = q.clone()
        run = lambda out: msa.paged_append(cache, table, seq, k, v, ki, freqs=f, rotate_index=False, q=q, q_out=out)  # noqa: B023,E731
        if dtype == torch.float32:
            with pytest.raises(msa.MsaError, match="in place"):
                run(q.view(torch.bfloat16)[:, :, :d])
            assert torch.equal(q, old)
            continue
        out = q.view(torch.bfloat16)
        run(out)
        msa.check_device_error()
        _close_rotated(out, old, ref.rotate(_np(old), np.arange(N), _np(f)), torch.bfloat16, 1.0, f"{dtype}")


# ------------------------------------------------------------------------------------ derivatives
def test_derivatives_that_would_be_dropped_are_refused(cuda_ok):
    """A tangent of any input (forward mode), and a gradient of the frequencies or the pages."""
    import torch.autograd.forward_ad as fw
    gen = _gen(45)
    cache, table, _, seq, q, qi = _filled(gen, [200, 100], 16, 2, 64, 32, 1, 8, 13)
    f, _ = msa.rope_frequencies(64)
    pos = torch.arange(2, device="cuda")
    k, v, ki = _randn(gen, 2, 2, 64), _randn(gen, 2, 2, 64), _randn(gen, 2, 2, 32)
    append = lambda **c: msa.paged_append(cache, table, seq, **{"k": k, "v": v, "k_idx": ki, "freqs": f, "rotate_index": False, **c})  # noqa: E731
    with fw.dual_level():
        dual = lambda t: fw.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: msa.rope(dual(k), pos, f), lambda: msa.rope((k, dual(v)), pos, f), lambda: msa.rope(k, pos, dual(f)),
                     lambda: append(k=dual(k)), lambda: append(q=dual(k)), lambda: append(freqs=dual(f)),
                     lambda: msa.paged_decode(cache, table, seq, dual(q), qi, 4),
                     lambda: msa.paged_decode(cache, table, seq, q, dual(qi), 4)):
            with pytest.raises(ValueError, match="tangent"):
                call()
        msa.rope(k, pos, f)   # nothing here carries one
        append()
        msa.paged_decode(cache, table, seq, q, qi, 4)
    learnt = f.clone().requires_grad_()
    for call in (lambda: msa.rope(k, pos, learnt), lambda: append(freqs=learnt)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    grown = msa.PagedCache(cache.k_pages.clone().requires_grad_(), cache.v_pages, cache.k_idx_pages)
    with pytest.raises(ValueError, match="gradient"):
        msa.paged_decode(grown, table, seq, q, qi, 4)
    with torch.no_grad():
        assert torch.equal(msa.paged_decode(grown, table, seq, q, qi, 4), msa.paged_decode(cache, table, seq, q, qi, 4))
    msa.check_device_error()


# ------------------------------------------------------------------------------------ refusals
def test_refusals_carry_the_librarys_status(cuda_ok):
    """A bad argument is MSA_ERR_INVALID_ARG (1), a valid shape that is not implemented MSA_ERR_UNSUPPORTED (2)."""
    gen = _gen(46)
    cache, table, _, seq, q, qi = _filled(gen, [200, 100], 16, 2, 64, 32, 1, 8, 13)
    run = lambda q=q, k=4, **more: msa.paged_decode(cache, table, seq, q, qi, k, **more)  # noqa: E731
    for call, status in ((lambda: run(scale=-1.0), 1), (lambda: run(scale=float("nan")), 1), (lambda: run(q=q[:, :, :7].contiguous()), 1),
                         (lambda: run(bk=48), 2), (lambda: run(k=33), 2),
                         (lambda: msa.paged_decode_workspace(cache, 2, 13, 7, 4), 1),
                         (lambda: msa.paged_decode_workspace(cache, 2, 0, 8, 4), 1),
                         (lambda: msa.paged_decode_workspace(cache, 2, 13, 8, 40), 2)):
        with pytest.raises(msa.MsaError) as e:
            call()
        assert e.value.status == status and len(str(e.value)) > len("MSA_ERR_INVALID_ARG: ")


# ------------------------------------------------------------------------------------ selections
def _poured(gen, lengths, ps, G, d, di, S, Hq, shared, keys, queries):
    """A cache that holds the sequences (shared: pages that all of them begin with), NaN in every other row;
    keys(n) gives n tokens' index keys, queries the index queries."""
    table, common = _deal(gen, lengths, ps, max(-(-L // ps) for L in lengths) + 1, sum(-(-L // ps) for L in lengths) + shared + 2, shared)
    cache = _cache(gen, sum(-(-L // ps) for L in lengths) + shared + 2, ps, G, d, di)
    for b, L in enumerate(lengths):
        first = shared if b else 0   # the shared pages with the first sequence
        n = L - first * ps
        if n <= 0:
            continue
        pages = table[b, first:-(-L // ps)].long()
        slots = (pages[:, None] * ps + torch.arange(ps, device="cuda")).flatten()[:n]
        for pool, new in ((cache.k_pages, _randn(gen, n, G, d)), (cache.v_pages, _randn(gen, n, G, d)), (cache.k_idx_pages, keys(n))):
            pool.view(-1, *pool.shape[2:])[slots] = new
    q = _randn(gen, len(lengths), S, Hq, d)
    return cache, table, common, torch.tensor(lengths, dtype=torch.int32, device="cuda"), q, queries


REAL = [
    # lengths, S, Hq, G, d, di, k, bk, ps, shared pages
    ([1500, 0, 700, 33], 1, 8, 2, 64, 32, 4, 32, 16, 0),
    ([9000, 2500], 2, 16, 4, 128, 128, 16, 128, 64, 0),
    ([40000], 1, 2, 1, 64, 64, 16, 32, 128, 0),                        # two chunks of Top-k
    ([2300, 2100, 2049] * 10, 1, 8, 4, 64, 128, 5, 128, 64, 32),       # the prefix scored once for 30 rows
    ([4200, 4097, 0, 5000] * 6, 8, 8, 2, 64, 128, 8, 64, 32, 128),     # for 192 rows
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lengths,S,Hq,G,d,di,k,bk,ps,shared", REAL)
def test_decode_of_real_index_inputs(cuda_ok, lengths, S, Hq, G, d, di, k, bk, ps, shared, wide):
    """Scores that are not exact: products of bf16 are exact in fp32 and a score is di of them added in some
    order, each addition off by at most 2^-23 of the terms' sum of absolutes, so a block's maximum is off by at
    most E = di 2^-23 max sum |q k|. Every chosen block's score reaches every other one's within the two E; the
    attention over the chosen blocks is held to fp64 as always."""
    gen = _gen(50 + k + bk)
    queries = _randn(gen, len(lengths), S, G, di)
    cache, table, common, seq, q, qi = _poured(gen, lengths, ps, G, d, di, S, Hq, shared, lambda n: _randn(gen, n, G, di), queries)
    full = table
    if wide:
        table = full = _wider(table, ps)
    if shared:
        table = table.clone()
        table[:, :shared] = -1
    ids = torch.full((len(lengths), S, G, k), -9, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, k, bk=bk, prefix_pages=common if shared else None, block_ids=ids)
    msa.check_device_error()
    tab, chosen, got, R = full.cpu().numpy(), ids.cpu().numpy(), _np(o), Hq // G
    qn, qin = _np(q), _np(qi)
    pools = [_np(t) for t in (cache.k_pages, cache.v_pages, cache.k_idx_pages)]
    for b, L in enumerate(lengths):
        pages = tab[b][:-(-L // ps)]
        kk, vv, ki = (t[pages].reshape(-1, G, t.shape[3])[:L] for t in pools)
        for s in range(S):
            p = L - S + s
            for g in range(G):
                row = chosen[b, s, g]
                if p < 0:
                    assert (row == -1).all() and (got[b, s] == 0).all()
                    continue
                local = p // bk
                take = row[row >= 0]
                assert len(take) == min(k, local + 1) and (np.diff(take) > 0).all() and take[-1] == local
                assert (row[len(take):] == -1).all()
                terms = ki[:local * bk, g] * qin[b, s, g]
                score = terms.sum(-1).reshape(local, bk).max(1)
                off = di * 2.0 ** -23 * np.abs(terms).sum(-1).reshape(local, bk).max(1)
                inside = np.zeros(local, dtype=bool)
                inside[take[:-1]] = True
                if inside.any() and not inside.all():
                    assert (score + off)[inside].min() >= (score - off)[~inside].max()
                tok = (take[:, None] * bk + np.arange(bk)).reshape(-1)
                tok = tok[tok <= p]
                z = qn[b, s, g * R:(g + 1) * R] @ kk[tok, g].T / np.sqrt(d)
                w = np.exp(z - z.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                want, weight = w @ vv[tok, g], w @ np.abs(vv[tok, g])
                err = np.abs(got[b, s, g * R:(g + 1) * R] - want)
                assert (err <= (2.0 ** -8 + 1e-4) * weight + 2.0 ** -8 * (np.abs(want) + 2.0 ** -8 * weight)).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("k", [2, 6, 7, 16, 32])
@pytest.mark.parametrize("length,low,high", [
    (2000, 0, 0), (5000, 0, 0), (40000, 0, 0), (2000, 0, 2), (5000, -3, 0), (40000, 0, 1), (40000, -1, 0), (70000, 0, 3)])
def test_decode_of_few_different_scores(cuda_ok, length, low, high, k, wide):
    """Blocks of 32 with scores from a few whole numbers, so that tens to thousands are equal: the lower blocks
    first, wherever the chunks of the Top-k begin."""
    gen = _gen(60 + k)
    G, di = 2, 32

    def keys(n):
        x = torch.zeros(n, G, di, dtype=torch.bfloat16, device="cuda")
        x[..., 0] = torch.randint(low, high + 1, (n // 32 + 1, G), generator=gen, device="cuda").repeat_interleave(32, 0)[:n].to(x.dtype)
        x[..., 0] += -0.0
        return x

    one = torch.zeros(1, 1, G, di, dtype=torch.bfloat16, device="cuda")
    one[..., 0] = 1.0
    cache, table, _, seq, q, qi = _poured(gen, [length], 128, G, 64, di, 1, 4, 0, keys, one)
    if wide:
        table = _wider(table, 128)
    ids = torch.empty(1, 1, G, k, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, k, bk=32, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, k, 32, None, o, ids)


@pytest.mark.parametrize("B,G,k,d", [(64, 8, 32, 64), (200, 4, 16, 128)])
def test_decode_behind_a_prefix_in_long_runs(cuda_ok, B, G, k, d):
    """More strips a CTA than one table holds (the first), and just fewer (the second), behind a prefix."""
    gen = _gen(70 + B)
    ps, di, shared = 64, 32, 80
    own = torch.randint(1, 300, (B,), generator=torch.Generator().manual_seed(5)).tolist()
    lengths = [shared * ps + n for n in own]
    cache, table, common, seq, q, qi = _poured(gen, lengths, ps, G, d, di, 1, G, shared, lambda n: _ints(gen, n, G, di),
                                               _ints(gen, B, 1, G, di))
    full = table.clone()
    table[:, :shared] = -1
    ids = torch.empty(B, 1, G, k, dtype=torch.int32, device="cuda")
    o = msa.paged_decode(cache, table, seq, q, qi, k, prefix_pages=common, block_ids=ids)
    msa.check_device_error()
    _check_decode(cache, table, seq, q, qi, k, 128, None, o, ids, full)
    assert torch.equal(o, msa.paged_decode(cache, table, seq, q, qi, k, prefix_pages=common))


# ------------------------------------------------------------------------------------ precision
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lengths,S,Hq,G,d,k,bk", [
    ([700, 3, 0, 129, 1], 1, 8, 2, 64, 4, 128), ([2500, 2, 1111], 4, 16, 1, 128, 5, 128), ([1300, 97], 1, 8, 8, 64, 8, 32),
    ([9000] * 12, 1, 64, 8, 128, 16, 128)])
def test_decode_outputs_are_off_by_their_own_rounding(cuda_ok, lengths, S, Hq, G, d, k, bk, wide):
    """Weights enter their product cut off to bf16 (8 bits: less than 2^-7 of each is left) and, for the rest and
    2^-20 of the weight, the bf16 number nearest to that: off by at most 2^-8 times 2^-7, and 2^-20, of each, in all
    (2^-15 + 2^-20) W (W: sum of weight * |v|); logits as in test_gpu_serving.py, 1e-4 W; then the output's own
    rounding, 2^-8 of the value. Weights in one bf16 number, off by up to 2^-8 each, do not pass."""
    gen = _gen(80 + k)
    ps, di = 16, 32
    cache, table, _, seq, q, qi = _poured(gen, lengths, ps, G, d, di, S, Hq, 0, lambda n: _ints(gen, n, G, di),
                                          _ints(gen, len(lengths), S, G, di))
    if wide:
        table = _wider(table, ps)
    o = msa.paged_decode(cache, table, seq, q, qi, k, bk=bk)
    msa.check_device_error()
    want, _, weight = ref.decode(_np(q), _np(qi), _np(cache.k_pages), _np(cache.v_pages), _np(cache.k_idx_pages),
                                 table.cpu().numpy(), seq.cpu().numpy(), k, bk)
    before = (2.0 ** -15 + 2.0 ** -20 + 1e-4) * weight
    err = np.abs(_np(o) - want)
    bad = ~(err <= before + 2.0 ** -8 * (np.abs(want) + before))
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, max err {err.max():.3e}"


@pytest.mark.parametrize("wide", [False, True])
def test_infinite_values_give_infinite_outputs(cuda_ok, wide):
    """A token's values of +inf or -inf, whatever its weight, 1 and powers of two among them: that infinity, as the
    formula has it; both signs in one place, or a NaN: NaN; the other elements as without them."""
    gen = _gen(90)
    lengths, ps, G, Hq, d, di, k = [1, 200, 700], 16, 2, 8, 64, 32, 8
    cache, table, _, seq, q, qi = _poured(gen, lengths, ps, G, d, di, 1, Hq, 0, lambda n: _ints(gen, n, G, di), _ints(gen, 3, 1, G, di))
    q *= 0.25
    if wide:
        table = _wider(table, ps)
    plain = msa.paged_decode(cache, table, seq, q, qi, k)
    want = plain.clone().view(3, G, Hq // G, d)
    inf = float("inf")
    for b, t, g, e, v, out in ((0, 0, 0, 3, inf, inf), (0, 0, 1, 63, -inf, -inf), (1, 0, 0, 0, inf, inf), (1, 199, 1, 17, -inf, -inf),
                               (2, 690, 0, 5, inf, inf), (2, 645, 1, 6, -inf, -inf), (1, 50, 0, 9, inf, inf), (1, 51, 0, 9, -inf, inf - inf),
                               (2, 699, 1, 40, inf - inf, inf - inf)):
        cache.v_pages[int(table[b, t // ps]), t % ps, g, e] = v
        want[b, g, :, e] = out
    got = msa.paged_decode(cache, table, seq, q, qi, k).view(3, G, Hq // G, d)
    msa.check_device_error()
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)
