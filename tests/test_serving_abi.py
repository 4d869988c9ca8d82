"""Refusals of the serving entry points (rotary positions, paged append, paged decode): checked on
the host before anything is enqueued, so without a GPU; and the frequency schemes."""
import ctypes
import math

import pytest
import torch

from block_sparse_long_tcgen05_b200 import build as msa_build
from block_sparse_long_tcgen05_b200 import msa

P = 1 << 12   # an aligned stand-in address: validation fails before it is used


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return msa.load_library()


def _with(struct, **changes):
    out = type(struct)()
    ctypes.pointer(out)[0] = struct
    for name, value in changes.items():
        setattr(out, name, value)
    return out


def _tensor(**changes):
    return _with(msa.MsaRopeTensor(P, P, 512, 64, 512, 64, 8, 64), **changes)


def _cache(**changes):
    return _with(msa.MsaPagedCache(P, P, P, 100, 16 * 2 * 64, 16 * 2 * 64, 16 * 2 * 32, 16, 2, 64, 32), **changes)


def test_rope_refusals(lib):
    good = msa.MsaRopeParams(0, 64, 0, 0, 1.0, 0, P, P)

    def call(p=good, t=None, count=1, n=4):
        t = _tensor() if t is None else t
        return lib.msa_rope(p, t, count, n, None)

    assert lib.msa_rope(None, _tensor(), 1, 4, None) == 1
    assert lib.msa_rope(good, None, 1, 4, None) == 1
    for changes, status in (({"dtype": 3}, 2), ({"rot": 0}, 1), ({"rot": 7}, 1), ({"rot": 66}, 1), ({"scale": math.inf}, 1),
                            ({"scale": math.nan}, 1), ({"freqs": None}, 1), ({"freqs": P + 4}, 1), ({"positions": None}, 1),
                            ({"positions": P + 2}, 1), ({"positions": P + 4, "positions_i64": 1}, 1)):
        assert call(p=_with(good, **changes)) == status, changes
        assert lib.msa_last_error_detail()
    for changes, status in (({"heads": 0}, 1), ({"heads": 2000}, 1), ({"dim": 65}, 2), ({"dim": 2048}, 2), ({"dim": 0}, 2),
                            ({"x": None}, 1), ({"y": None}, 1), ({"x": P + 1}, 1), ({"y_head_stride": 0}, 1), ({"y_token_stride": 0}, 1)):
        assert call(t=_tensor(**changes)) == status, changes
    assert call(count=0) == 1 and call(count=5) == 1 and call(n=-1) == 1 and call(n=1 << 26) == 1
    assert call(n=0) == 0   # nothing to do, nothing enqueued


def test_cache_refusals(lib):
    p = msa.MsaPagedDecodeParams(8, 3, 1, 128, 4, 10, 0, 0.0, 10, P, P, None)
    assert lib.msa_paged_decode_workspace(_cache(), p) > 0
    assert lib.msa_paged_decode_workspace(None, p) == 0 and lib.msa_paged_decode_workspace(_cache(), None) == 0
    for changes, status in (({"g": 0}, 1), ({"g": 65}, 1), ({"d": 96}, 2), ({"d_idx": 48}, 2), ({"page_size": 8}, 2),
                            ({"page_size": 24}, 2), ({"page_size": 2048}, 2), ({"num_pages": 0}, 1), ({"num_pages": 1 << 31}, 1),
                            ({"k": None}, 1), ({"v": P + 8}, 1), ({"k_page_stride": 16 * 2 * 64 - 8}, 1),
                            ({"v_page_stride": 16 * 2 * 64 + 4}, 1), ({"k_idx_page_stride": 0}, 1)):
        c = _cache(**changes)
        assert lib.msa_paged_decode(c, p, P, P, None, P, P, 1 << 40, None) == status, changes
        assert lib.msa_paged_decode_workspace(c, p) == 0, changes


def test_decode_refusals(lib):
    c = _cache()
    good = msa.MsaPagedDecodeParams(8, 3, 1, 128, 4, 10, 0, 0.0, 10, P, P, None)
    need = lib.msa_paged_decode_workspace(c, good)

    def call(p=good, q=P, qi=P, ids=None, o=P, ws=P, size=need):
        return lib.msa_paged_decode(c, p, q, qi, ids, o, ws, size, None)

    for changes, status in (({"hq": 0}, 1), ({"hq": 7}, 1), ({"hq": 34}, 2), ({"batch": 0}, 2), ({"batch": 4097}, 2), ({"n_new": 0}, 2),
                            ({"n_new": 9}, 2), ({"bk": 96}, 2), ({"k": 0}, 2), ({"k": 33}, 2), ({"scale": -1.0}, 1),
                            ({"scale": math.nan}, 1), ({"max_pages": 0}, 1), ({"max_pages": 1 << 22, "table_stride": 1 << 22}, 1),
                            ({"table_stride": 9}, 1), ({"page_table": None}, 1), ({"seqlens": None}, 1), ({"seqlens": P + 2}, 1),
                            ({"n_prefix_pages": -1, "prefix_pages": P}, 1), ({"n_prefix_pages": 11, "prefix_pages": P}, 1),
                            ({"n_prefix_pages": 3}, 1)):
        assert call(p=_with(good, **changes), size=1 << 40) == status, changes
    assert call(q=None) == 1 and call(qi=P + 2) == 1 and call(o=P + 8) == 1 and call(ids=P + 1) == 1 and call(ws=None) == 1
    assert call(size=need - 1) == 3


def test_append_refusals(lib):
    k = msa.MsaRopeTensor(P, None, 128, 64, 0, 0, 2, 64)
    ki = msa.MsaRopeTensor(P, None, 64, 32, 0, 0, 2, 32)
    good = msa.MsaPagedAppendParams(0, 3, 10, 0, 64, 32, 1.0, 10, P, P, None, P, P)

    def call(c=None, p=good, k_=k, v=k, i=ki, q=None, qi=None, n=3):
        return lib.msa_paged_append(c or _cache(), p, k_, v, i, q, qi, n, None)

    assert call(c=_cache(page_size=12)) == 2
    assert lib.msa_paged_append(None, good, k, k, ki, None, None, 3, None) == 1
    assert call(p=None) == 1 and call(k_=None) == 1 and call(v=None) == 1 and call(i=None) == 1
    for changes, status in (({"dtype": 9}, 2), ({"batch": 0}, 2), ({"max_pages": 0}, 1), ({"rot": 66}, 1), ({"rot": 3}, 1),
                            ({"idx_rot": 34}, 1), ({"scale": math.inf}, 1), ({"table_stride": 3}, 1), ({"page_table": None}, 1),
                            ({"seqlens": None}, 1), ({"cu_seqlens": P + 2}, 1), ({"freqs": P + 4}, 1)):
        assert call(p=_with(good, **changes)) == status, changes
    assert call(n=4) == 1                                   # not a multiple of the batch
    assert call(k_=_with(k, heads=3)) == 1 and call(i=_with(ki, dim=64)) == 1 and call(v=_with(k, x=None)) == 1
    assert call(q=_with(k, heads=8)) == 1                   # no destination
    assert call(q=_with(k, y=P, y_token_stride=128)) == 1   # one destination for both heads
    assert call(n=0) == 0


def test_results_in_place_only_where_they_replace_what_was_read(lib):
    """y == x with other strides, or of another element size: some results would fall on inputs not read yet."""
    good = msa.MsaRopeParams(0, 64, 0, 0, 1.0, 0, P, P)
    for changes in ({"y_token_stride": 1024}, {"y_head_stride": 128}, {"x_token_stride": 0}, {"x_head_stride": 0}):
        assert lib.msa_rope(good, _tensor(**changes), 1, 4, None) == 1, changes
        assert b"place" in lib.msa_last_error_detail()
    k = msa.MsaRopeTensor(P, None, 128, 64, 0, 0, 2, 64)
    ki = msa.MsaRopeTensor(P, None, 64, 32, 0, 0, 2, 32)
    c = _cache(k=2 * P, v=2 * P, k_idx=2 * P)
    for dtype, q, q_idx in ((2, _with(k, y=P, y_token_stride=128, y_head_stride=64), None),
                            (2, _with(k, y=P, y_token_stride=256, y_head_stride=128), None),
                            (2, None, _with(ki, y=P, y_token_stride=64, y_head_stride=32)),
                            (0, _with(k, y=P, y_token_stride=256, y_head_stride=64), None)):
        p = msa.MsaPagedAppendParams(dtype, 3, 10, 0, 64, 32, 1.0, 10, P, P, None, P, P)
        assert lib.msa_paged_append(c, p, k, k, ki, q, q_idx, 3, None) == 1
        assert b"place" in lib.msa_last_error_detail()


def test_a_pool_without_pages_is_refused(lib):
    pool = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16)  # noqa: E731
    for shape in ((0, 16, 2, 64), (4, 0, 2, 64), (4, 16, 0, 64)):
        with pytest.raises(ValueError, match="at least one"):
            msa.PagedCache(pool(*shape), pool(*shape), pool(*shape[:3], 32))
    with pytest.raises(ValueError, match="CUDA"):
        msa.PagedCache(pool(4, 16, 2, 64), pool(4, 16, 2, 64), pool(4, 16, 2, 32))


def test_frequency_schemes():
    """none: base^(-2i/rot). linear: all divided. ntk: the first pair unchanged, the last divided by the
    factor. yarn: fast pairs unchanged, slow ones divided, monotone between."""
    f, s = msa.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0 and f[0] == 1.0
    assert abs(float(f[31]) - 10000.0 ** (-62 / 64)) < 1e-18
    lin, _ = msa.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    assert torch.equal(lin, f / 8)
    ntk, _ = msa.rope_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(f[31] / ntk[31]) - 8.0) < 1e-9
    yarn, s = msa.rope_frequencies(64, scaling="yarn", factor=8.0, trained_length=4096, device="cpu")
    ratio = f / yarn
    assert ratio[0] == 1.0 and abs(float(ratio[31]) - 8.0) < 1e-12 and (ratio.diff() >= 0).all()
    assert abs(s - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    for bad in (dict(rot=0), dict(rot=5), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            msa.rope_frequencies(device="cpu", **bad)


@pytest.mark.parametrize("rot,base,trained,factor", [(128, 10000.0, 4096, 8.0), (64, 500000.0, 8192, 32.0), (32, 10000.0, 2048, 2.0)])
def test_yarn_pairs_between(rot, base, trained, factor):
    """The ramp's ends are the last pair of at least 32 turns in the trained length and the first of at most
    one; between them a pair's frequency goes from its own to the stretched one in equal steps."""
    own = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [trained * f / (2.0 * math.pi) for f in own]
    lo = max(i for i, t in enumerate(turns) if t >= 32.0)
    hi = min((i for i, t in enumerate(turns) if t <= 1.0), default=None)
    assert hi is not None and hi - lo > 2   # there are pairs between
    got, _ = msa.rope_frequencies(rot, base=base, scaling="yarn", factor=factor, trained_length=trained, device="cpu")
    for i, f in enumerate(own):
        part = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        assert abs(float(got[i]) / (f * (1.0 - part) + f / factor * part) - 1.0) < 1e-14, i
