"""The 4-bit KV cache on the host (no GPU): the plain definition the GPU tests compare
with, and argument checks that come before anything touches the GPU."""

import ctypes

import numpy as np
import pytest

import persistent_megakernel_02_b200 as mk
from persistent_megakernel_02_b200 import build, kv4
from tests import _kv4 as R


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("d", [64, 128])
def test_the_layout_uses_every_byte_once(d):
    kb, ks, km, vb, vs, vm = R.offsets(d)
    seen = sorted(set(kb.ravel()) | set(vb.ravel())
                  | {x + i for t in (ks, km, vs, vm) for x in t.ravel() for i in (0, 1)})
    assert seen == list(range(20 * d))
    assert mk.lib().mk_kv4_page_bytes(d) == 4 * 20 * d == kv4.page_bytes(d)


def test_quantisation_by_hand():
    x = np.zeros((1, 32))
    x[0, :3] = [-1.0, 6.5, 2.25]
    c, s, z = R.quantise(x)
    assert (s, z) == (0.5, -1.0)          # (6.5 + 1) / 15
    assert c[0, :4].tolist() == [0, 15, 6, 2]  # 6.5 -> 6 (even)
    assert R.quantised(x)[0, :4].tolist() == [-1.0, 6.5, 2.0, 0.0]
    rng = np.random.default_rng(1)
    y = rng.standard_normal((50, 64)) * 2.0 ** rng.integers(-10, 10, (50, 1))
    c, s, z = R.quantise(y)
    assert c.min() >= 0 and c.max() <= 15
    assert (np.abs(R.quantised(y) - y) <= np.repeat(s, 32, -1) / 2 * (1 + 1e-12)).all()


def test_page_bytes_refuses_other_head_sizes():
    for d in (0, 32, 96, 256, -64):
        assert mk.lib().mk_kv4_page_bytes(d) == 0
        with pytest.raises(mk.MkError, match="UNSUPPORTED"):
            kv4.page_bytes(d)


def _args(cache=(), batch=(), rows=()):
    fake = 1 << 20  # never dereferenced on the host
    c = dict(pool=fake, status=fake, n_layers=2, n_pages=10, n_kv_heads=2, head_dim=64)
    b = dict(block_table=fake, cu=fake, kv_lens=fake, n_seqs=2, max_pages=4, n_rows=3, max_new=2, max_len=200)
    r = dict(p=fake, row_stride=512, head_stride=64)
    c.update(cache), b.update(batch), r.update(rows)
    return mk.MkKv4CacheStruct(**c), mk.MkKv4Batch(**b), mk.MkKv4Rows(**r)


BAD_CACHE = [dict(pool=None), dict(pool=8), dict(status=None), dict(status=2), dict(n_layers=0), dict(n_pages=0),
             dict(n_kv_heads=0), dict(head_dim=32), dict(head_dim=96), dict(n_kv_heads=70000)]
BAD_BATCH = [dict(block_table=None), dict(cu=None), dict(kv_lens=None), dict(n_seqs=0), dict(max_pages=0),
             dict(n_rows=-1), dict(max_new=-1), dict(max_len=-1), dict(max_len=257), dict(n_seqs=70000)]
BAD_ROWS = [dict(p=None), dict(p=(1 << 20) + 8), dict(row_stride=4), dict(head_stride=4), dict(row_stride=-512)]


@pytest.mark.parametrize("cache,batch,rows", [(c, {}, {}) for c in BAD_CACHE] + [({}, b, {}) for b in BAD_BATCH]
                         + [({}, {}, r) for r in BAD_ROWS])
def test_calls_refuse_bad_arguments_before_the_gpu(cache, batch, rows):
    c, b, r = _args(cache, batch, rows)
    good = _args()[2]
    lib = mk.lib()
    refused = {mk.MkError(1, "").status, mk.MkError(2, "").status}
    assert lib.mk_kv4_append(c, 0, b, r, good, 0, None) in refused
    assert lib.mk_kv4_read(c, 0, b, r, good, 0, None) in refused
    assert lib.mk_kv4_attention(c, 0, b, r, good, 2, 0, 0.1, None, 0, None) in refused
    n = ctypes.c_int64()
    if not rows:
        assert lib.mk_kv4_attention_workspace(c, b, 2, 0, ctypes.byref(n)) in refused


def test_calls_refuse_bad_numbers():
    c, b, r = _args()
    lib = mk.lib()
    n = ctypes.c_int64()
    assert lib.mk_kv4_read(c, 0, b, r, r, 0, None) == 1  # one output for both
    for layer in (-1, 2):
        assert lib.mk_kv4_append(c, layer, b, r, r, 0, None) == 1
        assert lib.mk_kv4_attention(c, layer, b, r, r, 2, 0, 0.1, None, 0, None) == 1
    for dtype in (-1, 3):
        assert lib.mk_kv4_read(c, 0, b, r, r, dtype, None) == 1
        assert lib.mk_kv4_attention_workspace(c, b, 2, dtype, ctypes.byref(n)) == 1
    for heads, want in ((0, 1), (3, 1), (6, 2), (32, 2)):
        assert lib.mk_kv4_attention(c, 0, b, r, r, heads, 0, 0.1, None, 0, None) == want
    for scale in (float("nan"), float("inf"), 3e38):
        assert lib.mk_kv4_attention(c, 0, b, r, r, 2, 0, scale, None, 0, None) == 1
    overlap = _args(rows=dict(row_stride=64))[2]  # rows of two heads overlap
    assert lib.mk_kv4_read(c, 0, b, overlap, r, 0, None) == 1
    assert lib.mk_kv4_attention(c, 0, b, r, overlap, 2, 0, 0.1, None, 0, None) == 1
    assert lib.mk_kv4_attention_workspace(c, b, 2, 0, None) == 1
    for fn in (lib.mk_kv4_park, lib.mk_kv4_resume):
        assert fn(None, 0, 0, 1, c, 1 << 20, 4, None) == 1


def test_a_call_without_rows_is_done():
    c, b, _ = _args(batch=dict(n_rows=0, max_new=0))
    assert mk.lib().mk_kv4_append(c, 0, b, None, None, 0, None) == 0
    assert mk.lib().mk_kv4_attention(c, 0, b, None, None, 2, 0, 0.1, None, 0, None) == 0
