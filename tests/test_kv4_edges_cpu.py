"""Host-side checks of the 4-bit KV cache's calls (no GPU)."""

import pytest

import persistent_megakernel_02_b200 as mk
from persistent_megakernel_02_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def cache(**kw):
    fake = 1 << 20  # never dereferenced on the host
    return mk.MkKv4CacheStruct(**{**dict(pool=fake, status=fake, n_layers=2, n_pages=10, n_kv_heads=2, head_dim=64), **kw})


@pytest.mark.parametrize("bad", [dict(pool=None), dict(status=None), dict(status=2), dict(n_pages=0), dict(head_dim=32)])
def test_taking_the_status_refuses_a_bad_cache(bad):
    assert mk.lib().mk_kv4_take_status(cache(**bad), 1 << 20, None) in (1, 2)


@pytest.mark.parametrize("bits", [None, (1 << 20) + 2])
def test_taking_the_status_refuses_a_bad_place(bits):
    assert mk.lib().mk_kv4_take_status(cache(), bits, None) == 1
