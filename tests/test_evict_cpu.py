"""Host side of the eviction and of the append at a slot: their refusals and the workspace's size."""
import types

import pytest
import torch

from test_abi_cpu import FAKE, host_only, mla  # noqa: F401  (fixtures)

FAR = 1 << 40


def test_evict_workspace(mla):  # noqa: F811
    assert mla.evict_workspace_size(0, 5) == 0 and mla.evict_workspace_size(5, 0) == 0
    for batch, keep in ((1, 1), (3, 7), (128, 1024), (16384, 100000)):
        got = mla.evict_workspace_size(batch, keep)
        assert 4 * batch * (keep + 1) <= got < 4 * batch * (keep + 1) + 16 and got % 16 == 0


def test_evict_refusals(host_only):  # noqa: F811
    m, lib = host_only, host_only.lib
    d = m.contiguous_desc(8, 4096)
    need = m.evict_workspace_size(8, 256)

    def call(cache=FAKE, table=None, lens=FAKE, weights=FAKE, desc=d, batch=8, keep=256, sinks=4, recent=32, out=FAR,
             table_out=None, desc_out=d, kept=FAKE, lens_out=FAKE, weights_out=FAKE, ws=FAKE, nbytes=need):
        return lib.mla_cache_evict(cache, table, lens, weights, desc, batch, keep, sinks, recent, out, table_out,
                                   desc_out, kept, lens_out, weights_out, ws, nbytes, None)

    assert call(batch=0) == 0 and call(batch=0, out=FAKE) == 0
    assert call(batch=-1) == 1 and call(batch=9) == 1
    assert call(keep=0) == 1 and call(sinks=-1) == 1 and call(recent=-1) == 1
    assert call(sinks=200, recent=57) == 1 and call(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == 1
    assert call(keep=2049, nbytes=1 << 40, desc_out=m.contiguous_desc(8, 2048)) == 1
    assert call(keep=9000, nbytes=1 << 40, desc_out=m.contiguous_desc(8, 4095)) == 1
    assert call(batch=0, keep=9000) == 0      # more than a sequence can hold: nothing is ever evicted
    assert call(batch=0, keep=1 << 30) == 0 and call(batch=0, keep=(1 << 30) + 1) == 2
    assert call(keep=2 ** 31 - 1, nbytes=1 << 62) == 2
    assert call(desc_out=m.contiguous_desc(7, 4096)) == 1
    for name in ("lens", "weights", "kept", "lens_out", "weights_out", "cache", "out"):
        assert call(**{name: None}) == 1, name
    assert call(ws=None) == 3 and call(nbytes=need - 1) == 3 and call(ws=FAKE + 8) == 3
    assert call(cache=FAKE + 8) == 1 and call(out=FAR + 4) == 1
    # buffers that meet without being one cache
    assert call(out=FAKE + 1152 * 64) == 1
    assert call(cache=FAKE + 1152 * 64, out=FAKE) == 1
    assert call(out=FAKE, desc_out=m.contiguous_desc(8, 2048)) == 1
    assert call(out=FAKE, desc_out=m.paged_desc(8, 64, 512), table_out=FAKE) == 1
    many = m.contiguous_desc(16385, 512)
    assert call(desc=many, desc_out=many, batch=16385, nbytes=1 << 40) == 2

    def call8(scales=FAKE, scales_out=FAR, cache=FAKE, out=FAR, batch=0):
        return lib.mla_cache_evict_fp8(cache, scales, None, FAKE, FAKE, d, batch, 256, 4, 32, out, scales_out, None, d,
                                       FAKE, FAKE, FAKE, FAKE, need, None)

    assert call8() == 0
    assert call8(scales=None) == 1 and call8(scales_out=None) == 1
    assert call8(out=FAKE) == 1                              # one buffer of codes, two of scales
    assert call8(scales_out=FAKE + 64) == 1


def test_append_at_refusals(host_only):  # noqa: F811
    m, lib = host_only, host_only.lib
    d = m.contiguous_desc(4, 128)
    assert lib.mla_cache_append_at(FAKE, FAKE, None, FAKE, None, FAKE, None, d, 4, 10000.0, None) == 1
    assert lib.mla_cache_append_at(FAKE, FAKE, None, FAKE, None, FAKE, None, d, 0, 10000.0, None) == 0
    assert lib.mla_cache_append_at(FAKE, FAKE, None, None, FAKE, FAKE, None, d, 4, 10000.0, None) == 1
    assert lib.mla_cache_append_at(FAKE, FAKE, None, FAKE, FAKE, FAKE, None, d, 5, 10000.0, None) == 1
    assert lib.mla_cache_append_at_fp8(FAKE, FAKE, None, FAKE, None, FAKE, FAKE, None, d, 4, 10000.0, None) == 1
    assert lib.mla_cache_append_at_fp8(FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, d, 4, 10000.0, None) == 1


@pytest.fixture
def passed(mla, monkeypatch):  # noqa: F811
    """Calls the binding with a library that only notes what it is given."""
    def call(fp8, **kw):
        got = {}

        def note(*args):
            names = ["cache", *(["scales"] if fp8 else []), "table", "lens", "weights", "desc", "batch", "keep", "sinks",
                     "recent", "out", *(["scales_out"] if fp8 else []), "table_out", "desc_out"]
            got.update(zip(names, args))
            return 0

        monkeypatch.setattr(mla, "lib", types.SimpleNamespace(mla_cache_evict=note, mla_cache_evict_fp8=note))
        lens, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
        args = (lens, FAKE, mla.paged_desc(3, 8, 24), FAKE, FAKE, FAKE, ws)
        kw = dict(keep=64, block_table=0x200, stream=0, **kw)
        if fp8:
            mla.cache_evict_fp8(0x100, 0x110, *args, **kw)
        else:
            mla.cache_evict(0x100, *args, **kw)
        return got

    return call


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_in_place_takes_what_is_given(mla, passed, fp8):  # noqa: F811
    got = passed(fp8)
    assert got["out"] == 0x100 and got["table_out"] == 0x200 and got["desc_out"].max_blocks_per_seq == 8
    assert not fp8 or got["scales_out"] == 0x110
    # the same pool, other pages
    got = passed(fp8, desc_out=mla.paged_desc(3, 2, 24), block_table_out=0x300)
    assert got["out"] == 0x100 and got["table_out"] == 0x300 and got["desc_out"].max_blocks_per_seq == 2
    got = passed(fp8, block_table_out=0x300)   # as wide as the old table
    assert got["table_out"] == 0x300 and got["desc_out"].max_blocks_per_seq == 8
    # a narrower descriptor does not fit the source's table: no table, which the library refuses
    assert passed(fp8, desc_out=mla.paged_desc(3, 2, 24))["table_out"] is None
    assert passed(fp8, desc_out=mla.paged_desc(3, 8, 24))["table_out"] == 0x200
    if fp8:   # (and the library refuses one buffer of codes with two of scales)
        assert passed(fp8, scales_out=0x120)["scales_out"] == 0x120


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_into_another_cache(mla, passed, fp8):  # noqa: F811
    kw = dict(scales_out=0x410) if fp8 else {}
    got = passed(fp8, cache_out=0x400, desc_out=mla.paged_desc(3, 2, 6), block_table_out=0x300, **kw)
    assert got["out"] == 0x400 and got["table_out"] == 0x300 and got["desc_out"].num_rows == 6 * 64
    assert passed(fp8, cache_out=0x400, desc_out=mla.contiguous_desc(3, 128), **kw)["table_out"] is None
