"""Host side of the accumulated attention weights: refusals and the workspace's size."""
import ctypes

from test_abi_cpu import FAKE, host_only, mla  # noqa: F401  (fixtures)


def test_workspace_follows_the_ranges(mla):  # noqa: F811
    size = mla.prefill_attn_weights_workspace_size
    assert size(0, 64, 1) == 0 and size(1, 0, 1) == 0 and size(1, 64, -1) == 0
    one = 2 * (256 * 4 + 16)
    assert size(1, 64, 0) == one and size(1, 256, 1) == one and size(1, 257, 1) == 2 * one
    assert size(3, 256, 2) == 6 * one
    most = size(16384, 2 ** 31 - 1, 16384)
    assert most % one == 0 and most <= 1024 * one and size(128, 8192, 16) == most


def test_weights_refusals(host_only):  # noqa: F811
    m, lib = host_only, host_only.lib
    f = ctypes.c_float
    d = m.contiguous_desc(8, 4096)

    def call(q=FAKE, cache=FAKE, table=None, lens=FAKE, desc=d, batch=8, scale=0.07, lse=FAKE, prev=None, decay=1.0,
             out=FAKE):
        return lib.mla_attn_weights(q, cache, table, lens, desc, batch, f(scale), lse, prev, f(decay), out, None)

    assert call(batch=0) == 0 and call(batch=-1) == 1 and call(batch=9) == 1
    for name in ("q", "cache", "lens", "lse", "out"):
        assert call(**{name: None}) == 1, name
    assert call(q=FAKE + 8) == 1 and call(cache=FAKE + 8) == 1 and call(lse=FAKE + 4) == 1
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1
    assert call(decay=-0.5) == 1 and call(decay=float("nan")) == 1 and call(decay=float("inf")) == 1
    assert call(desc=m.paged_desc(8, 64, 512)) == 1 and call(table=FAKE) == 1
    assert call(desc=m.CacheDesc(32, 128, 2, 8, 1024), table=FAKE) == 2
    assert call(desc=m.contiguous_desc(16385, 64), batch=16385) == 2
    assert call(desc=m.contiguous_desc(8, 1 << 28)) == 2     # 2^31 rows
    assert lib.mla_attn_weights_fp8(FAKE, FAKE, None, None, FAKE, d, 8, f(0.07), FAKE, None, f(1.0), FAKE, None) == 1

    need = m.prefill_attn_weights_workspace_size(8, 4096, 40)

    def chunk(q=FAKE, lens=FAKE, start=FAKE, q_len=FAKE, batch=8, n=40, lse=FAKE, ws=FAKE, nbytes=need, out=FAKE):
        return lib.mla_prefill_attn_weights(q, FAKE, None, lens, start, q_len, d, batch, n, f(0.07), lse, None, f(1.0),
                                            ws, nbytes, out, None)

    assert chunk(batch=0) == 0 and chunk(n=-1) == 1 and chunk(n=16385, nbytes=1 << 40) == 2
    for name in ("q", "lens", "start", "q_len", "lse", "out"):
        assert chunk(**{name: None}) == 1, name
    assert chunk(nbytes=need - 16) == 3 and chunk(ws=None) == 3 and chunk(ws=FAKE + 8) == 3
    assert chunk(n=0, start=None) == 1 and chunk(n=0, lens=None) == 1
