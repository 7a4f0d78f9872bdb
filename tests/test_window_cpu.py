"""Host side of the windowed attention: the frame in which the kernel counts a row's visible tokens
(WindowRows in decode_common.cuh, restated here), the size of its workspace, and its refusals."""
import ctypes

import pytest

from test_abi_cpu import FAKE, host_only, mla  # noqa: F401  (fixtures)


def frame(L, window, sinks):
    """(span, frame token -> token, hidden range) of a row, as WindowRows forms them."""
    end = L if window > 0 else min(L, sinks)
    start = max(end - window, 0)
    if start <= sinks:
        return end, (lambda v: v), (0, 0)
    first = (sinks + 63) & ~63
    shift = max((start & ~63) - first, 0)
    return end - shift, (lambda v: v if v < first else v + shift), (sinks, start)


@pytest.mark.parametrize("sinks", [0, 1, 4, 63, 64, 65, 128, 300])
@pytest.mark.parametrize("window", [0, 1, 5, 63, 64, 65, 127, 200, 1000])
def test_frame_holds_each_visible_token_once(mla, window, sinks):  # noqa: F811
    for L in list(range(0, 200)) + [255, 256, 257, 511, 700, 1023, 1500]:
        span, real, (h0, h1) = frame(L, window, sinks)
        assert span <= mla.window_span(L, window, sinks) if L else span == 0
        tokens = [real(v) for v in range(span)]
        assert tokens == sorted(set(tokens)) and all(0 <= t < L for t in tokens)
        seen = [t for t in tokens if not h0 <= t < h1]
        assert seen == [t for t in range(L) if t < sinks or t >= L - window]
        for v in range(0, span, 64):   # a 64-token box is one run inside a page and holds a visible token
            box = tokens[v:v + 64]
            assert box == list(range(box[0], box[0] + len(box))) and box[0] % 64 == 0
            assert any(not h0 <= t < h1 for t in box)
        for v in range(0, span, 32):   # a thread's 32 tokens are one run
            assert real(v + 31) - real(v) == 31


def test_span_bounds_the_workspace(mla):  # noqa: F811
    assert mla.window_span(4096, 1000, 4) == 64 + 1000 + 63
    assert mla.window_span(500, 1000, 4) == 500
    assert mla.window_span(500, 0, 4) == 4 and mla.window_span(500, 0, 900) == 500
    assert mla.window_span(500, 0, 0) == 0
    big = 2 ** 31 - 1
    assert mla.window_span(big, big, big) == big
    for bad in ((0, 1, 1), (-5, 1, 1), (64, -1, 1), (64, 1, -1)):
        assert mla.window_span(*bad) == 0
    # the size for the full capacity also serves
    for cap, window, sinks in ((4096, 100, 4), (131072, 1024, 64), (64, 1, 0)):
        for batch in (1, 7, 128):
            assert mla.decode_workspace_size(batch, mla.window_span(cap, window, sinks)) <= \
                mla.decode_workspace_size(batch, cap)


def test_window_refusals(host_only):  # noqa: F811
    m, lib = host_only, host_only.lib
    f = ctypes.c_float
    d = m.contiguous_desc(8, 4096)
    need = m.decode_workspace_size(8, m.window_span(4096, 256, 4), 16)

    def decode(window=256, sinks=4, batch=8, scale=0.07, splits=16, ws=FAKE, nbytes=need, desc=d, q=FAKE, out=FAKE,
               lse=None, lens=FAKE, table=None):
        return lib.mla_decode_attn_window(q, FAKE, table, lens, desc, batch, window, sinks, f(scale), splits, ws,
                                          nbytes, out, lse, None)

    assert decode(window=-1) == 1 and decode(sinks=-1) == 1
    assert decode(nbytes=need - 16) == 3 and decode(ws=None) == 3
    assert decode(batch=9) == 1 and decode(batch=-1) == 1 and decode(batch=0) == 0
    assert decode(scale=0.0) == 1 and decode(scale=float("nan")) == 1 and decode(splits=-1) == 1
    assert decode(q=None) == 1 and decode(out=FAKE + 8) == 1 and decode(lse=FAKE + 4) == 1 and decode(lens=None) == 1
    assert decode(desc=m.CacheDesc(32, 128, 2, 8, 1024), table=FAKE) == 2
    assert decode(desc=m.paged_desc(8, 64, 512)) == 1      # pages without a block table
    assert decode(batch=16385, desc=m.contiguous_desc(16385, 64), nbytes=1 << 40) == 2
    assert lib.mla_decode_attn_window_fp8(FAKE, FAKE, None, None, FAKE, d, 8, 256, 4, f(0.07), 16, FAKE, need, FAKE,
                                          None, None) == 1
    assert lib.mla_decode_attn_window_fp8(FAKE, FAKE, FAKE, None, FAKE, m.contiguous_desc(8, 100), 8, 256, 4, f(0.07),
                                          16, FAKE, need, FAKE, None, None) == 1
    assert lib.mla_prefill_attn_window(FAKE, FAKE, None, None, FAKE, d, 40, 256, 4, f(0.07), 16, FAKE, 1 << 30, FAKE,
                                       None, None) == 1
    assert lib.mla_prefill_attn_window(FAKE, FAKE, None, FAKE, FAKE, d, 40, 256, -4, f(0.07), 16, FAKE, 1 << 30, FAKE,
                                       None, None) == 1
    assert lib.mla_prefill_attn_window(FAKE, FAKE, None, FAKE, FAKE, d, 0, 256, 4, f(0.07), 16, None, 0, FAKE, None,
                                       None) == 0
