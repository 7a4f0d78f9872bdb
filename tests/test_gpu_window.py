"""Attention with a sliding window and sinks (mla_decode_attn_window, _fp8, mla_prefill_attn_window)
against its definition in 64 bits: a row of cached length L attends to t < sinks and t >= L - window."""
import numpy as np
import pytest
import torch

import oracle
from bounded_common import SCALE, RowCache, assert_window_row, f64, launches, random_q, random_rows

pytestmark = pytest.mark.gpu

LENS = [0, 1, 63, 64, 65, 128, 129, 330, 700, 1000]
MASKS = [(1, 0), (64, 0), (100, 4), (129, 64), (200, 65), (5, 128), (0, 4), (0, 0), (1 << 30, 3), (64, 1 << 30),
         (333, 300)]


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available()
    import mla_latent_kv_20_b200 as lib
    return lib


def call(m, cache, q, window, sinks, splits=0, q_seq=None, q_len=None, stream=None, workspace=None):
    n = q.shape[0]
    out = torch.full((n, 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, 128), 7.0, dtype=torch.float32, device="cuda")
    nbytes = m.decode_workspace_size(n, m.window_span(cache.capacity, window, sinks), splits)
    ws = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device="cuda") if workspace is None else workspace
    kw = dict(window=window, sinks=sinks, lse=lse, block_table=cache.table, num_splits=splits, stream=stream)
    if q_seq is not None:
        m.prefill_attn_window(q, cache.data, q_seq, q_len, cache.desc, ws, out, **kw)
    elif cache.scales is not None:
        m.decode_attn_window_fp8(q, cache.data, cache.scales, cache.seq_lens, cache.desc, ws, out, **kw)
    else:
        m.decode_attn_window(q, cache.data, cache.seq_lens, cache.desc, ws, out, **kw)
    return out, lse


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_decode_matches_the_definition(m, window, sinks, fp8, paged):
    rng = np.random.default_rng(11)
    cache = RowCache(m, [random_rows(rng, L) for L in LENS], paged, 12, fp8=fp8)
    q = random_q(rng, len(LENS))
    out, lse = call(m, cache, q.cuda(), window, sinks)
    assert m.get_device_error() == 0
    out, lse = f64(out), f64(lse)
    for b in range(len(LENS)):
        assert_window_row(out[b], lse[b], oracle.window_rows(f64(q[b]), cache.values[b], window, sinks, SCALE, 512))


@pytest.mark.parametrize("splits", [1, 3, 17, 200])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_over_forced_ranges(m, paged, splits):
    rng = np.random.default_rng(21)
    lens = [5000, 77, 2600, 0, 300]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], paged, 22)
    q = random_q(rng, len(lens))
    out, lse = (f64(x) for x in call(m, cache, q.cuda(), 1500, 70, splits))
    assert m.get_device_error() == 0
    for b in range(len(lens)):
        assert_window_row(out[b], lse[b], oracle.window_rows(f64(q[b]), cache.values[b], 1500, 70, SCALE, 512))


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 0), (64, 65), (0, 5), (1 << 30, 0)])
def test_rows_of_a_chunk(m, window, sinks, paged):
    """Rows of several sequences mixed, lengths from 0, the same sequence and the same row twice."""
    rng = np.random.default_rng(31)
    lens = [400, 90, 650]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], paged, 32)
    q_seq = np.array([2, 0, 1, 0, 2, 2, 1, 0, 2, 2], np.int32)
    q_len = np.array([650, 400, 1, 399, 0, 130, 90, 64, 650, 300], np.int32)
    q = random_q(rng, len(q_seq))
    q[8] = q[0]
    out, lse = call(m, cache, q.cuda(), window, sinks, 0, torch.from_numpy(q_seq).cuda(), torch.from_numpy(q_len).cuda())
    assert m.get_device_error() == 0
    out, lse = f64(out), f64(lse)
    for i, (s, L) in enumerate(zip(q_seq, q_len)):
        assert_window_row(out[i], lse[i], oracle.window_rows(f64(q[i]), cache.values[s][:L], window, sinks, SCALE, 512))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(100, 4), (65, 0), (300, 130)])
def test_hidden_tokens_may_hold_anything(m, window, sinks, fp8):
    """NaN and infinities in every hidden token leave the bits of the outputs as they were."""
    rng = np.random.default_rng(41)
    lens = [700, 333, 200, 90]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 42, fp8=fp8)
    q = random_q(rng, len(lens)).cuda()
    a = call(m, cache, q, window, sinks)
    for b, L in enumerate(lens):
        hidden = np.flatnonzero(~oracle.window_visible(L, window, sinks))
        if len(hidden):
            rows = cache.rows_of(b, hidden).cuda()
            if fp8:
                cache.data[rows] = 0x7F
                cache.scales[rows] = 255
            else:
                cache.data[rows] = torch.tensor([float("inf"), float("-inf"), float("nan")] * 192,
                                                dtype=torch.bfloat16, device="cuda")
    b2 = call(m, cache, q, window, sinks)
    assert torch.equal(a[0].view(torch.int16), b2[0].view(torch.int16)) and torch.equal(a[1], b2[1])
    assert torch.isfinite(a[0].float()).all()


def test_paged_and_contiguous_give_the_same_bits(m):
    rng = np.random.default_rng(51)
    seqs = [random_rows(rng, L) for L in (64 * 20, 1000, 130, 640)]
    q = random_q(rng, len(seqs)).cuda()
    a, b = (call(m, RowCache(m, seqs, paged, 52), q, 200, 68, 5) for paged in (False, True))
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_a_window_over_everything_gives_the_bits_of_the_plain_decode(m):
    rng = np.random.default_rng(61)
    cache = RowCache(m, [random_rows(rng, L) for L in (700, 64, 1, 333)], True, 62)
    q = random_q(rng, 4).cuda()
    a = call(m, cache, q, 4096, 0, 6)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    ws = torch.empty((m.decode_workspace_size(4, cache.capacity, 6),), dtype=torch.uint8, device="cuda")
    m.decode_attn(q, cache.data, cache.seq_lens, cache.desc, ws, out, lse=lse, block_table=cache.table, num_splits=6)
    assert torch.equal(a[0].view(torch.int16), out.view(torch.int16)) and torch.equal(a[1], lse)


def test_capture_and_replay_with_other_lengths(m):
    """Captured on a side stream, replayed after the lengths and rows have changed on the device."""
    rng = np.random.default_rng(71)
    lens = [600, 250]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 72)
    q = random_q(rng, 2)
    qd = q.cuda()
    call(m, cache, qd, 128, 4)   # loads the kernel before the capture
    ws = torch.empty((m.decode_workspace_size(2, cache.capacity, 0),), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out, lse = call(m, cache, qd, 128, 4, workspace=ws)
    for new in ([600, 250], [150, 9], [0, 250]):
        cache.seq_lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for b in range(2):
            ref = oracle.window_rows(f64(q[b]), cache.values[b][:new[b]], 128, 4, SCALE, 512)
            assert_window_row(f64(out)[b], f64(lse)[b], ref)
    assert m.get_device_error() == 0


def test_bad_pages_and_lengths_are_reported(m):
    rng = np.random.default_rng(81)
    cache = RowCache(m, [random_rows(rng, 700), random_rows(rng, 700)], True, 82)
    q = random_q(rng, 2)
    table = cache.table.clone()
    table[0, 5] = 1 << 29          # hidden by the window: never looked up
    table[0, 3] = -1
    cache.table = table
    out, lse = call(m, cache, q.cuda(), 64, 64)
    assert m.get_device_error() == 0
    cache.table[0, 10] = 1 << 29   # in the window
    call(m, cache, q.cuda(), 64, 64)
    assert m.get_device_error() & m.DEVERR_BLOCK_RANGE
    cache.seq_lens[1] = 10 ** 6    # clamped to the capacity
    call(m, cache, q.cuda(), 0, 64)
    assert m.get_device_error() & m.DEVERR_SEQLEN_RANGE


@pytest.mark.parametrize("window,sinks", [(100, 4), (0, 0), (64, 65)])
def test_more_rows_than_ranges(m, window, sinks):
    """Rows by the hundred, empty ones among them: as a batch of sequences and as a chunk over one page
    table, whose plan and combine take other ways than those of a few rows."""
    rng = np.random.default_rng(91)
    lens = [int(x) for x in rng.integers(0, 400, 330)]
    lens[::17] = [0] * len(lens[::17])
    long = random_rows(rng, 400)
    cache = RowCache(m, [long], True, 92)
    n = len(lens)
    q = random_q(rng, n)
    out, lse = (f64(x) for x in call(m, cache, q.cuda(), window, sinks, 0, torch.zeros((n,), dtype=torch.int32).cuda(),
                                     torch.tensor(lens, dtype=torch.int32).cuda()))
    assert m.get_device_error() == 0
    for i in list(range(0, n, 7)) + list(range(0, n, 17)):
        ref = oracle.window_rows(f64(q[i]), cache.values[0][:lens[i]], window, sinks, SCALE, 512)
        assert_window_row(out[i], lse[i], ref)
    seqs = RowCache(m, [long[:L] for L in lens[:200]], False, 93)
    o2, l2 = (f64(x) for x in call(m, seqs, q[:200].cuda(), window, sinks))
    assert m.get_device_error() == 0
    for i in range(0, 200, 9):
        assert_window_row(o2[i], l2[i], oracle.window_rows(f64(q[i]), seqs.values[i], window, sinks, SCALE, 512))


@pytest.mark.parametrize("lens", [[0], [100], [0, 64], [64, 0], [0, 0]])
def test_calls_of_one_range(m, lens):
    """The smallest calls have one work range and no combine: empty rows beside short ones, and a forced one."""
    rng = np.random.default_rng(95)
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 96, max_len=64 if len(lens) == 2 else 128)
    q = random_q(rng, len(lens))
    for splits in (0, 1):
        out, lse = (f64(x) for x in call(m, cache, q.cuda(), 40, 3, splits))
        assert m.get_device_error() == 0
        for b, L in enumerate(lens):
            assert_window_row(out[b], lse[b], oracle.window_rows(f64(q[b]), cache.values[b], 40, 3, SCALE, 512))


def test_many_ranges_per_row(m):
    """One row over more ranges than the combine reads at a time, alone and beside others."""
    rng = np.random.default_rng(97)
    for lens, splits in (([12000], 60), ([9000, 100, 6000], 100), ([5000] * 12, 90)):
        cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 98)
        q = random_q(rng, len(lens))
        out, lse = (f64(x) for x in call(m, cache, q.cuda(), 11000, 40, splits))
        assert m.get_device_error() == 0
        for b in range(0, len(lens), 2):
            assert_window_row(out[b], lse[b], oracle.window_rows(f64(q[b]), cache.values[b], 11000, 40, SCALE, 512))


@pytest.mark.parametrize("filled", [0, 1, 2, 40])
def test_many_rows_almost_all_empty(m, filled):
    """More rows than ranges, but fewer tiles than ranges."""
    rng = np.random.default_rng(99)
    cache = RowCache(m, [random_rows(rng, 700)], True, 100)
    n = 200
    lens = np.zeros(n, np.int32)
    lens[rng.choice(n, filled, replace=False)] = 600 if filled < 40 else 130
    q = random_q(rng, n)
    out, lse = (f64(x) for x in call(m, cache, q.cuda(), 500, 4, 0, torch.zeros((n,), dtype=torch.int32).cuda(),
                                     torch.from_numpy(lens).cuda()))
    assert m.get_device_error() == 0
    for i in range(n):
        if lens[i] or i % 9 == 0:
            assert_window_row(out[i], lse[i], oracle.window_rows(f64(q[i]), cache.values[0][:lens[i]], 500, 4, SCALE, 512))


@pytest.mark.parametrize("window", [1 << 30, 200])
def test_fp8_rows_of_any_scale_have_the_bits_of_their_bf16_values(m, window):
    """Row scales from 2^-127 (values below bf16's normal range, rounded to it once) to 2^118."""
    rng = np.random.default_rng(91)
    exps, L = [-120, -119, -100, -7, 0, 7, 60, 124], 300
    seqs = [torch.from_numpy(rng.standard_normal((L, 576)) * 2.0 ** k).to(torch.bfloat16) for k in exps]
    coded = RowCache(m, seqs, True, 92, fp8=True)
    plain = RowCache(m, [torch.from_numpy(v).to(torch.bfloat16) for v in coded.values], True, 92)
    assert int(coded.scales.min()) == 0 and int(coded.scales.max()) > 240
    q = torch.stack([(r.double() * 2.0 ** -k).to(torch.bfloat16) for r, k in zip(random_q(rng, len(exps)), exps)]).cuda()
    a, b = call(m, coded, q, window, 4), call(m, plain, q, window, 4)
    assert torch.isfinite(a[1]).all() and (a[0] != 0).any(dim=2).all()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_the_default_stream_argument_is_the_current_stream(m):
    torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    assert m._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert m._stream(None) == side.cuda_stream
    assert m._stream(None) == torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("form", ["one range", "nothing visible", "many rows", "fewer rows than ranges"])
@pytest.mark.parametrize("fp8", [False, True])
def test_many_empty_rows_are_written_by_the_whole_device(m, form, fp8):
    """Zeros and -inf for every empty row, from blocks enough to write them quickly, and the other rows as ever."""
    rows = 40 if form == "fewer rows than ranges" else 500
    lens = [0] * rows
    if form != "nothing visible":
        lens[7], lens[rows - 1] = 130, 64
    rng = np.random.default_rng(71)
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 72, fp8=fp8,
                     max_len=4096 if form == "fewer rows than ranges" else None)
    q = random_q(rng, rows).cuda()
    out = torch.full((rows, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 128), float("nan"), device="cuda")
    ws = torch.empty((m.decode_workspace_size(rows, cache.capacity),), dtype=torch.uint8, device="cuda")
    kw = dict(lse=lse, block_table=cache.table, num_splits=1 if form == "one range" else 0)
    if form == "nothing visible":
        cache.seq_lens.fill_(64)
        kw.update(window=0, sinks=0)

    def call():
        args = (cache.seq_lens, cache.desc, ws, out)
        if fp8:
            f = m.decode_attn_window_fp8 if "window" in kw else m.decode_attn_fp8
            f(q, cache.data, cache.scales, *args, **kw)
        else:
            (m.decode_attn_window if "window" in kw else m.decode_attn)(q, cache.data, *args, **kw)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g, stream=side):
        call()
    out.fill_(float("nan"))
    lse.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert m.get_device_error() == 0
    full = [b for b, L in enumerate(lens) if L]
    empty = torch.ones(rows, dtype=torch.bool)
    empty[full] = False
    assert torch.all(out[empty.cuda()] == 0) and torch.all(torch.isneginf(lse[empty.cuda()]))
    for b in full:
        assert_window_row(f64(out[b]), f64(lse[b]),
                          oracle.window_rows(f64(q[b]), cache.values[b], 10 ** 6, 0, SCALE, 512))
    assert max(x * y for x, y, _ in launches(g)) >= rows
