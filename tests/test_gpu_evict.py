"""Eviction by accumulated attention weight (mla_cache_evict, _fp8) and the append at a slot of its own
(mla_cache_append_at, _fp8): every output is a copy or a whole number, so all comparisons are of bits."""
import numpy as np
import pytest
import torch

import oracle
from bounded_common import RowCache, launches, random_rows

pytestmark = pytest.mark.gpu

LENS = [0, 1, 5, 63, 64, 65, 100, 129, 300, 1000]


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available()
    import mla_latent_kv_20_b200 as lib
    return lib


def weights_like(rng, B, cap, kind):
    if kind == "heavy":
        w = np.exp(2 * rng.standard_normal((B, cap))) * (rng.random((B, cap)) > 0.125)
    elif kind == "equal":
        w = np.full((B, cap), 0.25)
    elif kind == "few":
        w = rng.integers(0, 3, (B, cap)).astype(float)
    else:   # signs, zeros of both signs, infinities, NaN of both signs, the smallest numbers
        w = rng.choice([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 1.0, -1.0, 3e38, -3e38], (B, cap))
    return torch.from_numpy(w.astype(np.float32))


def evict(m, cache, weights, keep, sinks, recent, out=None, weights_out=None, lens_out=None, stream=None):
    """out: a RowCache to move into, or None for in place."""
    B = len(cache.lens)
    dst = cache if out is None else out
    kept = torch.full((B, keep), 99, dtype=torch.int32, device="cuda")
    lens_out = torch.full((B,), 99, dtype=torch.int32, device="cuda") if lens_out is None else lens_out
    weights_out = torch.full((B, dst.capacity), 99.0, device="cuda") if weights_out is None else weights_out
    ws = torch.empty((m.evict_workspace_size(B, keep),), dtype=torch.uint8, device="cuda")
    kw = dict(keep=keep, sinks=sinks, recent=recent, block_table=cache.table, stream=stream)
    if out is not None:
        kw.update(cache_out=dst.data, desc_out=dst.desc, block_table_out=dst.table)
        if cache.scales is not None:
            kw["scales_out"] = dst.scales
    if cache.scales is not None:
        m.cache_evict_fp8(cache.data, cache.scales, cache.seq_lens, weights, cache.desc, kept, lens_out, weights_out,
                          ws, **kw)
    else:
        m.cache_evict(cache.data, cache.seq_lens, weights, cache.desc, kept, lens_out, weights_out, ws, **kw)
    return kept, lens_out, weights_out


def bits(t):
    return t.cpu().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy().copy()


def expected(cache, dst, before, weights, keep, sinks, recent, wo_before, lens):
    """The bits of the output cache (and scales), kept, lengths and weights."""
    B = len(lens)
    rows, scales = before["dst"].copy(), None if before["dst_scales"] is None else before["dst_scales"].copy()
    kept = np.full((B, keep), -1, np.int32)
    wo = wo_before.copy()
    for b, L in enumerate(lens):
        t = oracle.evict_keep(weights[b], L, keep, sinks, recent)
        n = len(t)
        kept[b, :n] = t
        if n:
            frm, to = cache.rows_of(b, t).numpy(), dst.rows_of(b, np.arange(n)).numpy()
            rows[to] = before["src"][frm]
            if scales is not None:
                scales[to] = before["src_scales"][frm]
        wo[b, :n] = weights[b][t].view(np.int32)
        wo[b, n:min(L, wo.shape[1])] = 0
    return rows, scales, kept, np.minimum(lens, keep).astype(np.int32), wo


def check(m, lens, paged, fp8, in_place, kind, keep, sinks, recent, seed, out_paged=None, max_len=None):
    rng = np.random.default_rng(seed)
    cache = RowCache(m, [random_rows(rng, L) for L in lens], paged, seed, fp8=fp8, max_len=max_len)
    dst = cache
    if not in_place:
        dst = RowCache(m, [random_rows(rng, keep) for _ in lens], paged if out_paged is None else out_paged, seed + 1,
                       fp8=fp8)
    w = weights_like(rng, len(lens), cache.capacity, kind).cuda()
    before = dict(src=bits(cache.data), dst=bits(dst.data), src_scales=None if not fp8 else bits(cache.scales),
                  dst_scales=None if not fp8 else bits(dst.scales))
    wo = torch.full((len(lens), dst.capacity), 99.0, device="cuda")
    want = expected(cache, dst, before, w.cpu().numpy(), keep, sinks, recent, bits(wo), lens)
    kept, lens_out, wo = evict(m, cache, w, keep, sinks, recent, None if in_place else dst, wo)
    assert m.get_device_error() == 0
    assert np.array_equal(kept.cpu().numpy(), want[2])
    assert np.array_equal(lens_out.cpu().numpy(), want[3])
    assert np.array_equal(bits(wo), want[4])
    assert np.array_equal(bits(dst.data), want[0])
    if fp8:
        assert np.array_equal(bits(dst.scales), want[1])
    if not in_place:
        assert np.array_equal(bits(cache.data), before["src"])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,sinks,recent", [(64, 4, 16), (1, 0, 0), (65, 0, 65), (65, 65, 0), (100, 40, 60),
                                               (33, 0, 1)])
def test_evict(m, keep, sinks, recent, in_place, paged, fp8):
    check(m, LENS, paged, fp8, in_place, "heavy", keep, sinks, recent, keep + 2 * recent)


@pytest.mark.parametrize("kind", ["equal", "few", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_ties_and_special_weights(m, in_place, kind):
    for keep, sinks, recent in ((50, 3, 7), (200, 0, 0), (257, 1, 64)):
        check(m, [700, 258, 64, 2, 999], True, False, in_place, kind, keep, sinks, recent, keep)


@pytest.mark.parametrize("in_place", [False, True])
def test_everything_fits(m, in_place):
    check(m, [5, 0, 64, 130], True, False, in_place, "heavy", 256, 4, 4, 5, max_len=512)
    check(m, [5, 0, 64, 130], True, False, in_place, "heavy", 1000, 4, 4, 6)   # more than a sequence can hold
    check(m, [5, 130], False, True, in_place, "heavy", 1000, 400, 4, 7)
    check(m, [5, 100], False, False, in_place, "heavy", 128, 0, 4, 8)


def test_between_layouts(m):
    check(m, [700, 100], True, False, False, "heavy", 96, 2, 30, 6, out_paged=False)
    check(m, [700, 100], False, False, False, "heavy", 96, 2, 30, 7, out_paged=True)


@pytest.mark.parametrize("lens,keep", [([40000], 3000), ([9000, 70000], 20000), ([140000], 64), ([5000] * 3, 4999)])
@pytest.mark.parametrize("kind", ["heavy", "few", "special"])
def test_long_sequences_shared_by_a_cluster(m, lens, keep, kind):
    """The selection alone at lengths that several CTAs share, over a cache of one page per sequence
    that every block-table entry names (its rows are moved onto themselves)."""
    rng = np.random.default_rng(len(lens) + keep)
    B, width = len(lens), (max(lens) + 63) // 64
    table = torch.arange(B, dtype=torch.int32)[:, None].repeat(1, width).cuda()
    cache = torch.zeros((B * 64, 576), dtype=torch.bfloat16, device="cuda")
    desc = m.paged_desc(B, width, B)
    w = weights_like(rng, B, width * 64, kind)
    kept = torch.zeros((B, keep), dtype=torch.int32, device="cuda")
    lens_out = torch.zeros((B,), dtype=torch.int32, device="cuda")
    wd = w.cuda()
    ws = torch.empty((m.evict_workspace_size(B, keep),), dtype=torch.uint8, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out_desc = m.paged_desc(B, (keep + 63) // 64, B)
    wo = torch.zeros((B, (keep + 63) // 64 * 64), device="cuda")
    m.cache_evict(cache, sl, wd, desc, kept, lens_out, wo, ws, keep=keep, sinks=5, recent=17, block_table=table,
                  cache_out=torch.zeros_like(cache), desc_out=out_desc,
                  block_table_out=table[:, :(keep + 63) // 64].contiguous())
    assert m.get_device_error() == 0
    got = kept.cpu().numpy()
    for b, L in enumerate(lens):
        t = oracle.evict_keep(w[b].numpy(), L, keep, 5, 17)
        assert np.array_equal(got[b, :len(t)], t) and np.all(got[b, len(t):] == -1)
        assert np.array_equal(bits(wo)[b, :len(t)], w[b].numpy()[t].view(np.int32))


def test_weights_and_lengths_in_place_and_twice(m):
    """weights_out = weights and lens_out = seq_lens; a second call finds nothing to evict."""
    rng = np.random.default_rng(3)
    lens = [300, 64, 17]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 4)
    first = bits(cache.data)
    w = weights_like(rng, 3, cache.capacity, "heavy").cuda()
    w0 = w.cpu().numpy()
    evict(m, cache, w, 40, 2, 10, None, w, cache.seq_lens)
    assert cache.seq_lens.tolist() == [40, 40, 17]
    got, rows = bits(w), bits(cache.data)
    for b, L in enumerate(lens):
        t = oracle.evict_keep(w0[b], L, 40, 2, 10)
        n = len(t)
        assert np.array_equal(got[b, :n], w0[b][t].view(np.int32)) and np.all(got[b, n:L] == 0)
        assert np.array_equal(got[b, L:], w0[b][L:].view(np.int32))
        assert np.array_equal(rows[cache.rows_of(b, np.arange(n)).numpy()], first[cache.rows_of(b, t).numpy()])
    kept, lens_out, _ = evict(m, cache, w, 40, 2, 10, None, w, cache.seq_lens)
    assert np.array_equal(bits(cache.data), rows) and np.array_equal(bits(w), got)
    assert kept[2].tolist() == list(range(17)) + [-1] * 23


@pytest.mark.parametrize("fp8", [False, True])
def test_into_fresh_pages_of_the_same_pool(m, fp8):
    """In place with another block table: the output's pages are pages of the pool that no token uses."""
    rng = np.random.default_rng(17)
    lens, keep = [500, 130, 64], 100
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 18, fp8=fp8)
    used = set(cache.table[cache.table >= 0].cpu().tolist())
    free = [p for p in range(cache.data.shape[0] // 64) if p not in used][:6]
    assert len(free) == 6
    table = torch.tensor(free, dtype=torch.int32).reshape(3, 2).cuda()
    desc = m.paged_desc(3, 2, cache.data.shape[0] // 64)
    w = weights_like(rng, 3, cache.capacity, "heavy").cuda()
    rows, scales = bits(cache.data), None if not fp8 else bits(cache.scales)
    kept = torch.zeros((3, keep), dtype=torch.int32, device="cuda")
    lens_out = torch.zeros((3,), dtype=torch.int32, device="cuda")
    wo = torch.zeros((3, 128), device="cuda")
    ws = torch.empty((m.evict_workspace_size(3, keep),), dtype=torch.uint8, device="cuda")
    kw = dict(keep=keep, sinks=2, recent=20, block_table=cache.table, cache_out=cache.data, desc_out=desc,
              block_table_out=table)
    if fp8:
        m.cache_evict_fp8(cache.data, cache.scales, cache.seq_lens, w, cache.desc, kept, lens_out, wo, ws,
                          scales_out=cache.scales, **kw)
    else:
        m.cache_evict(cache.data, cache.seq_lens, w, cache.desc, kept, lens_out, wo, ws, **kw)
    assert m.get_device_error() == 0
    tab = table.cpu().numpy()
    for b, L in enumerate(lens):
        t = oracle.evict_keep(w[b].cpu().numpy(), L, keep, 2, 20)
        to = tab[b][np.arange(len(t)) // 64].astype(np.int64) * 64 + np.arange(len(t)) % 64
        frm = cache.rows_of(b, t).numpy()
        rows[to] = rows[frm]
        if fp8:
            scales[to] = scales[frm]
    assert np.array_equal(bits(cache.data), rows)
    if fp8:
        assert np.array_equal(bits(cache.scales), scales)


def test_capture_replay_and_a_side_stream(m):
    rng = np.random.default_rng(8)
    cache = RowCache(m, [random_rows(rng, L) for L in (500, 200)], True, 9)
    out = RowCache(m, [random_rows(rng, 64) for _ in range(2)], True, 10)
    w = weights_like(rng, 2, cache.capacity, "heavy").cuda()
    evict(m, cache, w, 64, 4, 8, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kept, lens_out, wo = evict(m, cache, w, 64, 4, 8, out)
    for trial in range(3):
        new = weights_like(rng, 2, cache.capacity, "heavy")
        w.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        for b, L in enumerate((500, 200)):
            t = oracle.evict_keep(new[b].numpy(), L, 64, 4, 8)
            assert np.array_equal(kept[b].cpu().numpy(), t)
            assert np.array_equal(bits(out.data)[out.rows_of(b, np.arange(64)).numpy()],
                                  bits(cache.data)[cache.rows_of(b, t).numpy()])
    assert m.get_device_error() == 0


def test_bad_pages_and_lengths_are_reported_and_skipped(m):
    rng = np.random.default_rng(13)
    cache = RowCache(m, [random_rows(rng, 300), random_rows(rng, 300)], True, 14)
    out = RowCache(m, [random_rows(rng, 128) for _ in range(2)], True, 15)
    w = torch.ones((2, cache.capacity), device="cuda")
    before = bits(out.data)
    cache.table[0, 4] = 1 << 29     # tokens 256..299 of sequence 0, its recent ones
    out.table[1, 1] = -1            # slots 64..127 of sequence 1
    kept, lens_out, _ = evict(m, cache, w, 128, 4, 44, out)
    assert m.get_device_error() & m.DEVERR_BLOCK_RANGE
    got, src = bits(out.data), bits(cache.data)
    t = oracle.evict_keep(np.ones(300), 300, 128, 4, 44)
    assert kept[0].tolist() == list(t)
    good = np.flatnonzero(t < 256)
    rows = out.table.cpu().numpy()[0][good // 64].astype(np.int64) * 64 + good % 64
    assert np.array_equal(got[rows], src[cache.rows_of(0, t[good]).numpy()])
    bad = np.flatnonzero(t >= 256)
    rows = out.table.cpu().numpy()[0][bad // 64].astype(np.int64) * 64 + bad % 64
    assert np.array_equal(got[rows], before[rows])
    cache.seq_lens.copy_(torch.tensor([-3, 10 ** 6], dtype=torch.int32))
    kept, lens_out, _ = evict(m, cache, w, 128, 4, 44, out)
    assert m.get_device_error() & m.DEVERR_SEQLEN_RANGE
    assert lens_out.tolist() == [0, 128] and kept[0].tolist() == [-1] * 128


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_at_writes_the_row_of_the_position_to_the_slot(m, fp8, paged):
    rng = np.random.default_rng(21)
    n = 5
    c = torch.from_numpy(rng.standard_normal((n, 512))).to(torch.bfloat16).cuda()
    kr = torch.from_numpy(rng.standard_normal((n, 64))).to(torch.bfloat16).cuda()
    seq = torch.tensor([1, 0, 2, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([100000, 7, 0, 4096, 131071], dtype=torch.int32, device="cuda")   # beyond the capacity
    slots = torch.tensor([0, 9, 63, 64, 100], dtype=torch.int32, device="cuda")
    cache = RowCache(m, [random_rows(rng, 128) for _ in range(3)], paged, 22, fp8=fp8)
    before, sbefore = bits(cache.data), None if not fp8 else bits(cache.scales)
    # the rows themselves, as a plain append of tokens at these positions writes them
    long_desc = m.contiguous_desc(1, 131072)
    big = torch.zeros((131072, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    sbig = torch.zeros((131072,), dtype=torch.uint8, device="cuda")
    zero = torch.zeros((n,), dtype=torch.int32, device="cuda")
    if fp8:
        m.cache_append_fp8(c, kr, pos, big, sbig, long_desc, seq_ids=zero)
        m.cache_append_at_fp8(c, kr, pos, slots, cache.data, cache.scales, cache.desc, seq_ids=seq,
                              block_table=cache.table)
    else:
        m.cache_append(c, kr, pos, big, long_desc, seq_ids=zero)
        m.cache_append_at(c, kr, pos, slots, cache.data, cache.desc, seq_ids=seq, block_table=cache.table)
    assert m.get_device_error() == 0
    for i in range(n):
        r = int(cache.rows_of(int(seq[i]), int(slots[i])))
        before[r] = bits(big[int(pos[i])])
        if fp8:
            sbefore[r] = int(sbig[int(pos[i])])
    assert np.array_equal(bits(cache.data), before)
    if fp8:
        assert np.array_equal(bits(cache.scales), sbefore)


def test_append_at_refuses_slots_outside(m):
    cache = RowCache(m, [random_rows(np.random.default_rng(1), 64)], True, 2)
    before = bits(cache.data)
    c = torch.ones((2, 512), dtype=torch.bfloat16, device="cuda")
    kr = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    seq = torch.zeros((2,), dtype=torch.int32, device="cuda")
    for pos, slots in (([3, 3], [-1, 64]), ([-1, -5], [0, 1])):
        m.cache_append_at(c, kr, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                          torch.tensor(slots, dtype=torch.int32, device="cuda"), cache.data, cache.desc, seq_ids=seq,
                          block_table=cache.table)
        assert m.get_device_error() & m.DEVERR_POS_RANGE
        assert np.array_equal(bits(cache.data), before)


@pytest.mark.parametrize("fp8", [False, True])
def test_fresh_pages_named_without_the_cache(m, fp8):
    """block_table_out and desc_out alone: the rows land in those pages, the old ones keep theirs."""
    rng = np.random.default_rng(23)
    lens, keep = [500, 130, 64], 100
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 24, fp8=fp8)
    used = set(cache.table[cache.table >= 0].cpu().tolist())
    free = [p for p in range(cache.data.shape[0] // 64) if p not in used][:6]
    assert len(free) == 6
    tab = np.array(free, np.int32).reshape(3, 2)
    w = weights_like(rng, 3, cache.capacity, "heavy").cuda()
    rows, scales = bits(cache.data), None if not fp8 else bits(cache.scales)
    kept = torch.zeros((3, keep), dtype=torch.int32, device="cuda")
    lens_out = torch.zeros((3,), dtype=torch.int32, device="cuda")
    wo = torch.zeros((3, 128), device="cuda")
    ws = torch.empty((m.evict_workspace_size(3, keep),), dtype=torch.uint8, device="cuda")
    call = m.cache_evict_fp8 if fp8 else m.cache_evict
    call(cache.data, *([cache.scales] if fp8 else []), cache.seq_lens, w, cache.desc, kept, lens_out, wo, ws, keep=keep,
         sinks=2, recent=20, block_table=cache.table, block_table_out=torch.from_numpy(tab).cuda(),
         desc_out=m.paged_desc(3, 2, cache.data.shape[0] // 64))
    assert m.get_device_error() == 0
    for b, L in enumerate(lens):
        t = oracle.evict_keep(w[b].cpu().numpy(), L, keep, 2, 20)
        j = np.arange(len(t))
        to, frm = tab[b][j // 64].astype(np.int64) * 64 + j % 64, cache.rows_of(b, t).numpy()
        rows[to] = rows[frm]
        if fp8:
            scales[to] = scales[frm]
    assert np.array_equal(bits(cache.data), rows)
    if fp8:
        assert np.array_equal(bits(cache.scales), scales)


# Sequences whose selection a cluster of CTAs shares (more than 4096 tokens of capacity each): rows, scales and
# weights as they are after it, moved by the selection itself (up to 128 kept tokens) or by a second launch.
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep,sinks,recent", [([9000, 60, 0], 64, 4, 16), ([40000], 128, 0, 33),
                                                    ([9000, 129, 5000], 128, 60, 68), ([4100, 9000], 1, 0, 0),
                                                    ([9000, 300], 129, 3, 40), ([20000, 1500], 1000, 5, 100)])
def test_rows_of_sequences_shared_by_a_cluster(m, lens, keep, sinks, recent, in_place, fp8):
    check(m, lens, True, fp8, in_place, "heavy", keep, sinks, recent, keep + len(lens))


@pytest.mark.parametrize("kind", ["few", "special"])
def test_ties_of_sequences_shared_by_a_cluster(m, kind):
    check(m, [9000, 4500], False, False, True, kind, 100, 2, 10, 31)
    check(m, [9000, 4500], True, False, False, kind, 100, 0, 0, 32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("keep", [96, 200])
def test_weights_and_lengths_in_place_of_a_sequence_shared_by_a_cluster(m, keep, fp8):
    """weights_out = weights and lens_out = seq_lens."""
    rng = np.random.default_rng(41)
    lens = [9000, 150, 5000]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 42, fp8=fp8)
    first = bits(cache.data)
    w = weights_like(rng, 3, cache.capacity, "heavy").cuda()
    w0 = w.cpu().numpy()
    kept, _, _ = evict(m, cache, w, keep, 4, 30, None, w, cache.seq_lens)
    assert m.get_device_error() == 0
    assert cache.seq_lens.tolist() == [min(L, keep) for L in lens]
    got, rows = bits(w), bits(cache.data)
    for b, L in enumerate(lens):
        t = oracle.evict_keep(w0[b], L, keep, 4, 30)
        n = len(t)
        assert kept[b].tolist() == list(t) + [-1] * (keep - n)
        assert np.array_equal(got[b, :n], w0[b][t].view(np.int32)) and np.all(got[b, n:L] == 0)
        assert np.array_equal(got[b, L:], w0[b][L:].view(np.int32))
        assert np.array_equal(rows[cache.rows_of(b, np.arange(n)).numpy()], first[cache.rows_of(b, t).numpy()])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,blocks", [([100, 128], None), ([300, 1000], 32)])   # blocks of 32 of 1024 slots
def test_keep_beyond_the_capacity_costs_no_launches(m, lens, blocks, fp8):
    """What is launched follows min(keep, capacity): the slots that can hold a row."""
    rng = np.random.default_rng(51)
    keep = 1 << 18
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 52, fp8=fp8)
    out = RowCache(m, [random_rows(rng, cache.capacity) for _ in lens], True, 53, fp8=fp8)
    w = weights_like(rng, 2, cache.capacity, "heavy").cuda()
    evict(m, cache, w, keep, 4, 8, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g, stream=side):
        kept, lens_out, wo = evict(m, cache, w, keep, 4, 8, out)
    moves = [x for x in launches(g) if x[1] == len(lens)]   # (blocks of slots, sequences)
    g.replay()
    torch.cuda.synchronize()
    assert m.get_device_error() == 0 and lens_out.tolist() == lens
    for b, L in enumerate(lens):
        assert kept[b, :L].tolist() == list(range(L)) and torch.all(kept[b, L:] == -1)
        assert np.array_equal(bits(out.data)[out.rows_of(b, np.arange(L)).numpy()],
                              bits(cache.data)[cache.rows_of(b, np.arange(L)).numpy()])
    # (the selection itself moves the rows of a cache of at most 128 slots)
    assert moves == ([] if blocks is None else [(blocks, len(lens), 1)])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[1], [3, 2], [16, 0, 9]])
def test_caches_of_a_few_slots(m, lens, fp8):
    for in_place in (False, True):
        for keep, sinks, recent in ((1, 0, 0), (1, 1, 0), (2, 0, 1)):
            check(m, lens, False, fp8, in_place, "special", keep, sinks, recent, 61)
