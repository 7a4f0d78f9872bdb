"""Attention weights accumulated per cached token (mla_attn_weights, _fp8, mla_prefill_attn_weights)
against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from bounded_common import SCALE, RowCache, U, f64, random_q, random_rows, weight_sums

pytestmark = pytest.mark.gpu

LENS = [0, 1, 63, 64, 65, 128, 129, 255, 256, 257, 700, 1000]


@pytest.fixture(scope="module")
def m():
    assert torch.cuda.is_available()
    import mla_latent_kv_20_b200 as lib
    return lib


def row_lse(q, rows, scale=SCALE):
    """The row's log-sum-exps as the attention would leave them, rounded to fp32."""
    s = scale * (q @ rows.T)
    if s.shape[1] == 0:
        return np.full(len(q), -np.inf, np.float32)
    top = s.max(axis=1)
    return (top + np.log(np.exp(s - top[:, None]).sum(axis=1))).astype(np.float32)


def call(m, cache, q, lse, prev=None, decay=1.0, out=None, q_start=None, q_len=None, stream=None, ws=None,
         scale=SCALE):
    B = len(cache.lens)
    out = torch.full((B, cache.capacity), 7.0, device="cuda") if out is None else out
    kw = dict(prev=prev, decay=decay, block_table=cache.table, stream=stream, softmax_scale=scale)
    if q_start is not None:
        n = m.prefill_attn_weights_workspace_size(B, cache.capacity, len(q))
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        m.prefill_attn_weights(q, cache.data, cache.seq_lens, q_start, q_len, cache.desc, lse, ws, out, **kw)
    elif cache.scales is not None:
        m.attn_weights_fp8(q, cache.data, cache.scales, cache.seq_lens, cache.desc, lse, out, **kw)
    else:
        m.attn_weights(q, cache.data, cache.seq_lens, cache.desc, lse, out, **kw)
    return out


def check(got, lens, sums, bounds, prev, decay, untouched):
    for b, L in enumerate(lens):
        base = np.zeros(L) if prev is None else float(np.float32(decay)) * prev[b, :L]
        want = base + sums[b]
        bound = bounds[b] + 4 * U * (np.abs(base) + sums[b])
        err = np.abs(got[b, :L] - want)
        assert np.all(err <= bound), f"sequence {b} of {L}: {(err > bound).sum()} out, worst {(err - bound).max():.3e}"
        assert np.array_equal(got[b, L:], untouched[b, L:])


@pytest.mark.parametrize("form", ["contiguous", "odd stride", "paged"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("before", ["none", "other", "same"])
def test_one_row_per_sequence(m, form, fp8, before):
    rng = np.random.default_rng(11)
    cache = RowCache(m, [random_rows(rng, L) for L in LENS], form == "paged", 12, fp8=fp8,
                     max_len=1003 if form == "odd stride" else None, align=1 if form == "odd stride" else 16)
    q = random_q(rng, len(LENS))
    qf = f64(q)
    lse = np.stack([row_lse(qf[b], cache.values[b]) for b in range(len(LENS))])
    prev = torch.from_numpy(rng.exponential(2.0, (len(LENS), cache.capacity)).astype(np.float32)).cuda()
    p = None if before == "none" else f64(prev)
    out = prev if before == "same" else None
    untouched = f64(prev) if before == "same" else np.full((len(LENS), cache.capacity), 7.0)
    got = call(m, cache, q.cuda(), torch.from_numpy(lse).cuda(), None if before == "none" else prev, 0.875, out)
    assert m.get_device_error() == 0
    pairs = [weight_sums(qf[b], cache.values[b], lse[b].astype(float)) for b in range(len(LENS))]
    check(f64(got), LENS, [x for x, _ in pairs], [x for _, x in pairs], p, 0.875, untouched)


def test_many_short_sequences(m):
    """More sequences than lanes and CTA pairs, most of them one tile, some empty."""
    rng = np.random.default_rng(21)
    lens = [int(x) for x in rng.integers(0, 300, 200)]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 22)
    q = random_q(rng, len(lens))
    qf = f64(q)
    lse = np.stack([row_lse(qf[b], cache.values[b]) for b in range(len(lens))])
    got = call(m, cache, q.cuda(), torch.from_numpy(lse).cuda())
    assert m.get_device_error() == 0
    pairs = [weight_sums(qf[b], cache.values[b], lse[b].astype(float)) for b in range(len(lens))]
    check(f64(got), lens, [x for x, _ in pairs], [x for _, x in pairs], None, 1.0, np.full(got.shape, 7.0))


CHUNKS = {
    # lengths, rows of each sequence, how far they reach
    "last tokens": ([700, 300, 64], [3, 5, 2], "last"),
    "one tile over many ranges": ([200], [150], "last"),
    "two tiles over many ranges": ([400], [97], "last"),
    "sequences without rows or tokens": ([300, 0, 513, 129, 0], [0, 0, 9, 0, 3], "last"),
    "any reach": ([600, 257, 1000], [20, 1, 33], "any"),
    "whole prompt": ([130], [130], "last"),
    "more sequences than ranges": ([70] * 90, [2] * 90, "any"),
}


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("name", list(CHUNKS))
def test_rows_of_a_chunk(m, name, paged):
    lens, counts, reach = CHUNKS[name]
    rng = np.random.default_rng(31)
    cache = RowCache(m, [random_rows(rng, L) for L in lens], paged, 32)
    n = sum(counts)
    q = random_q(rng, n)
    qf = f64(q)
    q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    seq = np.repeat(np.arange(len(lens)), counts)
    q_len = np.zeros(n, np.int32)
    for b, c in enumerate(counts):
        L = lens[b]
        q_len[q_start[b]:q_start[b + 1]] = np.maximum(L - c + 1 + np.arange(c), 0) if reach == "last" else \
            rng.integers(-3, L + 200, c)   # nothing, some, and more than there is
    prev = rng.exponential(2.0, (len(lens), cache.capacity)).astype(np.float32)
    lse = np.zeros((n, 128), np.float32)
    sums, bounds = [np.zeros(L) for L in lens], [np.zeros(L) for L in lens]
    for i, b in enumerate(seq):
        L = min(max(int(q_len[i]), 0), lens[b])
        lse[i] = row_lse(qf[i], cache.values[b][:L])
        w, e = weight_sums(qf[i], cache.values[b][:L], lse[i].astype(float))
        sums[b][:L] += w
        bounds[b][:L] += e
    for b, c in enumerate(counts):
        bounds[b] += c * 2 * U * sums[b]
    for p in (None, prev):
        got = call(m, cache, q.cuda(), torch.from_numpy(lse).cuda(), None if p is None else torch.from_numpy(p).cuda(),
                   0.5, None, torch.from_numpy(q_start).cuda(), torch.from_numpy(q_len).cuda())
        assert m.get_device_error() == 0
        check(f64(got), lens, sums, bounds, None if p is None else p.astype(float), 0.5, np.full(got.shape, 7.0))


def test_no_rows_at_all(m):
    """n_queries = 0: the weights fade, and nothing else is read."""
    rng = np.random.default_rng(41)
    lens = [300, 0, 64]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 42)
    prev = torch.rand((3, cache.capacity), device="cuda")
    out = torch.full_like(prev, 7.0)
    ws = torch.empty((m.prefill_attn_weights_workspace_size(3, cache.capacity, 0),), dtype=torch.uint8, device="cuda")
    m.prefill_attn_weights(None, cache.data, cache.seq_lens, torch.zeros((4,), dtype=torch.int32, device="cuda"), None,
                           cache.desc, None, ws, out, prev=prev, decay=0.25, block_table=cache.table, n_queries=0)
    assert m.get_device_error() == 0
    for b, L in enumerate(lens):
        assert torch.equal(out[b, :L], 0.25 * prev[b, :L]) and torch.all(out[b, L:] == 7.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_after_the_attention_the_weights_of_a_row_sum_to_the_heads(m, fp8):
    """lse as decode_attn writes it: 128 for every sequence, within its own and this call's errors."""
    rng = np.random.default_rng(51)
    lens = [1, 500, 3000]
    cache = RowCache(m, [random_rows(rng, L) for L in lens], True, 52, fp8=fp8)
    q = random_q(rng, 3)
    qd = q.cuda()
    out = torch.empty((3, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 128), device="cuda")
    ws = torch.empty((m.decode_workspace_size(3, cache.capacity),), dtype=torch.uint8, device="cuda")
    if fp8:
        m.decode_attn_fp8(qd, cache.data, cache.scales, cache.seq_lens, cache.desc, ws, out, lse=lse,
                          block_table=cache.table)
    else:
        m.decode_attn(qd, cache.data, cache.seq_lens, cache.desc, ws, out, lse=lse, block_table=cache.table)
    got = f64(call(m, cache, qd, lse))
    assert m.get_device_error() == 0
    for b, L in enumerate(lens):
        w, e = weight_sums(f64(q[b]), cache.values[b], f64(lse[b]))
        assert np.all(np.abs(got[b, :L] - w) <= e + 4 * U * w)
        ds = 576 * 2 * U * (SCALE * (np.abs(f64(q[b])) @ np.abs(cache.values[b]).T)).max()
        assert abs(got[b, :L].sum() - 128) <= e.sum() + 128 * (ds + 2.0 ** -16 + 4 * U)


def test_large_scores_and_heads_without_tokens(m):
    """Scores of tens, so that most terms are far below 1; a head whose lse is -inf adds nothing, one
    whose lse is +inf neither."""
    rng = np.random.default_rng(61)
    cache = RowCache(m, [random_rows(rng, 300, 6.0), random_rows(rng, 90, 6.0)], True, 62)
    q = random_q(rng, 2)
    qf = f64(q)
    lse = np.stack([row_lse(qf[b], cache.values[b]) for b in range(2)])
    lse[0, 5], lse[0, 77], lse[1, 127] = -np.inf, np.inf, -np.inf
    got = f64(call(m, cache, q.cuda(), torch.from_numpy(lse).cuda()))
    pairs = [weight_sums(qf[b], cache.values[b], lse[b].astype(float)) for b in range(2)]
    check(got, [300, 90], [x for x, _ in pairs], [x for _, x in pairs], None, 1.0, np.full(got.shape, 7.0))


def test_a_token_of_nan_spoils_only_itself(m):
    rng = np.random.default_rng(71)
    cache = RowCache(m, [random_rows(rng, 300)], True, 72)
    q = random_q(rng, 1)
    lse = torch.from_numpy(row_lse(f64(q[0]), cache.values[0])[None]).cuda()
    a = call(m, cache, q.cuda(), lse).clone()
    cache.data[cache.rows_of(0, [17, 290]).cuda()] = float("nan")
    b = call(m, cache, q.cuda(), lse)
    assert torch.isnan(b[0, [17, 290]]).all()
    keep = torch.ones_like(a[0], dtype=torch.bool)
    keep[[17, 290]] = False
    assert torch.equal(a[0][keep], b[0][keep])


def test_layouts_and_calls_give_the_same_bits(m):
    rng = np.random.default_rng(81)
    seqs = [random_rows(rng, L) for L in (64 * 20, 1000, 130, 640)]
    q = random_q(rng, 12)
    lse = torch.from_numpy(rng.uniform(5, 7, (12, 128)).astype(np.float32)).cuda()
    q_start = torch.tensor([0, 5, 5, 7, 12], dtype=torch.int32, device="cuda")
    q_len = torch.full((12,), 1280, dtype=torch.int32, device="cuda")
    outs, rows = [], []
    for form in (True, False, True):
        cache = RowCache(m, seqs, form, 82)
        outs.append(call(m, cache, q[:4].cuda(), lse[:4])[:, :1280])
        rows.append(call(m, cache, q.cuda(), lse, None, 1.0, None, q_start, q_len)[:, :1280])
    for x in outs[1:]:
        assert torch.equal(outs[0], x)
    for x in rows[1:]:
        assert torch.equal(rows[0], x)


def test_capture_and_replay_with_other_lengths(m):
    rng = np.random.default_rng(91)
    cache = RowCache(m, [random_rows(rng, 600), random_rows(rng, 250)], True, 92)
    q = random_q(rng, 6)
    qf, qd = f64(q), q.cuda()
    lse = torch.from_numpy(rng.uniform(5, 7, (6, 128)).astype(np.float32)).cuda()
    q_start = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    q_len = torch.full((6,), 1000, dtype=torch.int32, device="cuda")
    call(m, cache, qd, lse, q_start=q_start, q_len=q_len)
    ws = torch.empty((m.prefill_attn_weights_workspace_size(2, cache.capacity, 6),), dtype=torch.uint8, device="cuda")
    out = torch.full((2, cache.capacity), 7.0, device="cuda")
    acc = torch.zeros((2, cache.capacity), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(m, cache, qd, lse, None, 1.0, out, q_start, q_len, ws=ws)
        call(m, cache, qd[:2], lse[:2], acc, 1.0, acc)
    total = np.zeros((2, cache.capacity))
    bound = np.zeros_like(total)
    for starts, lens in (([0, 4, 6], [600, 250]), ([0, 1, 6], [100, 9]), ([0, 0, 6], [0, 250])):
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        sums, bounds = [], []
        for b, L in enumerate(lens):
            pairs = [weight_sums(qf[i], cache.values[b][:L], f64(lse[i])) for i in range(starts[b], starts[b + 1])]
            sums.append(sum((x for x, _ in pairs), np.zeros(L)))
            bounds.append(sum((x for _, x in pairs), np.zeros(L)) + 6 * 2 * U * sums[-1])
            w, e = weight_sums(qf[b], cache.values[b][:L], f64(lse[b]))
            total[b, :L] += w
            bound[b, :L] += e + 4 * U * total[b, :L]
        check(f64(out), lens, sums, bounds, None, 1.0, np.full(out.shape, 7.0))
        assert np.all(np.abs(f64(acc) - total) <= bound)
    assert m.get_device_error() == 0


def test_bad_pages_lengths_and_starts_are_reported(m):
    rng = np.random.default_rng(95)
    cache = RowCache(m, [random_rows(rng, 300), random_rows(rng, 300)], True, 96)
    q = random_q(rng, 4)
    qf = f64(q)
    lse = np.full((4, 128), 5.0, np.float32)
    ld = torch.from_numpy(lse).cuda()
    cache.table[0, 2] = 1 << 29
    got = f64(call(m, cache, q[:2].cuda(), ld[:2]))
    assert m.get_device_error() & m.DEVERR_BLOCK_RANGE
    vals = [v.copy() for v in cache.values]
    vals[0][128:192] = 0.0   # reads as zeros
    pairs = [weight_sums(qf[b], vals[b], lse[b].astype(float)) for b in range(2)]
    check(got, [300, 300], [x for x, _ in pairs], [x for _, x in pairs], None, 1.0, np.full(got.shape, 7.0))
    cache.table[0, 2] = cache.table[1, 0]
    for starts in ([0, 3, 2], [-1, 0, 2], [0, 2, 5], [2, 1, 2]):   # one good range at most
        out = f64(call(m, cache, q.cuda(), ld, None, 1.0, None, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       torch.full((4,), 300, dtype=torch.int32, device="cuda")))
        assert m.get_device_error() & m.DEVERR_SEQLEN_RANGE
        for b in range(2):
            if not 0 <= starts[b] < starts[b + 1] <= 4:
                assert np.all(out[b, :300] == 0)
    cache.seq_lens.copy_(torch.tensor([-1, 10 ** 6], dtype=torch.int32))
    cache.table.copy_(torch.from_numpy(cache.full_table))
    out = call(m, cache, q[:2].cuda(), ld[:2])
    assert m.get_device_error() & m.DEVERR_SEQLEN_RANGE
    assert torch.all(out[0] == 7.0) and not torch.any(out[1] == 7.0)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_bounded_conversation(m, fp8, paged):
    """A prompt observed by its last rows, its cache cut to 96 tokens, then decode steps that append, attend
    and accumulate, with a second cut on the way: followed by an oracle that holds the same rows."""
    rng = np.random.default_rng(101)
    lens, keep, sinks, recent = [300, 150], 96, 4, 24
    cache = RowCache(m, [random_rows(rng, L) for L in lens], paged, 102, fp8=fp8, max_len=320)
    if paged:
        cache.table.copy_(torch.from_numpy(cache.full_table))
    cap, B = cache.capacity, 2
    acc = torch.zeros((B, cap), device="cuda")
    kept = torch.zeros((B, keep), dtype=torch.int32, device="cuda")
    ews = torch.empty((m.evict_workspace_size(B, keep),), dtype=torch.uint8, device="cuda")
    dws = torch.empty((m.decode_workspace_size(B, cap),), dtype=torch.uint8, device="cuda")
    true_len = list(lens)
    rows = [v.copy() for v in cache.values]

    def evict():
        before = f64(acc)
        kw = dict(keep=keep, sinks=sinks, recent=recent, block_table=cache.table)
        if fp8:
            m.cache_evict_fp8(cache.data, cache.scales, cache.seq_lens, acc, cache.desc, kept, cache.seq_lens, acc, ews,
                              **kw)
        else:
            m.cache_evict(cache.data, cache.seq_lens, acc, cache.desc, kept, cache.seq_lens, acc, ews, **kw)
        for b in range(B):
            t = oracle.evict_keep(before[b], len(rows[b]), keep, sinks, recent)
            assert kept[b, :len(t)].tolist() == list(t)
            rows[b] = rows[b][t]
        assert cache.seq_lens.tolist() == [len(r) for r in rows]

    def step():
        n = B
        q = random_q(rng, n)
        c = torch.from_numpy(rng.standard_normal((n, 512))).to(torch.bfloat16)
        kr = torch.from_numpy(rng.standard_normal((n, 64))).to(torch.bfloat16)
        pos = torch.tensor(true_len, dtype=torch.int32, device="cuda")
        slots = cache.seq_lens.clone()
        kw = dict(block_table=cache.table)
        if fp8:
            m.cache_append_at_fp8(c.cuda(), kr.cuda(), pos, slots, cache.data, cache.scales, cache.desc, **kw)
        else:
            m.cache_append_at(c.cuda(), kr.cuda(), pos, slots, cache.data, cache.desc, **kw)
        cache.seq_lens.add_(1)
        out = torch.empty((n, 128, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((n, 128), device="cuda")
        before = f64(acc)
        if fp8:
            m.decode_attn_fp8(q.cuda(), cache.data, cache.scales, cache.seq_lens, cache.desc, dws, out, lse=lse, **kw)
            m.attn_weights_fp8(q.cuda(), cache.data, cache.scales, cache.seq_lens, cache.desc, lse, acc, prev=acc, **kw)
        else:
            m.decode_attn(q.cuda(), cache.data, cache.seq_lens, cache.desc, dws, out, lse=lse, **kw)
            m.attn_weights(q.cuda(), cache.data, cache.seq_lens, cache.desc, lse, acc, prev=acc, **kw)
        for b in range(B):
            if fp8:
                codes, sc = oracle.fp8_cache_rows(f64(c[b:b + 1]), f64(kr[b:b + 1]), np.array([true_len[b]]))
                new = oracle.dequantize_rows(codes, sc)
            else:   # the row as the cache holds it (its rounding is the append's own test)
                at = cache.rows_of(b, np.array([len(rows[b])]))
                new = f64(cache.data[at.cuda()])
                exact = oracle.cache_rows(f64(c[b:b + 1]), f64(kr[b:b + 1]), np.array([true_len[b]]))
                assert np.all(np.abs(new - exact) <= 2.0 ** -8 * np.abs(exact) + 1e-30)
            rows[b] = np.concatenate([rows[b], new])
            true_len[b] += 1
            w, e = weight_sums(f64(q[b]), rows[b], f64(lse[b]))
            L = len(rows[b])
            want = before[b, :L] + w
            assert np.all(np.abs(f64(acc)[b, :L] - want) <= e + 4 * U * want)
            assert np.all(f64(acc)[b, L:] == 0)

    if not fp8:   # the prompt's last 16 tokens observe it (FP8 has no chunk form: its first cut is by order)
        n = 16 * B
        q = random_q(rng, n)
        q_seq = np.repeat(np.arange(B), 16).astype(np.int32)
        q_len = np.concatenate([L - 15 + np.arange(16) for L in lens]).astype(np.int32)
        out = torch.empty((n, 128, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((n, 128), device="cuda")
        ws = torch.empty((m.decode_workspace_size(n, cap),), dtype=torch.uint8, device="cuda")
        m.prefill_attn(q.cuda(), cache.data, torch.from_numpy(q_seq).cuda(), torch.from_numpy(q_len).cuda(), cache.desc,
                       ws, out, lse=lse, block_table=cache.table)
        call(m, cache, q.cuda(), lse, acc, 1.0, acc, torch.tensor([0, 16, 32], dtype=torch.int32, device="cuda"),
             torch.from_numpy(q_len).cuda())
        want, err = np.zeros((B, cap)), np.zeros((B, cap))
        for i in range(n):
            w, e = weight_sums(f64(q[i]), rows[q_seq[i]][:q_len[i]], f64(lse[i]))
            want[q_seq[i], :q_len[i]] += w
            err[q_seq[i], :q_len[i]] += e + 16 * 2 * U * w
        assert np.all(np.abs(f64(acc) - want) <= err + 4 * U * want)
    evict()
    for _ in range(8):
        step()
    evict()
    for _ in range(3):
        step()
    assert m.get_device_error() == 0


@pytest.mark.parametrize("capacity", [1, 3, 8, 9, 16, 60])
@pytest.mark.parametrize("fp8", [False, True])
def test_caches_smaller_than_a_copy(m, fp8, capacity):
    """Buffers of fewer rows than the boxes that are copied from them."""
    for lens in ([capacity], [capacity, 0, (capacity + 1) // 2]):
        rng = np.random.default_rng(111)
        cache = RowCache(m, [random_rows(rng, L) for L in lens], False, 112, fp8=fp8, max_len=capacity, align=1)
        assert cache.capacity == capacity
        q = random_q(rng, len(lens))
        qf = f64(q)
        lse = np.stack([row_lse(qf[b], cache.values[b]) for b in range(len(lens))])
        got = call(m, cache, q.cuda(), torch.from_numpy(lse).cuda())
        assert m.get_device_error() == 0
        pairs = [weight_sums(qf[b], cache.values[b], lse[b].astype(float)) for b in range(len(lens))]
        check(f64(got), lens, [x for x, _ in pairs], [x for _, x in pairs], None, 1.0, np.full(got.shape, 7.0))
        if not fp8:
            n = len(lens)
            got = call(m, cache, q.cuda(), torch.from_numpy(lse).cuda(),
                       q_start=torch.arange(n + 1, dtype=torch.int32, device="cuda"), q_len=cache.seq_lens.clone())
            check(f64(got), lens, [x for x, _ in pairs], [x for _, x in pairs], None, 1.0, np.full(got.shape, 7.0))
