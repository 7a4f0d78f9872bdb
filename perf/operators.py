"""Cases of the bounded latent cache: attention with a sliding window and sinks, attention weights
accumulated per cached token, and eviction by those weights.

A cached row is [c (512) | rotated key (64)], bf16 or FP8 (E4M3 codes with an E8M0 scale byte per
row), in a contiguous cache or in 64-token pages.  A query row holds 128 heads of 576 values.

  window   out = softmax over the visible tokens (the first `sinks` and the last `window`) . c, and
           its log-sum-exp; one row per sequence, or the rows of a chunk of new tokens
  weights  decay * prev[t] + the sum over heads (and the chunk's rows) of token t's attention weight
  evict    the `sinks` first and `recent` last tokens and the heaviest others, `keep` in all, moved
           in order to the front of the same cache or into another one
"""
import math
import random

import torch

own = False

HEADS, LAT, ROW, PAGE = 128, 512, 576, 64
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # window: one short conversation on its own, where latency counts
        dict(name="window_one", op="window", batch=1, lo=256, hi=256, window=128, sinks=4, paged=False, fp8=False,
             rows=0, lens_seed=1),
        # the batch-128 paged workload with a window of odd size and one page of sinks
        dict(name="window_b128_paged", op="window", batch=128, lo=1024, hi=8192, window=2001, sinks=64, paged=True,
             fp8=False, rows=0, lens_seed=2),
        # four long documents, a window of a quarter of each
        dict(name="window_long", op="window", batch=4, lo=131072, hi=131072, window=32768, sinks=128, paged=False,
             fp8=False, rows=0, lens_seed=3),
        # an FP8 cache in pages, few sinks, a window that starts inside a page
        dict(name="window_fp8_paged", op="window", batch=128, lo=1024, hi=8192, window=1000, sinks=5, paged=True,
             fp8=True, rows=0, lens_seed=4),
        # a chunk of a prompt: 256 new tokens of each of four sequences, each row with its own window
        dict(name="window_chunk", op="window", batch=4, lo=1500, hi=2500, window=512, sinks=4, paged=True, fp8=False,
             rows=256, lens_seed=5),
        # weights: one short conversation, one new token
        dict(name="weights_one", op="weights", batch=1, lo=256, hi=256, paged=False, fp8=False, rows=0, decay=1.0,
             lens_seed=6),
        # one decode step of the batch-128 paged workload
        dict(name="weights_b128_paged", op="weights", batch=128, lo=1024, hi=8192, paged=True, fp8=False, rows=0,
             decay=1.0, lens_seed=7),
        # an FP8 cache, contiguous, older weights fading
        dict(name="weights_fp8_b32", op="weights", batch=32, lo=4000, hi=4096, paged=False, fp8=True, rows=0,
             decay=0.99, lens_seed=8),
        # the last 32 tokens of eight prompts observed before their caches are cut
        dict(name="weights_observed", op="weights", batch=8, lo=1024, hi=8192, paged=True, fp8=False, rows=32,
             decay=1.0, lens_seed=9),
        # evict: one short conversation
        dict(name="evict_one", op="evict", batch=1, lo=300, hi=300, keep=128, sinks=4, recent=32, paged=False,
             in_place=False, lens_seed=10),
        # prompts of the batch-128 workload cut into a smaller pool of pages
        dict(name="evict_b128_paged", op="evict", batch=128, lo=1024, hi=8192, keep=1024, sinks=4, recent=127,
             paged=True, in_place=False, lens_seed=11),
        # branches of 32 conversations: restored from their snapshots, then cut to half in place
        dict(name="evict_branch_b32", op="evict", batch=32, lo=3500, hi=4096, keep=2048, sinks=4, recent=256,
             paged=True, in_place=True, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "weights", "evict"])
    paged = rng.random() < 0.6
    fp8 = rng.random() < 0.3
    batch = _log_int(rng, 1, 128)
    hi = min(_log_int(rng, 64, 131072), 500000 // batch)
    in_place = rng.random() < 0.4
    if op == "evict" and in_place:   # the restored branch is written whole
        hi = min(hi, 250000 // batch)
    lo = 1 if rng.random() < 0.2 else max(1, int(hi * rng.uniform(0.1, 1.0)))
    case = dict(op=op, batch=batch, lo=lo, hi=hi, paged=paged, lens_seed=rng.randrange(1 << 30))
    chunk = rng.random() < 0.25
    if op == "evict":
        keep = min(_log_int(rng, 16, 8192), 200000 // batch)
        sinks = rng.randint(0, min(64, keep // 2))
        case.update(keep=keep, sinks=sinks, recent=rng.randint(0, (keep - sinks) // 2), in_place=in_place)
        return case
    rows = 0
    if chunk:   # a few sequences, several rows each, over caches of ordinary length
        fp8 = False
        batch = rng.randint(1, 4)
        hi = _log_int(rng, 64, 4096)
        rows = _log_int(rng, 2, 64)
        case.update(batch=batch, hi=hi, lo=max(1, hi // 2))
    case.update(fp8=fp8, rows=rows)
    if op == "window":
        case.update(window=_log_int(rng, 1, 32768), sinks=rng.choice([0, 1, 4, 5, 16, 63, 64, 65, 128]))
    else:
        case.update(decay=rng.choice([1.0, 0.9, 0.5]))
    return case


# ----------------------------------------------------------------------------- a case's geometry
def lengths(case):
    rng = random.Random(case["lens_seed"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def row_lengths(case):
    """Per query row: (its sequence, the tokens it may attend).  One row per sequence, or the chunk's
    rows: the last `rows` tokens of each sequence, each up to itself."""
    lens = lengths(case)
    if not case["rows"]:
        return [(b, L) for b, L in enumerate(lens)]
    return [(b, t + 1) for b, L in enumerate(lens) for t in range(max(0, L - case["rows"]), L)]


def _layout(gen, lens, paged, device, align=16):
    """(rows of the buffer, block table or None, tokens a sequence can hold) of a cache for lens."""
    if not paged:
        cap = (max(lens) + align - 1) // align * align
        return len(lens) * cap, None, cap
    pages = [(L + PAGE - 1) // PAGE for L in lens]
    perm = torch.randperm(sum(pages), generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=device)
    o = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[o:o + n]
        o += n
    return sum(pages) * PAGE, table, max(pages) * PAGE


def _random_rows(gen, rows, device):
    """Latent rows: N(0, 1) values, and a few tokens (1 in 64) of twice the size, which draw more attention."""
    data = torch.empty((rows, ROW), dtype=torch.bfloat16, device=device)
    for i in range(0, rows, 1 << 17):
        x = torch.randn((min(1 << 17, rows - i), ROW), generator=gen, device=device)
        x *= 1.0 + (torch.rand((x.shape[0], 1), generator=gen, device=device) < 1.0 / 64).float()
        data[i:i + x.shape[0]] = x.to(torch.bfloat16)
    return data


def _to_fp8(rows):
    """(codes, scale bytes): per row the power of two 2^k, k the smallest with amax <= 448 * 2^k."""
    codes = torch.empty(rows.shape, dtype=torch.uint8, device=rows.device)
    scales = torch.empty((rows.shape[0],), dtype=torch.uint8, device=rows.device)
    for i in range(0, rows.shape[0], 1 << 17):
        x = rows[i:i + (1 << 17)].double()
        k = torch.ceil(torch.log2(x.abs().amax(1).clamp_min(1e-30) / 448.0))
        codes[i:i + x.shape[0]] = (x * torch.exp2(-k)[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + x.shape[0]] = (k + 127).to(torch.uint8)
    return codes, scales


def _index(st, b, t):
    """Rows of the buffer that hold tokens t (a tensor) of sequence b."""
    if st["table"] is None:
        return b * st["cap"] + t
    return st["table"][b, t // PAGE].long() * PAGE + t % PAGE


def _values(st, idx, dtype):
    rows = st["cache"][idx]
    if st["scales"] is None:
        return rows.to(dtype)
    return rows.view(torch.float8_e4m3fn).to(dtype) * torch.exp2(st["scales"][idx].to(dtype) - 127)[:, None]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = lengths(case)
    st = dict(case=case, lens=lens)
    rows, st["table"], st["cap"] = _layout(gen, lens, case["paged"], dev)
    st["cache"], st["scales"] = _random_rows(gen, rows, dev), None
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] == "evict":
        _prepare_evict(st, gen, dev)
    else:
        if case["fp8"]:
            st["cache"], st["scales"] = _to_fp8(st["cache"])
        st["rows"] = row_lengths(case)
        n = len(st["rows"])
        # an absorbed query: latent part of variance 1/4 (N(0, 1) times N(0, 1/512) weights over 128), rotary part 1
        q = torch.randn((n, HEADS, ROW), generator=gen, device=dev)
        q[:, :, :LAT] *= 0.5
        st["q"] = q.to(torch.bfloat16)
        st["q_seq"] = torch.tensor([b for b, _ in st["rows"]], dtype=torch.int32, device=dev)
        st["q_len"] = torch.tensor([m for _, m in st["rows"]], dtype=torch.int32, device=dev)
        counts = [sum(1 for s, _ in st["rows"] if s == b) for b in range(case["batch"])] if case["rows"] else []
        st["q_start"] = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32, device=dev)
        st["out"] = torch.zeros((n, HEADS, LAT), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros((n, HEADS), dtype=torch.float32, device=dev)
        if case["op"] == "weights":   # the attention before this call left its log-sum-exp
            for i, s in _scores(st, torch.float32):
                st["lse"][i] = torch.logsumexp(s, 1)
            age = torch.rand((case["batch"], st["cap"]), generator=gen, device=dev)
            st["prev"] = 4.0 * age ** 4
            st["weights"] = torch.zeros_like(st["prev"])
    if own:
        _prepare_own(st, dev)
    return st


def _prepare_evict(st, gen, dev):
    case, B = st["case"], st["case"]["batch"]
    # accumulated weights: heavy-tailed, and some tokens (1 in 8) that nothing has looked at yet
    w = torch.exp(2.0 * torch.randn((B, st["cap"]), generator=gen, device=dev))
    st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.125, torch.zeros_like(w), w)
    st["kept"] = torch.zeros((B, case["keep"]), dtype=torch.int32, device=dev)
    st["lens_out"] = torch.zeros((B,), dtype=torch.int32, device=dev)
    if case["in_place"]:
        st["snapshot"] = st["cache"]
        st["cache"] = st["snapshot"].clone()
        st["cache_out"], st["table_out"], st["cap_out"] = st["cache"], st["table"], st["cap"]
    else:
        rows, st["table_out"], st["cap_out"] = _layout(gen, [case["keep"]] * B, case["paged"], dev)
        st["cache_out"] = torch.zeros((rows, ROW), dtype=torch.bfloat16, device=dev)
    st["weights_out"] = torch.zeros((B, st["cap_out"]), dtype=torch.float32, device=dev)


def _prepare_own(st, dev):
    import mla_latent_kv_20_b200 as m
    case, B = st["case"], st["case"]["batch"]
    st["m"] = m

    def desc(table, cap, rows):
        return m.contiguous_desc(B, cap) if table is None else m.paged_desc(B, table.shape[1], rows // PAGE)

    st["desc"] = desc(st["table"], st["cap"], st["cache"].shape[0])
    if case["op"] == "evict":
        st["desc_out"] = desc(st["table_out"], st["cap_out"], st["cache_out"].shape[0])
        nbytes = m.evict_workspace_size(B, case["keep"])
    elif case["op"] == "window":
        nbytes = m.decode_workspace_size(len(st["rows"]), m.window_span(st["cap"], case["window"], case["sinks"]))
    else:
        nbytes = m.prefill_attn_weights_workspace_size(B, st["cap"], len(st["rows"])) if case["rows"] else 0
    st["workspace"] = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=dev)


# ----------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if case["op"] == "window":
        return _window_own(st) if own else _window(st)
    if case["op"] == "weights":
        return _weights_own(st) if own else _weights(st)
    if case["in_place"]:
        st["cache"].copy_(st["snapshot"])
    return _evict_own(st) if own else _evict(st)


def _window_own(st):
    m, case = st["m"], st["case"]
    kw = dict(window=case["window"], sinks=case["sinks"], lse=st["lse"], block_table=st["table"], softmax_scale=SCALE)
    if case["rows"]:
        m.prefill_attn_window(st["q"], st["cache"], st["q_seq"], st["q_len"], st["desc"], st["workspace"], st["out"],
                              **kw)
    elif case["fp8"]:
        m.decode_attn_window_fp8(st["q"], st["cache"], st["scales"], st["seq_lens"], st["desc"], st["workspace"],
                                 st["out"], **kw)
    else:
        m.decode_attn_window(st["q"], st["cache"], st["seq_lens"], st["desc"], st["workspace"], st["out"], **kw)
    return st["out"], st["lse"]


def _weights_own(st):
    m, case = st["m"], st["case"]
    kw = dict(prev=st["prev"], decay=case["decay"], block_table=st["table"], softmax_scale=SCALE)
    if case["rows"]:
        m.prefill_attn_weights(st["q"], st["cache"], st["seq_lens"], st["q_start"], st["q_len"], st["desc"], st["lse"],
                               st["workspace"], st["weights"], **kw)
    elif case["fp8"]:
        m.attn_weights_fp8(st["q"], st["cache"], st["scales"], st["seq_lens"], st["desc"], st["lse"], st["weights"],
                           **kw)
    else:
        m.attn_weights(st["q"], st["cache"], st["seq_lens"], st["desc"], st["lse"], st["weights"], **kw)
    return st["weights"]


def _evict_own(st):
    m, case = st["m"], st["case"]
    m.cache_evict(st["cache"], st["seq_lens"], st["weights"], st["desc"], st["kept"], st["lens_out"], st["weights_out"],
                  st["workspace"], keep=case["keep"], sinks=case["sinks"], recent=case["recent"],
                  block_table=st["table"], cache_out=st["cache_out"], desc_out=st["desc_out"],
                  block_table_out=st["table_out"])
    return st["cache_out"], st["weights_out"], st["lens_out"], st["kept"]


# ----------------------------------------------------------------------------- the plain forms
def _visible(L, window, sinks, dev):
    start = max(L - window, 0)
    return torch.cat([torch.arange(0, min(sinks, start), device=dev), torch.arange(start, L, device=dev)])


def _window(st):
    case, out, lse = st["case"], st["out"], st["lse"]
    for i, (b, L) in enumerate(st["rows"]):
        t = _visible(L, case["window"], case["sinks"], out.device)
        rows = _values(st, _index(st, b, t), torch.float32)
        s = SCALE * (st["q"][i].float() @ rows.T)
        top = s.amax(1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(1, keepdim=True)
        out[i] = (p @ rows[:, :LAT] / total).to(torch.bfloat16)
        lse[i] = (top + torch.log(total))[:, 0]
    return out, lse


def _scores(st, dtype):
    """Per query row i: its scores [heads, tokens it may attend]."""
    held, rows = -1, None
    for i, (b, L) in enumerate(st["rows"]):
        if b != held:
            held = b
            rows = _values(st, _index(st, b, torch.arange(st["lens"][b], device=st["q"].device)), dtype)
        yield i, SCALE * (st["q"][i].to(dtype) @ rows[:L].T)


def _weights(st):
    out = st["weights"]
    for b, L in enumerate(st["lens"]):
        out[b, :L] = st["case"]["decay"] * st["prev"][b, :L]
    for i, s in _scores(st, torch.float32):
        b, L = st["rows"][i]
        out[b, :L] += torch.exp(s - st["lse"][i][:, None]).sum(0)
    return out


def _evict(st):
    case, dev = st["case"], st["cache"].device
    keep, sinks, recent = case["keep"], case["sinks"], case["recent"]
    for b, L in enumerate(st["lens"]):
        n = min(L, keep)
        if L <= keep:
            t = torch.arange(L, device=dev)
        else:
            middle = st["weights"][b, sinks:L - recent]
            heavy = torch.sort(middle, descending=True, stable=True).indices[:keep - sinks - recent] + sinks
            t = torch.cat([torch.arange(sinks, device=dev), torch.sort(heavy).values,
                           torch.arange(L - recent, L, device=dev)])
        moved = st["cache"][_index(st, b, t)]
        slots = torch.arange(n, device=dev)
        if st["table_out"] is None:
            st["cache_out"][b * st["cap_out"] + slots] = moved
        else:
            st["cache_out"][st["table_out"][b, slots // PAGE].long() * PAGE + slots % PAGE] = moved
        st["weights_out"][b, :n] = st["weights"][b, t]
        st["weights_out"][b, n:min(L, st["cap_out"])] = 0.0
        st["kept"][b, :n] = t.to(torch.int32)
        st["kept"][b, n:] = -1
        st["lens_out"][b] = n
    return st["cache_out"], st["weights_out"], st["lens_out"], st["kept"]


# ----------------------------------------------------------------------------- work and exact values
def work(case):
    lens = lengths(case)
    row_bytes = 2 * ROW if not case.get("fp8") else ROW + 1
    if case["op"] == "evict":
        n = [min(L, case["keep"]) for L in lens]
        cached = sum(n)
        if case["in_place"]:   # the snapshot read and the branch written, whole
            cached = sum((L + PAGE - 1) // PAGE * PAGE for L in lens) if case["paged"] else \
                len(lens) * ((max(lens) + 15) // 16 * 16)
        return dict(bytes=2 * row_bytes * cached + 4 * sum(lens) + 8 * sum(n) + 8 * len(lens), flops=0)
    rows = row_lengths(case)
    if case["op"] == "window":
        seen = [set() for _ in lens]
        pairs = 0
        for b, L in rows:
            start = max(L - case["window"], 0)
            spans = ((0, min(case["sinks"], start)), (start, L))
            pairs += sum(e - s for s, e in spans)
            seen[b].update(spans)
        tokens = 0
        for spans in seen:   # tokens of a sequence that any of its rows sees
            end = 0
            for s, e in sorted(spans):
                tokens += max(0, e - max(s, end))
                end = max(end, e)
        return dict(bytes=tokens * row_bytes + len(rows) * HEADS * (2 * ROW + 2 * LAT + 4),
                    flops=2 * HEADS * (ROW + LAT) * pairs)
    pairs = sum(L for _, L in rows)
    return dict(bytes=sum(lens) * (row_bytes + 8) + len(rows) * HEADS * (2 * ROW + 4), flops=2 * HEADS * ROW * pairs)


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["cache"].device
    if case["op"] == "window":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=dev)
        for i, s in _scores(st, torch.float64):
            b, L = st["rows"][i]
            t = torch.arange(L, device=dev)
            hidden = (t >= case["sinks"]) & (t < L - case["window"])
            s = s.masked_fill(hidden[None, :], -math.inf)
            lse[i] = torch.logsumexp(s, 1)
            out[i] = torch.exp(s - lse[i][:, None]) @ _values(st, _index(st, b, t), torch.float64)[:, :LAT]
        return out, lse
    if case["op"] == "weights":
        out = torch.zeros(st["weights"].shape, dtype=torch.float64, device=dev)
        for i, s in _scores(st, torch.float64):
            b, L = st["rows"][i]
            out[b, :L] += (s - st["lse"][i].double()[:, None]).exp().sum(0)
        for b, L in enumerate(st["lens"]):
            out[b, :L] += case["decay"] * st["prev"][b, :L].double()
        return out
    return _exact_evict(st)


def _exact_evict(st):
    case = st["case"]
    keep, sinks, recent = case["keep"], case["sinks"], case["recent"]
    w_in, table = st["weights"].double().cpu().tolist(), None if st["table"] is None else st["table"].cpu().tolist()
    table_out = None if st["table_out"] is None else st["table_out"].cpu().tolist()

    def row(tab, cap, b, t):
        return b * cap + t if tab is None else tab[b][t // PAGE] * PAGE + t % PAGE

    weights = torch.zeros(st["weights_out"].shape, dtype=torch.float64)
    kept = torch.full(st["kept"].shape, -1, dtype=torch.int32)
    src, dst = [], []
    for b, L in enumerate(st["lens"]):
        tokens = list(range(L))
        if L > keep:
            order = sorted(range(sinks, L - recent), key=lambda t: (-w_in[b][t], t))
            tokens = sorted(list(range(sinks)) + order[:keep - sinks - recent] + list(range(L - recent, L)))
        for j, t in enumerate(tokens):
            weights[b, j] = w_in[b][t]
            kept[b, j] = t
            src.append(row(table, st["cap"], b, t))
            dst.append(row(table_out, st["cap_out"], b, j))
    cache = st["cache_out"].clone()
    dev = cache.device
    cache[torch.tensor(dst, device=dev)] = st["cache"][torch.tensor(src, device=dev)]
    lens = torch.tensor([min(L, keep) for L in st["lens"]], dtype=torch.int32)
    return cache.double(), weights.to(dev), lens.to(dev), kept.to(dev)
