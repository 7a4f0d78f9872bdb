"""Helpers of the bounded-cache tests: caches filled with given rows, and error bounds.

Bounds, from the arithmetic of the kernels (u = 2^-24, half a step of fp32):
  * a score is 576 exact products of bf16 values summed in fp32; one step of fp32 (2u) per addition
    covers truncating accumulators: |ds| <= 576 * 2u * scale * sum |q_j row_j| =: ds;
  * a softmax weight: e^(ds from the score, ds from the log-sum-exp or maximum), and exp2 with its
    argument formed in fp32 of size <= 2^7: 2^7 * 2u + 2^-21 relative, together <= 2 ds + EXP;
  * out_lat: the weights' error times pc = sum_t p_t |c_t|, the weights' rounding to bf16 (half a
    step, 2^-8, relative) times pc, and the output's rounding to bf16, 2^-8 relative;
  * lse: ds plus the fp32 arithmetic around it, <= 2^-16;
  * a sum of weights e^(s - l): each term within ds, and the fp32 argument of exp2: the factor scale log2(e)
    within 3u, l log2(e) within 2u, the fused product within u, so (6u (|s| + |l|) log2(e)) ln 2 + 2^-21 of
    exp2 itself, relative; the additions of n terms within n * 2u of the sum.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

SCALE = 1.0 / 192 ** 0.5
U = 2.0 ** -24
EXP = 2.0 ** 7 * 2 * U + 2.0 ** -21


def score_err(sabs):
    return 576 * 2 * U * sabs


def assert_window_row(g_out, g_lse, ref):
    if np.all(np.isneginf(ref["lse"])):
        assert np.all(g_out == 0) and np.all(np.isneginf(g_lse))
        return
    ds = score_err(ref["sabs"])
    bound = 2.0 ** -8 * np.abs(ref["out_lat"]) + (2.0 ** -8 + 2 * ds + EXP)[:, None] * ref["pc"]
    err = np.abs(g_out - ref["out_lat"])
    assert np.all(err <= bound), f"{(err > bound).sum()} out of bound, worst excess {(err - bound).max():.3e}"
    lerr = np.abs(g_lse - ref["lse"])
    assert np.all(lerr <= ds + 2.0 ** -16), f"lse off by {lerr.max():.3e}"


def weight_sums(q, rows, lse, scale=SCALE):
    """(sum over heads of e^(s - lse) for each row, its error bound); q [H, 576], rows [L, 576], lse [H]."""
    s = scale * (q @ rows.T)
    l = np.where(np.isneginf(lse), np.inf, lse)[:, None]
    w = np.exp(s - l)
    rel = score_err(scale * (np.abs(q) @ np.abs(rows).T)) + 6 * U * (np.abs(s) + np.abs(np.where(np.isinf(l), 0, l))) + \
        2.0 ** -21
    return w.sum(axis=0), (w * rel).sum(axis=0) + len(q) * 2 * U * w.sum(axis=0) + 1e-35


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def random_rows(rng, n, size=1.0):
    """n cached rows of bf16 values, as a CPU tensor."""
    return (torch.from_numpy(rng.standard_normal((n, 576))) * size).to(torch.bfloat16)


def random_q(rng, n):
    q = rng.standard_normal((n, 128, 576))
    q[:, :, :512] *= 0.5
    return torch.from_numpy(q).to(torch.bfloat16)


class RowCache:
    """A cache holding the given rows ([L_b, 576] bf16 CPU tensors), in pages or contiguous; every row
    and block-table entry no sequence uses holds NaN / -1.  fp8: rows coded by their oracle form."""

    def __init__(self, m, seqs, paged, seed=0, max_len=None, fp8=False, device="cuda",
                 align=16):
        import oracle
        lens = [len(s) for s in seqs]
        B, L = len(seqs), max(max(lens + [1]) if max_len is None else max_len, 1)
        rng = np.random.default_rng(seed)
        if paged:
            width = (L + 63) // 64
            used = [(n + 63) // 64 for n in lens]
            blocks = B * width + 3
            perm = rng.permutation(blocks).astype(np.int32)
            table = np.full((B, width), -1, np.int32)
            for b in range(B):
                table[b, :used[b]] = perm[b * width:b * width + used[b]]
            self.full_table = perm[:B * width].reshape(B, width).copy()   # every page a sequence may grow into
            self.desc = m.paged_desc(B, width, blocks)
            rows, self.table = blocks * 64, torch.from_numpy(table)
        else:
            L = (L + align - 1) // align * align
            rows, self.table, self.desc = B * L, None, m.contiguous_desc(B, L)
        self.paged, self.stride, self.lens = paged, L, lens
        self.capacity = L if not paged else width * 64
        data = torch.full((rows, 576), float("nan"), dtype=torch.bfloat16)
        for b, s in enumerate(seqs):
            if len(s):
                data[self.rows_of(b, np.arange(len(s)))] = s
        self.values = [f64(s) for s in seqs]   # what attention sees
        self.scales = None
        if fp8:
            codes = np.full((rows, 576), 0x7F, np.uint8)   # E4M3 NaN
            scales = np.full((rows,), 127, np.uint8)
            for b, s in enumerate(seqs):
                if len(s):
                    c, sc = oracle.quantize_rows(f64(s))
                    idx = self.rows_of(b, np.arange(len(s))).numpy()
                    codes[idx], scales[idx] = c, (np.log2(sc) + 127).astype(np.uint8)
                    self.values[b] = oracle.dequantize_rows(c, sc)
            data, self.scales = torch.from_numpy(codes), torch.from_numpy(scales).to(device)
        self.data = data.to(device)
        if self.table is not None:
            self.table = self.table.to(device)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)

    def rows_of(self, b, t):
        t = np.asarray(t)
        if not self.paged:
            return torch.as_tensor(b * self.stride + t)
        table = self.table.cpu().numpy()
        return torch.as_tensor(table[b, t // 64].astype(np.int64) * 64 + t % 64)


class KernelNodeParams(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(graph):
    """The grids of the kernels of a captured graph."""
    cu = ctypes.CDLL("libcuda.so.1")
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    grids = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), KernelNodeParams()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:   # a kernel
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            grids.append(tuple(p.grid))
    return grids
