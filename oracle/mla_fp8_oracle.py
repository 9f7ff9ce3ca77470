"""CPU oracle for the 8-bit paged latent KV cache and the attention over it.

TEST INFRASTRUCTURE ONLY, like the other oracles: it shares no code with the CUDA
library and never reads a value the library produced.

The cache holds e4m3fn codes [pages, page_size, 1, 576] and one fp32 scale per page
(value = code * scale), the page table is the MLA decode call's. Definitions:
  * the scale of a set of rows: 0 if every finite entry is 0, else the smallest power of
    two s >= 2^-110 with |x| <= 448 s for all finite entries x;
  * append: sequence b's new rows are the last n_b of its L_b tokens, in the pages the
    table gives them. A page written from its first slot has no earlier contents; any
    other page keeps its earlier rows and its scale only grows. Where it grows, an earlier
    code c becomes e4m3(c * old / new); a new row's entry x becomes e4m3(x / scale) (x
    itself where the scale is 0), saturating, NaN staying NaN;
  * gather: bf16(code * scale) of a sequence's first tokens;
  * attention: query i of a sequence's n sees its first L - n + i + 1 tokens; softmax of
    sm_scale <q, k> (soft-capped), values the first 512 entries; no token: o = 0, lse = -inf.
Attention is in fp64 on the exact values. Pinned by tests/test_oracle_mla_fp8.py.
"""
from __future__ import annotations

import math

import torch

from oracle.fp8moe_oracle import bf16_round, e4m3_decode, e4m3_encode

F64 = torch.float64


def scale_of(x: torch.Tensor) -> float:
    """The scale of the rows x: found by trying every power of two from the smallest on."""
    x = x.to(F64)
    finite = x[torch.isfinite(x)].abs()
    amax = float(finite.max()) if finite.numel() else 0.0
    if amax == 0.0:
        return 0.0
    e = -110
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def codes_of(x: torch.Tensor) -> torch.Tensor:
    """The nearest codes of the fp64 values x, ties to even, saturating; NaN stays NaN."""
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    step = torch.exp2((torch.frexp(finite)[1] - 1).clamp(min=-6).to(F64) - 3)
    return e4m3_encode(torch.where(torch.isfinite(x), torch.round(finite / step) * step, x))


def lengths(kv_indptr, kv_last_page_lens, page_size: int) -> list[int]:
    out = []
    for b in range(len(kv_last_page_lens)):
        n = int(kv_indptr[b + 1]) - int(kv_indptr[b])
        out.append(0 if n == 0 else (n - 1) * page_size + int(kv_last_page_lens[b]))
    return out


def append(kv_new, append_indptr, codes, scales, kv_indptr, kv_indices, kv_last_page_lens):
    """(codes uint8, scales fp32) after the append; codes uint8 [pages, ps, 1, 576] is the cache before."""
    codes, scales = codes.clone(), scales.clone()
    ps = codes.shape[1]
    for b, L in enumerate(lengths(kv_indptr, kv_last_page_lens, ps)):
        r0, r1 = int(append_indptr[b]), int(append_indptr[b + 1])
        start = L - (r1 - r0)
        pos = start
        while pos < L:
            j = pos // ps
            end = min(L, (j + 1) * ps)
            page = int(kv_indices[int(kv_indptr[b]) + j])
            rows = kv_new[r0 + pos - start:r0 + end - start].float()
            slot = pos - j * ps
            old = float(scales[page, 0]) if slot > 0 else 0.0
            s = max(old, scale_of(rows))
            if slot > 0 and old < s:
                codes[page, :slot, 0] = codes_of(e4m3_decode(codes[page, :slot, 0]).to(F64) * old / s)
            codes[page, slot:slot + rows.shape[0], 0] = codes_of(rows.to(F64) / s if s > 0 else rows.to(F64))
            scales[page, 0] = s
            pos = end
    return codes, scales


def sequence_values(codes, scales, kv_indptr, kv_indices, b: int, upto: int) -> torch.Tensor:
    """fp64 values [upto, 576] of the first tokens of sequence b."""
    ps = codes.shape[1]
    lo = int(kv_indptr[b])
    rows = []
    for i in range(upto):
        page = int(kv_indices[lo + i // ps])
        rows.append(e4m3_decode(codes[page, i % ps, 0]) * float(scales[page, 0]))
    return torch.stack(rows) if rows else torch.zeros(0, codes.shape[-1], dtype=F64)


def gather(codes, scales, kv_indptr, kv_indices, out_indptr, out):
    """out (bf16, its other rows kept) with the sequences' first tokens, each rounded once."""
    out = out.clone()
    for b in range(len(out_indptr) - 1):
        lo, hi = int(out_indptr[b]), int(out_indptr[b + 1])
        if hi > lo:
            out[lo:hi] = bf16_round(sequence_values(codes, scales, kv_indptr, kv_indices, b, hi - lo)).to(torch.bfloat16)
    return out


def extend(q, qo_indptr, codes, scales, kv_indptr, kv_indices, kv_last_page_lens, sm_scale=None, logit_cap=0.0):
    """o [T, H, 512], lse [T, H], and for error bounds mag = sum_j p_j |v_j| [T, H, 512], size =
    max_j sm_scale * <|q|, |k_j|> [T, H] and coded = max_j (p_j s_j) sum_j |v_j / s_j| [T, H, 512]
    (s_j the scale of token j's page); fp64. Rows of no sequence are NaN."""
    T, H, Dk = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(Dk)
    o = torch.full((T, H, 512), math.nan, dtype=F64)
    lse = torch.full((T, H), math.nan, dtype=F64)
    mag, size, coded = torch.zeros_like(o), torch.zeros_like(lse), torch.zeros_like(o)
    for b, L in enumerate(lengths(kv_indptr, kv_last_page_lens, codes.shape[1])):
        lo, hi = int(qo_indptr[b]), int(qo_indptr[b + 1])
        if hi == lo:
            continue
        kv = sequence_values(codes, scales, kv_indptr, kv_indices, b, L)
        first, ps = int(kv_indptr[b]), codes.shape[1]
        pages = [int(kv_indices[first + i // ps]) for i in range(L)]
        sc = scales[pages, 0].to(F64)
        sums = e4m3_decode(codes[pages, [i % ps for i in range(L)], 0, :512]).to(F64).abs().cumsum(0)
        for i in range(hi - lo):
            sees = max(0, L - (hi - lo) + i + 1)
            t = lo + i
            if sees == 0:
                o[t], lse[t] = 0.0, -math.inf
                continue
            k = kv[:sees]
            s = sm_scale * (q[t].to(F64) @ k.T)
            if logit_cap > 0:
                s = logit_cap * torch.tanh(s / logit_cap)
            m = s.max(dim=1, keepdim=True).values
            e = torch.exp(s - m)
            den = e.sum(1, keepdim=True)
            o[t] = (e / den) @ k[:, :512]
            mag[t] = (e / den) @ k[:, :512].abs()
            lse[t] = m[:, 0] + torch.log(den[:, 0])
            coded[t] = (e / den * sc[:sees]).max(dim=1, keepdim=True).values * sums[sees - 1]
            size[t] = sm_scale * (q[t].to(F64).abs() @ k.abs().T).max(1).values
    return o, lse, mag, size, coded


def decode(q, codes, scales, kv_indptr, kv_indices, kv_last_page_lens, sm_scale=None, logit_cap=0.0):
    return extend(q, torch.arange(q.shape[0] + 1), codes, scales, kv_indptr, kv_indices, kv_last_page_lens, sm_scale,
                  logit_cap)
