"""The operators on an 8-bit paged latent KV cache, as cases to measure: appending tokens to it, reading
tokens back from it, attention of one decode step over it and attention of several new tokens per
sequence over it (multi-head latent attention, 576-wide keys whose first 512 entries are the values).

The cache is float8_e4m3fn [pages, page_size, 1, 576] with one fp32 scale per page and KV head
([pages, 1]); a stored value is code * scale. Scales are powers of two, the smallest one with which no
finite value of the page exceeds 448. The page table is kv_indptr / kv_indices / kv_last_page_lens.

`run` computes each operator in its plain form with elementary torch operations, or (`own`) by the calls a
user makes of the package. `exact` gives the definition in 64 bits.
"""
import math

import torch

own = False

DK, DV = 576, 512
DEV = "cuda"
BIG = 448.0           # the largest e4m3fn value


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's write: a new token for each of 64 sequences around 544 tokens
        dict(name="append_step_b64", op="append", B=64, L=544, spread=60, n=1, n_spread=0, page=64),
        # the write of a prefill batch: eight whole prompts, about 4096 tokens, ragged
        dict(name="append_prompt_t4096", op="append", B=8, L=600, spread=177, n=600, n_spread=177, page=64),
        # chunks of about 16K tokens written behind prefixes that end inside a page
        dict(name="append_chunk_t16k", op="append", B=12, L=4000, spread=333, n=1500, n_spread=211, page=16),
        # cached prefixes read back for the up-projection of a short prompt's keys and values
        dict(name="gather_prefix_b8", op="gather", B=8, L=500, spread=123, page=16),
        # the same for 32 long prefixes
        dict(name="gather_long_b32", op="gather", B=32, L=4096, spread=1001, page=64),
        # a single user's short context on a tensor-parallel rank's 16 heads, a page per token
        dict(name="decode_b1_h16_l97", op="decode", B=1, H=16, L=97, spread=0, page=1),
        # the decode batch of 64 sequences of about 544 tokens on 16 heads
        dict(name="decode_b64_h16_l544", op="decode", B=64, H=16, L=544, spread=60, page=64),
        # the same batch at an 8K context
        dict(name="decode_b64_h16_l8192", op="decode", B=64, H=16, L=8192, spread=300, page=64),
        # data-parallel attention: all 128 heads on one GPU, ragged contexts
        dict(name="decode_b24_h128_l4096", op="decode", B=24, H=128, L=4096, spread=1500, page=64),
        # checking one drafted token: two query tokens per sequence
        dict(name="extend_b64_q2_h16", op="extend", B=64, H=16, L=546, spread=60, n=2, n_spread=0, page=64),
        # a chunk of about 500 prompt tokens behind a cached prefix
        dict(name="extend_b4_q500_h16", op="extend", B=4, H=16, L=2000, spread=401, n=500, n_spread=77, page=64),
        # short questions after a long shared document, all 128 heads
        dict(name="extend_b5_q33_h128", op="extend", B=5, H=128, L=3001, spread=999, n=33, n_spread=9, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "extend", "extend"])
    page = rng.choice([1, 7, 16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 200)
        n = _log(rng, 1, max(1, 16000 // B))
        L = n + (0 if rng.random() < 0.3 else _log(rng, 1, 2000))
        return dict(op=op, B=B, L=L, spread=rng.randint(0, max(0, L - n) // 2), n=n, n_spread=rng.randint(0, n // 3), page=page)
    if op == "gather":
        B = _log(rng, 1, 64)
        L = _log(rng, 1, max(2, 100000 // B))
        return dict(op=op, B=B, L=L, spread=rng.randint(0, L // 2), page=page)
    if op == "decode":
        H = rng.choice([8, 16, 16, 32, 64, 128])
        B = _log(rng, 1, 128)
        L = _log(rng, 1, max(2, 64 * 8192 * 16 // (B * max(H, 16))))
        return dict(op=op, B=B, H=H, L=L, spread=rng.randint(0, L // 2), page=page)
    H = rng.choice([8, 16, 16, 32, 64, 128])
    B = _log(rng, 1, 32)
    n = _log(rng, 1, max(2, 32000 // (B * H)))
    L = n + _log(rng, 1, 2500)
    return dict(op=op, B=B, H=H, L=L, spread=rng.randint(0, (L - n) // 2), n=n, n_spread=rng.randint(0, n // 3), page=page)


def _lengths(case):
    """Tokens in the cache of each sequence (the new ones among them), and new tokens of each."""
    B, spread = case["B"], case["spread"]
    total = [max(1, case["L"] - (b * 7919 + 13 * (b % 5)) % (spread + 1)) for b in range(B)]
    new = [0] * B
    if "n" in case:
        new = [max(1, case["n"] - (b * 104729) % (case["n_spread"] + 1)) for b in range(B)]
        if case["L"] == case["n"]:
            total = new                   # whole prompts
        total = [max(t, n) for t, n in zip(total, new)]
    return total, new


def work(case):
    total, new = _lengths(case)
    page, op = case["page"], case["op"]
    cached, fresh = sum(total), sum(new)
    if op == "append":
        pages = sum((t - 1) // page - (t - n) // page + 1 for t, n in zip(total, new))
        return {"bytes": fresh * DK * 3 + pages * 4, "flops": fresh * DK * 2}
    if op == "gather":
        return {"bytes": cached * DK * 3, "flops": cached * DK}
    H = case["H"]
    tables = 4 * sum(-(-t // page) * 2 for t in total)      # page indices and scales
    if op == "decode":
        rows, pairs = case["B"], cached
    else:
        rows, pairs = fresh, sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(total, new))
    return {"bytes": cached * DK + tables + rows * H * (2 * DK + 2 * DV + 4), "flops": 2 * H * pairs * (DK + DV)}


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-110; 0 where amax is 0."""
    m, e = torch.frexp(amax)              # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-110)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _rows(n, g):
    """Latent rows as a layer makes them: a normalised latent whose size varies a little from token to
    token, and a rotary part of larger entries; bf16."""
    x = torch.randn(n, DK, generator=g, device=DEV)
    x *= torch.exp(0.25 * torch.randn(n, 1, generator=g, device=DEV))
    x[:, DV:] *= 3.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    total, new = _lengths(case)
    page, B = case["page"], case["B"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    counts = [-(-t // page) for t in total]
    used = sum(counts)
    n_pages = used + 3                    # a few pages that no sequence lists
    # earlier contents of every page, quantised page by page
    chunk = max(1, 65536 // page)
    codes, scales = [], []
    for p in range(0, n_pages, chunk):
        k = min(chunk, n_pages - p)
        x = _rows(k * page, g).float().view(k, page * DK)
        s = _pow2_scale(x.abs().amax(1))
        codes.append((x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
    kv_cache = torch.cat(codes).view(torch.float8_e4m3fn).view(n_pages, page, 1, DK)
    kv_scale = torch.cat(scales).view(n_pages, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    indptr = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), **i32)
    order = torch.randperm(n_pages, generator=g, device=DEV)[:used].to(torch.int32)
    last = torch.tensor([t - (c - 1) * page for t, c in zip(total, counts)], **i32)
    s = dict(op=case["op"], kv_cache=kv_cache, kv_scale=kv_scale, kv_indptr=indptr, kv_indices=order,
             kv_last_page_lens=last, max_len=max(total), max_new=max(new), page=page)
    fresh = sum(new)
    if fresh:
        s["new_indptr"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), **i32)
    if case["op"] == "append":
        s["kv_new"] = _rows(fresh, g)
    elif case["op"] == "gather":
        s["out_indptr"] = torch.tensor([0] + torch.tensor(total).cumsum(0).tolist(), **i32)
        s["out"] = torch.empty(sum(total), DK, dtype=torch.bfloat16, device=DEV)
    else:
        rows = fresh or B
        s["q"] = torch.randn(rows, case["H"], DK, generator=g, device=DEV).to(torch.bfloat16)
        s["o"] = torch.empty(rows, case["H"], DV, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(rows, case["H"], dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_attention,
            "extend": _plain_attention}[s["op"]](s)


def _run_own(s):
    from fp8_block_scaled_biased_b200 import binding as K
    table = (s["kv_indptr"], s["kv_indices"], s["kv_last_page_lens"])
    if s["op"] == "append":
        K.mla_kv_append_fp8(s["kv_new"], s["new_indptr"], s["kv_cache"], s["kv_scale"], *table)
        return {"kv_cache": s["kv_cache"], "kv_scale": s["kv_scale"]}
    if s["op"] == "gather":
        return K.mla_kv_gather_fp8(s["kv_cache"], s["kv_scale"], *table, s["out_indptr"], s["out"])
    if s["op"] == "decode":
        K.mla_decode_fp8_fwd(s["q"], s["kv_cache"], s["kv_scale"], s["o"], *table, lse=s["lse"])
    else:
        K.mla_extend_fp8_fwd(s["q"], s["new_indptr"], s["kv_cache"], s["kv_scale"], s["o"], *table, lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def _table_lengths(s):
    n = s["kv_indptr"][1:] - s["kv_indptr"][:-1]
    return torch.where(n > 0, (n - 1) * s["page"] + s["kv_last_page_lens"], 0).long()


def _token_pages(s, b, pos):
    """The page of position `pos` of sequence `b` (positions past the end: some page of the buffer)."""
    at = s["kv_indptr"].long()[b] + pos // s["page"]
    return s["kv_indices"].long()[at.clamp(max=s["kv_indices"].numel() - 1)]


def _of_indptr(indptr, rows):
    """The sequence of each of the rows 0..rows-1, and its place among that sequence's rows."""
    t = torch.arange(rows, device=DEV)
    b = torch.searchsorted(indptr[1:].long(), t, right=True)
    return b, t - indptr.long()[b]


def _values(s, page, slot):
    """fp32 values of the cache's rows (page, slot)."""
    codes = s["kv_cache"].view(torch.uint8).view(-1, DK)[page * s["page"] + slot]
    return codes.view(torch.float8_e4m3fn).float() * s["kv_scale"][page]


def _plain_append(s):
    page_size, cache, scale = s["page"], s["kv_cache"], s["kv_scale"]
    x = s["kv_new"].float()
    b, i = _of_indptr(s["new_indptr"], x.shape[0])
    count = (s["new_indptr"][1:] - s["new_indptr"][:-1]).long()
    start = _table_lengths(s) - count                       # tokens each sequence held before
    pos = start[b] + i
    page, slot = _token_pages(s, b, pos), pos % page_size
    finite = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(1)
    amax = torch.zeros(scale.shape[0], device=DEV).scatter_reduce(0, page, finite, "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV).index_fill(0, page, True)
    first = torch.full((scale.shape[0],), page_size, device=DEV).scatter_reduce(0, page, slot, "amin")
    old = torch.where(first == 0, 0.0, scale[:, 0])         # a page written from its first slot starts afresh
    grown = torch.where(touched, torch.maximum(old, _pow2_scale(amax)), scale[:, 0])
    # the rows that a sequence's first page held before, in the page's new scale
    flat = cache.view(torch.uint8).view(-1, DK)
    head = _token_pages(s, torch.arange(start.numel(), device=DEV), start)
    rows = head[:, None] * page_size + torch.arange(page_size, device=DEV)
    keep = (count > 0)[:, None] & (torch.arange(page_size, device=DEV) < (start % page_size)[:, None])
    ratio = torch.where(grown[head] > 0, old[head] / grown[head], 0.0)
    again = (flat[rows].view(torch.float8_e4m3fn).float() * ratio[:, None, None]).to(torch.float8_e4m3fn)
    flat[rows] = torch.where(keep[:, :, None], again.view(torch.uint8), flat[rows])
    g = grown[page][:, None]
    code = torch.where(g > 0, x / g, x).clamp(-BIG, BIG)
    flat[page * page_size + slot] = code.to(torch.float8_e4m3fn).view(torch.uint8)
    scale[:, 0] = grown
    return {"kv_cache": cache, "kv_scale": scale}


def _plain_gather(s):
    b, pos = _of_indptr(s["out_indptr"], s["out"].shape[0])
    s["out"].copy_(_values(s, _token_pages(s, b, pos), pos % s["page"]))
    return s["out"]


def _plain_attention(s):
    """Sequences padded to the longest; query token i of n sees the first L - n + i + 1 tokens."""
    q, page_size = s["q"], s["page"]
    H, L = q.shape[1], _table_lengths(s)
    B = L.numel()
    pos = torch.arange(s["max_len"], device=DEV)
    kv = _values(s, _token_pages(s, torch.arange(B, device=DEV)[:, None], pos), pos % page_size)
    kv = torch.where((pos < L[:, None])[:, :, None], kv, 0.0)
    if s["op"] == "decode":
        b, i, n, count = torch.arange(B, device=DEV), 0, 1, torch.ones_like(L)
    else:
        b, i = _of_indptr(s["new_indptr"], q.shape[0])
        n, count = s["max_new"], (s["new_indptr"][1:] - s["new_indptr"][:-1]).long()
    padded = torch.zeros(B, n, H, DK, device=DEV)
    padded[b, i] = q.float()
    t = torch.matmul(padded.view(B, n * H, DK), kv.transpose(1, 2)) * (1.0 / math.sqrt(DK))
    sees = (L - count)[:, None] + torch.arange(1, n + 1, device=DEV)            # [B, n]
    t = t.view(B, n, H, -1).masked_fill_((pos >= sees[:, :, None])[:, :, None, :], -math.inf)
    top = t.amax(3, keepdim=True)
    e = torch.exp_(t.sub_(torch.where(torch.isfinite(top), top, 0.0)))
    den = e.sum(3)
    o = torch.matmul(e.view(B, n * H, -1), kv[:, :, :DV]).view(B, n, H, DV) / den[..., None]
    o = torch.where(den[..., None] > 0, o, 0.0)
    s["o"].copy_(o[b, i])
    s["lse"].copy_((top[..., 0] + torch.log(den))[b, i])
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ 64 bits
def _sequence(s, b, upto):
    """(flat row, page) of the first `upto` tokens of sequence b."""
    lo = int(s["kv_indptr"][b])
    pages = s["kv_indices"][lo:lo + -(-upto // s["page"])].long().repeat_interleave(s["page"])[:upto]
    return pages * s["page"] + torch.arange(upto, device=DEV) % s["page"], pages


def _e4m3(x):
    """fp64 values rounded to the nearest e4m3fn value, ties to even, at most 448."""
    e = torch.frexp(x)[1].double().clamp(min=-5) - 1        # the binade, or the subnormals' one
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-BIG, BIG)


def exact(case, seed):
    total, new = _lengths(case)
    s = prepare(case, seed)
    value = s["kv_cache"].view(-1, DK).double()
    scale = s["kv_scale"].double()
    if case["op"] == "gather":
        parts = [_sequence(s, b, n) for b, n in enumerate(total)]
        return torch.cat([value[r] * scale[p] for r, p in parts])
    if case["op"] == "append":
        at = 0
        for b, n in enumerate(new):
            rows, pages = _sequence(s, b, total[b])
            x, start = s["kv_new"][at:at + n].double(), total[b] - n
            at += n
            for j in range(start // case["page"], -(-total[b] // case["page"])):
                lo, hi = max(start, j * case["page"]), min(total[b], (j + 1) * case["page"])
                p, piece = pages[j * case["page"]], x[lo - start:hi - start]
                want = torch.exp2(torch.ceil(torch.log2(piece.abs().max() / BIG)))
                if lo > j * case["page"]:
                    want = torch.maximum(want, scale[p, 0])
                    before = rows[j * case["page"]:lo]
                    value[before] = _e4m3(value[before] * (scale[p, 0] / want))
                value[rows[lo:hi]] = _e4m3(piece / want)
                scale[p, 0] = want
        return {"kv_cache": value.view(s["kv_cache"].shape), "kv_scale": scale}
    outs, lses, at = [], [], 0
    for b, n in enumerate(new):
        n = n or 1
        rows, pages = _sequence(s, b, total[b])
        kv = value[rows] * scale[pages]
        t = torch.einsum("ihd,ld->ihl", s["q"][at:at + n].double(), kv) / math.sqrt(DK)
        at += n
        hidden = torch.arange(total[b], device=DEV) >= torch.arange(total[b] - n + 1, total[b] + 1, device=DEV)[:, None]
        t = t.masked_fill(hidden[:, None, :], -math.inf)
        lses.append(torch.logsumexp(t, 2))
        outs.append(torch.einsum("ihl,ld->ihd", torch.softmax(t, 2), kv[:, :DV]))
    return {"o": torch.cat(outs), "lse": torch.cat(lses)}
