"""GPU parity of the 8-bit latent cache (append, gather) and the attention over it, against the oracle.

Append and gather are exact: codes, scales and bf16 values must match bit for bit.

Attention, from the kernel's arithmetic. With S = sm_scale * max_j <|q|, |k_j|>:
  * a query entry is split into two e4m3 codes, off by at most 2^-22 of its row's largest
    magnitude; products of codes are exact, and their fp32 sums of 18 matrix steps (each a
    truncation, 2^-23) and a few more roundings are off by less than 2^-18 S. A row's
    largest magnitude is below 16 times its mean here, so the split adds less than
    16 * 2^-22 S. Score error: below 2^-17 S; with the fp32 exponent's rounding (2^-22 of
    the argument, itself within 2 S) below 2^-17 (1 + S);
  * so a softmax weight and its normaliser are each off by 2^-17 (1 + S), together
    2^-16 (1 + S) relatively;
  * a weight times its page's scale is rounded to fp16's 11 bits, 2^-12 relatively, and becomes
    three e4m3 codes, hi + lo / 32 + lo2 / 1024: 4, 4 and 3 of the bits, exactly, until lo2 is
    subnormal (steps of 2^-9 / 1024 = 2^-19): then 2^-20 absolutely. The reference is coded as
    2^2 (2^4 above 2^14 tokens, 2^6 above 2^16), and nothing that set it is larger than the
    largest weight times scale, M = max_j p_j s_j: 2^-22 M (2^-24, 2^-26) a token, and with the
    codes v_j / s_j that it multiplies `faint` = 2^-22 M sum_j |v_j / s_j| in all;
  * fp32 sums of L/32 steps: L * 2^-28;
  * the bf16 output: half a step, 2^-8 relatively.
|o - o_ref| <= (2^-16 (1 + S) + 2^-12 + 2^-28 L) * sum_j p_j |v_j| + faint + 2^-8 |o_ref| + 1e-30,
|lse - lse_ref| <= 2^-17 (1 + S) + 2^-21 (1 + |lse_ref|).
"""
import ctypes
import math

import pytest
import torch

from oracle import mla_fp8_oracle as M8
from oracle.fp8moe_oracle import e4m3_encode
from fp8_block_scaled_biased_b200 import binding as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device"),
              pytest.mark.filterwarnings("ignore")]

DEV = "cuda"


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert B.device_status() == 0


class Batch:
    """A cache (CPU codes and scales), a page table with shuffled pages, and their device copies."""

    def __init__(self, lens, ps, seed=0, spare=2, scale_exp=(-6, -5), poison=True, codes=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.ps, self.lens = g, ps, list(lens)
        counts = [-(-n // ps) for n in self.lens]
        n = sum(counts) + spare
        self.codes = e4m3_encode(torch.randn(n, ps, 1, 576, generator=g) * 40) if codes is None else codes(n, ps, g)
        self.scales = torch.exp2(torch.randint(scale_exp[0], scale_exp[1] + 1, (n, 1), generator=g).float())
        self.indptr = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
        self.indices = torch.randperm(n, generator=g)[:sum(counts)].to(torch.int32)
        self.last = torch.tensor([L - (c - 1) * ps if c else 0 for L, c in zip(self.lens, counts)], dtype=torch.int32)
        if poison:                                       # NaN codes wherever no token lies
            used = torch.zeros(n, ps, dtype=torch.bool)
            for b, L in enumerate(self.lens):
                for j in range(counts[b]):
                    used[self.indices[self.indptr[b] + j], :min(ps, L - j * ps)] = True
            self.codes[~used] = 0x7F

    @property
    def table(self):
        return self.indptr, self.indices, self.last

    def device(self, wide=False):
        """wide: a table with room for 144K tokens, as a serving program keeps it. The call then
        takes a long work list's 32 columns per CTA where a sequence has more than 16."""
        self.dc = self.codes.view(torch.float8_e4m3fn).to(DEV)
        self.ds = self.scales.to(DEV)
        indptr, indices, last = self.table
        if wide:
            indices = torch.cat([indices, torch.full((-(-144 * 1024 // self.ps),), -1, dtype=torch.int32)])
        self.dt = (indptr.to(DEV), indices.to(DEV), last.to(DEV))
        return self

    def q(self, rows, H, std=1.0):
        return (torch.randn(rows, H, 576, generator=self.g) * std).to(torch.bfloat16)


def _indptr(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)


def _codes(t):
    return t.view(torch.uint8).cpu()


def _bound(ref, mag, size, coded, L):
    c = 2.0 ** -16 * (1 + size) + 2.0 ** -12 + 2.0 ** -28 * L
    faint = 2.0 ** (-22 if L <= 2 ** 14 else -24 if L <= 2 ** 16 else -26)
    return c[..., None] * mag + faint * coded + 2.0 ** -8 * ref.abs() + 1e-30


def _check(b, q, qo, o, lse, **kw):
    ref, ref_lse, mag, size, coded = M8.extend(q, qo, b.codes, b.scales, *b.table, **kw)
    o, lse = o.cpu().double(), lse.cpu().double()
    rows = ~torch.isnan(ref_lse)
    bound = _bound(ref, mag, size, coded, max(b.lens))
    assert torch.isfinite(o[rows]).all()
    d = (o - ref).abs()
    worst = (d / bound)[rows].max().item()
    assert worst <= 1, f"worst |d|/bound {worst:.3f}"
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse) & rows, empty)
    assert (o[empty] == 0).all()
    fin = rows & ~empty
    dl = (lse - ref_lse).abs()[fin] - (2.0 ** -17 * (1 + size) + 2.0 ** -21 * (1 + ref_lse.abs()))[fin]
    assert (dl <= 0).all(), f"lse over its bound by {dl.max().item():.3e}"


def _decode(b, q, **kw):
    o = torch.full((q.shape[0], q.shape[1], 512), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float32, device=DEV)
    B.mla_decode_fp8_fwd(q.to(DEV), b.dc, b.ds, o, *b.dt, lse=lse, **kw)
    return o, lse


def _extend(b, q, qo, fill=math.nan, **kw):
    o = torch.full((q.shape[0], q.shape[1], 512), fill, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], fill, dtype=torch.float32, device=DEV)
    B.mla_extend_fp8_fwd(q.to(DEV), qo.to(DEV), b.dc, b.ds, o, *b.dt, lse=lse, **kw)
    return o, lse


# ---------------------------------------------------------------- append
def _append_and_check(b, x, counts, stride=576):
    ip = _indptr(counts)
    want_c, want_s = M8.append(x, ip, b.codes, b.scales, *b.table)
    wide = torch.zeros(max(x.shape[0], 1), stride, dtype=torch.bfloat16, device=DEV)
    wide[:x.shape[0], :576] = x.to(DEV)
    B.mla_kv_append_fp8(wide[:x.shape[0], :576], ip.to(DEV), b.dc, b.ds, *b.dt)
    assert torch.equal(b.ds.cpu(), want_s)
    got = _codes(b.dc)
    nan = (want_c & 0x7F) == 0x7F                         # a NaN's sign says nothing
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], want_c[~nan])
    b.codes, b.scales = want_c, want_s


@pytest.mark.parametrize("ps", [1, 3, 16, 64, 130])
@pytest.mark.parametrize("stride", [576, 640])
def test_append_matches_the_oracle_on_ragged_batches(ps, stride):
    new = [1, 0, 5, 64, 65, 130, 17, 1]
    old = [0, 9, 3, 0, 63, 1, 128, 200]
    b = Batch([n + o for n, o in zip(new, old)], ps, seed=ps, poison=False).device()
    x = (torch.randn(sum(new), 576, generator=b.g) * 2).to(torch.bfloat16)
    _append_and_check(b, x, new, stride)


def test_append_grows_scales_repeatedly_and_keeps_dead_rows():
    """Four calls on one page table that grows; magnitudes rise, fall and vanish, so pages are
    re-coded (down to subnormal codes), kept, and started afresh over old contents."""
    ps = 8
    full = Batch([40, 33], ps, seed=5, poison=False).device()
    pages = [full.indices[:5].clone(), full.indices[5:10].clone()]
    have = [0, 0]
    for step, (n, mag) in enumerate([((3, 1), 1e-3), ((4, 2), 5.0), ((20, 17), 1e4), ((13, 13), 0.0)]):
        have = [h + k for h, k in zip(have, n)]
        counts = [-(-h // ps) for h in have]
        full.indptr = _indptr(counts)
        full.indices = torch.cat([pages[0][:counts[0]], pages[1][:counts[1]]])
        full.last = torch.tensor([h - (c - 1) * ps for h, c in zip(have, counts)], dtype=torch.int32)
        full.dt = tuple(t.to(DEV) for t in full.table)
        x = (torch.randn(sum(n), 576, generator=full.g) * mag).to(torch.bfloat16)
        _append_and_check(full, x, n)


def test_append_infinities_nan_zeros_and_tiny_rows():
    b = Batch([6, 2, 3], 4, seed=9, poison=False).device()
    x = torch.randn(11, 576, generator=b.g)
    x[0, 5], x[1, 7], x[2, 9] = math.inf, -math.inf, math.nan
    x[6:8] = 0.0                                          # a page of zeros: scale 0
    x[8] = 1e-38                                          # below the smallest scale's codes
    x[9], x[10, 0] = 0.0, 3e38
    _append_and_check(b, x.to(torch.bfloat16), [6, 2, 3])
    b2 = Batch([2], 4, seed=10, poison=False).device()    # nothing finite and non-zero
    y = torch.zeros(2, 576)
    y[0, 0], y[1, 1] = math.inf, math.nan
    _append_and_check(b2, y.to(torch.bfloat16), [2])


def test_append_large_page_and_many_sequences():
    b = Batch([700], 512, seed=3, poison=False).device()  # more rows than a CTA holds in registers
    _append_and_check(b, torch.randn(650, 576, generator=b.g).to(torch.bfloat16), [650])
    b = Batch([1 + i % 3 for i in range(1500)], 2, seed=4, poison=False).device()
    counts = [i % 2 for i in range(1500)]
    _append_and_check(b, torch.randn(sum(counts), 576, generator=b.g).to(torch.bfloat16), counts)


@pytest.mark.parametrize("B_", [97, 513, 20000])
def test_append_and_gather_of_many_short_sequences(B_):
    """More sequences than a CTA has threads, some of them empty or without new tokens."""
    g = torch.Generator().manual_seed(B_)
    lens = torch.randint(0, 4, (B_,), generator=g)
    new = torch.minimum(torch.randint(0, 3, (B_,), generator=g), lens)
    pages = (lens + 1) // 2
    n = int(pages.sum())
    indptr = _indptr(pages.tolist())
    last = torch.where(lens > 0, lens - (pages - 1) * 2, 0).to(torch.int32)
    table = (indptr.to(DEV), torch.randperm(n, generator=g).to(torch.int32).to(DEV), last.to(DEV))
    cache = torch.zeros(n, 2, 1, 576, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.zeros(n, 1, device=DEV)
    want = torch.zeros(int(lens.sum()), 576, dtype=torch.bfloat16)
    full = _indptr(lens.tolist())
    for counts, offset in ((lens - new, torch.zeros_like(lens)), (new, lens - new)):
        # small integers: exact in the cache whatever the page's scale
        x = torch.randint(-7, 8, (int(counts.sum()), 576), generator=g).to(torch.bfloat16)
        done = offset + counts
        used = (done + 1) // 2
        at = torch.cat([torch.arange(int(u)) + int(i) for u, i in zip(used, indptr[:-1])]) if int(used.sum()) else torch.zeros(0)
        now = (_indptr(used.tolist()).to(DEV), table[1][at.long().to(DEV)].contiguous(),
               torch.where(done > 0, done - (used - 1) * 2, 0).to(torch.int32).to(DEV))
        B.mla_kv_append_fp8(x.to(DEV), _indptr(counts.tolist()).to(DEV), cache, scale, *now)
        seq = torch.repeat_interleave(torch.arange(B_), counts)
        place = torch.arange(len(x)) - torch.repeat_interleave(_indptr(counts.tolist())[:-1].long(), counts)
        want[full[:-1].long()[seq] + offset[seq] + place] = x
    out = torch.full((len(want) + 2, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(cache, scale, *table, full.to(DEV), out)
    assert torch.equal(out[:-2].cpu(), want) and (out[-2:] == 9).all()


def test_append_and_gather_of_nothing():
    b = Batch([3, 0], 4).device()
    before = _codes(b.dc)
    B.mla_kv_append_fp8(torch.empty(0, 576, dtype=torch.bfloat16, device=DEV), _indptr([0, 0]).to(DEV), b.dc, b.ds, *b.dt)
    assert torch.equal(_codes(b.dc), before)
    out = torch.empty(0, 576, dtype=torch.bfloat16, device=DEV)
    assert B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, _indptr([0, 0]).to(DEV), out) is out


# ---------------------------------------------------------------- gather
@pytest.mark.parametrize("ld, off", [(576, 0), (584, 0), (592, 0), (592, 8), (640, 24)])
def test_gather_into_rows_of_any_stride_and_alignment(ld, off):
    b = Batch([70, 0, 33], 16, seed=3).device()
    ip = _indptr([70, 0, 30])
    buf = torch.full((100 * ld + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = torch.as_strided(buf, (100, 576), (ld, 1), off)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip.to(DEV), out)
    want = M8.gather(b.codes, b.scales, b.indptr, b.indices, ip, torch.full((100, 576), 5.0, dtype=torch.bfloat16))
    assert torch.equal(out.cpu(), want)
    out.fill_(5.0)
    assert (buf == 5.0).all()                              # nothing between the rows


@pytest.mark.parametrize("ps", [1, 7, 64])
def test_gather_matches_the_oracle_and_leaves_other_rows(ps):
    lens, take = [5, 0, 70, 33, 64, 1], [5, 0, 41, 33, 0, 1]
    b = Batch(lens, ps, seed=ps, scale_exp=(-8, 3)).device()
    ip = _indptr(take) + 3                                # three rows before the first sequence, some behind the last
    out = torch.full((sum(take) + 9, 640), 5.0, dtype=torch.bfloat16)
    dev = out.to(DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip.to(DEV), dev[:, :576])
    want = M8.gather(b.codes, b.scales, b.indptr, b.indices, ip, out[:, :576])
    assert torch.equal(dev[:, :576].cpu(), want) and (dev[:, 576:] == 5).all()


# ---------------------------------------------------------------- decode
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ps", [1, 7, 64, 200])
@pytest.mark.parametrize("H", [1, 8, 16, 24, 128])
def test_decode_ragged_lengths_heads_and_pages(ps, H, wide):
    b = Batch([0, 1, 127, 128, 129, 2, 300, 64], ps, seed=H + ps).device(wide)
    q = b.q(8, H)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(9), o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ps", [3, 64])
@pytest.mark.parametrize("H", [2, 16, 40, 128])
def test_decode_short_beside_long(ps, H, wide):
    """Sequences cut into parts beside whole ones, and alone in a share beside empty ones."""
    for lens in ([0, 1, 900, 128, 129, 2, 640, 0], [500, 0, 0, 505], [130] * 30 + [0] * 6, [200] * 40):
        b = Batch(lens, ps, seed=H + ps + len(lens)).device(wide)
        q = b.q(len(lens), H)
        o, lse = _decode(b, q)
        _check(b, q, torch.arange(len(lens) + 1), o, lse)


def test_decode_long_and_many():
    b = Batch([3000, 5, 1711], 64, seed=1).device()
    q = b.q(3, 16)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(4), o, lse)
    b = Batch([1 + (i * 7) % 5 for i in range(700)], 2, seed=2).device()
    q = b.q(700, 2)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(701), o, lse)


def test_decode_sharp_scores_explicit_scale_and_soft_cap():
    b = Batch([40, 300, 77, 1], 16, seed=5).device()
    q = b.q(4, 16, std=6.0)
    for kw in (dict(sm_scale=0.11), dict(sm_scale=0.11, logit_cap=2.0), dict(sm_scale=0.02, logit_cap=30.0)):
        o, lse = _decode(b, q, **kw)
        _check(b, q, torch.arange(5), o, lse, **kw)


def test_decode_rising_scores_renormalise_every_tile():
    """Keys whose scores rise steadily over the sequence, and the same falling: the running
    maximum moves in every tile, or never after the first."""
    def codes(n, ps, g):
        c = torch.randn(n, ps, 1, 576, generator=g) * 40
        c[:, :, 0, 0] = 400.0
        return e4m3_encode(c)
    for sign in (1, -1):
        b = Batch([1000], 1, seed=6, codes=codes)
        at = torch.arange(1000)
        b.codes[b.indices[at].long(), 0, 0, 0] = e4m3_encode(sign * (at - 500).float() * 0.8)
        b.device()
        q = b.q(1, 16)
        q[:, :, 0] = 60.0
        o, lse = _decode(b, q)
        _check(b, q, torch.arange(2), o, lse)


def test_decode_one_dominant_token_over_a_long_faint_rest():
    """A sink: one token whose score stands about 11.5 nats above 4000 others of one size."""
    b = Batch([4001], 32, seed=7, scale_exp=(-6, -6))
    lat = b.codes.view(torch.float8_e4m3fn)
    b.codes[:, :, 0, 575] = e4m3_encode(torch.zeros(1))
    first = int(b.indices[0])
    b.codes[first, 0, 0, 575] = e4m3_encode(torch.full((1,), 256.0))
    b.device()
    q = torch.zeros(1, 16, 576)
    q[:, :, 575] = 11.5 * 24 / (256 * 2.0 ** -6)
    q[:, :, :8] = torch.randn(1, 16, 8, generator=b.g) * 0.5
    q = q.to(torch.bfloat16)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(2), o, lse)


def test_decode_pages_of_very_different_scales_and_a_zero_page():
    b = Batch([200, 512, 40], 8, seed=8, scale_exp=(-14, 2))
    b.scales[b.indices[3].long()] = 0.0                    # a page of zeros inside the first sequence
    b.scales[b.indices[b.indptr[2]:].long()] = 0.0         # a sequence of nothing else
    b.device()
    q = b.q(3, 16, std=0.05)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(4), o, lse)


def test_decode_zero_query_and_queries_of_any_size():
    b = Batch([150, 150, 150], 16, seed=11).device()
    q = b.q(3, 16).float()
    q[0] = 0.0
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 40
    q = q.to(torch.bfloat16)
    o, lse = _decode(b, q, sm_scale=0.05 * 2.0 ** -40)
    _check(b, q, torch.arange(4), o, lse, sm_scale=0.05 * 2.0 ** -40)


def test_decode_nan_stays_with_its_sequence_and_head():
    b = Batch([130, 200, 50], 16, seed=12)
    bad = int(b.indices[b.indptr[1] + 3])
    b.codes[bad, 2, 0, 100] = 0x7F                         # a token of the second sequence
    b.device()
    q = b.q(3, 16)
    q[0, 5, 17] = math.nan
    q[2, 7, 3] = math.inf
    o, lse = _decode(b, q)
    nan = torch.isnan(lse.cpu())
    want = torch.zeros(3, 16, dtype=torch.bool)
    want[0, 5] = want[2, 7] = True
    want[1] = True
    assert torch.equal(nan, want)
    assert torch.equal(torch.isnan(o.cpu()).all(2), want) and torch.equal(torch.isnan(o.cpu()).any(2), want)
    ref, ref_lse, mag, size, coded = M8.decode(torch.nan_to_num(q, posinf=0.0), b.codes, b.scales, *b.table)
    fine = ~want
    bound = _bound(ref, mag, size, coded, 200)
    assert ((o.cpu().double() - ref).abs()[fine] <= bound[fine]).all()


@pytest.mark.parametrize("L, H, ps", [(17000, 3, 64), (17000, 40, 16), (70000, 2, 128), (70000, 1, 8)])
def test_decode_long_contexts(L, H, ps):
    """Contexts long enough for the two higher references, joined from a hundred and more parts; one
    token stands 9 nats above the rest, so that most of the mass lies in faint weights."""
    b = Batch([L], ps, seed=L + H, scale_exp=(-6, -6))
    lat = b.codes.view(-1, 576)
    lat[:, 575] = e4m3_encode(torch.zeros(1))
    lat[int(b.indices[0]) * ps, 575] = e4m3_encode(torch.full((1,), 256.0))
    b.device()
    q = torch.zeros(1, H, 576)
    q[:, :, 575] = 9.0 * 24 / (256 * 2.0 ** -6)
    q[:, :, :8] = torch.randn(1, H, 8, generator=b.g) * 0.5
    q = q.to(torch.bfloat16)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(2), o, lse)


def test_decode_and_gather_of_a_shared_prefix():
    """Two sequences whose tables begin with the same pages, and one that names a page twice."""
    b = Batch([200, 90, 64], 32, seed=17)
    b.indices[7:9] = b.indices[:2]
    b.indices[11] = b.indices[10]
    b.codes[b.indices.long()] = e4m3_encode(torch.randn(12, 32, 1, 576, generator=b.g) * 40)
    b.device()
    q = b.q(3, 16)
    o, lse = _decode(b, q)
    _check(b, q, torch.arange(4), o, lse)
    out = torch.zeros(354, 576, dtype=torch.bfloat16, device=DEV)
    ip = _indptr(b.lens)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip.to(DEV), out)
    assert torch.equal(out.cpu(), M8.gather(b.codes, b.scales, b.indptr, b.indices, ip, torch.zeros_like(out).cpu()))


@pytest.mark.parametrize("H, bad", [(8, 0), (5, 0), (16, 3), (24, 17)])
def test_decode_nan_in_one_head_leaves_the_others(H, bad):
    b = Batch([130, 300], 16, seed=13).device(wide=True)
    q = b.q(2, H)
    clean = q.clone()
    q[:, bad, 40] = math.nan
    o, lse = _decode(b, q)
    assert torch.isnan(o[:, bad]).all() and torch.isnan(lse[:, bad]).all()
    o2, lse2 = _decode(b, clean)
    keep = [h for h in range(H) if h != bad]
    assert torch.equal(o[:, keep], o2[:, keep]) and torch.equal(lse[:, keep], lse2[:, keep])


@pytest.mark.parametrize("H", [1, 8, 16, 32])
def test_extend_a_nan_query_leaves_the_other_queries(H):
    b = Batch([200, 40], 64, seed=14).device(wide=H != 16)
    qo = _indptr([6, 3])
    q = b.q(9, H)
    clean = q.clone()
    q[1], q[6] = math.nan, math.inf
    o, lse = _extend(b, q, qo)
    o2, lse2 = _extend(b, clean, qo)
    bad, keep = [1, 6], [0, 2, 3, 4, 5, 7, 8]
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])


def test_decode_scales_at_the_ends_of_their_range():
    """The smallest scale an append writes, under scores that rise after the first tile by just
    less than what moves a reference: the weights' sum stays finite. Any output is a mean of
    values, so it is off by at most twice the largest, 448 * 2^-110."""
    b = Batch([1600], 64, seed=15, scale_exp=(-110, -110))
    late = torch.arange(1600) >= 128
    flat = b.codes.view(-1, 576)
    at = b.indices[torch.arange(1600) // 64].long() * 64 + torch.arange(1600) % 64
    flat[at, 575] = e4m3_encode(torch.where(late, 128.0, 0.0))
    b.device()
    q = torch.zeros(1, 16, 576)
    q[:, :, 575] = 2.0 ** 103 * 5.75 * math.log(2.0)
    q = q.to(torch.bfloat16)
    ref, ref_lse, _, size, _ = M8.decode(q, b.codes, b.scales, *b.table, sm_scale=1.0)
    many = 160                                             # so many on the same pages that none is cut up
    b.dt = (torch.arange(many + 1, dtype=torch.int32, device=DEV) * 25, b.dt[1].repeat(many), b.dt[2].repeat(many))
    o, lse = _decode(b, q.expand(many, 16, 576).contiguous(), sm_scale=1.0)
    dl = (lse.cpu().double() - ref_lse).abs()
    assert (dl <= 2.0 ** -17 * (1 + size) + 2.0 ** -21 * (1 + ref_lse.abs())).all()
    assert ((o.cpu().double() - ref).abs() <= 2 * 448 * 2.0 ** -110).all()
    for e in (-88, 100):                                   # where the weights still have their full precision
        b = Batch([300, 90], 16, seed=16, scale_exp=(e, e)).device()
        q = b.q(2, 16)
        o, lse = _decode(b, q, sm_scale=2.0 ** (-5 - e) / 24)
        _check(b, q, torch.arange(3), o, lse, sm_scale=2.0 ** (-5 - e) / 24)


# ---------------------------------------------------------------- extend
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ps", [2, 8, 16, 32, 96, 128, 256])
@pytest.mark.parametrize("H", [5, 48])
def test_extend_by_page_size(ps, H, wide):
    b = Batch([129, 1, 400, 128, 257], ps, seed=ps + H).device(wide)
    new = [9, 1, 4, 0, 13]
    qo = _indptr(new)
    q = b.q(sum(new), H)
    o, lse = _extend(b, q, qo)
    _check(b, q, qo, o, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H", [3, 16, 40, 128])
@pytest.mark.parametrize("ps", [1, 48])
def test_extend_ragged(ps, H, wide):
    lens, new = [5, 0, 140, 260, 33, 128, 9], [5, 0, 2, 37, 0, 128, 1]
    if H == 128:
        new = [5, 0, 2, 7, 0, 20, 1]
    b = Batch(lens, ps, seed=ps + H).device(wide)
    qo = _indptr(new)
    q = b.q(sum(new) + 3, H)                               # three rows behind the last sequence
    o, lse = _extend(b, q, qo, fill=3.0)
    assert (o[sum(new):] == 3).all() and (lse[sum(new):] == 3).all()
    _check(b, q, qo, o, lse)


def test_extend_with_more_queries_than_tokens_leaves_the_first_ones_empty():
    b = Batch([3, 0, 130], 4, seed=2).device()
    qo = _indptr([7, 4, 135])
    q = b.q(146, 2)
    o, lse = _extend(b, q, qo)
    assert torch.isneginf(lse.cpu()[:4]).all() and torch.isneginf(lse.cpu()[7:11]).all()
    _check(b, q, qo, o, lse)


def test_extend_of_one_token_each_is_a_decode():
    b = Batch([77, 300, 5], 16, seed=3).device()
    q = b.q(3, 32)
    o1, l1 = _decode(b, q, logit_cap=20.0)
    o2, l2 = _extend(b, q, torch.arange(4, dtype=torch.int32), logit_cap=20.0)
    _check(b, q, torch.arange(4), o1, l1, logit_cap=20.0)
    _check(b, q, torch.arange(4), o2, l2, logit_cap=20.0)


def test_extend_a_nan_token_stays_hidden_from_earlier_queries():
    """NaN in a later token's row must not reach the queries that do not see it, though they
    share its tile."""
    b = Batch([140, 20], 16, seed=4)
    page = int(b.indices[b.indptr[0] + 135 // 16])
    b.codes[page, 135 % 16, 0, 300] = 0x7F                 # token 135 of 140
    b.device()
    qo = _indptr([12, 3])
    q = b.q(15, 16)
    o, lse = _extend(b, q, qo)
    sees = torch.arange(12) + 129                          # token 135 is seen from 136 on
    nan = torch.isnan(lse.cpu()).any(1)
    assert torch.equal(nan[:12], sees >= 136) and not nan[12:].any()
    assert torch.isnan(o.cpu()[:12][sees >= 136]).all()
    clean = Batch([140, 20], 16, seed=4)
    clean.codes = b.codes.clone()
    clean.codes[page, 135 % 16, 0, 300] = 0x20
    ref, ref_lse, mag, size, coded = M8.extend(q, qo, clean.codes, clean.scales, *clean.table)
    fine = ~nan
    bound = _bound(ref, mag, size, coded, 140)
    assert ((o.cpu().double() - ref).abs()[fine] <= bound[fine]).all()


# ---------------------------------------------------------------- as a user runs them
def test_a_prompt_then_steps_then_a_prefix_read_back():
    """Append a prompt, attend over it, append and decode token by token, read the prefix back:
    every stage against the oracle's own cache."""
    ps, H = 16, 16
    b = Batch([64, 64], ps, seed=21, poison=False)
    final = [37 + 4, 20 + 4]
    pages = [b.indices[:4].clone(), b.indices[4:8].clone()]
    b.device()

    def grow(have):
        counts = [-(-h // ps) for h in have]
        b.lens = list(have)
        b.indptr, b.indices = _indptr(counts), torch.cat([p[:c] for p, c in zip(pages, counts)])
        b.last = torch.tensor([h - (c - 1) * ps for h, c in zip(have, counts)], dtype=torch.int32)
        b.dt = tuple(t.to(DEV) for t in b.table)

    have = [37, 20]
    grow(have)
    _append_and_check(b, torch.randn(57, 576, generator=b.g).to(torch.bfloat16), have)
    q = b.q(57, H)
    qo = _indptr(have)
    o, lse = _extend(b, q, qo)
    _check(b, q, qo, o, lse)
    for step in range(4):
        have = [h + 1 for h in have]
        grow(have)
        _append_and_check(b, (torch.randn(2, 576, generator=b.g) * (1 + 3 * step)).to(torch.bfloat16), [1, 1])
        q = b.q(2, H)
        o, lse = _decode(b, q)
        _check(b, q, torch.arange(3), o, lse)
    assert have == final
    ip = _indptr([30, 24])
    out = torch.zeros(54, 576, dtype=torch.bfloat16)
    got = B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip.to(DEV), out.to(DEV))
    assert torch.equal(got.cpu(), M8.gather(b.codes, b.scales, b.indptr, b.indices, ip, out))


def test_same_bits_again_with_a_dirty_workspace_and_without_lse():
    b = Batch([700, 33, 1200, 5], 16, seed=30).device()
    q = b.q(4, 64)
    o1, l1 = _decode(b, q)
    need = B.mla_fp8_workspace_bytes(64, 4)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    o2, l2 = _decode(b, q, workspace=ws)
    ws.fill_(0x7F)
    o3 = torch.empty_like(o1)
    B.mla_decode_fp8_fwd(q.to(DEV), b.dc, b.ds, o3, *b.dt, workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2) and torch.equal(o1, o3)


def test_captured_step_replays_on_new_contents():
    """An append and the attention over it, captured once and replayed with other rows, queries
    and a page table that has grown within its buffers."""
    ps, H = 8, 16
    b = Batch([60, 60], ps, seed=40, poison=False).device()
    pages = [b.indices[:8].clone(), b.indices[8:16].clone()]
    x = torch.zeros(2, 576, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, H, 576, dtype=torch.bfloat16, device=DEV)
    o = torch.zeros(2, H, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(2, H, device=DEV)
    ip = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    indptr = torch.zeros(3, dtype=torch.int32, device=DEV)
    indices = torch.zeros(16, dtype=torch.int32, device=DEV)
    last = torch.ones(2, dtype=torch.int32, device=DEV)

    def step():
        B.mla_kv_append_fp8(x, ip, b.dc, b.ds, indptr, indices, last)
        B.mla_decode_fp8_fwd(q, b.dc, b.ds, o, indptr, indices, last, lse=lse)

    def table(have):
        counts = [-(-h // ps) for h in have]
        b.lens, b.indptr = list(have), _indptr(counts)
        b.indices = torch.cat([pages[0][:counts[0]], pages[1][:counts[1]]])
        b.last = torch.tensor([h - (c - 1) * ps for h, c in zip(have, counts)], dtype=torch.int32)
        indptr.copy_(b.indptr)
        indices[:b.indices.numel()].copy_(b.indices)
        last.copy_(b.last)

    have = [59, 30]
    table(have)
    step()                                                 # warm-up outside the capture
    torch.cuda.synchronize()
    b.codes, b.scales = _codes(b.dc), b.ds.cpu()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        have = [h + 1 for h in have] if k else have
        have = [min(have[0], 60), have[1]]
        table(have)
        rows = (torch.randn(2, 576, generator=b.g) * (k + 1)).to(torch.bfloat16)
        qs = b.q(2, H)
        x.copy_(rows)
        q.copy_(qs)
        graph.replay()
        torch.cuda.synchronize()
        b.codes, b.scales = M8.append(rows, [0, 1, 2], b.codes, b.scales, *b.table)
        assert torch.equal(_codes(b.dc), b.codes) and torch.equal(b.ds.cpu(), b.scales)
        _check(b, qs, torch.arange(3), o, lse)


def test_calls_wait_for_the_work_before_them():
    """Kernels are launched early and wait by themselves: for copies, fills, another stream's work and
    each other, captured and not."""
    b = Batch([300, 40, 129, 700], 64, seed=53).device()
    H, lens = 16, b.lens
    q, x = b.q(4, H).to(DEV), torch.randn(4, 576, generator=b.g).to(torch.bfloat16).to(DEV)
    ip, full = _indptr([1] * 4).to(DEV), _indptr(lens).to(DEV)
    codes, scales = b.dc.clone(), b.ds.clone()
    q_in, x_in = torch.zeros_like(q), torch.zeros_like(x)
    big = torch.zeros(32 << 20, device=DEV)
    o = torch.zeros(4, H, 512, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(sum(lens), 576, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()

    def step():
        b.dc.copy_(codes)
        b.ds.copy_(scales)
        big.zero_()
        x_in.copy_(x)
        B.mla_kv_append_fp8(x_in, ip, b.dc, b.ds, *b.dt)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            big.add_(1.0)
            q_in.copy_(q)
        here.wait_stream(side)
        B.mla_decode_fp8_fwd(q_in, b.dc, b.ds, o, *b.dt)
        B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, full, out)
        x_in.zero_()
        q_in.zero_()

    step()
    torch.cuda.synchronize()
    want_codes, want_scales = M8.append(x.cpu(), _indptr([1] * 4), b.codes, b.scales, *b.table)
    assert torch.equal(_codes(b.dc), want_codes) and torch.equal(b.ds.cpu(), want_scales)
    first = o.clone()
    b.codes, b.scales = want_codes, want_scales
    _check(b, q.cpu(), torch.arange(5), o, _decode(b, q.cpu())[1])
    want = M8.gather(want_codes, want_scales, b.indptr, b.indices, _indptr(lens), torch.zeros_like(out).cpu())
    assert torch.equal(out.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for run in [step] * 10 + [g.replay] * 10:
        o.fill_(math.nan)
        out.zero_()
        run()
        assert torch.equal(o, first) and torch.equal(out.cpu(), want)


def test_two_captured_graphs_share_a_workspace():
    b = Batch([700, 30, 300], 64, seed=52).device()
    ws = torch.empty(B.mla_fp8_workspace_bytes(128, 3), dtype=torch.uint8, device=DEV)
    runs = []
    for H in (16, 128):
        q = b.q(3, H).to(DEV)
        o = torch.zeros(3, H, 512, dtype=torch.bfloat16, device=DEV)
        want = _decode(b, q)[0]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            B.mla_decode_fp8_fwd(q, b.dc, b.ds, o, *b.dt, workspace=ws)
        runs.append((g, q, o, want))
    for _ in range(5):
        for g, _, o, _ in runs:
            o.zero_()
            g.replay()
    for _, _, o, want in runs:
        assert torch.equal(o, want)


def test_two_streams_with_a_workspace_each():
    b = Batch([900, 411, 1300], 16, seed=50).device()
    q = b.q(3, 32)
    want, want_l = _decode(b, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(_decode(b, q))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want) and torch.equal(lse, want_l)


def test_cache_beyond_four_gigabytes():
    """Pages whose byte offsets pass 2^32."""
    ps = 64
    n = (1 << 32) // (ps * 576) + 40
    cache = torch.empty(n, ps, 1, 576, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.full((n, 1), 2.0 ** -6, device=DEV)
    b = Batch([100, 200], ps, seed=60, scale_exp=(-6, -6))
    at = torch.tensor([n - 1 - i for i in range(b.indices.numel())], dtype=torch.int32)
    cache.view(torch.uint8)[at.long().to(DEV)] = b.codes[b.indices.long()].to(DEV)
    table = (b.dt if hasattr(b, "dt") else tuple(t.to(DEV) for t in b.table))
    table = (table[0], at.to(DEV), table[2])
    q = b.q(2, 16)
    o = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 16, device=DEV)
    B.mla_decode_fp8_fwd(q.to(DEV), cache, scale, o, *table, lse=lse)
    _check(b, q, torch.arange(3), o, lse)
    out = torch.zeros(300, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(cache, scale, *table, _indptr([100, 200]).to(DEV), out)
    assert torch.equal(out.cpu(), M8.gather(b.codes, b.scales, b.indptr, b.indices, _indptr([100, 200]),
                                            torch.zeros(300, 576, dtype=torch.bfloat16)))
    x = torch.ones(1, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_append_fp8(x, _indptr([0, 1]).to(DEV), cache, scale, *table)
    row = cache[int(at[int(b.indptr[2]) - 1]), int(b.last[1]) - 1, 0]
    assert (row.float() * 2.0 ** -6 == 1).all()


# ---------------------------------------------------------------- refusals
def test_table_entries_out_of_range_are_flagged_not_followed():
    b = Batch([20, 30], 8, seed=70, poison=False).device()
    q = b.q(2, 16).to(DEV)
    o = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    before = _codes(b.dc)
    x = torch.ones(2, 576, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(50, 576, dtype=torch.bfloat16, device=DEV)
    ip, full = _indptr([1, 1]).to(DEV), _indptr([20, 30]).to(DEV)

    def everything(table, append=ip, take=full):
        B.mla_decode_fp8_fwd(q, b.dc, b.ds, o, *table)
        assert B.device_status() == 32
        B.mla_extend_fp8_fwd(q, ip, b.dc, b.ds, o, *table)
        assert B.device_status() == 32
        B.mla_kv_gather_fp8(b.dc, b.ds, *table, take, out)
        assert B.device_status() == 32
        B.mla_kv_append_fp8(x, append, b.dc, b.ds, *table)
        assert B.device_status() == 32

    for entry in (-1, b.codes.shape[0], 2 ** 31 - 1):
        bad = b.dt[1].clone()
        bad[2] = entry                                     # the first sequence's last page
        everything((b.dt[0], bad, b.dt[2]))
    assert torch.equal(_codes(b.dc)[b.indices[:2].long()], before[b.indices[:2].long()])
    for indptr in ([0, 3, 9], [0, -1, 7], [0, 8, 7]):
        everything((torch.tensor(indptr, dtype=torch.int32, device=DEV), b.dt[1], b.dt[2]))
    for last in ([0, 6], [9, 6]):
        everything((b.dt[0], b.dt[1], torch.tensor(last, dtype=torch.int32, device=DEV)))


def test_ranges_out_of_bounds_are_flagged_not_followed():
    b = Batch([20, 30], 8, seed=71, poison=False).device()
    before = _codes(b.dc)
    x = torch.ones(2, 576, dtype=torch.bfloat16, device=DEV)
    q = b.q(2, 16).to(DEV)
    o = torch.full((2, 16, 512), 4.0, dtype=torch.bfloat16, device=DEV)
    out = torch.full((4, 576), 4.0, dtype=torch.bfloat16, device=DEV)
    for bad in ([0, 1, 3], [0, -5, 2], [-2, 1, 2]):
        ip = torch.tensor(bad, dtype=torch.int32, device=DEV)
        B.mla_kv_append_fp8(x, ip, b.dc, b.ds, *b.dt)
        B.mla_extend_fp8_fwd(q, ip, b.dc, b.ds, o, *b.dt)
        assert B.device_status() == 32
    ip = torch.tensor([0, 21, 22], dtype=torch.int32, device=DEV)   # 21 of 20 tokens
    big = torch.ones(22, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_append_fp8(big, ip, b.dc, b.ds, *b.dt)
    assert B.device_status() == 32
    rows = torch.zeros(22, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip, rows)
    assert B.device_status() == 32 and (rows[20] == 0).all()


def test_append_ranges_that_decrease_are_flagged():
    """A later range that begins before an earlier one: no page before a sequence's first is looked up."""
    b = Batch([60, 60, 60, 60], 1, seed=72, poison=False).device()
    x = torch.ones(60, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_append_fp8(x, torch.tensor([0, 50, 55, 3, 9], dtype=torch.int32, device=DEV), b.dc, b.ds, *b.dt)
    assert B.device_status() == 32


def test_decode_of_an_empty_table():
    for H in (16, 128):
        b = Batch([0, 0], 64, seed=73).device()
        assert b.dt[1].numel() == 0
        o, lse = _decode(b, b.q(2, H))
        assert (o == 0).all() and torch.isneginf(lse).all()


# ---------------------------------------------------------------- calls that follow one another at once
def test_each_call_sees_what_the_one_before_it_wrote():
    """Steps in which every page's scale and codes change, run without a pause and with one after every
    call: neighbouring pages' scales share memory lines that other SMs have read a call earlier."""
    seqs, ps, H, steps = 96, 4, 16, 12
    b = Batch([ps * 3] * seqs, ps, seed=90, poison=False).device()
    rows = [(torch.randn(seqs, 576, generator=b.g) * 4.0 ** k).to(torch.bfloat16).to(DEV) for k in range(steps)]
    q, ip = b.q(seqs, H, std=0.01).to(DEV), _indptr([1] * seqs).to(DEV)
    tables = []
    for k in range(steps):
        counts = -(-(k + 1) // ps)
        idx = b.dt[1].view(seqs, 3)[:, :counts].contiguous().view(-1)
        tables.append((torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * counts, idx,
                       torch.full((seqs,), k + 1 - (counts - 1) * ps, dtype=torch.int32, device=DEV),
                       torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * (k + 1)))

    def run(pause):
        cache, scale, got = b.dc.clone(), b.ds.clone(), []
        outs = [torch.empty(seqs * (k + 1), 576, dtype=torch.bfloat16, device=DEV) for k in range(steps)]
        os_ = [torch.empty(seqs, H, 512, dtype=torch.bfloat16, device=DEV) for _ in range(steps)]
        torch.cuda.synchronize()
        for k, (indptr, idx, last, full) in enumerate(tables):
            B.mla_kv_append_fp8(rows[k], ip, cache, scale, indptr, idx, last)
            pause()
            B.mla_kv_gather_fp8(cache, scale, indptr, idx, last, full, outs[k])
            pause()
            B.mla_decode_fp8_fwd(q, cache, scale, os_[k], indptr, idx, last)
            pause()
            got += [outs[k], os_[k]]
        torch.cuda.synchronize()
        return got + [scale, cache.view(torch.uint8)]

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        for x, y in zip(run(lambda: None), want):
            assert torch.equal(x, y)


# ---------------------------------------------------------------- pages whose scale was 0
def test_append_after_a_row_of_infinities_and_zeros():
    """The page's scale is 0 and its codes +-448: the value 0, which the next rows must not change."""
    ps = 8
    full = Batch([8], ps, seed=91, poison=False).device()
    page = int(full.indices[0])

    def step(have, x):
        full.last = torch.tensor([have], dtype=torch.int32)
        full.dt = tuple(t.to(DEV) for t in full.table)
        _append_and_check(full, x.to(torch.bfloat16), [x.shape[0]])

    x = torch.zeros(2, 576)
    x[0, 0], x[0, 1], x[1, 2], x[1, 575] = math.inf, -math.inf, math.nan, math.inf
    step(2, x)
    assert float(full.ds[page]) == 0
    step(3, torch.zeros(1, 576))                           # still nothing finite
    step(4, torch.randn(1, 576, generator=full.g))
    out = torch.full((4, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(full.dc, full.ds, *full.dt, _indptr([4]).to(DEV), out)
    got = out[:3].cpu().float()
    assert torch.isnan(got[1, 2]) and (torch.nan_to_num(got) == 0).all() and torch.isnan(got).sum() == 1


def test_append_to_a_callers_page_of_scale_zero():
    """Any codes under a scale of 0 stand for 0."""
    b = Batch([20, 9], 16, seed=92, poison=False)
    b.scales[:] = 0.0
    b.device()
    _append_and_check(b, torch.randn(5, 576, generator=b.g).to(torch.bfloat16), [3, 2])


# ---------------------------------------------------------------- ranges, one call at a time
def _gather_flagged(b, ip, rows, behind=0):
    """One gather of `rows` rows with ranges that are wrong: flagged; returns what it left in the rows."""
    out = torch.full((rows + behind, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, torch.tensor(ip, dtype=torch.int32, device=DEV), out[:rows])
    assert B.device_status() == 32, ip
    assert (out[rows:] == 9).all()
    return out[:rows].cpu()


def test_gather_ranges_out_of_bounds_are_flagged_and_their_rows_left():
    b = Batch([20, 30, 40], 8, seed=93).device()
    want = [M8.gather(b.codes, b.scales, b.indptr, b.indices, [0] * (s + 1) + [4] * (3 - s),
                      torch.zeros(4, 576, dtype=torch.bfloat16)) for s in range(3)]
    # the last range ends behind the output: its rows are left, the first one's written
    got = _gather_flagged(b, [0, 1, 1, 3], 2, behind=4)
    assert torch.equal(got[0], want[0][0]) and (got[1] == 9).all()
    # it begins at or behind the end, so that no row belongs to it
    got = _gather_flagged(b, [0, 0, 2, 5], 2, behind=4)
    assert torch.equal(got, want[1][:2])
    got = _gather_flagged(b, [0, 2, 7, 9], 2, behind=8)
    assert torch.equal(got, want[0][:2])
    # negative starts
    assert (_gather_flagged(b, [0, -5, 2, 2], 2, behind=4) == 9).all()
    got = _gather_flagged(b, [-2, 1, 2, 4], 4)
    assert (got[0] == 9).all() and torch.equal(got[1:2], want[1][:1]) and torch.equal(got[2:], want[2][:2])
    # ranges that decrease: rows claimed twice may be either's
    got = _gather_flagged(b, [0, 3, 1, 4], 6)
    assert (got[4:] == 9).all()
    # all of them, far out
    assert (_gather_flagged(b, [2 ** 31 - 1] * 4, 3, behind=4) == 9).all()
    assert (_gather_flagged(b, [-2 ** 31, 0, 0, 0], 3, behind=4) == 9).all()


def test_gather_a_bad_range_among_many_sequences():
    """More sequences than one CTA's threads, few rows: the wrong range has none of them."""
    n = 5000
    b = Batch([1] * 3, 4, seed=94).device()
    indptr = torch.full((n + 1,), 3, dtype=torch.int32)
    indptr[:3] = torch.arange(3)
    table = (indptr.to(DEV), b.dt[1], torch.cat([b.dt[2], torch.zeros(n - 3, dtype=torch.int32, device=DEV)]))
    ip = indptr.clone()
    out = torch.full((3, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *table, ip.to(DEV), out)
    assert B.device_status() == 0
    want = M8.gather(b.codes, b.scales, b.indptr, b.indices, [0, 1, 2, 3], torch.zeros(3, 576, dtype=torch.bfloat16))
    assert torch.equal(out.cpu(), want)
    for at, value in ((n, 4), (4000, 2), (300, 2 ** 31 - 1)):
        bad = ip.clone()
        bad[at] = value
        out.fill_(9.0)
        B.mla_kv_gather_fp8(b.dc, b.ds, *table, bad.to(DEV), out)
        assert B.device_status() == 32, (at, value)


def test_extend_ranges_out_of_bounds_are_flagged_and_their_rows_left():
    b = Batch([20, 30], 8, seed=95, poison=False).device()
    q = b.q(2, 16).to(DEV)
    for bad, left in (([0, 1, 3], [1]), ([0, -5, 2], [0, 1]), ([-2, 1, 2], [0]), ([0, 2, 5], []), ([0, 2, 1], [])):
        o = torch.full((2, 16, 512), 4.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((2, 16), 4.0, device=DEV)
        B.mla_extend_fp8_fwd(q, torch.tensor(bad, dtype=torch.int32, device=DEV), b.dc, b.ds, o, *b.dt, lse=lse)
        assert B.device_status() == 32, bad
        for r in range(2):
            assert (o[r] == 4).all() == (r in left) and (lse[r] == 4).all() == (r in left), (bad, r)


def test_append_ranges_out_of_bounds_are_flagged_and_their_pages_left():
    b = Batch([20, 30], 8, seed=96, poison=False).device()
    before, scales = _codes(b.dc), b.ds.cpu()
    x = torch.ones(2, 576, dtype=torch.bfloat16, device=DEV)
    last = [int(b.indices[2]), int(b.indices[-1])]         # the page that each sequence's last token lies in
    for bad, left in (([0, 1, 3], [1]), ([0, -5, 2], [0, 1]), ([-2, 1, 2], [0]), ([0, 2, 5], [1]), ([0, 1, 0], [1])):
        b.device()
        B.mla_kv_append_fp8(x, torch.tensor(bad, dtype=torch.int32, device=DEV), b.dc, b.ds, *b.dt)
        assert B.device_status() == 32, bad
        got, now = _codes(b.dc), b.ds.cpu()
        mine = torch.zeros(len(scales), dtype=torch.bool)
        for s in (0, 1):
            if s not in left:
                mine[last[s]] = True
                assert not torch.equal(got[last[s]], before[last[s]])
        assert torch.equal(got[~mine], before[~mine]) and torch.equal(now[~mine], scales[~mine]), bad


@pytest.mark.parametrize("ranges, rows, ps", [
    ([5, 3, 5], 7, 1), ([0, 2, 0, 2, 2], 2, 1), ([1, 2, 0, 0], 2, 1), ([10, 7, 10], 20, 2), ([16, 19, 14, 17, 20], 25, 2),
    ([9, 0, 4, 4], 13, 4), ([0, 0, 40, 40, 4, 5], 60, 4), ([0, 60, 0, 60, 0, 60], 60, 1), ([0, 9, 9, 9, -1, 9], 60, 1)])
def test_append_every_range_that_decreases_is_flagged(ranges, rows, ps):
    """One that decreases by several pages has no block of its own: the next sequence's begin first."""
    b = Batch([60] * (len(ranges) - 1), ps, seed=97, poison=False).device()
    x = torch.ones(rows, 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_append_fp8(x, torch.tensor(ranges, dtype=torch.int32, device=DEV), b.dc, b.ds, *b.dt)
    assert B.device_status() == 32
    b.device()
    ranges = sorted(max(0, r) for r in ranges)
    B.mla_kv_append_fp8(x, torch.tensor(ranges, dtype=torch.int32, device=DEV), b.dc, b.ds, *b.dt)
    assert B.device_status() == 0


# ---------------------------------------------------------------- soft caps of any size
# Capping a score t is off by less than 2^-19.5 of it: below half the cap by a few 2^-24. Above, with x = t / cap,
# u = 1 / (1 + e^2x) is relatively off by 2^-22 + 2^-24 (quotient, sum) and by 1 - u times e^2x's 2^-22 +
# 3 * 2^-24: 1 - 2 u by 2.6 * 2^-22 at most, where it is 0.46 or more. Together with the 18 * 2^-23 = 2^-18.8 S
# of the scores' sums that is still below 2^-18 S.
@pytest.mark.parametrize("cap", [1e-40, 1e-3, 0.5, 50.0, 1e4, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("H, ps", [(16, 64), (40, 3)])
def test_soft_cap_keeps_the_scores_precision(cap, H, ps):
    b = Batch([40, 300, 77, 1], ps, seed=98).device(wide=H > 16)
    cap = float(torch.tensor(cap, dtype=torch.float32))    # the call takes it in 32 bits
    for std, sm_scale in ((6.0, 0.11), (1.0, None), (1e-3, None)):
        q = b.q(4, H, std=std)
        o, lse = _decode(b, q, logit_cap=cap, sm_scale=sm_scale)
        _check(b, q, torch.arange(5), o, lse, logit_cap=cap, sm_scale=sm_scale)
    q = b.q(4, H, std=6.0)
    q[1] = 0.0
    o, lse = _extend(b, q, _indptr([0, 3, 1, 0]), logit_cap=cap)
    _check(b, q, _indptr([0, 3, 1, 0]), o, lse, logit_cap=cap)


# ---------------------------------------------------------------- a caller's scales: no powers of two
def _single_token_batch(scales, seed, slots=1):
    """A sequence per scale, a page each of `slots` + 1 slots, one of them still free."""
    n = len(scales)
    b = Batch([slots + 1] * n, slots + 1, seed=seed, spare=0, poison=False)
    b.scales[b.indices.long(), 0] = torch.tensor(scales, dtype=torch.float32)
    return b


def test_gather_rounds_once_under_any_scale():
    """Products next to the middle of two bf16 values, which fp32 would round to the middle: tie / c with a
    last bit, times c; beside arbitrary scales, and ones below fp32's normal range."""
    scales = [t / c for c in (9, 11, 13, 15) for t in range(257, 512, 2)] + [1.37e-3, 3.1e5, 1e-38, 3e-39, 1e-44, 2.0 ** -130, 0.0,
                                                                             3e38, 1.5 * 2.0 ** 119]
    b = _single_token_batch(scales, 100)
    b.device()
    ip = _indptr(b.lens)
    out = torch.zeros(sum(b.lens), 576, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *b.dt, ip.to(DEV), out)
    want = M8.gather(b.codes, b.scales, b.indptr, b.indices, ip, torch.zeros_like(out).cpu())
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


def test_append_rounds_once_into_pages_of_any_scale():
    """New rows x / scale next to the middle of two codes, into pages whose scale stays: 7 (ties themselves), and
    x / tie with a last bit; then codes times old / scale next to it, into pages whose scale grows."""
    g = torch.Generator().manual_seed(101)
    # (quotients stay below 31 / 16 * 2^6: twice that is below 448, so no scale grows)
    pairs = [(float(x), x * 16 / t) for x in range(128, 256, 3) for t in range(17, 32, 2)] + [(10.9375, 7.0), (12.6875, 7.0)]
    b = _single_token_batch([s for _, s in pairs], 101).device()
    x = torch.tensor([[x] for x, _ in pairs]) * torch.exp2(torch.randint(-8, 7, (len(pairs), 576), generator=g).float())
    x[:, ::2] *= -1
    x[:, 1], x[:, 3], x[:, 5] = math.inf, math.nan, 0.0
    before = b.scales.clone()
    _append_and_check(b, x.to(torch.bfloat16), [1] * len(pairs))
    assert torch.equal(b.scales, before)
    pairs = [(c, t) for c in (9, 11, 13, 15) for t in range(17, 32, 2)]
    b = _single_token_batch([t / c for c, t in pairs], 102, slots=5).device()
    x = torch.randn(len(pairs), 576, generator=g)
    x[:, 7] = 448.0 * 3
    _append_and_check(b, x.to(torch.bfloat16), [1] * len(pairs))
    assert (b.scales == 4).all()


# ---------------------------------------------------------------- whole sequences, bad tables call by call
@pytest.mark.parametrize("many", [1, 100, 148])
def test_decode_whole_sequences_of_the_smallest_scale(many):
    """Up to as many sequences as CTAs, all of 13 tiles: each is taken whole by one CTA (alone it is cut).
    Their scores rise after the first tile by just less than what moves a reference, under the
    smallest scale that an append writes: the sum of 1472 weights stays finite in one place. Any output is
    a mean of values, so it is off by at most twice the largest, 448 * 2^-110."""
    b = Batch([1600], 64, seed=15, scale_exp=(-110, -110))
    flat = b.codes.view(-1, 576)
    at = b.indices[torch.arange(1600) // 64].long() * 64 + torch.arange(1600) % 64
    flat[at, 575] = e4m3_encode(torch.where(torch.arange(1600) >= 128, 128.0, 0.0))
    b.device()
    q = torch.zeros(1, 16, 576)
    q[:, :, 575] = 2.0 ** 103 * 5.75 * math.log(2.0)
    q = q.to(torch.bfloat16)
    ref, ref_lse, _, size, _ = M8.decode(q, b.codes, b.scales, *b.table, sm_scale=1.0)
    b.dt = (torch.arange(many + 1, dtype=torch.int32, device=DEV) * 25, b.dt[1].repeat(many), b.dt[2].repeat(many))
    o, lse = _decode(b, q.expand(many, 16, 576).contiguous(), sm_scale=1.0)
    dl = (lse.cpu().double() - ref_lse).abs()
    assert (dl <= 2.0 ** -17 * (1 + size) + 2.0 ** -21 * (1 + ref_lse.abs())).all()
    assert ((o.cpu().double() - ref).abs() <= 2 * 448 * 2.0 ** -110).all()


@pytest.mark.parametrize("kind", ["page below", "page above", "table end", "table start", "last 0", "last above"])
def test_a_bad_table_leaves_the_other_sequences_right(kind):
    """One sequence's entries are out of range: each call flags it, the others' results are right, and rows and
    pages that are not the bad sequence's stay as they were."""
    lens = [20, 30, 17]
    b = Batch(lens, 8, seed=103, poison=False).device()
    indptr, indices, last = (t.clone() for t in b.table)
    if kind.startswith("page"):
        indices[2] = -1 if kind == "page below" else b.codes.shape[0]       # the first sequence's last page
    elif kind == "table end":                              # the last sequence's pages pass the table's end
        indptr[3] = indices.numel() + 1
    elif kind == "table start":
        indptr[0] = -1
    else:
        last[0] = 0 if kind == "last 0" else 9
    bad = 2 if kind == "table end" else 0
    fine = [s for s in range(3) if s != bad]
    table = tuple(t.to(DEV) for t in (indptr, indices, last))
    ip, full = _indptr([1, 1, 1]), _indptr(lens)
    q = b.q(3, 16)
    ref, ref_lse, mag, size, coded = M8.decode(q, b.codes, b.scales, *b.table)
    bound = _bound(ref, mag, size, coded, 30)
    for qo in (None, ip.to(DEV)):
        o = torch.full((3, 16, 512), 4.0, dtype=torch.bfloat16, device=DEV)
        if qo is None:
            B.mla_decode_fp8_fwd(q.to(DEV), b.dc, b.ds, o, *table)
        else:
            B.mla_extend_fp8_fwd(q.to(DEV), qo, b.dc, b.ds, o, *table)
        assert B.device_status() == 32
        assert ((o.cpu().double() - ref).abs()[fine] <= bound[fine]).all()
    out = torch.full((sum(lens) + 3, 576), 4.0, dtype=torch.bfloat16, device=DEV)
    B.mla_kv_gather_fp8(b.dc, b.ds, *table, full.to(DEV), out)
    assert B.device_status() == 32
    want = M8.gather(b.codes, b.scales, b.indptr, b.indices, full, torch.full((sum(lens) + 3, 576), 4.0, dtype=torch.bfloat16))
    for s in fine:
        assert torch.equal(out[full[s]:full[s + 1]].cpu(), want[full[s]:full[s + 1]])
    assert (out[sum(lens):] == 4).all()
    x = torch.randn(3, 576, generator=b.g).to(torch.bfloat16)
    want_c, want_s = M8.append(x, ip, b.codes, b.scales, *b.table)
    B.mla_kv_append_fp8(x.to(DEV), ip.to(DEV), b.dc, b.ds, *table)
    assert B.device_status() == 32
    own = b.indices[b.indptr[bad]:b.indptr[bad + 1]].long()
    other = torch.ones(b.codes.shape[0], dtype=torch.bool)
    other[own] = False
    assert torch.equal(_codes(b.dc)[other], want_c[other]) and torch.equal(b.ds.cpu()[other], want_s[other])
