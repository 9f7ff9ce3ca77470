"""Pins for the 8-bit latent cache's oracle: cases by hand and against other definitions."""
import math
from fractions import Fraction

import pytest
import torch

from oracle import mla_fp8_oracle as M8
from oracle import mla_oracle as M
from oracle.fp8moe_oracle import e4m3_decode, e4m3_encode


def test_scale_is_the_smallest_power_of_two_that_fits():
    for amax, s in ((448.0, 1.0), (448.5, 2.0), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (1.0, 2.0 ** -8),
                    (0.0, 0.0), (3e38, 2.0 ** 120), (1e-38, 2.0 ** -110)):
        assert M8.scale_of(torch.tensor([[amax, -amax / 2]], dtype=torch.float64)) == s
    assert M8.scale_of(torch.tensor([[math.inf, 2.0, math.nan]])) == 2.0 ** -7


def _table(L, ps, pages):
    n = -(-L // ps)
    return torch.tensor([0, n]), torch.tensor(pages[:n]), torch.tensor([L - (n - 1) * ps])


def test_append_by_hand_growth_and_a_fresh_page():
    ps, codes = 4, torch.full((3, 4, 1, 576), 0x11, dtype=torch.uint8)
    scales = torch.tensor([[8.0], [8.0], [8.0]])
    # two tokens from the start: the page's earlier scale is forgotten
    x = torch.zeros(2, 576)
    x[0, 0], x[1, 1] = 448.0, 3.0
    c, s = M8.append(x, [0, 2], codes, scales, *_table(2, ps, [1]))
    assert s.flatten().tolist() == [8.0, 1.0, 8.0]
    assert e4m3_decode(c[1, 0, 0])[0] == 448 and e4m3_decode(c[1, 1, 0])[1] == 3
    assert (c[1, 2:] == 0x11).all() and (c[0] == 0x11).all() and (c[2] == 0x11).all()
    # three more, of which one needs scale 4: the rows before are divided by 4, and the last opens page 2
    y = torch.zeros(3, 576)
    y[0, 0], y[1, 0], y[2, 0] = 1.0, 1000.0, 0.875
    c2, s2 = M8.append(y, [0, 3], c, s, *_table(5, ps, [1, 2]))
    assert s2.flatten().tolist() == [8.0, 4.0, 2.0 ** -9]
    v = e4m3_decode(c2[1, :, 0]) * 4
    assert v[0, 0] == 448 and v[1, 1] == 3 and v[2, 0] == 1 and v[3, 0] == 1024   # 250 -> 256
    assert e4m3_decode(c2[2, 0, 0])[0] == 448


def test_append_in_one_call_or_token_by_token_agree_where_no_code_falls_to_subnormals():
    g = torch.Generator().manual_seed(0)
    ps, T = 5, 13
    x = torch.exp2(torch.randint(-3, 4, (T, 576), generator=g).float()) * torch.where(
        torch.rand(T, 576, generator=g) < 0.5, -1.0, 1.0)
    pages = [4, 0, 2]
    codes, scales = torch.zeros(5, ps, 1, 576, dtype=torch.uint8), torch.zeros(5, 1)
    one_c, one_s = M8.append(x, [0, T], codes, scales, *_table(T, ps, pages))
    c, s = codes, scales
    for t in range(T):
        c, s = M8.append(x[t:t + 1], [0, 1], c, s, *_table(t + 1, ps, pages))
    assert torch.equal(one_s, s)
    got = e4m3_decode(c) * s[:, :, None, None]
    assert torch.equal(got, e4m3_decode(one_c) * one_s[:, :, None, None])


def test_attention_equals_the_bf16_oracle_on_exact_values_and_is_causal():
    g = torch.Generator().manual_seed(1)
    ps, L, H = 3, 10, 2
    codes = e4m3_encode(torch.randn(6, ps, 1, 576, generator=g) * 16)
    scales = torch.full((6, 1), 2.0 ** -4)
    q = torch.randn(4, H, 576, generator=g).to(torch.bfloat16)
    table = _table(L, ps, [5, 0, 3, 1])
    o, lse, mag, _, _ = M8.extend(q, [0, 4], codes, scales, *table, logit_cap=3.0)
    values = e4m3_decode(codes) * 2.0 ** -4
    for i in range(4):
        ref, ref_lse = M.mla_decode(q[i:i + 1], values, *_table(L - 3 + i, ps, [5, 0, 3, 1]), logit_cap=3.0)
        assert torch.allclose(o[i], ref[0], rtol=1e-12, atol=1e-14) and torch.allclose(lse[i], ref_lse[0], rtol=1e-12)
    assert (mag >= o.abs() - 1e-12).all()


def test_queries_before_the_first_token_see_nothing_and_gather_rounds_once():
    codes = torch.full((1, 2, 1, 576), 0x39, dtype=torch.uint8)                     # 1.125
    scales = torch.tensor([[0.5]])
    q = torch.ones(3, 1, 576, dtype=torch.bfloat16)
    o, lse, *_ = M8.extend(q, [0, 3], codes, scales, *_table(2, 2, [0]))
    assert (o[0] == 0).all() and lse[0, 0] == -math.inf
    assert o[1, 0, 0] == 0.5625 and lse[1, 0].item() == pytest.approx(576 * 0.5625 / 24)
    out = M8.gather(codes, scales, [0, 1], [0], [1, 3], torch.full((4, 576), 7.0, dtype=torch.bfloat16))
    assert (out[1:3] == 0.5625).all() and (out[0] == 7).all() and (out[3] == 7).all()


def test_append_clears_codes_of_a_page_whose_scale_was_zero():
    """A row of zeros and infinities has scale 0 and codes of +-448, which stand for 0; they still stand
    for 0 (and NaN for NaN) once a later row raises the page's scale."""
    ps, codes, scales = 4, torch.zeros(1, 4, 1, 576, dtype=torch.uint8), torch.zeros(1, 1)
    x = torch.zeros(1, 576)
    x[0, 0], x[0, 1], x[0, 2] = math.inf, -math.inf, math.nan
    c, s = M8.append(x, [0, 1], codes, scales, *_table(1, ps, [0]))
    assert s[0, 0] == 0 and e4m3_decode(c[0, 0, 0])[:2].tolist() == [448.0, -448.0]
    c, s = M8.append(torch.full((1, 576), 1.75), [0, 1], c, s, *_table(2, ps, [0]))
    assert s[0, 0] == 2.0 ** -8
    v = e4m3_decode(c[0, :2, 0]) * 2.0 ** -8
    assert (v[0, :2] == 0).all() and math.isnan(v[0, 2]) and (v[0, 3:] == 0).all() and (v[1] == 1.75).all()


def test_append_rounds_once_where_a_page_came_with_a_scale_that_is_no_power_of_two():
    """Quotients at or next to the middle of two codes, which a rounding before the code's would move there."""
    ps = 2

    def nearest(q, step):                                          # of the fraction q, ties to even
        n = q / step
        lo = n.numerator // n.denominator
        up = n - lo > Fraction(1, 2) or (n - lo == Fraction(1, 2) and lo % 2)
        return float((lo + up) * step)

    for x, old in ((10.9375, 7.0), (12.6875, 7.0), (128.0, 128 * 16 / 19), (128.0, 128 * 16 / 29), (129.0, 129 * 16 / 21)):
        scale = torch.tensor([[old]], dtype=torch.float32)
        q = Fraction(x) / Fraction(scale.item())
        assert 1 < q < 2 and abs(q * 16 - round(q * 16)) < Fraction(1, 2 ** 18) and round(q * 16) % 2
        c, s = M8.append(torch.full((1, 576), x), [0, 1], torch.zeros(1, 2, 1, 576, dtype=torch.uint8), scale,
                         *_table(2, ps, [0]))
        assert s[0, 0] == scale[0, 0] and (e4m3_decode(c[0, 1, 0]) == nearest(q, Fraction(1, 8))).all()
    # and codes carried over to a larger scale
    for code, tie in ((9, 29), (9, 31), (11, 23), (13, 19), (15, 31)):
        scale = torch.tensor([[tie / code]], dtype=torch.float32)
        q = code * Fraction(scale.item()) / 4
        c, s = M8.append(torch.full((1, 576), 1000.0), [0, 1], e4m3_encode(torch.full((1, 2, 1, 576), float(code))), scale,
                         *_table(2, ps, [0]))
        assert s[0, 0] == 4.0 and q * 4 != tie and (e4m3_decode(c[0, 0, 0]) == nearest(q, Fraction(1, 2))).all()
