"""Pins of the serving oracle (rotary embedding, 4-bit records, modified scores): closed forms,
hand-worked values, the float64 attention oracle and torch in float64."""
import numpy as np
import pytest
import torch

from oracle import cp_oracle as orc
from oracle import serving_oracle as so


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_rotation_and_relative(pairs):
    r = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(16) / 16)
    q, k = r.normal(size=(1, 1, 48)), r.normal(size=(1, 1, 48))
    dots = []
    for a, b in [(7, 3), (107, 103), (100007, 100003)]:
        x, y = so.rotate(q, [a], f, pairs), so.rotate(k, [b], f, pairs)
        assert np.isclose((x ** 2).sum(), (q ** 2).sum(), rtol=1e-12)
        assert np.array_equal(x[..., 32:], q[..., 32:])      # dims past rot_dim stay
        dots.append(float((x * y).sum()))
    assert np.allclose(dots, dots[0], rtol=1e-9)             # only the distance matters
    assert np.allclose(so.rotate(q, [0], f, pairs), q)
    one = so.rotate(np.eye(4)[None, :1], [1], [np.pi / 2], pairs)[0, 0]
    assert np.allclose(one, np.eye(4)[1 if pairs else 1])    # (1, 0) a quarter turn on: (0, 1)


def test_bf16_rounding_is_torchs():
    x = np.random.default_rng(2).normal(size=4096) * 10.0 ** np.arange(-8, 8).repeat(256)
    want = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(so.to_bf16(x), want)


@pytest.mark.parametrize("d", [64, 128])
def test_record_layout_by_hand(d):
    rec = np.zeros(9 * d, np.uint8)
    row = np.zeros(d)
    row[0], row[9], row[d - 1] = 15.0, 7.0, 3.0   # minimum 0; scales 1, and 0.2 in the last group
    so.q4_write(rec, 2, row)
    base = 2 * (d // 2)
    assert rec[base] == 15                                    # dim 0: word 0, lowest nibble
    second = 8 if d == 128 else 4                             # dims 8..15: word 2 (d = 128) or 1
    assert rec[base + second] == 7 << 4                       # dim 9: its second nibble
    if d == 128:
        assert rec[base + 63] == 15 << 4                      # dim 127: word 15, highest nibble
        s = so.to_bf16(0.2)
        assert np.allclose(so.q4_read(rec, 2, d)[127], 15 * s)
    assert rec[8 * d + 2 * (d // 16):8 * d + 2 * (d // 16) + 4].tolist() == [0x80, 0x3f, 0, 0]  # 1.0, 0.0
    assert rec[:base].max() == 0 and rec[base + d // 2:8 * d].max() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_record_round_trip_error(d):
    r = np.random.default_rng(3)
    rec = np.full(9 * d, 0xA5, np.uint8)
    for t in range(16):
        row = r.normal(size=d) * 10.0 ** r.uniform(-3, 3) + r.normal() * 5
        so.q4_write(rec, t, row)
        _, sc, mn = so.q4_codes(row)
        # half a step, and what rounding the minimum and the scale to bf16 can cut off the ends
        tol = np.repeat(sc / 2 + 2.0 ** -8 * (np.abs(mn) + 15 * sc), 64)
        assert (np.abs(so.q4_read(rec, t, d) - row) <= tol).all()
    so.q4_write(rec, 0, np.full(d, 2.5))
    assert np.array_equal(so.q4_read(rec, 0, d), np.full(d, 2.5))    # a constant row: scale 0
    bad = np.ones(d)
    bad[5] = np.inf
    so.q4_write(rec, 0, bad)
    assert np.isnan(so.q4_read(rec, 0, d)[:64]).all()
    assert d == 64 or np.array_equal(so.q4_read(rec, 0, d)[64:], np.ones(64))


@pytest.mark.parametrize("cp,I", [(1, 8), (2, 8), (3, 5), (4, 1)])
def test_slots_are_the_deal(cp, I):
    L = 200
    deal = {}
    for r in range(cp):
        for loc, p in enumerate(orc.rank_positions(L, r, cp, I)):
            deal[int(p)] = (r, loc)
    table = np.tile(np.arange(20), (cp, 1))
    for p in range(L):
        r, page, row = so.slot(p, cp, I, table)
        assert (r, page * 16 + row) == deal[p]


def test_attention_reduces_to_the_plain_oracle():
    r = np.random.default_rng(4)
    T, Hq, Hkv, d = 40, 6, 2, 64
    q, k, v = r.normal(size=(T, Hq, d)), r.normal(size=(T, Hkv, d)), r.normal(size=(T, Hkv, d))
    O, L = orc.attention(q, k, v, 0.125)
    for i in range(T):
        lo, hi = so.bounds(i, T)
        o, l, _, _ = so.attend(q[i], k.transpose(1, 0, 2), v.transpose(1, 0, 2), i, lo, hi, 0.125)
        assert np.allclose(o, O[i], atol=1e-12) and np.allclose(l, L[i], atol=1e-12)


def test_modified_attention_against_torch():
    g = torch.Generator().manual_seed(5)
    T, Hq, Hkv, d, cap, W = 33, 4, 2, 64, 3.0, 9
    q, k, v = (torch.randn(T, h, d, generator=g, dtype=torch.float64) for h in (Hq, Hkv, Hkv))
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], dtype=torch.float64)
    start = torch.tensor([0] * 11 + [11] * 15 + [40] * 3 + [26] * 4)   # three rows see nothing
    prefix = 13
    i, j = torch.arange(T)[:, None], torch.arange(T)[None]
    mask = (j >= (i - W + 1)) & (j >= start[:, None]) & ((j <= i) | (j < prefix))
    kk, vv = (x.repeat_interleave(2, 1).permute(1, 0, 2) for x in (k, v))
    s = cap * torch.tanh(q.permute(1, 0, 2) @ kk.transpose(1, 2) * 0.2 / cap)
    s = s - slopes[:, None, None] * (i - j).abs()
    s = s.masked_fill(~mask, -torch.inf)
    O = torch.softmax(s, -1).nan_to_num(0.0) @ vv
    L = torch.logsumexp(s, -1)
    for row in range(T):
        lo, hi = so.bounds(row, T, W, int(start[row]), prefix)
        o, l, _, _ = so.attend(q[row].numpy(), k.permute(1, 0, 2).numpy(), v.permute(1, 0, 2).numpy(), row, lo,
                               hi, 0.2, cap, slopes.numpy())
        assert np.allclose(o, O[:, row].numpy(), atol=1e-12)
        assert np.allclose(l, L[:, row].numpy(), atol=1e-12)
    assert not mask[26:29].any() and np.isneginf(L[:, 26:29].numpy()).all()
