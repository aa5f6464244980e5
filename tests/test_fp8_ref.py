"""The plain forms that the 8-bit products and the routed rows are tested against, on closed forms (no GPU)."""
import pytest
import torch

import fp8_ref as ref

F64 = torch.float64


def test_rounding_hits_every_code_and_breaks_ties_to_even():
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]
    v = ref.decode(codes)
    assert torch.equal(ref.e4m3(v), v)
    pos = v[v > 0].sort().values
    mid = (pos[:-1] + pos[1:]) / 2
    even = torch.where((codes[v > 0][pos.argsort()][:-1] & 1) == 0, pos[:-1], pos[1:])
    assert torch.equal(ref.e4m3(mid), even)
    assert torch.equal(ref.e4m3(mid * (1 + 1e-9)), pos[1:]) and torch.equal(ref.e4m3(mid * (1 - 1e-9)), pos[:-1])
    assert ref.e4m3(torch.tensor([500.0, -1e9, 2.0**-10, 2.0**-11], dtype=F64)).tolist() == [448, -448, 0, 0]


def test_scales_of_known_blocks():
    x = torch.zeros((2, 130), dtype=torch.bfloat16)
    x[0, 3], x[1, 129] = -448.0, 896.0
    q, s = ref.quantize(x, (1, 128))
    assert s[0, 0] == 1 and s[1, 1] == 2 and s[1, 0] == float(torch.tensor(2.0**-50 / 448).float())
    assert q[0, 3] == -448 and q[1, 129] == 448
    q, s = ref.quantize(x, (128, 128))
    assert s.shape == (1, 2) and s[0, 0] == 1 and s[0, 1] == 2
    x[0, 0] = float("inf")
    q, s = ref.quantize(x, (1, 128))
    assert torch.isnan(s[0, 0]) and torch.isnan(q[0, :128]).all() and q[1, 129] == 448 and not torch.isnan(q[0, 128:]).any()


@pytest.mark.parametrize("block", [(1, 128), (128, 128)])
def test_values_are_near(block):
    x = torch.randn((200, 300), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q, s = ref.quantize(x, block)
    v = ref.values(q, s, block)
    # half a step: 2^-4 of the value, or of the smallest normal's step (2^-9, half of it) times the scale
    big = ref.values(torch.ones_like(q), s, block)
    assert ((v - x.to(F64)).abs() <= x.to(F64).abs() * 2.0**-4 * (1 + 1e-6) + big * 2.0**-10).all()


def test_layout_of_a_known_routing():
    ids = torch.tensor([[1, 0], [1, 7], [2, 1]], dtype=torch.int32)
    row, segments, end = ref.layout(ids, 4)
    assert row.tolist() == [[128, 0], [129, -1], [256, 130]]
    assert segments == [(0, 1), (128, 3), (256, 1), (384, 0)] and end == 384


def test_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    ids = torch.tensor([[1, 0], [1, 1], [2, 9]], dtype=torch.int32)
    row, _, end = ref.layout(ids, 3)
    n = lambda *s: torch.randn(s, generator=g, dtype=F64)  # noqa: E731
    rows, w, dout = n(end, 5), n(3, 2), n(3, 5)
    drows, dw, _ = ref.combine_grads(rows, dout, row, w)
    loss = lambda r, v: (ref.combine(r, row, v)[0] * dout).sum()  # noqa: E731
    for i, j in ((0, 2), (129, 4), (130, 0), (5, 1)):
        e = torch.zeros_like(rows)
        e[i, j] = 1
        assert abs(loss(rows + e, w) - loss(rows, w) - drows[i, j]) < 1e-10
    for t in range(3):
        for k in range(2):
            e = torch.zeros_like(w)
            e[t, k] = 1
            assert abs(loss(rows, w + e) - loss(rows, w) - dw[t, k]) < 1e-10
    # dispatch's gradient is the sum of the rows
    x, d = n(3, 5), n(end, 5)
    assert abs((ref.dispatch(x, row, end) * d).sum() - (x * ref.combine(d, row)[0]).sum()) < 1e-10
