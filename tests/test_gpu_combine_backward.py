"""Gradient of the combine against a plain 64-bit form.

A row of dy is one fp32 product rounded once to bf16: equal bit for bit.  A weight's gradient is a sum of products
that a lane adds one after the other, at most 8 * 32 here, then 5 + 8 additions: 2^-16 of the sum of magnitudes.
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def case(N, K, E, A, H, masked, seed, extra=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    idx = torch.rand((N, E), generator=g, device=DEV).argsort(1)[:, :K] if K <= E else torch.randint(0, E, (N, K), generator=g, device=DEV)
    idx = torch.where(torch.rand((N, K), generator=g, device=DEV) < masked, -1, idx).long()
    cap = N * K + E * (A - 1) + extra
    lay = binding.Layout(binding.LayoutDesc(N, K, E, 1, A), cap).build(idx.contiguous())
    dout = torch.randn((N, H), generator=g, device=DEV).to(BF16)
    y = torch.randn((cap, H), generator=g, device=DEV).to(BF16)
    w = torch.randn((N, K), generator=g, device=DEV)
    return lay, dout, y, w


def check(lay, dout, y, w, dy, dw, zero_pad=True):
    N, K = w.shape
    slot = lay.dst_slot[:N * K].view(N, K).long()
    want = torch.full(dy.shape, 7.0, dtype=BF16, device=DEV)
    off, cnt = lay.expert_offset.tolist(), lay.expert_count.tolist()
    if zero_pad:
        for e, c in enumerate(cnt):
            want[off[e] + c:off[e + 1]] = 0
    t, k = torch.nonzero(slot >= 0, as_tuple=True)
    want[slot[t, k]] = (w[t, k].unsqueeze(1) * dout[t].float()).to(BF16)
    assert torch.equal(dy, want)
    if dw is not None:
        prod = torch.zeros((N, K, dout.shape[1]), dtype=torch.float64, device=DEV)
        prod[t, k] = y[slot[t, k]].double() * dout[t].double()
        assert torch.all((dw.double() - prod.sum(2)).abs() <= 2.0 ** -16 * prod.abs().sum(2))
        assert torch.all(dw[slot < 0] == 0)


CASES = [
    (1, 1, 1, 1, 8, 0.0), (1, 8, 256, 16, 7168, 0.0), (5, 3, 8, 4, 264, 0.3), (40, 9, 16, 16, 1040, 0.2), (33, 32, 8, 1, 512, 0.5),
    (700, 2, 8, 128, 2056, 0.1), (2000, 8, 64, 64, 256, 0.05), (1500, 4, 33, 8, 4096, 0.9), (3, 2, 4, 128, 8192, 1.0),
]


@pytest.mark.parametrize("N,K,E,A,H,masked", CASES)
def test_rows_and_weights(N, K, E, A, H, masked):
    lay, dout, y, w = case(N, K, E, A, H, masked, N + K + H)
    for zero_pad in (True, False):
        dy, dw = torch.full(y.shape, 7.0, dtype=BF16, device=DEV), torch.full((N, K), 9.0, device=DEV)
        lay.combine_backward(dout, w, dy, y, dw, zero_pad=zero_pad)
        assert lay.error() == 0
        check(lay, dout, y, w, dy, dw, zero_pad)
        again = torch.empty_like(dw)
        lay.combine_backward(dout, w, dy, y, again, zero_pad=zero_pad)
        assert torch.equal(again, dw)
    dy.fill_(7.0)
    lay.combine_backward(dout, w, dy)
    check(lay, dout, y, w, dy, None)


@pytest.mark.parametrize("N,H", [(20, 1040), (1500, 512)])
def test_in_place(N, H):
    """dy written over the expert outputs, which each column's reader has by then."""
    lay, dout, y, w = case(N, 5, 16, 16, H, 0.1, 3)
    dy, dw = y.clone(), torch.empty_like(w)
    lay.combine_backward(dout, w, dy, y, dw)
    own, dw2 = y.clone(), torch.empty_like(w)
    lay.combine_backward(dout, w, own, own, dw2)
    assert torch.equal(own, dy) and torch.equal(dw, dw2) and lay.error() == 0


def test_slots_past_the_rows_are_recorded():
    lay, dout, y, w = case(30, 2, 4, 1, 256, 0.0, 4)
    short = y[:50].contiguous()
    dy, dw = torch.full_like(short, 7.0), torch.full_like(w, 9.0)
    lay.combine_backward(dout, w, dy, short, dw)
    assert lay.error() == 4
    slot = lay.dst_slot[:60].view(30, 2).long()
    assert torch.all(dw[slot >= 50] == 0)
    t, k = torch.nonzero(slot < 50, as_tuple=True)
    assert torch.equal(dy[slot[t, k]], (w[t, k].unsqueeze(1) * dout[t].float()).to(BF16))


def test_layout_that_overflowed():
    """A layout without room has no slots: nothing of a row is written."""
    N, K, E = 30, 2, 4
    idx = torch.randint(0, E, (N, K), device=DEV)
    lay = binding.Layout(binding.LayoutDesc(N, K, E, 1, 16), 40).build(idx)
    assert lay.error() == 4
    dy, dw = torch.full((40, 64), 7.0, dtype=BF16, device=DEV), torch.full((N, K), 9.0, device=DEV)
    lay.combine_backward(torch.ones((N, 64), dtype=BF16, device=DEV), torch.ones((N, K), device=DEV), dy, dy.clone(), dw, zero_pad=False)
    assert torch.all(dy == 7.0) and torch.all(dw == 0.0) and lay.error() == 0


def test_no_tokens():
    lay = binding.Layout(binding.LayoutDesc(0, 2, 4, 1, 8), 16).build(torch.empty((0, 2), dtype=torch.int64, device=DEV))
    dy = torch.full((16, 64), 7.0, dtype=BF16, device=DEV)
    lay.combine_backward(torch.empty((0, 64), dtype=BF16, device=DEV), torch.empty((0, 2), device=DEV), dy)
    assert torch.all(dy == 7.0) and lay.error() == 0


def test_against_differences():
    """<out, dout> moved in one weight, and in the expert outputs along dy, changes as the gradient says.

    Both are linear, so a difference is the derivative up to rounding: of out to bf16 (2^-8 of each value's magnitude)."""
    lay, dout, y, w = case(50, 3, 8, 8, 512, 0.1, 6)
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    lay.combine_backward(dout, w, dy, y, dw)
    out = lambda w, y: (lambda o: (lay.combine(y, w, o), o)[1])(torch.empty((50, 512), dtype=BF16, device=DEV)).double()
    at = lay.dst_slot[:150].view(50, 3).long()
    base = out(w, y)
    for k in range(3):
        moved = w.clone()
        moved[:, k] += 1.0
        diff = (out(moved, y) - base) * dout.double()
        off = 2.0 ** -8 * ((out(moved, y).abs() + base.abs()) * dout.double().abs()).sum(1) + 2.0 ** -16 * (diff.abs().sum(1) + 1)
        real = at[:, k] >= 0
        assert torch.all(((diff.sum(1) - dw[:, k].double()).abs() <= off)[real])
    step = torch.randn(y.shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF16)
    moved = (y.float() + step.float()).to(BF16)
    delta = moved.double() - y.double()
    delta[torch.isin(torch.arange(len(y), device=DEV), at[at >= 0], invert=True)] = 0
    want = (delta * dy.double()).sum()
    a, b = out(w, moved), base
    off = 2.0 ** -8 * ((a.abs() + b.abs()) * dout.double().abs()).sum() + 2.0 ** -8 * (delta * dy.double()).abs().sum()
    assert (((a - b) * dout.double()).sum() - want).abs() <= off


def test_graph_and_stream():
    lay, dout, y, w = case(64, 4, 8, 16, 512, 0.1, 7)
    dy, dw = torch.full(y.shape, 7.0, dtype=BF16, device=DEV), torch.empty_like(w)
    lay.combine_backward(dout, w, dy, y, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.combine_backward(dout, w, dy, y, dw)
    dout.copy_(dout.flip(0))
    w.copy_(w.flip(0))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph.replay()
    s.synchronize()
    check(lay, dout, y, w, dy, dw)
    assert lay.error() == 0
