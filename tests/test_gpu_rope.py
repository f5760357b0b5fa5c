"""Rotary positions on the GPU against the float64 definition.

attn_rope computes in float32 and rounds once: |y - exact| <= half a step of
the type at |exact| (eps / 2 relative; fp16 never finer than 2^-25) plus the
float32 error of two products and a sum, 3 * 2^-24 (|a c| + |b s|).
attn_rope_tables: the fraction of a turn is exact to 2^-32 turns, its float32
conversion to 2^-25 of an eighth of a turn, sincospif to 2 units of 2^-24:
below 2e-7 in total (2^-32 turns are 1.5e-9).
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_73_gb300 import binding as L
from exact_attention_73_gb300 import inputs, rope
from oracle import score as S

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def tables(n, rot):
    a = np.arange(n, dtype=np.float64)[:, None] * rope.inv_freq(rot).numpy()[None]
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def check(y, x, cos, sin, interleaved, inverse, dtype):
    ref = S.rotate(x, cos, sin, interleaved, inverse)
    mag = np.abs(S.rotate(np.abs(x.double().numpy()), np.abs(cos), -np.abs(sin), interleaved))   # >= |a c| + |b s| on one of the two
    big = np.maximum(mag, np.abs(S.rotate(np.abs(x.double().numpy()), np.abs(cos), np.abs(sin), interleaved)))
    half = torch.finfo(DT[dtype]).eps / 2
    tol = np.maximum(half * np.abs(ref), 2.0 ** -25 if dtype == "fp16" else 0.0) + (1 + half) * 3 * 2.0 ** -24 * big
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("B,H,N,d,rot", [(1, 1, 1, 64, 64), (2, 3, 37, 128, 128), (1, 40, 5, 128, 64), (3, 9, 130, 64, 16),
                                         (1, 17, 300, 256, 256), (2, 8, 1025, 256, 32), (1, 2, 64, 128, 112), (5, 33, 1, 256, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rotation(B, H, N, d, rot, interleaved, inverse, dtype):
    (x,) = inputs.normal(1, [(B, H, N, d)], dtype)
    cos, sin = tables(N, rot)
    y = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
    L.attn_rope(x.cuda(), y, torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), interleaved=interleaved, inverse=inverse)
    check(y, x, cos, sin, interleaved, inverse, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_strides_padding_and_in_place(interleaved):
    B, H, N, d, rot = 3, 5, 50, 128, 96
    (x,) = inputs.normal(2, [(B, N, H + 4, d)])
    r = np.random.default_rng(3)
    pos = r.integers(0, 500, (B, N)).astype(np.int32)
    pos[1, 20:] = -1
    pos[2, 7] = 500          # one past the tables
    cos, sin = tables(500, rot)
    c, s = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    buf = x.cuda()
    view = buf[:, :, 2:2 + H].transpose(1, 2)              # [B, H, N, d] inside a projection's rows
    y = torch.full((B, H, N, d), 7.0, dtype=x.dtype, device="cuda")
    p = torch.from_numpy(pos).cuda()
    L.attn_rope(view, y, c, s, positions=p, interleaved=interleaved)
    assert L.attn_get_device_status() == 3 and L.attn_get_device_status() == 0
    ok = (pos >= 0) & (pos < 500)
    at = np.where(ok, pos, 0)
    xv = x[:, :, 2:2 + H].transpose(1, 2)
    keep = torch.from_numpy(ok)[:, None, :, None].expand(B, H, N, d)
    assert (y.cpu()[~keep] == 7.0).all()
    yy = torch.where(keep, y.cpu(), torch.zeros((), dtype=y.dtype))
    xx = torch.where(keep, xv, torch.zeros((), dtype=y.dtype))
    check(yy, xx, cos[at][:, None], sin[at][:, None], interleaved, False, "bf16")
    # in place, through the same strided view: the rest of the buffer stays
    L.attn_rope(view, view, c, s, positions=p, interleaved=interleaved)
    assert torch.equal(torch.where(keep.cuda(), view, y), y)
    after, before = buf.cpu(), x
    assert torch.equal(after[:, :, :2], before[:, :, :2]) and torch.equal(after[:, :, 2 + H:], before[:, :, 2 + H:])
    assert torch.equal(after[2, 7], before[2, 7]) and torch.equal(after[1, 20:], before[1, 20:])
    L.attn_get_device_status()


def test_the_inverse_is_the_gradient():
    """<rotate(x), g> = <x, rotate back(g)>, as the product of float64 sums of the two results."""
    x, g = inputs.normal(4, [(2, 6, 77, 128)] * 2, "fp16")
    cos, sin = tables(77, 128)
    c, s = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    y, dx = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    L.attn_rope(x.cuda(), y, c, s, interleaved=True)
    L.attn_rope(g.cuda(), dx, c, s, interleaved=True, inverse=True)
    a, b = (y.double() * g.cuda().double()).sum().item(), (x.cuda().double() * dx.double()).sum().item()
    # each of 2 * numel roundings is off by at most 2^-11 of a value below 6, against a factor below 6, at random signs
    assert abs(a - b) <= 6 * 2.0 ** -11 * 36 * math.sqrt(2 * x.numel())


def test_far_offsets_past_32_bits():
    n = 2 ** 25 + 3                       # (n, 64) elements: offsets up to 2^31 + 192
    x = torch.zeros((1, 1, n, 64), dtype=torch.float16, device="cuda")
    x[0, 0, -1] = 1.0
    c, s = torch.full((4, 32), 0.6, device="cuda"), torch.full((4, 32), 0.8, device="cuda")
    pos = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    L.attn_rope(x, x, c, s, positions=pos)
    tail = x[0, 0, -1].float().cpu()
    assert (tail[:32] - (0.6 - 0.8)).abs().max() <= 2e-4 and (tail[32:] - 1.4).abs().max() <= 2e-3
    assert not x[0, 0, :-1].any()


@pytest.mark.parametrize("first,n,rot,amp", [(0, 1, 16, 1.0), (0, 4097, 128, 1.0), (131072, 33, 64, 1.25), (1 << 40, 9, 16, 1.0),
                                             (5, 70000, 256, 1.0)])
def test_tables(first, n, rot, amp):
    f = rope.inv_freq(rot, 500000.0, "parts", 8.0, trained=8192)
    c, s = (torch.full((n, rot // 2), float("nan"), device="cuda") for _ in range(2))
    L.attn_rope_tables(c, s, f.cuda(), first_position=first, amplitude=amp)
    # the angle in whole and fractional turns: position * (f / 2 pi) with f / 2 pi cut to 2^-50 turns is exact
    p = np.arange(first, first + n, dtype=object)
    turns = np.array([[float((int(q) * int(t * 2 ** 62)) % 2 ** 62) / 2 ** 62 for t in (f / (2 * math.pi)).tolist()] for q in p[:200]])
    # the step itself is a float64: position * 2^-53 of its turns
    tol = 2e-7 * amp + 2 * math.pi * (first + n) * 2.0 ** -53 * amp
    assert np.abs(c[:200].double().cpu().numpy() - amp * np.cos(2 * math.pi * turns)).max() <= tol
    assert np.abs(s[:200].double().cpu().numpy() - amp * np.sin(2 * math.pi * turns)).max() <= tol
    one = c.double() ** 2 + s.double() ** 2
    assert (one - amp * amp).abs().max().item() <= 1e-6 * amp * amp


def test_tables_of_frequencies_above_a_turn_and_zero():
    f = torch.tensor([0.0, 7.0, 2 * math.pi, 1e-12, 3.0, 100.5, 1.0, 0.5], dtype=torch.float64)
    c, s = (torch.empty((50, 8), device="cuda") for _ in range(2))
    L.attn_rope_tables(c, s, f.cuda())
    a = np.arange(50)[:, None] * f.numpy()[None]
    assert np.abs(c.double().cpu().numpy() - np.cos(a)).max() <= 2e-7 and np.abs(s.double().cpu().numpy() - np.sin(a)).max() <= 2e-7


def test_captured_and_replayed_on_another_stream():
    (x,) = inputs.normal(5, [(2, 8, 65, 128)])
    xd = x.cuda()
    f = rope.inv_freq(128).cuda()
    c, s = (torch.empty((65, 64), device="cuda") for _ in range(2))
    y = torch.empty_like(xd)

    def step():
        L.attn_rope_tables(c, s, f)
        L.attn_rope(xd, y, c, s)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    want = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    y.fill_(0)
    xd.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -want)
