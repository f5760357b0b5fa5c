"""Score-modified attention on the GPU against the float64 definition: tanh
cap, distance bias, documents, prefixes, padding, windows; forward, backward
and the row masks.

Tolerances. Forward and LSE, with A = sum_j p_j |v_j| (per element) and
X = scale log2(e) max_j sum |q||k| (per row): a score in log2 units is off by
at most dx = (d + 8) 2^-24 X + 6e-7 X' + 2^-22 (X' + slope distance), X' =
min(X, cap log2(e)) (the tanh's 6e-7 of the score only with a cap); O by
A (h + 2 dx ln 2 + 2^-20) + h |O| with h half a step of the type (P and O
rounded once each), LSE by dx ln 2 + 2^-20 (1 + |LSE|).
Backward: those of attn_bwd, relative RMS <= 1e-2 on each gradient.
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_73_gb300 import binding as L
from exact_attention_73_gb300 import inputs
from oracle import attention as A
from oracle import score as S

pytestmark = pytest.mark.gpu
I32 = torch.int32
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def slopes_of(H):
    return (2.0 ** (-8.0 * (np.arange(H) + 1) / H)).astype(np.float32)


def run_fwd(q, k, v, ranges=None, slopes=None, cap=0.0, window=(-1, -1)):
    B, Hq, N, d = q.shape
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, Hq, N), float("nan"), device="cuda")
    ws = None if ranges is None else torch.full((L.attn_score_workspace_size(B, N),), 0xff, dtype=torch.uint8, device="cuda")
    L.attn_fwd_score(q, k, v, o, lse, workspace=ws, row_ranges=ranges, slopes=slopes, score_cap=cap, window=window)
    return o, lse


def run_bwd(q, k, v, o, lse, do, ranges=None, slopes=None, cap=0.0, window=(-1, -1)):
    B, Hq, N, d = q.shape
    g = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    ws = torch.full((L.attn_bwd_score_workspace_size(B, Hq, k.shape[1], N, d),), 0xff, dtype=torch.uint8, device="cuda")
    L.attn_bwd_score(q, k, v, o, lse, do, *g, ws, row_ranges=ranges, slopes=slopes, score_cap=cap, window=window)
    return g


def check(seed, B, Hq, Hkv, N, d, dtype="bf16", ranges=None, slopes=False, cap=0.0, window=(-1, -1), gain=1.0, backward=True):
    q, k, v, do = inputs.normal(seed, [(B, Hq, N, d), (B, Hkv, N, d), (B, Hkv, N, d), (B, Hq, N, d)], dtype)
    q = q * gain
    sl = slopes_of(Hq) if slopes else None
    scale = d ** -0.5
    dev = [x.cuda() for x in (q, k, v, do)]
    r = None if ranges is None else torch.from_numpy(np.ascontiguousarray(ranges)).to(I32).cuda()
    mods = (r, None if sl is None else torch.from_numpy(sl).cuda(), cap, window)
    o, lse = run_fwd(*dev[:3], *mods)
    assert L.attn_get_device_status() == 0
    ro, rl = S.forward(q, k, v, scale, ranges, window, cap, sl)
    mag, _ = S.forward(q, k, v.abs(), scale, ranges, window, cap, sl)
    G = Hq // Hkv
    X = np.stack([[1.4427 * scale * (np.abs(q[b, h].double().numpy()) @ np.abs(k[b, h // G].double().numpy()).T).max(1)
                   for h in range(Hq)] for b in range(B)])
    Xc = np.minimum(X, cap * 1.4427) if cap else X
    dx = (d + 8) * 2.0 ** -24 * X + (6e-7 * Xc if cap else 0) + 2.0 ** -22 * Xc
    if slopes:
        dx = dx + 2.0 ** -22 * 1.4427 * sl[None, :, None] * N
    h = torch.finfo(DT[dtype]).eps / 2
    tol = mag * (h + (2 * dx * math.log(2) + 2.0 ** -20)[..., None]) * (1 + h) + h * np.abs(ro) + 2.0 ** -25
    err = np.abs(o.double().cpu().numpy() - ro)
    assert (err <= tol).all(), (err - tol).max()
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert (np.abs(gl[fin] - rl[fin]) <= dx[fin] * math.log(2) + 2.0 ** -20 * (1 + np.abs(rl[fin]))).all()
    if not backward:
        return
    got = run_bwd(*dev[:3], o, lse, dev[3], *mods)
    assert L.attn_get_device_status() == 0
    # fp32 sums of dP and D cancel where a row sees one key: (d + 8) 2^-24 of their magnitude is left, times the other operand
    floor = (d + 8) * 2.0 ** -24 * scale * float(do.abs().double().max() * v.abs().double().max()) * d * float(max(q.abs().max(), k.abs().max()))
    vis = [S._visible(N, None if ranges is None else ranges[b], window) for b in range(B)]
    alone = {"dq": np.stack([~m.any(1) for m in vis]), "dk": np.stack([~m.any(0) for m in vis])}
    alone["dv"] = alone["dk"]
    for name, x, ref in zip(("dq", "dk", "dv"), got, S.backward(q, k, v, do, scale, ranges, window, cap, sl)):
        x = x.double().cpu().numpy()
        assert np.isfinite(x).all(), name
        n = np.linalg.norm(ref)
        assert np.linalg.norm(x - ref) <= 1e-2 * n + floor * math.sqrt(ref.size), (name, np.linalg.norm(x - ref) / max(n, 1e-30))
        # rows that see nothing and keys that nobody sees have an exact zero
        assert not x.transpose(0, 2, 1, 3)[alone[name]].any(), name


def documents(seed, B, N, docs, pad=0):
    r = np.random.default_rng(seed)
    ids = np.zeros((B, N), np.int32)
    for b in range(B):
        cuts = np.sort(r.integers(1, N, docs - 1)) if docs > 1 and N > 1 else []
        for c in cuts:
            ids[b, c:] += 1
        if pad:
            ids[b, N - r.integers(0, pad + 1):] = -1
    return ids


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 1023, 1024, 1025, 5000])
@pytest.mark.parametrize("docs", [None, 1, 4, 900])
@pytest.mark.parametrize("causal,prefix", [(True, None), (True, [0, 700, 10 ** 6]), (False, None), (False, [5, 5, 5])])
def test_mask_rows(N, docs, causal, prefix):
    ids = None if docs is None else documents(1, 3, N, min(docs, N), pad=N // 3)
    want = S.mask_rows(3, N, ids, prefix, causal)
    got = torch.full((3, N, 2), -7, dtype=I32, device="cuda")
    L.attn_mask_rows(got, doc_ids=None if ids is None else torch.from_numpy(ids).cuda(),
                     prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=I32, device="cuda"), causal=causal)
    assert np.array_equal(got.cpu().numpy(), want)


def test_mask_rows_of_alternating_and_long_documents():
    N = 300000
    ids = np.zeros((2, N), np.int32)
    ids[0, 1::2] = 1
    ids[1, 123456:] = -4
    ids[1, 200000:] = 9
    got = torch.empty((2, N, 2), dtype=I32, device="cuda")
    L.attn_mask_rows(got, doc_ids=torch.from_numpy(ids).cuda(), causal=False)
    g = got.cpu().numpy()
    assert (g[0] == np.stack([np.arange(N), np.arange(N) + 1], 1)).all()
    assert (g[1, :123456] == [0, 123456]).all() and not g[1, 123456:200000].any() and (g[1, 200000:] == [200000, N]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap,slopes,gain", [(0.0, False, 1.0), (30.0, False, 1.0), (8.0, False, 3.0), (2.0, False, 6.0),
                                             (0.0, True, 1.0), (20.0, True, 2.0)])
@pytest.mark.parametrize("window", [(-1, 0), (-1, -1)])
def test_cap_and_bias(d, dtype, cap, slopes, gain, window):
    check(10, 1, 4, 2, 333, d, dtype, None, slopes, cap, window, gain)


@pytest.mark.parametrize("N", [1, 2, 17, 64, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("masked", [False, True])
def test_lengths(N, masked):
    ranges = S.mask_rows(2, N, documents(11, 2, N, min(3, N), pad=N // 2), None, True) if masked else None
    check(12, 2, 3, 1, N, 128, ranges=ranges, cap=25.0, slopes=True, window=(-1, -1) if masked else (-1, 0))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,prefix,docs,pad", [(True, None, 5, 0), (False, None, 5, 0), (True, [300, 0], 1, 200), (True, [500, 90], 3, 100),
                                                    (False, None, 40, 300), (True, None, 600, 0)])
def test_documents_prefixes_and_padding(d, causal, prefix, docs, pad):
    ranges = S.mask_rows(2, 600, documents(13, 2, 600, docs, pad), prefix, causal)
    check(14, 2, 4, 2, 600, d, "fp16", ranges)
    check(15, 2, 4, 4, 600, d, "bf16", ranges, True, 15.0, gain=2.0)


@pytest.mark.parametrize("window", [(100, 0), (-1, 30), (7, 7), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1), (64, -1)])
@pytest.mark.parametrize("masked", [False, True])
def test_windows(window, masked):
    ranges = S.mask_rows(1, 500, documents(16, 1, 500, 3, 50), None, False) if masked else None
    w = tuple(min(x, 500) for x in window)
    q, k, v = (x.cuda() for x in inputs.normal(17, [(1, 2, 500, 64)] * 3))
    r = None if ranges is None else torch.from_numpy(ranges).to(I32).cuda()
    if window[0] > 1000:   # the widest windows mask nothing
        a, b = run_fwd(q, k, v, r, window=window), run_fwd(q, k, v, r)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ga, gb = (run_bwd(q, k, v, *a, q, r, window=x) for x in (window, (-1, -1)))
        assert all(torch.equal(x, y) for x, y in zip(ga[1:], gb[1:]))
    check(18, 1, 4, 2, 500, 64, "bf16", ranges, True, 10.0, w)


def test_any_ranges_of_the_callers_own():
    """Ranges out of [0, N], empty and reversed ones, rows that see one far key, tiles that see nothing."""
    N = 520
    r = np.random.default_rng(19)
    ranges = r.integers(-50, N + 50, (2, N, 2))
    ranges[0, :256] = (40, 40)                 # two query tiles that see nothing
    ranges[0, 256:384] = (500, 501)            # one far key
    ranges[1, 100:300, 1] = ranges[1, 100:300, 0] - 5
    ranges[1, 400:] = (0, 1)                   # everybody on the first key
    cut = np.stack([ranges[..., 0].clip(0, N), ranges[..., 1].clip(0, N)], -1)
    q, k, v, do = inputs.normal(20, [(2, 4, N, 128), (2, 2, N, 128), (2, 2, N, 128), (2, 4, N, 128)])
    dev = [x.cuda() for x in (q, k, v, do)]
    rg = torch.from_numpy(ranges).to(I32).cuda()
    o, lse = run_fwd(*dev[:3], rg, cap=9.0)
    o2, lse2 = run_fwd(*dev[:3], torch.from_numpy(cut).to(I32).cuda(), cap=9.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(20, 2, 4, 2, N, 128, "bf16", cut, False, 9.0)


def test_without_changes_it_is_attn_fwd_and_attn_bwd():
    q, k, v, do = (x.cuda() for x in inputs.normal(21, [(2, 4, 700, 128), (2, 2, 700, 128), (2, 2, 700, 128), (2, 4, 700, 128)]))
    o, lse = run_fwd(q, k, v, window=(-1, 0))
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    L.attn_fwd(q, k, v, o2, lse2, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = run_bwd(q, k, v, o, lse, do, window=(-1, 0))
    g2 = [torch.empty_like(x) for x in (q, k, v)]
    ws = torch.empty(L.attn_bwd_workspace_size(2, 4, 2, 700, 128), dtype=torch.uint8, device="cuda")
    L.attn_bwd(q, k, v, o, lse, do, *g2, ws, causal=True)
    assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])


def test_extreme_scores():
    """Scores far beyond the cap (tanh at +-1), tiny and huge scales and caps."""
    q, k, v = inputs.normal(22, [(1, 2, 300, 64)] * 3)
    for gain, cap, scale in ((300.0, 5.0, 0.125), (1.0, 1e-3, 0.125), (1.0, 1e5, 0.125), (3.0, 4.0, 0.5), (1.0, 20.0, 1e-9), (1.0, 1e-6, 40.0)):
        o, lse = torch.empty_like(q, device="cuda"), torch.empty((1, 2, 300), device="cuda")
        qg = q * gain
        L.attn_fwd_score(qg.cuda(), k.cuda(), v.cuda(), o, lse, score_cap=cap, window=(-1, 0), scale=scale)
        ro, rl = S.forward(qg, k, v, scale, None, (-1, 0), cap)
        mag, _ = S.forward(qg, k, v.abs(), scale, None, (-1, 0), cap)
        X = min(cap, abs(scale) * gain * 64 * 12.0) * 1.4427       # |q.k| < 64 * 12 for these inputs
        d_ = 1e-6 * X + 2.0 ** -18 * min(X, 40.0) + 2.0 ** -20
        assert (np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * d_) * mag * 1.01).all(), (gain, cap, scale)
        assert np.abs(lse.double().cpu().numpy() - rl).max() <= d_ + 2.0 ** -20 * (1 + np.abs(rl).max()), (gain, cap, scale)


def test_gradients_against_differences():
    """The kernel's own gradients against differences of its own forward: d/dt of sum(dO o O(x + t dx)) along a
    direction, in fp16 with a step that keeps the rounding of O (2^-11 of each of 2 * numel values, random) below a hundredth."""
    q, k, v, do = inputs.normal(23, [(1, 2, 256, 64)] * 4, "fp16")
    ids = documents(24, 1, 256, 3, 40)
    r = torch.from_numpy(S.mask_rows(1, 256, ids, [60], True)).to(I32).cuda()
    mods = (r, torch.from_numpy(slopes_of(2)).cuda(), 3.0)
    dev = [x.cuda() for x in (q * 2, k, v)]
    o, lse = run_fwd(*dev, *mods)
    grads = run_bwd(*dev, o, lse, do.cuda(), *mods)
    for i in range(3):
        step = torch.sign(grads[i].float()) * 2.0 ** -5          # uphill
        up, down = [x.clone() for x in dev], [x.clone() for x in dev]
        up[i] = (dev[i].float() + step).half()
        down[i] = (dev[i].float() - step).half()
        moved = up[i].double() - down[i].double()
        f = [(run_fwd(*x, *mods)[0].double() * do.cuda().double()).sum().item() for x in (up, down)]
        want = (moved * grads[i].double()).sum().item()
        assert abs((f[0] - f[1]) - want) <= 0.02 * abs(want), (i, f[0] - f[1], want)


def test_a_training_run_captured_and_replayed():
    """Rotate q and k, attend over packed documents with a cap, go back through both: against float64, and captured into a graph."""
    B, Hq, Hkv, N, d = 1, 4, 2, 400, 128
    x = inputs.normal(25, [(B, N, Hq + 2 * Hkv, d), (B, Hq, N, d)])
    ids = documents(26, B, N, 4, 30)
    pos = np.zeros((B, N), np.int32)             # positions restart with each document; padding has none
    rows = S.mask_rows(B, N, ids, None, False)
    pos[0] = np.where(ids[0] < 0, -1, np.arange(N) - rows[0, :, 0])
    from oracle import fp8 as F
    cos, sin = F.rope_tables(N, d)
    c, s, p, di = (torch.from_numpy(t).cuda() for t in (cos, sin, pos, ids))
    qkv, do = (t.cuda() for t in x)
    q, k = torch.zeros((B, Hq, N, d), dtype=qkv.dtype, device="cuda"), torch.zeros((B, Hkv, N, d), dtype=qkv.dtype, device="cuda")
    v = torch.empty_like(k)
    rr = torch.empty((B, N, 2), dtype=I32, device="cuda")
    ws = torch.empty(L.attn_score_workspace_size(B, N), dtype=torch.uint8, device="cuda")
    wb = torch.empty(L.attn_bwd_score_workspace_size(B, Hq, Hkv, N, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, Hq, N), device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    dqkv = torch.zeros_like(qkv)

    def heads(t, a, n):
        return t[:, :, a:a + n].transpose(1, 2)

    def step():
        L.attn_rope(heads(qkv, 0, Hq), q, c, s, positions=p)
        L.attn_rope(heads(qkv, Hq, Hkv), k, c, s, positions=p)
        v.copy_(heads(qkv, Hq + Hkv, Hkv))
        L.attn_mask_rows(rr, doc_ids=di)
        L.attn_fwd_score(q, k, v, o, lse, workspace=ws, row_ranges=rr, score_cap=20.0)
        L.attn_bwd_score(q, k, v, o, lse, do, dq, dk, dv, wb, row_ranges=rr, score_cap=20.0)
        L.attn_rope(dq, heads(dqkv, 0, Hq), c, s, positions=p, inverse=True)
        L.attn_rope(dk, heads(dqkv, Hq, Hkv), c, s, positions=p, inverse=True)

    step()
    torch.cuda.synchronize()
    assert L.attn_get_device_status() == 0
    first = [t.clone() for t in (o, lse, dqkv, dv)]
    xx = x[0].double().numpy()
    at = np.maximum(pos[0], 0)
    qf, kf, vf = (xx[:, :, a:b].transpose(0, 2, 1, 3) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    qr, kr = (S.rotate(t, cos[at], sin[at]) for t in (qf, kf))
    ranges = S.mask_rows(B, N, ids, None, True)
    gq, gk, gv = S.backward(qr, kr, vf, x[1], d ** -0.5, ranges, cap=20.0)
    gq, gk = (S.rotate(t, cos[at], sin[at], inverse=True) for t in (gq, gk))
    got = dqkv.double().cpu().numpy().transpose(0, 2, 1, 3)
    for a, ref in ((got[:, :Hq], gq), (got[:, Hq:Hq + Hkv], gk), (dv.double().cpu().numpy(), gv)):
        assert np.linalg.norm(a - ref) <= 1.5e-2 * np.linalg.norm(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (o, lse, dqkv, dv, q, k, rr, ws, wb):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1]) and torch.equal(dv, first[3])
    # dQ is summed with atomic adds, whose order may differ: one rounding of the type at most
    assert (dqkv.float() - first[2].float()).abs().max().item() <= 2.0 ** -7 * first[2].float().abs().max().item()


def test_two_streams_with_workspaces_of_their_own():
    q, k, v, do = (x.cuda() for x in inputs.normal(27, [(1, 4, 900, 64)] * 4))
    masks = [torch.from_numpy(S.mask_rows(1, 900, documents(28 + i, 1, 900, 4, 100), None, True)).to(I32).cuda() for i in range(2)]
    want = [run_fwd(q, k, v, m, cap=5.0) for m in masks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            got[i] = run_fwd(q, k, v, masks[i], cap=5.0)
    torch.cuda.synchronize()
    for (a, b), (x, y) in zip(got, want):
        assert torch.equal(a, x) and torch.equal(b, y)
