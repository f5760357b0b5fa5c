"""The rotary, score-modified and 8-bit cache operators side by side (GPU only):
what they write and what they leave alone, workspaces used again at once and by
two captured graphs, calls on a stream that is not the current one, and masks
of more rows than one block's tile facts.

Outputs and workspaces are views into the middle of larger buffers whose
margins hold a sentinel. Repeated and replayed forward calls give the same
bits; dQ is summed with atomic additions in any order, so a repeated one may be
a rounding of the type off (2^-7 of the largest element for bf16: one step).
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_73_gb300 import binding as L
from exact_attention_73_gb300 import inputs
from exact_attention_73_gb300 import rope as R
from oracle import score as S

pytestmark = pytest.mark.gpu

I32, U8 = torch.int32, torch.uint8
PAD = 4096


class Guard:
    """Tensors in the middle of buffers with sentinel margins."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype, fill=None):
        n = math.prod(shape)
        s = 0x5A if dtype == U8 else -7
        buf = torch.full((PAD + n + PAD,), s, dtype=dtype, device="cuda")
        view = buf[PAD:PAD + n].view(shape)
        view.fill_(fill if fill is not None else float("nan") if dtype.is_floating_point else s)
        self.bufs.append((buf, s))
        return view

    def check(self):
        torch.cuda.synchronize()
        assert L.attn_get_device_status() == 0
        for buf, s in self.bufs:
            assert (buf[:PAD] == s).all() and (buf[-PAD:] == s).all()


def masks(seed, B, N, n, pad=0):
    r = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        ids = np.sort(r.integers(0, 5, (B, N)), 1).astype(np.int32)
        if pad:
            ids[:, N - pad:] = -1
        out.append(S.mask_rows(B, N, ids, None, True))
    return [torch.from_numpy(m).to(I32).cuda() for m in out]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap,slopes,ranges", [(9.0, False, False), (0.0, True, True), (9.0, True, True), (0.0, False, True)])
def test_score_attention_writes_its_outputs_only(d, cap, slopes, ranges):
    B, Hq, Hkv, N = 2, 4, 2, 333
    q, k, v, do = (x.cuda() for x in inputs.normal(40, [(B, Hq, N, d), (B, Hkv, N, d), (B, Hkv, N, d), (B, Hq, N, d)]))
    g = Guard()
    o, lse = g(q.shape, q.dtype), g((B, Hq, N), torch.float32)
    sl = torch.tensor([0.5, 0.25, 0.1, 0.01], device="cuda") if slopes else None
    m = masks(41, B, N, 1)[0] if ranges else None
    ws = g((L.attn_score_workspace_size(B, N),), U8)
    mods = dict(row_ranges=m, slopes=sl, score_cap=cap, window=(-1, 0))
    L.attn_fwd_score(q, k, v, o, lse, workspace=ws, **mods)
    grads = [g(x.shape, x.dtype) for x in (q, k, v)]
    L.attn_bwd_score(q, k, v, o, lse, do, *grads, g((L.attn_bwd_score_workspace_size(B, Hq, Hkv, N, d),), U8), **mods)
    g.check()
    for t in (o, lse, *grads):
        assert torch.isfinite(t.float()).all()
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    L.attn_fwd_score(q, k, v, o2, l2, workspace=ws, **mods)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("N", [1, 100, 1024, 2500])
def test_rotation_tables_and_masks_write_their_outputs_only(N):
    B, H, d, rot = 2, 3, 128, 48
    g = Guard()
    c, s = g((N, rot // 2), torch.float32), g((N, rot // 2), torch.float32)
    L.attn_rope_tables(c, s, R.inv_freq(rot).cuda())
    (x,) = (t.cuda() for t in inputs.normal(42, [(B, H, N, d)]))
    y = g(x.shape, x.dtype)
    L.attn_rope(x, y, c, s)
    r = g((B, N, 2), I32)
    ids = torch.zeros((B, N), dtype=I32, device="cuda")
    ids[:, N // 2:] = 3
    L.attn_mask_rows(r, doc_ids=ids, prefix_lens=torch.tensor([0, N], dtype=I32, device="cuda"))
    g.check()
    for t in (c, s, y):
        assert torch.isfinite(t.float()).all()
    assert np.array_equal(r.cpu().numpy(), S.mask_rows(B, N, ids.cpu().numpy(), [0, N], True))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pages", [False, True])
def test_cache_operators_write_their_rows_only(d, pages):
    B, H, n, rows = 3, 2, 70, 384
    lens, news = [0, 100, 250], [70, 33, 0]
    kv = [x.cuda() for x in inputs.normal(43, [(B, H, n, d)] * 2)]
    g = Guard()
    shape, fac = ((B * 3, H, 128, d), (B * 3, H)) if pages else ((B, H, rows, d), (B, H, 3))
    x8, f = [g(shape, U8, 0x11) for _ in range(2)], [g(fac, torch.float32, 1.0) for _ in range(2)]
    t = torch.arange(B * 3, dtype=I32, device="cuda").view(B, 3) if pages else None
    L.attn_cache_append_fp8(*kv, *x8, *f, torch.tensor(lens, dtype=I32, device="cuda"),
                            new_lens=torch.tensor(news, dtype=I32, device="cuda"), block_table=t)
    total = [a + b for a, b in zip(lens, news)]
    for c in x8:   # rows behind the last new one, and the sequence without new rows, stay
        flat = c.view(B, 3, H, 128, d).transpose(1, 2).reshape(B, H, rows, d) if pages else c
        for b in range(B):
            assert (flat[b, :, total[b]:] == 0x11).all()
        assert (flat[2] == 0x11).all()
    q, seen = kv[0][:, :, 0].contiguous(), torch.tensor(total, dtype=I32, device="cuda")
    for splits in (1, 3):
        o, lse = g((B, H, d), torch.bfloat16), g((B, H), torch.float32)
        L.attn_decode_cache_fp8(q, *x8, *f, seen, o, lse, g((L.attn_decode_cache_fp8_workspace_size(B, H, d, splits),), U8),
                                splits, block_table=t)
        g.check()
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("cap,slopes", [(0.0, False), (6.0, True)])
def test_masks_of_more_rows_than_one_block_takes(cap, slopes):
    """17 sequences of 1000 rows: bounds, key tiles and order come from kernels of their own."""
    B, N, d = 17, 1000, 64
    q, k, v, do = inputs.normal(44, [(B, 1, N, d)] * 4)
    m = masks(45, B, N, 1, pad=130)[0]
    sl = np.array([0.03], np.float32) if slopes else None
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = torch.full_like(dev[0], float("nan")), torch.full((B, 1, N), float("nan"), device="cuda")
    mods = dict(row_ranges=m, slopes=None if sl is None else torch.from_numpy(sl).cuda(), score_cap=cap)
    L.attn_fwd_score(*dev[:3], o, lse, workspace=torch.full((L.attn_score_workspace_size(B, N),), 0xff, dtype=U8, device="cuda"), **mods)
    grads = [torch.full_like(dev[0], float("nan")) for _ in range(3)]
    L.attn_bwd_score(*dev[:3], o, lse, dev[3], *grads,
                     torch.full((L.attn_bwd_score_workspace_size(B, 1, 1, N, d),), 0xff, dtype=U8, device="cuda"), **mods)
    assert L.attn_get_device_status() == 0
    r = m.cpu().numpy()
    ro, rl = S.forward(q, k, v, d ** -0.5, r, (-1, -1), cap, sl)
    mag, _ = S.forward(q, k, v.abs(), d ** -0.5, r, (-1, -1), cap, sl)
    # P and O rounded once each to bf16 (2^-8), the scores' own errors far below that
    assert (np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * 1.05 * (mag + np.abs(ro)) + 2.0 ** -25).all()
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert np.abs(gl[fin] - rl[fin]).max() <= 1e-4
    for x, ref in zip(grads, S.backward(q, k, v, do, d ** -0.5, r, (-1, -1), cap, sl)):
        assert np.linalg.norm(x.double().cpu().numpy() - ref) <= 1e-2 * np.linalg.norm(ref)
        assert not x[:, :, N - 130:].any()


@pytest.mark.parametrize("cap", [5.0, 55.0, 56.0, 300.0])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (128, "fp16"), (256, "bf16")])
@pytest.mark.parametrize("ranges", [False, True])
def test_scores_at_either_end_of_the_cap(cap, d, dtype, ranges):
    """Every score of a head at -cap, at +cap, or the rows' own half at one and the rest at the other, whatever the
    cap: weights without a running max (small caps) or with one give the same attention."""
    B, H, N = 1, 3, 300
    r = np.random.default_rng(54)
    q = np.abs(r.standard_normal((B, H, N, d))) + 0.5
    k = np.abs(r.standard_normal((B, H, N, d))) + 0.5
    q *= 8 * cap / d ** 0.5               # q.k / sqrt(d) is at least 2 cap: tanh within 4 % of one, mostly at one
    k[:, 0] *= -1
    k[:, 2, ::2] *= -1
    q, k, v = (torch.from_numpy(x).to({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype])
               for x in (q, k, r.standard_normal((B, H, N, d))))
    m = masks(55, B, N, 1)[0] if ranges else None
    o, lse = torch.full_like(q, float("nan")).cuda(), torch.full((B, H, N), float("nan"), device="cuda")
    L.attn_fwd_score(q.cuda(), k.cuda(), v.cuda(), o, lse, row_ranges=m, score_cap=cap, window=(-1, 0),
                     workspace=torch.empty(L.attn_score_workspace_size(B, N), dtype=U8, device="cuda"))
    assert L.attn_get_device_status() == 0
    rm = None if m is None else m.cpu().numpy()
    ro, rl = S.forward(q, k, v, d ** -0.5, rm, (-1, 0), cap)
    mag, _ = S.forward(q, k, v.abs(), d ** -0.5, rm, (-1, 0), cap)
    # the capped score is off by 6e-7 of itself (cap) and 2^-22 of it (float32), both in the exponent
    half, dx = torch.finfo(q.dtype).eps / 2, cap * (6e-7 + 2.0 ** -22)
    tol = (half + 2 * dx + 2.0 ** -20) * (1 + half) * mag + half * np.abs(ro) + 2.0 ** -25
    assert (np.abs(o.double().cpu().numpy() - ro) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= dx + 2.0 ** -20 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_smallest_and_the_largest_cap(d):
    """1e-12: uniform weights and no gradient of the scores; 1e30: no cap at all."""
    q, k, v, do = (x.cuda() for x in inputs.normal(56, [(1, 2, 200, d)] * 4))
    ws = torch.empty(L.attn_bwd_score_workspace_size(1, 2, 2, 200, d), dtype=U8, device="cuda")

    def step(cap):
        o, lse, g = torch.empty_like(q), torch.empty((1, 2, 200), device="cuda"), [torch.empty_like(q) for _ in range(3)]
        L.attn_fwd_score(q, k, v, o, lse, score_cap=cap, window=(-1, 0))
        L.attn_bwd_score(q, k, v, o, lse, do, *g, ws, score_cap=cap, window=(-1, 0))
        return [x.double() for x in (o, lse, *g)]

    plain, small, large = step(0.0), step(1e-12), step(1e30)
    assert L.attn_get_device_status() == 0
    n = torch.arange(1, 201, device="cuda", dtype=torch.float64)
    assert (small[1] - n.log()).abs().max() <= 2.0 ** -20 * (1 + math.log(200))
    mean = v.double().cumsum(2) / n[:, None]
    size = v.double().abs().cumsum(2) / n[:, None]
    assert ((small[0] - mean).abs() <= 2.0 ** -8 * 1.05 * (mean.abs() + size)).all()
    for i in (2, 3):   # 1 - tanh^2 is zero but for the rounding of its square, 2^-22
        assert small[i].norm() <= 2.0 ** -20 * plain[i].norm()
    # the same scores by another way: each output within two roundings (2^-8 of its sums; gradients as against float64)
    assert (large[1] - plain[1]).abs().max() <= 2.0 ** -18
    assert ((large[0] - plain[0]).abs() <= 2.0 ** -7 * (plain[0].abs() + v.double().abs().max())).all()
    for a, b in zip(large[2:], plain[2:]):
        assert (a - b).norm() <= 1e-2 * b.norm()


@pytest.mark.parametrize("B,N", [(2, 500), (20, 1000)])
def test_one_workspace_used_again_at_once(B, N):
    """Calls behind one another with other masks and one workspace: each sees its own tile facts."""
    q, k, v, do = (x.cuda() for x in inputs.normal(46, [(B, 2, N, 64)] * 4))
    ms = masks(47, B, N, 3, pad=17)
    big = torch.empty(L.attn_bwd_score_workspace_size(B, 2, 2, N, 64), dtype=U8, device="cuda")

    def step(m, ws, wb):
        o, lse, grads = torch.empty_like(q), torch.empty((B, 2, N), device="cuda"), [torch.empty_like(q) for _ in range(3)]
        L.attn_fwd_score(q, k, v, o, lse, workspace=ws, row_ranges=m, score_cap=4.0)
        L.attn_bwd_score(q, k, v, o, lse, do, *grads, wb, row_ranges=m, score_cap=4.0)
        return o, lse, *grads

    want = []
    for m in ms:
        want.append(step(m, torch.empty(L.attn_score_workspace_size(B, N), dtype=U8, device="cuda"), torch.empty_like(big)))
        torch.cuda.synchronize()
    got = [step(ms[i % 3], big, big) for i in range(12)]
    torch.cuda.synchronize()
    assert L.attn_get_device_status() == 0
    for i, g in enumerate(got):
        w = want[i % 3]
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) and torch.equal(g[3], w[3]) and torch.equal(g[4], w[4])
        assert (g[2].float() - w[2].float()).abs().max() <= 2.0 ** -7 * w[2].float().abs().max()


def test_two_graphs_that_share_workspaces():
    B, H, N, d, rows = 2, 2, 400, 64, 1024
    q, k, v = (x.cuda() for x in inputs.normal(48, [(B, H, N, d)] * 3))
    ms = masks(49, B, N, 2)
    (tok,) = (x.cuda() for x in inputs.normal(50, [(B, H, d)]))
    x8 = [torch.empty((B, H, rows, d), dtype=U8, device="cuda") for _ in range(2)]
    f = [torch.empty((B, H, 8), device="cuda") for _ in range(2)]
    (kn, vn) = (x.cuda() for x in inputs.normal(51, [(B, H, rows, d)] * 2))
    L.attn_cache_append_fp8(kn, vn, *x8, *f, torch.zeros(B, dtype=I32, device="cuda"))
    ws = torch.empty(L.attn_score_workspace_size(B, N), dtype=U8, device="cuda")
    wd = torch.empty(L.attn_decode_cache_fp8_workspace_size(B, H, d, 8), dtype=U8, device="cuda")
    seen = [torch.tensor(n, dtype=I32, device="cuda") for n in ([1000, 3], [77, 640])]
    outs = [[torch.empty_like(q), torch.empty((B, H, N), device="cuda"), torch.empty_like(tok), torch.empty((B, H), device="cuda")]
            for _ in range(2)]

    def step(i):
        o, lse, ot, lt = outs[i]
        L.attn_fwd_score(q, k, v, o, lse, workspace=ws, row_ranges=ms[i], score_cap=4.0)
        L.attn_decode_cache_fp8(tok, *x8, *f, seen[i], ot, lt, wd, 8)

    want = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[i]])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            step(i)
    for o in outs:
        for t in o:
            t.zero_()
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert L.attn_get_device_status() == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_calls_on_a_stream_that_is_not_the_current_one():
    """Every entry point launches all of its kernels on the stream it is given: behind a long copy there, results follow it."""
    B, H, N, d, rows = 1, 2, 300, 64, 512
    src = [x.cuda() for x in inputs.normal(52, [(B, H, N, d)] * 4)]
    m = masks(53, B, N, 1)[0]
    st = torch.cuda.Stream()
    pad = [torch.empty(1 << 28, dtype=U8, device="cuda") for _ in range(2)]
    ins = [torch.zeros_like(x) for x in src]
    c, s = torch.zeros((N, d // 2), device="cuda"), torch.zeros((N, d // 2), device="cuda")
    freq = R.inv_freq(d).cuda()
    ids = torch.zeros((B, N), dtype=I32, device="cuda")
    ids[:, 150:] = 1

    def buffers():
        return dict(q=torch.empty_like(src[0]), o=torch.empty_like(src[0]), lse=torch.empty((B, H, N), device="cuda"),
                    g=[torch.empty_like(src[0]) for _ in range(3)], rr=torch.empty((B, N, 2), dtype=I32, device="cuda"),
                    ws=torch.empty(L.attn_score_workspace_size(B, N), dtype=U8, device="cuda"),
                    wb=torch.empty(L.attn_bwd_score_workspace_size(B, H, H, N, d), dtype=U8, device="cuda"),
                    x8=[torch.zeros((B, H, rows, d), dtype=U8, device="cuda") for _ in range(2)],
                    f=[torch.ones((B, H, 4), device="cuda") for _ in range(2)], tok=torch.empty((B, H, d), dtype=src[0].dtype, device="cuda"),
                    ot=torch.empty((B, H, d), dtype=src[0].dtype, device="cuda"), lt=torch.empty((B, H), device="cuda"),
                    wd=torch.empty(L.attn_decode_cache_fp8_workspace_size(B, H, d, 4), dtype=U8, device="cuda"),
                    held=torch.zeros(B, dtype=I32, device="cuda"), seen=torch.full((B,), N, dtype=I32, device="cuda"))

    def run(b, x, stream):
        kw = dict(stream=stream)
        L.attn_rope_tables(c, s, freq, **kw)
        L.attn_rope(x[0], b["q"], c, s, **kw)
        L.attn_mask_rows(b["rr"], doc_ids=ids, **kw)
        L.attn_fwd_score(b["q"], x[1], x[2], b["o"], b["lse"], workspace=b["ws"], row_ranges=b["rr"], score_cap=5.0, **kw)
        L.attn_bwd_score(b["q"], x[1], x[2], b["o"], b["lse"], x[3], *b["g"], b["wb"], row_ranges=b["rr"], score_cap=5.0, **kw)
        L.attn_cache_append_fp8(x[1], x[2], *b["x8"], *b["f"], b["held"], rope_cos=c, rope_sin=s, **kw)
        L.attn_decode_cache_fp8(b["tok"], *b["x8"], *b["f"], b["seen"], b["ot"], b["lt"], b["wd"], 4, **kw)

    want, got = buffers(), buffers()
    for b in (want, got):
        b["tok"].copy_(src[0][:, :, 0])
    run(want, src, None)
    torch.cuda.synchronize()
    c.zero_()
    s.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(8):
            pad[0].copy_(pad[1])
        for a, x in zip(ins, src):
            a.copy_(x)
    run(got, ins, st)
    torch.cuda.synchronize()
    assert L.attn_get_device_status() == 0
    for n in ("q", "o", "lse", "rr", "ot", "lt"):
        assert torch.equal(want[n], got[n]), n
    for n in ("x8", "f"):
        assert all(torch.equal(a, b) for a, b in zip(want[n], got[n])), n
    assert torch.equal(want["g"][1], got["g"][1]) and torch.equal(want["g"][2], got["g"][2])
    assert (want["g"][0].float() - got["g"][0].float()).abs().max() <= 2.0 ** -7 * want["g"][0].float().abs().max()
