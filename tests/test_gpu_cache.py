"""Appending to a block-quantised cache and attention of single tokens over it,
against the float64 definitions (GPU only).

Append: codes and factors equal the oracle's exactly (float32 rotation, then
the power-of-two rule and round to nearest even are fixed steps).
Decode: with A = sum_j p_j |v_j| (per head dim) and X = scale log2(e) max_j
sum |q||k| the score in log2 units is off by at most
  dx = (d + 8) 2^-24 X (float32 sum of exact products) + 2^-20 cap log2(e)
       + 2^-22 (slope distance) (their float32 terms),
the weights by 2^-11 (P in FP16, at least 2^-10 normal) + 2 dx ln 2 + 2^-20
(exp2), and o by that times A plus half a step of its type at |o|; lse by
dx ln 2 + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from exact_attention_73_gb300 import binding as L
from exact_attention_73_gb300 import inputs
from oracle import fp8 as F
from oracle import score as S

pytestmark = pytest.mark.gpu
U8, I32 = torch.uint8, torch.int32
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def paged(x8, s, seed, spare=3):
    """Dense codes [B, H, nb * 128, d] and factors [B, H, nb] as shuffled pages, spare ones among them."""
    B, H, n, d = x8.shape
    nb = n // 128
    at = np.random.default_rng(seed).permutation(B * nb + spare)[:B * nb].reshape(B, nb)
    p8, ps = np.full((B * nb + spare, H, 128, d), 0x7f, np.uint8), np.full((B * nb + spare, H), np.nan, np.float32)
    for b in range(B):
        for t in range(nb):
            p8[at[b, t]], ps[at[b, t]] = x8[b, :, t * 128:(t + 1) * 128], s[b, :, t]
    return p8, ps, at.astype(np.int32)


def append_case(seed, B, H, d, nmax, lens, news, n, dtype="bf16", rot=0, interleaved=False, pages=False, gain=1.0):
    r = np.random.default_rng(seed)
    old = r.standard_normal((2, B, H, nmax, d)).astype(np.float32)
    cache = [F.quantize_blocks(o) for o in old]
    kv = inputs.normal(seed + 1, [(B, n, H, d)] * 2, dtype)
    kv = [x * gain for x in kv]
    cos = sin = None
    if rot:
        a = np.arange(nmax, dtype=np.float64)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
        cos, sin = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    want = []
    for i in range(2):
        c, f = (x.copy() for x in cache[i])
        for b in range(B):
            rows = kv[i][b, :news[b]].float().numpy().transpose(1, 0, 2)
            if i == 0 and rot:
                rows = S.rotate_fp32(rows, cos[lens[b]:lens[b] + news[b]], sin[lens[b]:lens[b] + news[b]], interleaved)
            c[b], f[b] = S.append_sequence(c[b], f[b], lens[b], rows)
        want += [c, f]
    t = None
    if pages:
        k8, sk, at = paged(*cache[0], seed)
        v8, sv, _ = paged(*cache[1], seed)
        w = [paged(want[0], want[1], seed), paged(want[2], want[3], seed)]
        want = [w[0][0], w[0][1], w[1][0], w[1][1]]
        t = torch.from_numpy(at).cuda()
    else:
        (k8, sk), (v8, sv) = cache
    dev = [torch.from_numpy(x).cuda() for x in (k8, v8, sk, sv)]
    L.attn_cache_append_fp8(kv[0].cuda().transpose(1, 2), kv[1].cuda().transpose(1, 2), *dev,
                            torch.tensor(lens, dtype=I32, device="cuda"),
                            new_lens=torch.tensor(news, dtype=I32, device="cuda"), block_table=t,
                            rope_cos=None if cos is None else torch.from_numpy(cos).cuda(),
                            rope_sin=None if sin is None else torch.from_numpy(sin).cuda(), interleaved=interleaved)
    assert L.attn_get_device_status() == 0
    for got, ref, name in zip((dev[0], dev[2], dev[1], dev[3]), want, ("k8", "sk", "v8", "sv")):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=name[0] == "s"), name


@pytest.mark.parametrize("pages", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gain", [1.0, 30.0, 1e-3])
def test_one_new_token_at_every_kind_of_place(pages, d, gain):
    append_case(10, 6, 2, d, 384, [0, 1, 127, 128, 200, 383], [1] * 6, 1, rot=d, pages=pages, gain=gain)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, True), (64, False), (128, True), (112, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ragged_pieces_of_prompt(rot, interleaved, dtype):
    append_case(11, 5, 3, 128, 640, [0, 100, 128, 3, 300], [640 - 0, 29, 128, 0, 1], 640, dtype, rot, interleaved)


@pytest.mark.parametrize("nmax,lens,news", [(130, [0, 129], [130, 1]), (1, [0], [1]), (257, [126, 255], [3, 2])])
def test_a_dense_cache_that_ends_inside_a_block(nmax, lens, news):
    append_case(12, len(lens), 2, 64, nmax, lens, news, max(news), rot=32)


def test_what_does_not_fit_is_dropped_and_reported():
    B, H, d, nb = 4, 2, 64, 2
    k, v = inputs.normal(13, [(B, H, 5, d)] * 2)
    k8, v8 = (torch.full((7, H, 128, d), 9, dtype=U8, device="cuda") for _ in range(2))
    sk, sv = (torch.full((7, H), 3.0, device="cuda") for _ in range(2))
    table = torch.tensor([[0, 1], [7, 2], [3, -1], [4, 5]], dtype=I32, device="cuda")
    lens = torch.tensor([254, 10, 126, -3], dtype=I32, device="cuda")
    L.attn_cache_append_fp8(k.cuda(), v.cuda(), k8, v8, sk, sv, lens, block_table=table)
    assert L.attn_get_device_status() == 3 and L.attn_get_device_status() == 0
    for x8, s, x in ((k8, sk, k), (v8, sv, v)):
        touched = [(1, 0, 254, 256), (3, 2, 126, 128)]     # page, sequence, rows that fitted
        for page in range(7):
            hit = [q for q in touched if q[0] == page]
            if not hit:
                assert (x8[page] == 9).all() and (s[page] == 3.0).all()
                continue
            _, b, lo, hi = hit[0]
            for h in range(H):
                c, f = S.append_block(np.full((128, d), 9, np.uint8), np.float32(3.0), lo % 128, x[b, h, :hi - lo].float().numpy())
                got = x8[page, h].cpu().numpy()
                assert np.array_equal(got[:lo % 128 + hi - lo], c) and s[page, h].item() == f
                assert (got[lo % 128 + hi - lo:] == 9).all()
    # tables that end before the cache does
    c = torch.ones((100, 32), device="cuda")
    k8.fill_(9)
    L.attn_cache_append_fp8(k[:1].cuda(), v[:1].cuda(), k8, v8, sk, sv, torch.tensor([98], dtype=I32, device="cuda"),
                            block_table=table[:1], rope_cos=c, rope_sin=c)
    assert L.attn_get_device_status() == 3
    assert (k8[0, :, 100:] == 9).all() and not (k8[0, :, 98:100] == 9).all()


def test_zeros_and_saturated_codes():
    """A block of zeros has factor 1 until a value comes; a NaN code counts as 448 and stays NaN."""
    d = 64
    k8 = torch.zeros((1, 1, 128, d), dtype=U8, device="cuda")
    v8 = torch.full_like(k8, 0x7f)
    sk, sv = torch.ones((1, 1, 1), device="cuda"), torch.full((1, 1, 1), 0.5, device="cuda")
    x = torch.full((1, 1, 1, d), 2.0 ** -20, dtype=torch.bfloat16, device="cuda")
    L.attn_cache_append_fp8(x, torch.zeros_like(x), k8, v8, sk, sv, torch.tensor([2], dtype=I32, device="cuda"))
    assert sk.item() == 2.0 ** -28 and (k8[0, 0, 2] == 0x78).all() and not k8[0, 0, :2].any()
    assert sv.item() == 0.5 and (v8[0, 0, :2] == 0x7f).all() and not v8[0, 0, 2].any()


def decode_case(seed, B, Hq, Hkv, d, nmax, lens, splits, dtype="bf16", cap=0.0, slopes=False, left=-1, pages=False,
                gain=1.0, poison=True, vgain=1.0):
    (q,) = inputs.normal(seed, [(B, Hq, d)], dtype)
    q = q * gain
    r = np.random.default_rng(seed + 1)
    kv = r.standard_normal((2, B, Hkv, nmax, d)).astype(np.float32)
    kv[1] *= vgain
    (k8, sk), (v8, sv) = F.quantize_blocks(kv[0]), F.quantize_blocks(kv[1])
    nb = sk.shape[2]
    kf, vf = (F.e4m3_decode(c) * np.repeat(s.astype(np.float64), 128, 2)[:, :, :nmax, None] for c, s in ((k8, sk), (v8, sv)))
    scale = d ** -0.5
    sl = np.float32(2.0) ** (-8.0 * (np.arange(Hq) + 1) / Hq).astype(np.float32) if slopes else None
    if poison:   # nothing behind the length may matter: NaN codes, NaN factors
        for b in range(B):
            n = max(0, lens[b])
            k8[b, :, n:], v8[b, :, n:] = 0x7f, 0xff
            sk[b, :, -(-n // 128):], sv[b, :, -(-n // 128):] = np.nan, np.nan
    t = None
    if pages:
        pk, ps, at = paged(k8, sk, seed)
        pv, psv, _ = paged(v8, sv, seed)
        k8, sk, v8, sv, t = pk, ps, pv, psv, torch.from_numpy(at).cuda()
    o = torch.full((B, Hq, d), float("nan"), dtype=DT[dtype], device="cuda")
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    ws = torch.full((L.attn_decode_cache_fp8_workspace_size(B, Hq, d, splits),), 0xff, dtype=U8, device="cuda")
    L.attn_decode_cache_fp8(q.cuda(), *(torch.from_numpy(x).cuda() for x in (k8, v8, sk, sv)),
                            torch.tensor(lens, dtype=I32, device="cuda"), o, lse, ws, splits, block_table=t,
                            slopes=None if sl is None else torch.from_numpy(sl).cuda(), score_cap=cap, window_left=left)
    assert L.attn_get_device_status() == 0
    seen = [min(max(n, 0), nmax) for n in lens]
    ro, rl, mag = S.decode(q, kf, vf, seen, scale, cap, sl, left)
    X = scale * 1.4427 * np.einsum("bhgd,bhnd->bhgn", np.abs(q.double().numpy()).reshape(B, Hkv, Hq // Hkv, d), np.abs(kf)).max(-1).reshape(B, Hq)
    dx = (d + 8) * 2.0 ** -24 * X + 2.0 ** -20 * cap * 1.4427
    if slopes:
        dx = dx + 2.0 ** -22 * sl[None] * nmax * 1.4427
    half = torch.finfo(DT[dtype]).eps / 2
    rel = 2.0 ** -11 + 2 * dx * math.log(2) + 2.0 ** -20
    tol = rel[..., None] * mag + half * (np.abs(ro) + rel[..., None] * mag) + 2.0 ** -25
    err = np.abs(o.double().cpu().numpy() - ro)
    assert (err <= tol).all(), (err - tol).max()
    gl = lse.double().cpu().numpy()
    fin = np.isfinite(rl)
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    assert (np.abs(gl[fin] - rl[fin]) <= (dx * math.log(2))[fin] + 2.0 ** -20 * (1 + np.abs(rl[fin]))).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (8, 1), (9, 1), (16, 1), (40, 2), (35, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_head_groups(d, Hq, Hkv, dtype):
    decode_case(20, 3, Hq, Hkv, d, 700, [700, 1, 333], 3, dtype)


@pytest.mark.parametrize("splits", [1, 2, 5, 9])
@pytest.mark.parametrize("pages", [False, True])
@pytest.mark.parametrize("cap,slopes,left", [(0.0, False, -1), (20.0, False, -1), (0.0, True, -1), (5.0, True, 100), (0.0, False, 0),
                                             (0.0, False, 511)])
def test_decode_score_changes_lengths_and_splits(splits, pages, cap, slopes, left):
    decode_case(21, 8, 6, 2, 128, 1152, [0, 1, 16, 17, 128, 129, 1000, 1152], splits, cap=cap, slopes=slopes, left=left, pages=pages)


@pytest.mark.parametrize("nmax", [1, 15, 127, 130])
def test_decode_small_dense_caches(nmax):
    decode_case(22, 2, 4, 2, 64, nmax, [nmax, max(1, nmax - 1)], 1)


def test_decode_peaked_scores_and_small_values():
    decode_case(23, 2, 8, 2, 128, 2000, [2000, 1500], 4, gain=12.0)
    decode_case(24, 2, 8, 2, 128, 2000, [2000, 1500], 4, gain=12.0, cap=50.0, vgain=1e-6)


def test_decode_blocks_with_far_apart_factors():
    """Values of 1e-6 next to a block of zeros (factor 1) and a block of 300s: each at its own place in the sum."""
    B, H, d, nmax = 1, 1, 64, 512
    r = np.random.default_rng(25)
    kv = r.standard_normal((2, B, H, nmax, d)).astype(np.float32) * 0.01
    kv[1, :, :, :128] = 0
    kv[1, :, :, 128:256] *= 1e-4
    kv[1, :, :, 384:] *= 3e4
    (k8, sk), (v8, sv) = F.quantize_blocks(kv[0]), F.quantize_blocks(kv[1])
    kf, vf = (F.e4m3_decode(c) * np.repeat(s.astype(np.float64), 128, 2)[..., None] for c, s in ((k8, sk), (v8, sv)))
    (q,) = inputs.normal(26, [(B, 4, d)])
    dev = [torch.from_numpy(x).cuda() for x in (k8, v8, sk, sv)]
    for n in (256, 384, 512):
        o, lse = torch.empty((B, 4, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 4), device="cuda")
        ws = torch.empty(256, dtype=U8, device="cuda")
        L.attn_decode_cache_fp8(q.cuda(), *dev, torch.tensor([n], dtype=I32, device="cuda"), o, lse, ws, 1)
        ro, _, mag = S.decode(q, kf, vf, [n], d ** -0.5)
        assert (np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * mag).all()


@pytest.mark.parametrize("tiny", [(1, 2), (0, 1), (2, 4), (4,)])
def test_decode_factors_past_the_range_of_a_float(tiny):
    """Values of 1e-37 between values of 1e4: the sum in units of the small ones would pass 2^127."""
    H, d, n = 2, 128, 640
    r = np.random.default_rng(34)
    kv = r.standard_normal((2, 1, H, n, d)).astype(np.float32) * 0.01
    kv[1] *= 1e6
    for t in tiny:
        kv[1, :, :, 128 * t:128 * (t + 1)] *= 1e-41
    (k8, sk), (v8, sv) = F.quantize_blocks(kv[0]), F.quantize_blocks(kv[1])
    kf, vf = (F.e4m3_decode(c) * np.repeat(s.astype(np.float64), 128, 2)[..., None] for c, s in ((k8, sk), (v8, sv)))
    (q,) = inputs.normal(35, [(1, 8, d)])
    dev = [torch.from_numpy(x).cuda() for x in (k8, v8, sk, sv)]
    for m in (256, 384, 640):
        o, lse = torch.empty((1, 8, d), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 8), device="cuda")
        ws = torch.empty(256, dtype=U8, device="cuda")
        L.attn_decode_cache_fp8(q.cuda(), *dev, torch.tensor([m], dtype=I32, device="cuda"), o, lse, ws, 1)
        ro, rl, mag = S.decode(q, kf, vf, [m], d ** -0.5)
        assert (np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * mag).all()
        assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-5


def test_decode_lengths_out_of_range_and_missing_pages():
    B, H, d, nmax = 3, 2, 64, 256
    r = np.random.default_rng(27)
    x = r.standard_normal((B, H, nmax, d)).astype(np.float32)
    c, s = F.quantize_blocks(x)
    p8, ps, at = paged(c, s, 28)
    at[1, 0], at[2, 1] = -1, p8.shape[0]
    (q,) = inputs.normal(29, [(B, 4, d)])
    o, lse = torch.empty((B, 4, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 4), device="cuda")
    ws = torch.empty(L.attn_decode_cache_fp8_workspace_size(B, 4, d, 2), dtype=U8, device="cuda")
    k, f, t = (torch.from_numpy(v).cuda() for v in (p8, ps, at))
    L.attn_decode_cache_fp8(q.cuda(), k, k, f, f, torch.tensor([-5, 100, 4000], dtype=I32, device="cuda"), o, lse, ws, 2, block_table=t)
    assert L.attn_get_device_status() == 3 and L.attn_get_device_status() == 0
    xf = F.e4m3_decode(c) * np.repeat(s.astype(np.float64), 128, 2)[..., None]
    assert not o[:2].any() and torch.isneginf(lse[:2]).all()
    ro, rl, mag = S.decode(q[2:], xf[2:], xf[2:], [128], d ** -0.5)
    assert (np.abs(o[2:].double().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * mag).all()
    assert np.abs(lse[2:].double().cpu().numpy() - rl).max() <= 1e-5


def test_offsets_past_32_bits():
    """A cache of 2^31 + bytes: the last sequence's last page and block."""
    H, d, n = 8, 256, 2 ** 17 + 128            # 8 * 256 * (2^17 + 128) bytes each
    B = 9
    x8 = torch.zeros((B, H, n, d), dtype=U8, device="cuda")
    s = torch.ones((B, H, n // 128), device="cuda")
    (row,) = inputs.normal(30, [(B, H, 1, d)])
    L.attn_cache_append_fp8(row.cuda(), row.cuda(), x8, x8.clone(), s, s.clone(), torch.full((B,), n - 1, dtype=I32, device="cuda"))
    c, f = F.quantize_blocks(row.float().numpy())
    assert np.array_equal(x8[-1, :, -1].cpu().numpy(), c[-1, :, 0]) and np.array_equal(s[-1, :, -1].cpu().numpy(), f[-1, :, 0])
    (q,) = inputs.normal(31, [(B, H, d)])
    o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H), device="cuda")
    sp = L.attn_decode_cache_fp8_splits(B, H, H, n // 128)
    ws = torch.empty(L.attn_decode_cache_fp8_workspace_size(B, H, d, sp), dtype=U8, device="cuda")
    L.attn_decode_cache_fp8(q.cuda(), x8, x8, s, s, torch.full((B,), n, dtype=I32, device="cuda"), o, lse, ws, sp, window_left=0)
    want = F.e4m3_decode(c[:, :, 0]) * f[:, :, 0][..., None].astype(np.float64)
    assert (np.abs(o.double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all()


def test_a_serving_run_captured_and_replayed():
    """Append a prompt, then a captured step (rotate the query, append a token, attend) replayed with growing lengths
    equals direct calls and the attention of the whole row."""
    B, Hq, Hkv, d, nmax, prompt, steps = 2, 8, 2, 128, 512, 120, 12
    kv = inputs.normal(32, [(B, prompt + steps, Hkv, d)] * 2)
    (q,) = inputs.normal(33, [(B, prompt + steps, Hq, d)])
    cos, sin = (torch.from_numpy(t).cuda() for t in F.rope_tables(nmax, d))
    table = torch.tensor([[5, 2, 0, 7], [1, 6, 3, 4]], dtype=I32, device="cuda")
    dev = [x.cuda() for x in kv]

    def fresh():
        return ([torch.full((8, Hkv, 128, d), 0x7f, dtype=U8, device="cuda") for _ in range(2)]
                + [torch.full((8, Hkv), float("nan"), device="cuda") for _ in range(2)])

    def fill(c):
        L.attn_cache_append_fp8(*(x[:, :prompt].transpose(1, 2) for x in dev), *c, torch.zeros(B, dtype=I32, device="cuda"),
                                block_table=table, rope_cos=cos, rope_sin=sin)

    kt, vt, qt = (torch.empty((B, h, 1, d), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    held, pos = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros((B, 1), dtype=I32, device="cuda")
    seen = torch.zeros(B, dtype=I32, device="cuda")
    qr, o, lse = torch.empty_like(qt), torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, Hq), device="cuda")
    ws = torch.empty(L.attn_decode_cache_fp8_workspace_size(B, Hq, d, 2), dtype=U8, device="cuda")

    def step(c):
        L.attn_rope(qt, qr, cos, sin, positions=pos)
        L.attn_cache_append_fp8(kt, vt, *c, held, block_table=table, rope_cos=cos, rope_sin=sin)
        L.attn_decode_cache_fp8(qr[:, :, 0], *c, seen, o, lse, ws, 2, block_table=table, score_cap=30.0)

    def run(c, go):
        fill(c)
        out = []
        for i in range(prompt, prompt + steps):
            for dst, src in ((kt, dev[0]), (vt, dev[1]), (qt, q.cuda())):
                dst.copy_(src[:, i, :, None])
            held.fill_(i)
            pos.fill_(i)
            seen.fill_(i + 1)
            go()
            out.append((o.clone(), lse.clone()))
        return out

    a = fresh()
    direct = run(a, lambda: step(a))
    b = fresh()
    g = torch.cuda.CUDAGraph()
    fill(b)
    with torch.cuda.graph(g):
        step(b)
    replayed = run(b, g.replay)
    torch.cuda.synchronize()
    assert L.attn_get_device_status() == 0
    for (x, y), (u, w) in zip(direct, replayed):
        assert torch.equal(x, u) and torch.equal(y, w)
    # the cache rounds keys and values to E4M3 (2^-4 relative, twice where a factor moved): against the unrounded row
    # the output is off by no more than that of |v| and of the weights, whose scores are off by 2^-3 X
    i = prompt + steps - 1
    kr = S.rotate(dev[0].cpu().double().numpy().transpose(0, 2, 1, 3), *(t[:i + 1].cpu().numpy() for t in (cos, sin)))
    qrow = S.rotate(q[:, i].double().numpy()[:, :, None], cos[i:i + 1].cpu().numpy(), sin[i:i + 1].cpu().numpy())[:, :, 0]
    ro, _, mag = S.decode(qrow, kr, dev[1].cpu().double().numpy().transpose(0, 2, 1, 3), [i + 1] * B, d ** -0.5, 30.0)
    err = np.abs(direct[-1][0].double().cpu().numpy() - ro)
    assert np.sqrt((err ** 2).mean()) <= 0.1 * np.sqrt((mag ** 2).mean())
