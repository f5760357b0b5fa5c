"""Refusals of the rotary, cache and score-modified attention entry points
(CPU only): the C checks return before any device work, and the binding
refuses tensors the library would read out of bounds."""
import ctypes as C
import math
import types

import pytest
import torch

from exact_attention_73_gb300 import binding as L
from exact_attention_73_gb300 import rope

STREAM = types.SimpleNamespace(cuda_stream=0)
BF, U8, F32, F64, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.float64, torch.int32
P = lambda x=16: C.c_void_p(x)  # noqa: E731
ST = (C.c_longlong * 3)(64, 64, 64)


def test_rope_refusals(lib):
    def call(x=P(), y=P(), c=P(), s=P(), pos=None, sx=ST, sy=ST, B=1, H=1, N=4, d=64, rot=64, n_pos=4, dt=0):
        return lib.attn_rope(x, y, c, s, pos, sx, sy, B, H, N, d, rot, n_pos, 0, 0, dt, None)
    assert call(x=None) == 1 and call(s=None) == 1 and call(sx=None) == 1
    assert call(y=P(24)) == 2 and call(pos=P(20)) == 2 and call(sx=(C.c_longlong * 3)(64, 12, 64)) == 2
    assert call(B=0) == 3 and call(H=0) == 3 and call(N=0) == 3 and call(B=65536) == 3
    assert call(N=5) == 3                                         # past the tables, without positions
    assert call(d=96) == 4
    assert call(rot=0) == 3 and call(rot=24) == 3 and call(rot=80) == 3
    assert call(dt=2) == 6
    assert lib.attn_rope_tables(None, P(), P(), 0, 4, 64, 1.0, None) == 1
    assert lib.attn_rope_tables(P(), P(), P(8), 0, 4, 64, 1.0, None) == 2
    for first, n, rot in ((-1, 4, 64), (0, 0, 64), (0, 4, 20), (0, 4, 272), (2 ** 40 + 1, 4, 64)):
        assert lib.attn_rope_tables(P(), P(), P(), first, n, rot, 1.0, None) == 3


def test_cache_refusals(lib):
    def app(k=P(), k8=P(), sk=P(), lens=P(), table=None, cos=None, sin=None, st=ST, B=1, H=1, n=1, nmax=128, pages=0, d=64, rot=0,
            n_pos=0, dt=0):
        return lib.attn_cache_append_fp8(k, P(), st, ST, k8, P(), sk, P(), lens, None, table, cos, sin, B, H, n, nmax, pages, d,
                                         rot, n_pos, 0, dt, None)
    assert app(k=None) == 1 and app(lens=None) == 1 and app(cos=P()) == 1 and app(st=None) == 1
    assert app(k8=P(8)) == 2 and app(st=(C.c_longlong * 3)(4, 64, 64)) == 2
    assert app(B=0) == 3 and app(B=32768) == 3 and app(n=0) == 3 and app(nmax=0) == 3 and app(H=65536) == 3
    assert app(table=P(), pages=0) == 3 and app(table=P(), pages=2, nmax=130) == 3
    assert app(cos=P(), sin=P(), rot=24, n_pos=9) == 3 and app(cos=P(), sin=P(), rot=32, n_pos=0) == 3
    assert app(d=32) == 4 and app(dt=2) == 6
    w = L.attn_decode_cache_fp8_workspace_size(2, 8, 128, 3)
    assert w == L.attn_decode_fp8_workspace_size(2, 8, 128, 3) + 256 and L.attn_decode_cache_fp8_workspace_size(2, 8, 128, 1) == 256

    def dec(q=P(), o=P(), lens=P(), table=None, ws=P(), wb=w, B=2, Hq=8, Hkv=2, nmax=300, pages=0, d=128, cap=0.0, left=-1, splits=3,
            dt=0):
        return lib.attn_decode_cache_fp8(q, P(), P(), P(), P(), table, lens, None, o, P(), ws, wb, B, Hq, Hkv, nmax, pages, d, 0.1,
                                         cap, left, splits, dt, None)
    assert dec(q=None) == 1 and dec(lens=None) == 1 and dec(ws=None) == 1
    assert dec(o=P(24)) == 2
    assert dec(B=0) == 3 and dec(nmax=0) == 3 and dec(left=-2) == 3 and dec(splits=0) == 3 and dec(splits=4) == 3
    assert dec(cap=-1.0) == 3 and dec(cap=math.nan) == 3 and dec(cap=math.inf) == 3
    assert dec(table=P(), pages=5) == 3 and dec(table=P(), pages=0, nmax=384) == 3
    assert dec(d=96) == 4 and dec(Hkv=3) == 5 and dec(dt=2) == 6 and dec(wb=w - 1) == 7
    # sizes that suit: within the documented range, and more for fewer sequences
    for b, hq, hkv, nb in ((1, 1, 1, 1), (1, 32, 8, 256), (16, 32, 8, 256), (64, 64, 1, 7), (500, 8, 8, 2)):
        assert 1 <= L.attn_decode_cache_fp8_splits(b, hq, hkv, nb) <= nb
    assert L.attn_decode_cache_fp8_splits(1, 3, 2, 4) == 0 and L.attn_decode_cache_fp8_splits(1, 4, 2, 0) == 0


def test_score_refusals(lib):
    assert lib.attn_mask_rows(P(), None, None, 1, 8, 1, None) == 1
    assert lib.attn_mask_rows(P(8), None, P(), 1, 8, 1, None) == 2 and lib.attn_mask_rows(None, P(8), P(), 1, 8, 1, None) == 2
    for b, n in ((0, 8), (65536, 8), (1, 0), (1, 2 ** 24 + 1)):
        assert lib.attn_mask_rows(P(), None, P(), b, n, 1, None) == 3
    w = L.attn_score_workspace_size(2, 300)
    assert w == 256 and L.attn_score_workspace_size(2, 8192) == 2 * (128 * 8 + 64 * 16) and L.attn_score_workspace_size(0, 8) == 0

    def fwd(q=P(), lse=P(), ranges=None, slopes=None, ws=P(), wb=w, B=2, Hq=4, Hkv=2, N=300, d=64, scale=0.1, cap=0.0, left=-1,
            right=-1, dt=0):
        return lib.attn_fwd_score(q, P(), P(), P(), lse, ranges, slopes, ws, wb, B, Hq, Hkv, N, d, scale, cap, left, right, dt, None)
    assert fwd(q=None) == 1 and fwd(ranges=P(), ws=None) == 1
    assert fwd(lse=P(20)) == 2 and fwd(ranges=P(8)) == 2 and fwd(slopes=P(4)) == 2
    assert fwd(B=0) == 3 and fwd(N=0) == 3 and fwd(N=2 ** 24 + 1) == 3 and fwd(left=-2) == 3 and fwd(right=-7) == 3
    assert fwd(cap=-0.5) == 3 and fwd(cap=math.nan) == 3 and fwd(cap=math.inf) == 3 and fwd(scale=math.nan) == 3
    assert fwd(scale=0.0) == 3 and fwd(scale=-0.1) == 3
    assert fwd(d=96) == 4 and fwd(Hkv=3) == 5 and fwd(dt=2) == 6 and fwd(ranges=P(), wb=w - 1) == 7
    wb_ = L.attn_bwd_score_workspace_size(2, 4, 2, 300, 64)
    assert wb_ == L.attn_bwd_workspace_size(2, 4, 2, 300, 64) + w and L.attn_bwd_score_workspace_size(0, 4, 2, 300, 64) == 0

    def bwd(do=P(), ranges=None, ws=P(), wb=wb_, B=2, Hq=4, Hkv=2, N=300, d=64, scale=0.1, cap=0.0, left=-1, right=-1, dt=0):
        return lib.attn_bwd_score(P(), P(), P(), P(), P(), do, P(), P(), P(), ranges, None, ws, wb, B, Hq, Hkv, N, d, scale, cap, left,
                                  right, dt, None)
    assert bwd(do=None) == 1 and bwd(ws=None) == 1 and bwd(ranges=P(8)) == 2
    assert bwd(N=0) == 3 and bwd(left=-2) == 3 and bwd(cap=-1.0) == 3 and bwd(scale=math.inf) == 3
    assert bwd(d=32) == 4 and bwd(Hkv=3) == 5 and bwd(dt=2) == 6 and bwd(wb=wb_ - 1) == 7


def test_caps_out_of_range(lib):
    """Caps whose square, or whose ratio to the scale, leaves float32."""
    w = L.attn_bwd_score_workspace_size(1, 1, 1, 64, 64)

    def calls(cap, scale=0.1):
        return (lib.attn_fwd_score(P(), P(), P(), P(), P(), None, None, None, 0, 1, 1, 1, 64, 64, scale, cap, -1, -1, 0, None),
                lib.attn_bwd_score(P(), P(), P(), P(), P(), P(), P(), P(), P(), None, None, P(), w, 1, 1, 1, 64, 64, scale, cap, -1, -1,
                                   0, None),
                lib.attn_decode_cache_fp8(P(), P(), P(), P(), P(), None, P(), None, P(), P(), P(), 256, 1, 1, 1, 128, 0, 64, scale,
                                          cap, -1, 1, 0, None))
    for cap, scale in ((1e-13, 0.1), (1e-45, 0.1), (2e30, 0.1), (3e38, 0.1), (-1e-13, 0.1), (1e-12, 1e30), (1e10, 1e-25), (math.nan, 0.1)):
        assert calls(cap, scale) == (3, 3, 3), (cap, scale)


class _Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = _Lib()
    monkeypatch.setattr(L, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(L, "load", lambda build_if_missing=True: f)
    return f


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_binding_takes_strided_rows_and_refuses_the_rest(fake):
    x = z(2, 9, 6, 128)[:, :, 1:5].transpose(1, 2)          # [2, 4, 9, 128]
    y, c = z(2, 4, 9, 128), z(9, 32, dtype=F32)
    L.attn_rope(x, y, c, c, positions=z(2, 9, dtype=I32), stream=STREAM)
    (name, a), = fake.calls
    assert name == "attn_rope" and list(a[5]) == [9 * 6 * 128, 128, 6 * 128] and list(a[6]) == [4 * 9 * 128, 9 * 128, 128]
    assert a[7:13] == (2, 4, 9, 128, 64, 9)
    # the strides of dimensions of one element are never used: any value there is fine
    L.attn_rope(torch.as_strided(x, (1, 4, 1, 128), (3, 128, 5, 1)), y[:1, :, :1], c, c, stream=STREAM)
    assert list(fake.calls[1][1][5]) == [0, 128, 0]
    fake.calls.clear()
    for err, call in (
            (ValueError, lambda: L.attn_rope(x.transpose(2, 3), y, c, c, stream=STREAM)),
            (ValueError, lambda: L.attn_rope(z(2, 4, 128, 9).transpose(2, 3), y, c, c, stream=STREAM)),
            (ValueError, lambda: L.attn_rope(x, y[:1], c, c, stream=STREAM)),
            (TypeError, lambda: L.attn_rope(x, y.half(), c, c, stream=STREAM)),
            (TypeError, lambda: L.attn_rope(x.float(), y.float(), c, c, stream=STREAM)),
            (ValueError, lambda: L.attn_rope(x, y, c, c[:, :16], stream=STREAM)),
            (ValueError, lambda: L.attn_rope(x, y, c, c, positions=z(2, 8, dtype=I32), stream=STREAM)),
            (TypeError, lambda: L.attn_rope(x, y, c, c, positions=z(2, 9, dtype=torch.int64), stream=STREAM)),
            (TypeError, lambda: L.attn_rope_tables(c, c, z(32, dtype=F32), stream=STREAM)),
            (ValueError, lambda: L.attn_rope_tables(c, c, z(31, dtype=F64), stream=STREAM))):
        with pytest.raises(err):
            call()
    assert fake.calls == []


def test_binding_checks_caches(fake):
    k = z(3, 5, 2, 64).transpose(1, 2)
    dense = (z(3, 2, 200, 64, dtype=U8), z(3, 2, 200, 64, dtype=U8), z(3, 2, 2, dtype=F32), z(3, 2, 2, dtype=F32))
    pages = (z(7, 2, 128, 64, dtype=U8), z(7, 2, 128, 64, dtype=U8), z(7, 2, dtype=F32), z(7, 2, dtype=F32))
    lens, table = z(3, dtype=I32), z(3, 4, dtype=I32)
    q, o, lse, ws = z(3, 4, 64), z(3, 4, 64), z(3, 4, dtype=F32), z(256, dtype=U8)
    L.attn_cache_append_fp8(k, k, *dense, lens, stream=STREAM)
    L.attn_cache_append_fp8(k, k, *pages, lens, block_table=table, new_lens=lens, stream=STREAM)
    L.attn_decode_cache_fp8(q, *dense, lens, o, lse, ws, 1, stream=STREAM)
    L.attn_decode_cache_fp8(q, *pages, lens, o, lse, ws, 1, block_table=table, slopes=z(4, dtype=F32), stream=STREAM)
    assert [n for n, _ in fake.calls] == ["attn_cache_append_fp8"] * 2 + ["attn_decode_cache_fp8"] * 2
    assert fake.calls[0][1][15:18] == (5, 200, 0) and fake.calls[1][1][15:18] == (5, 512, 7)
    fake.calls.clear()
    for call in (lambda: L.attn_cache_append_fp8(k, k, *pages, lens, stream=STREAM),
                 lambda: L.attn_cache_append_fp8(k, k, *dense, lens, block_table=table, stream=STREAM),
                 lambda: L.attn_cache_append_fp8(k, k[:, :, :4], *dense, lens, stream=STREAM),
                 lambda: L.attn_cache_append_fp8(k, k, *dense, lens[:2], stream=STREAM),
                 lambda: L.attn_cache_append_fp8(k, k, *dense, lens, rope_cos=z(200, 32, dtype=F32), stream=STREAM),
                 lambda: L.attn_cache_append_fp8(k, k, *pages, lens, block_table=table[:2], stream=STREAM),
                 lambda: L.attn_decode_cache_fp8(q, *dense, lens, o[:, :2], lse, ws, 1, stream=STREAM),
                 lambda: L.attn_decode_cache_fp8(q, *dense, lens, o, lse, ws, 1, slopes=z(3, dtype=F32), stream=STREAM),
                 lambda: L.attn_decode_cache_fp8(q, dense[0], dense[1], dense[2], dense[3][:, :, :1], lens, o, lse, ws, 1, stream=STREAM)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.attn_decode_cache_fp8(q, *dense, lens.long(), o, lse, ws, 1, stream=STREAM)
    with pytest.raises(TypeError):
        L.attn_decode_cache_fp8(q, *dense, lens, o.half(), lse, ws, 1, stream=STREAM)
    assert fake.calls == []


def test_binding_checks_score_calls(fake):
    q, kv, lse = z(2, 4, 70, 64), z(2, 2, 70, 64), z(2, 4, 70, dtype=F32)
    rr, sl, ws = z(2, 70, 2, dtype=I32), z(4, dtype=F32), z(4096, dtype=U8)
    L.attn_mask_rows(rr, doc_ids=z(2, 70, dtype=I32), prefix_lens=z(2, dtype=I32), stream=STREAM)
    L.attn_fwd_score(q, kv, kv, q, lse, stream=STREAM)
    L.attn_fwd_score(q, kv, kv, q, lse, workspace=ws, row_ranges=rr, slopes=sl, score_cap=30.0, window=(5, 0), stream=STREAM)
    L.attn_bwd_score(q, kv, kv, q, lse, q, q, kv, kv, ws, row_ranges=rr, slopes=sl, score_cap=30.0, stream=STREAM)
    assert [n for n, _ in fake.calls] == ["attn_mask_rows", "attn_fwd_score", "attn_fwd_score", "attn_bwd_score"]
    assert fake.calls[1][1][7:9] == (None, 0) and fake.calls[2][1][8] == 4096
    fake.calls.clear()
    for call in (lambda: L.attn_mask_rows(rr, doc_ids=z(2, 69, dtype=I32), stream=STREAM),
                 lambda: L.attn_mask_rows(z(2, 70, 3, dtype=I32), stream=STREAM),
                 lambda: L.attn_mask_rows(rr, prefix_lens=z(3, dtype=I32), stream=STREAM),
                 lambda: L.attn_fwd_score(q, kv, kv, q, lse, workspace=ws, row_ranges=rr[:1], stream=STREAM),
                 lambda: L.attn_fwd_score(q, kv, kv, q, lse, slopes=sl[:2], stream=STREAM),
                 lambda: L.attn_fwd_score(q, kv, kv[:, :, :9], q, lse, stream=STREAM),
                 lambda: L.attn_bwd_score(q, kv, kv, q, lse, q, q, kv[:1], kv, ws, stream=STREAM)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.attn_mask_rows(rr.long(), stream=STREAM)
    assert fake.calls == []


def test_frequencies():
    f = rope.inv_freq(64)
    assert f.dtype == F64 and f.shape == (32,) and f[0] == 1.0 and abs(f[16].item() - 10000.0 ** -0.5) < 1e-15
    assert torch.equal(rope.inv_freq(64, scaling="linear", factor=4.0), f / 4)
    b = rope.inv_freq(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and abs((b[-1] * 4 / f[-1]).item() - 1) < 1e-12
    p = rope.inv_freq(64, scaling="parts", factor=4.0, trained=4096)
    assert p[0] == f[0] and abs((p[-1] * 4 / f[-1]).item() - 1) < 1e-12 and ((p <= f) & (p >= f / 4)).all()
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="x"), dict(rot_dim=8, scaling="parts"),
                dict(rot_dim=8, scaling="linear", factor=0.0)):
        with pytest.raises(ValueError):
            rope.inv_freq(**bad)
