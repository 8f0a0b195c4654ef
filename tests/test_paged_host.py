"""Host side of the paged-cache operators and the token log probabilities: every refusal comes before any
device work (no call here launches a kernel), the described rotation against the float64 definition, and the
oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import tpx
from oracle import paged_oracle as PO

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below fails its checks first
FAKE2 = ctypes.c_void_p(1 << 30)
FAKE3 = ctypes.c_void_p(1 << 32)
ODD = ctypes.c_void_p((1 << 20) + 2)
SH = tpx.make_shape(1024, n_q=8, n_kv=4, hd=128, t=2)
PG = tpx.make_pages(16, 100, 10)


@pytest.fixture(scope="module", autouse=True)
def built():
    from megatron_tensor_transformer_gb300 import build
    build.build_library()
    tpx.lib()


def tables(pages=PG, lens=FAKE, add=FAKE, M=4, free=FAKE, n_free=5, head=None, table=FAKE2, lens_out=FAKE2, cu=FAKE2,
           pos=FAKE2, slots=FAKE2, rows=8, counts=FAKE2):
    return tpx.lib().tp_paged_tables(ctypes.byref(pages) if pages else None, lens, add, M, free, n_free, head, table,
                                     lens_out, cu, pos, slots, rows, counts, None)


def append(sh=SH, rope=None, pages=PG, qkv=FAKE, pos=FAKE, slots=FAKE, M=4, q=FAKE2, k=FAKE3, v=FAKE3, ks=None, vs=None):
    return tpx.lib().tp_rope_append(ctypes.byref(sh), None if rope is None else ctypes.byref(rope), ctypes.byref(pages),
                                    qkv, pos, slots, M, q, k, v, ks, vs, None)


def attn(sh=SH, pages=PG, q=FAKE, k=FAKE3, v=FAKE3, ks=None, vs=None, table=FAKE3, lens=FAKE3, M=4, scale=0.0, window=0,
         o=FAKE2, lse=None, ws=FAKE3, ws_bytes=1 << 30):
    return tpx.lib().tp_paged_attn_decode(ctypes.byref(sh), ctypes.byref(pages), q, k, v, ks, vs, table, lens, M, scale,
                                          window, o, lse, ws, ws_bytes, None)


def logprobs(logits=FAKE, ldl=100, M=4, V=100, ids=FAKE, k=2, lp=FAKE, rank=FAKE, ent=FAKE, tl=FAKE, ti=FAKE):
    return tpx.lib().tp_token_logprobs(logits, ldl, M, V, ids, k, lp, rank, ent, tl, ti, None)


@pytest.mark.parametrize("page_size,n_pages,max_pages,kv,stride,status", [
    (8, 10, 10, 0, 10, tpx.TP_ERR_SHAPE), (48, 10, 10, 0, 10, tpx.TP_ERR_SHAPE), (512, 10, 10, 0, 10, tpx.TP_ERR_SHAPE),
    (16, 0, 10, 0, 10, tpx.TP_ERR_SHAPE), (16, 10, 0, 0, 10, tpx.TP_ERR_SHAPE), (16, 10, 10, 0, 9, tpx.TP_ERR_SHAPE),
    (16, 10, 10, 2, 10, tpx.TP_ERR_INVALID_ARG), (256, 1 << 23, 10, 0, 10, tpx.TP_ERR_UNSUPPORTED)])
def test_bad_pages(page_size, n_pages, max_pages, kv, stride, status):
    bad = tpx.make_pages(page_size, n_pages, max_pages, kv, stride)
    assert tables(bad) == append(pages=bad) == attn(pages=bad) == status


def test_tables_refusals():
    E = tpx.TP_ERR_INVALID_ARG
    assert tables(pages=None) == E and tables(M=-1) == E and tables(n_free=-1) == E and tables(rows=-1) == E
    for kw in (dict(lens=None), dict(add=None), dict(free=None), dict(table=None), dict(lens_out=None), dict(cu=None),
               dict(pos=None), dict(slots=None), dict(counts=None)):
        assert tables(**kw) == E
    assert tables(lens=ODD) == tables(slots=ODD) == tables(head=ODD) == tpx.TP_ERR_ALIGN
    assert tables(lens_out=FAKE) == E                                     # over the lengths
    assert tables(lens_out=ctypes.c_void_p((1 << 20) + 12)) == E          # partly over them
    assert tables(head=FAKE2, counts=ctypes.c_void_p((1 << 30) - 8)) == E  # counts over head
    assert tables(M=0, lens=None) == tpx.TP_OK


def test_rope_refusals():
    E = tpx.TP_ERR_INVALID_ARG
    ok = dict(rot_dim=64, theta=10000.0)

    def status(**kw):
        with pytest.raises(tpx.TpxError) as e:
            tpx.make_rope(**{**ok, **kw})
        return e.value.status
    assert status(rot_dim=24) == status(rot_dim=0) == status(rot_dim=272) == tpx.TP_ERR_SHAPE
    assert status(layout=2) == status(scaling=4) == status(theta=1.0) == status(theta=math.inf) == E
    assert status(scaling=tpx.TP_ROPE_LINEAR, factor=0.0) == E
    assert status(scaling=tpx.TP_ROPE_LINEAR, factor=math.nan) == E
    assert status(scaling=tpx.TP_ROPE_LINEAR, factor=5e-324) == E                     # 1 / factor is infinite
    assert status(scaling=tpx.TP_ROPE_WAVELENGTH, factor=8.0) == E                   # no original length
    assert status(scaling=tpx.TP_ROPE_WAVELENGTH, factor=8.0, original_len=4096, low_freq_factor=4.0) == E
    assert status(scaling=tpx.TP_ROPE_YARN, factor=8.0, original_len=4096, beta_fast=0.0) == E
    rope = tpx.make_rope(64)
    bad = tpx.make_rope(64)
    bad.magic = 0
    assert append(rope=bad) == tpx.TP_ERR_LAYOUT_MISMATCH
    assert append(rope=tpx.make_rope(256)) == tpx.TP_ERR_SHAPE                        # wider than the head
    assert append(sh=tpx.make_shape(1024, n_q=8, n_kv=4, hd=72, t=2), rope=rope) == tpx.TP_ERR_UNSUPPORTED
    assert append(sh=tpx.make_shape(1024, n_q=8, n_kv=4, hd=512, t=2), rope=rope) == tpx.TP_ERR_UNSUPPORTED
    assert append(sh=tpx.make_shape(1024, n_q=8, n_kv=2, hd=128, t=4), rope=rope) == tpx.TP_ERR_SHAPE
    assert append(sh=tpx.make_shape(1024, n_q=65536, n_kv=4, hd=128, t=2), rope=rope) == tpx.TP_ERR_UNSUPPORTED
    for kw in (dict(qkv=None), dict(pos=None), dict(slots=None), dict(q=None), dict(k=None), dict(v=None), dict(M=-1),
               dict(ks=FAKE), dict(vs=FAKE), dict(q=FAKE), dict(q=ctypes.c_void_p((1 << 20) + 4 * 2048 * 2 - 16))):
        assert append(rope=rope, **kw) == E, kw
    for kw in (dict(qkv=ODD), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(pos=ODD), dict(slots=ODD)):
        assert append(rope=rope, **kw) == tpx.TP_ERR_ALIGN, kw
    assert append(rope=rope, M=0) == tpx.TP_OK
    L = tpx.lib()
    f = lambda r, src, pos, dst, M=4: L.tp_rope_forward(ctypes.byref(SH), r, src, pos, M, dst, None)
    r = ctypes.byref(rope)
    assert f(None, FAKE, FAKE, FAKE2) == f(r, None, FAKE, FAKE2) == f(r, FAKE, None, FAKE2) == E
    assert f(r, FAKE, FAKE, None) == f(r, FAKE, FAKE, FAKE2, -1) == E
    assert f(r, FAKE, FAKE, ctypes.c_void_p((1 << 20) + 32)) == E                     # overlaps, not in place
    assert f(r, FAKE, FAKE, ODD) == f(r, FAKE, ODD, FAKE2) == tpx.TP_ERR_ALIGN
    assert f(r, FAKE, FAKE, FAKE, 0) == tpx.TP_OK


def test_attention_refusals():
    E, U = tpx.TP_ERR_INVALID_ARG, tpx.TP_ERR_UNSUPPORTED
    shape = lambda **kw: tpx.make_shape(1024, **{**dict(n_q=8, n_kv=4, hd=128, t=2), **kw})
    assert attn(sh=shape(hd=96)) == attn(sh=shape(n_q=128)) == U
    assert attn(pages=tpx.make_pages(256, 1 << 21, 10)) == U                         # page rows: int32
    assert attn(sh=shape(t=8)) == tpx.TP_ERR_SHAPE
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(o=None), dict(M=-1),
               dict(window=-1), dict(scale=math.inf), dict(scale=math.nan), dict(ks=FAKE), dict(vs=FAKE), dict(o=FAKE)):
        assert attn(**kw) == E, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(ws=ODD), dict(table=ODD), dict(lens=ODD),
               dict(lse=ODD)):
        assert attn(**kw) == tpx.TP_ERR_ALIGN, kw
    need = tpx.tp_paged_attn_workspace_bytes(SH)
    assert need > 0 and attn(ws=None) == attn(ws_bytes=need - 1) == tpx.TP_ERR_WORKSPACE
    assert tpx.tp_paged_attn_workspace_bytes(shape(hd=96)) == 0
    assert attn(M=0, ws=None) == tpx.TP_OK


def test_logprobs_refusals():
    E = tpx.TP_ERR_INVALID_ARG
    for kw in (dict(M=-1), dict(V=0), dict(ldl=99), dict(k=-1), dict(k=101), dict(logits=None), dict(ids=None),
               dict(ids=None, lp=None), dict(tl=None), dict(ti=None)):
        assert logprobs(**kw) == E, kw
    assert logprobs(k=33) == logprobs(V=1 << 30, ldl=1 << 30) == tpx.TP_ERR_UNSUPPORTED
    for kw in (dict(logits=ODD), dict(ids=ODD), dict(lp=ODD), dict(rank=ODD), dict(ent=ODD), dict(tl=ODD), dict(ti=ODD)):
        assert logprobs(**kw) == tpx.TP_ERR_ALIGN, kw
    assert logprobs(M=0) == tpx.TP_OK


def test_logprobs_binding_refusals():
    """What the C call cannot see: logits that are not next to one another, one half of the alternatives alone."""
    x = torch.zeros((4, 100))
    f, n = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    tl, ti = torch.zeros((4, 3)), torch.zeros((4, 3), dtype=torch.int32)
    for args in ((torch.zeros((100, 4)).t(), n, f, f, n), (torch.zeros((4, 200))[:, ::2], n, f, f, n),
                 (torch.zeros((1, 200))[:, ::2], n, f, f, n),
                 (x, n, f, f, n, tl, None), (x, n, f, f, n, None, ti), (x, n, f, f, n, tl, ti[:, :2])):
        with pytest.raises(tpx.TpxError) as e:
            tpx.tp_token_logprobs(*args)
        assert e.value.status == tpx.TP_ERR_INVALID_ARG


def test_block_refusals():
    E = tpx.TP_ERR_INVALID_ARG
    sh = tpx.make_shape(1024, n_q=8, n_kv=4, hd=128, t=2)
    q, o = tpx.tp_describe(sh, tpx.TP_W_QKV), tpx.tp_describe(sh, tpx.TP_W_O)
    BUF = [ctypes.c_void_p((1 << 34) + (i << 28)) for i in range(6)]

    def block(qd=q, od=o, x=FAKE, M=4, rope=None, pages=PG, pos=FAKE, slots=FAKE, k=FAKE3, v=FAKE3, ks=None, table=FAKE,
              lens=FAKE, window=0, y=BUF[0], qkv=BUF[1], qo=BUF[2], oi=BUF[3], ws=BUF[4], n=1 << 27, flags=0):
        return tpx.lib().tp_paged_attn_block_forward(
            ctypes.byref(qd), FAKE, ctypes.byref(od), FAKE, x, None, M, rope, ctypes.byref(pages), pos, slots, k, v, ks, None,
            table, lens, window, y, qkv, qo, oi, ws, n, flags, None)
    other = tpx.tp_describe(tpx.make_shape(1024, n_q=8, n_kv=4, hd=128, t=4), tpx.TP_W_O)
    assert block(od=other) == tpx.TP_ERR_LAYOUT_MISMATCH and block(qd=o) == tpx.TP_ERR_LAYOUT_MISMATCH
    assert block(pages=tpx.make_pages(8, 4, 4)) == tpx.TP_ERR_SHAPE
    for kw in (dict(x=None), dict(M=-1), dict(slots=None), dict(k=None), dict(v=None), dict(ks=FAKE), dict(table=None),
               dict(lens=None), dict(window=-1), dict(y=None), dict(qkv=None), dict(qo=None), dict(oi=None),
               dict(flags=0x1000), dict(oi=BUF[2]), dict(qo=BUF[1])):
        assert block(**kw) == E, kw
    for kw in (dict(x=ODD), dict(y=ODD), dict(qkv=ODD), dict(qo=ODD), dict(oi=ODD), dict(slots=ODD), dict(lens=ODD)):
        assert block(**kw) == tpx.TP_ERR_ALIGN, kw
    need = tpx.tp_paged_attn_block_workspace_bytes(sh, 4)
    assert need > tpx.tp_workspace_bytes(sh, 4) and block(ws=None) == block(n=need - 1) == tpx.TP_ERR_WORKSPACE
    assert block(M=0, x=None, ws=None, n=0) == tpx.TP_OK


@pytest.mark.parametrize("scaling", ["none", "linear", "wavelength", "yarn"])
@pytest.mark.parametrize("rot,theta,factor", [(128, 500000.0, 8.0), (64, 10000.0, 1.0), (32, 1e6, 40.0), (256, 2.0, 0.1)])
def test_described_rotation(scaling, rot, theta, factor):
    """step[i] / 2^64 is f_i / 2 pi modulo 1 to a few parts in 2^53 of f_i."""
    r = tpx.make_rope(rot, theta, scaling=getattr(tpx, "TP_ROPE_" + scaling.upper()), factor=factor, original_len=8192)
    f, mscale = PO.rope_freqs(rot, theta, scaling, factor, 8192)
    turn = np.array([r.step[i] for i in range(rot // 2)], dtype=np.float64) / 2.0 ** 64
    want = np.mod(f / (2 * math.pi), 1.0)
    # eight roundings (pow, divisions, products, the blend), each 2^-53 of the largest term; then the fraction
    # is cut to 64 bits, which takes away up to 2^-64 however small f is
    assert np.all(np.abs(turn - want) <= 16 * 2.0 ** -53 * (f + f / min(1.0, factor)) + 2.0 ** -64)
    assert abs(r.mscale - mscale) <= 2.0 ** -23
    assert list(r.step[rot // 2:]) == [0] * (128 - rot // 2)


def test_oracle_rotation_is_relative():
    """q at position a against k at position b depends on a - b only, and lengths stay."""
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    f, _ = PO.rope_freqs(32, 10000.0)
    for layout in ("half", "interleaved"):
        dots = [float((PO.rope(q, [a], f, 1.0, layout) * PO.rope(k, [b], f, 1.0, layout)).sum())
                for a, b in ((5, 2), (105, 102), (3, 0))]
        assert max(dots) - min(dots) < 1e-10
        assert abs(np.linalg.norm(PO.rope(q, [77], f, 1.0, layout)) - np.linalg.norm(q)) < 1e-12
    # by hand: one pair a quarter turn on
    y = PO.rope(np.array([[[3.0, 5.0, 7.0]]]), [1], np.array([math.pi / 2]), 1.0, "interleaved")
    assert np.allclose(y[0, 0], [-5.0, 3.0, 7.0])


def test_oracle_tables_by_hand():
    """Pages of 16: request 0 grows inside its page, 1 into a new one, 2 is too long for a row of 2 pages, 3 needs
    two of the one page left, 4 needs none and is served."""
    table = np.array([[7, -1], [3, -1], [4, 5], [-1, -1], [2, -1]])
    got = PO.tables([3, 16, 32, 0, 5], [2, 1, 1, 20, 1], [9, 8], 0, table, 16, 2, 10, 25)
    assert got[0].tolist() == [[7, -1], [3, 9], [4, 5], [-1, -1], [2, -1]]
    assert got[1].tolist() == [5, 17, 32, 0, 6]
    assert got[2].tolist() == [0, 2, 3, 4, 24, 25]
    assert got[4].tolist() == [7 * 16 + 3, 7 * 16 + 4, 9 * 16, -1] + [-1] * 20 + [2 * 16 + 5]
    assert got[5].tolist() == [1, 25, 2]
