"""Host side of the attention with shared prefixes and of the sampled tokens: refusals before any device work (no call
here launches a kernel), the workspaces' sizes, and the oracle's own pins."""
import ctypes
import glob
import math
import os
import re

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import tpx
from oracle import paged_oracle as PO
from tests.test_paged_host import FAKE, FAKE2, FAKE3, ODD, PG, SH


@pytest.fixture(scope="module", autouse=True)
def built():
    from megatron_tensor_transformer_gb300 import build
    build.build_library()
    tpx.lib()


def attn(sh=SH, pages=PG, q=FAKE, k=FAKE3, v=FAKE3, ks=None, vs=None, table=FAKE3, lens=FAKE3, M=4, cu=FAKE3, prefix=FAKE3,
         n=2, scale=0.0, window=0, o=FAKE2, lse=None, ws=FAKE3, ws_bytes=1 << 40):
    return tpx.lib().tp_prefix_attn_decode(ctypes.byref(sh), ctypes.byref(pages), q, k, v, ks, vs, table, lens, M, cu, prefix,
                                           n, scale, window, o, lse, ws, ws_bytes, None)


def sample(logits=FAKE, ldl=100, M=4, V=100, u=FAKE, T=FAKE, k=FAKE, p=FAKE, q=FAKE, ids=FAKE2, lp=FAKE2):
    return tpx.lib().tp_sample_tokens(logits, ldl, M, V, u, T, k, p, q, ids, lp, None)


def test_prefix_attention_refusals():
    E, U = tpx.TP_ERR_INVALID_ARG, tpx.TP_ERR_UNSUPPORTED
    shape = lambda **kw: tpx.make_shape(1024, **{**dict(n_q=8, n_kv=4, hd=128, t=2), **kw})
    assert attn(sh=shape(hd=96)) == attn(sh=shape(n_q=128)) == U
    assert attn(pages=tpx.make_pages(256, 1 << 21, 10)) == U
    assert attn(sh=shape(t=8)) == attn(pages=tpx.make_pages(24, 10, 10)) == tpx.TP_ERR_SHAPE
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(o=None), dict(M=-1),
               dict(window=-1), dict(scale=math.inf), dict(scale=math.nan), dict(ks=FAKE), dict(vs=FAKE), dict(o=FAKE),
               dict(n=-1), dict(n=5), dict(cu=None), dict(prefix=None)):
        assert attn(**kw) == E, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(ws=ODD), dict(table=ODD), dict(lens=ODD),
               dict(lse=ODD), dict(cu=ODD), dict(prefix=ODD)):
        assert attn(**kw) == tpx.TP_ERR_ALIGN, kw
    need = tpx.tp_prefix_attn_workspace_bytes(SH, 4)
    assert attn(ws=None) == attn(ws_bytes=need - 1) == tpx.TP_ERR_WORKSPACE
    assert attn(M=0, n=0, ws=None) == tpx.TP_OK


def test_prefix_attention_workspace_sizes():
    """Grows with M, holds a paged call's, and is 0 for shapes that the attention does not take."""
    for hd in (64, 128, 256):
        sh = tpx.make_shape(1024, n_q=16, n_kv=2, hd=hd)
        sizes = [tpx.tp_prefix_attn_workspace_bytes(sh, M) for M in (0, 1, 7, 300, 100000)]
        assert sizes == sorted(sizes) and sizes[0] >= tpx.tp_paged_attn_workspace_bytes(sh) > 0
    assert tpx.tp_prefix_attn_workspace_bytes(tpx.make_shape(1024, n_q=8, n_kv=4, hd=96), 4) == 0
    assert tpx.tp_prefix_attn_workspace_bytes(SH, -1) == 0


def test_prefix_attention_binding_refusals():
    """Group bounds that are not one more than the prefixes, which the C call cannot see."""
    x, n = torch.zeros((4, 1024), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for cu, prefix in ((n[:2], n[:2]), (n[:3], n[:1]), (n[:1], n[:3])):
        with pytest.raises(tpx.TpxError) as e:
            tpx.tp_prefix_attn_decode(SH, PG, x, x, x, n, n, cu, prefix, x, x)
        assert e.value.status == tpx.TP_ERR_INVALID_ARG


def test_sample_refusals():
    E = tpx.TP_ERR_INVALID_ARG
    for kw in (dict(M=-1), dict(V=0), dict(ldl=99), dict(logits=None), dict(u=None), dict(ids=None)):
        assert sample(**kw) == E, kw
    assert sample(V=(1 << 19) + 1, ldl=1 << 20) == tpx.TP_ERR_UNSUPPORTED
    for kw in (dict(logits=ODD), dict(u=ODD), dict(T=ODD), dict(k=ODD), dict(p=ODD), dict(q=ODD), dict(ids=ODD), dict(lp=ODD)):
        assert sample(**kw) == tpx.TP_ERR_ALIGN, kw
    assert sample(M=0, logits=None, u=None, ids=None) == tpx.TP_OK


def test_sample_binding_refusals():
    f, n = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    for x in (torch.zeros((100, 4)).t(), torch.zeros((4, 200))[:, ::2], torch.zeros((1, 200))[:, ::2]):
        with pytest.raises(tpx.TpxError) as e:
            tpx.tp_sample_tokens(x, f, n)
        assert e.value.status == tpx.TP_ERR_INVALID_ARG


def test_oracle_sample_by_hand():
    """Weights 1, 1/2, 1/4, 1/8 (of ids 2, 0, 3, 1): sums by id 1/2, 5/8, 13/8, 15/8."""
    x = np.log([0.5, 0.125, 1.0, 0.25])
    pick = lambda u, **kw: PO.sample(x, u, **kw)[0]
    assert [pick(u)[0] for u in (0.0, 0.26, 0.27, 0.33, 0.34, 0.86, 0.87, 0.999, 1.5)] == [0, 0, 1, 1, 2, 2, 3, 3, 3]
    assert [pick(u, k=2)[0] for u in (0.0, 0.33, 0.34, 0.99)] == [0, 0, 2, 2]
    assert [pick(u, p=0.5)[0] for u in (0.0, 0.5)] == [2, 2]           # the first rank weighs more than half
    assert [pick(u, p=0.54)[0] for u in (0.0, 0.5)] == [0, 2]
    assert [pick(u, q=0.3)[0] for u in (0.0, 0.5)] == [0, 2]
    assert pick(0.99, T=0.0) == [2] and abs(PO.sample(x, 0.5, k=2)[1][0] - math.log(2 / 3)) < 1e-12
    assert pick(0.1, T=0.5)[0] == 0 and pick(0.195, T=0.5)[0] == 1   # weights 1/4, 1/64, 1, 1/16
    assert PO.sample(np.array([1.0, np.nan]), 0.5)[0] == [-1]
    assert sorted(set(pick(1 / 3 + 1e-9, slack=1e-6))) == [1, 2]


def test_oracle_shared_rows():
    got = PO.shared_by([0, 1, 3, 3, 6], [50, 40, 9, 31], 8, 16, 10)
    assert got == [(0, 0), (32, 1), (32, 1), (16, 3), (16, 3), (16, 3), (0, 6), (0, 7)]
    assert PO.shared_by([2, 1, 9], [50, 40], 8, 16, 10) == [(0, m) for m in range(8)]
    assert PO.shared_by([0, 4], [161], 4, 16, 10) == [(0, m) for m in range(4)]


def test_oracle_sample_min_p_above_one_and_infinite_temperature():
    x = np.array([0.0, 2.0, 2.0, -np.inf])
    assert [PO.sample(x, u, q=1.5) for u in (0.0, 0.9)] == [([1], [0.0])] * 2
    assert [PO.sample(x, u, q=1.0)[0] for u in (0.4, 0.6)] == [[1], [2]]
    assert [PO.sample(x, u, T=np.inf, q=q)[0][0] for q in (0.0, 0.5, 1.0) for u in (0.0, 0.4, 0.7, 0.999)] == [0, 1, 2, 2] * 3


def test_error_words_name_their_kernel():
    """A wait that runs out leaves a word by which its file is known."""
    from megatron_tensor_transformer_gb300 import build
    words = {}
    for f in glob.glob(os.path.join(build.CSRC, "*.cu")):
        with open(f) as src:
            for w in set(re.findall(r"err(?:or)?,\s*(\d+)u", src.read())):
                words.setdefault(int(w), []).append(os.path.basename(f))
    assert len(words) > 20 and all(len(f) == 1 for f in words.values()), words


def test_sample_binding_refuses_what_the_call_would_misread():
    """A column of a table of settings, another type, too few elements: data_ptr() alone says nothing of them."""
    x, f, n = torch.zeros((4, 100)), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    column, far = torch.zeros((4, 5))[:, 0], torch.zeros((4, 5), dtype=torch.int32)[:, 1]
    good = dict(u=f, ids=n, temperature=f, top_k=n, top_p=f, min_p=f, logprob=f)
    bad = [{k: far if k in ("ids", "top_k") else column} for k in good] + [{k: f.double()} for k in good] + [{k: n[:3]} for k in good]
    bad += [{k: (n if k in ("ids", "top_k") else f)[:3]} for k in good]
    for b in bad + [dict(logits=x.double())]:
        a = {**good, "logits": x, **b}
        with pytest.raises(tpx.TpxError) as e:
            tpx.tp_sample_tokens(a.pop("logits"), a.pop("u"), a.pop("ids"), **a)
        assert e.value.status == tpx.TP_ERR_INVALID_ARG, b


def test_prefix_attention_binding_refuses_what_the_call_would_misread():
    M, row = 4, SH.n_q_heads * SH.head_dim
    pages = tpx.make_pages(16, 5, 3, table_stride=7)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    n32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = bf(SH.t, 5, SH.n_kv_heads // SH.t, 16, SH.head_dim)
    good = dict(q=bf(M, row), k_pages=pool, v_pages=pool, block_table=n32(M, 7)[:, :3], lens=n32(M), cu_groups=n32(3),
                prefix_lens=n32(2), o_in=bf(M, row), lse=torch.zeros((M, SH.n_q_heads)))
    for b in (dict(q=bf(M, 2 * row)[:, :row]), dict(q=torch.zeros((M, row))), dict(o_in=bf(row, M).t()), dict(o_in=bf(M - 1, row)),
              dict(k_pages=pool.view(torch.uint8)), dict(v_pages=pool.transpose(3, 4)), dict(k_pages=pool[:, :4].contiguous()),
              dict(lens=n32(M, 2)[:, 0]), dict(lens=n32(M).long()), dict(lens=n32(M - 1)), dict(cu_groups=n32(6)[::2]),
              dict(prefix_lens=n32(4)[::2]), dict(prefix_lens=n32(2).float()), dict(lse=torch.zeros((SH.n_q_heads, M)).t()),
              dict(block_table=n32(M, 3)), dict(block_table=n32(7, M).t()), dict(block_table=n32(M, 7)[:, :2]),
              dict(block_table=n32(M - 1, 7)), dict(block_table=n32(M, 7).long()), dict(block_table=n32(M * 7))):
        with pytest.raises(tpx.TpxError) as e:
            tpx.tp_prefix_attn_decode(SH, pages, ws=torch.zeros(1, dtype=torch.uint8), **{**good, **b})
        assert e.value.status == tpx.TP_ERR_INVALID_ARG, list(b)
    with pytest.raises(tpx.TpxError) as e:                             # the good ones reach the call, which sees the workspace
        tpx.tp_prefix_attn_decode(SH, pages, ws=torch.zeros(1, dtype=torch.uint8), **good)
    assert e.value.status == tpx.TP_ERR_WORKSPACE
