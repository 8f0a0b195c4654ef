"""Decode attention with shared prefixes where the tests against the paged call's tolerances would not tell: the bits that
weights keep, long runs of one CTA, long sums.  The reference is the formula in 64 bits, on the device."""
import ctypes
import math

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import tpx
from oracle import tp_oracle as O
from tests.test_gpu_paged import HALF, assert_within, dev, i32, sync  # noqa: F401
from tests.test_gpu_parity import bits
from tests.test_gpu_prefix import BOTH, Shared, tails

pytestmark = pytest.mark.gpu


def reference(c, scale=0.0, window=0):
    """o [M, n_q, hd] and lse [M, n_q] of a Shared case whose requests' pages are all there; sum p |v| and the largest sum
    |q| |k| times the scale, for the bounds."""
    M, G = len(c.lens), c.n_q // c.n_kv
    q = c.q.double().view(M, c.n_kv, G, c.hd) * (scale or 1 / math.sqrt(c.hd))
    out = [[], [], [], []]
    for m, n in enumerate(c.lens):
        ids = torch.tensor(c.table[m, : -(-n // c.page)], device=c.dev)

        def rows(x, s):
            raw = x if c.kv == tpx.TP_BF16 else x.view(torch.uint8)
            y = raw[:, ids].view(x.dtype).double().permute(0, 2, 1, 3, 4).reshape(c.n_kv, -1, c.hd)[:, max(0, n - window) if window else 0: n]
            return y if s is None else y * s.double()[:, None, None]
        k, v = rows(c.k, c.ks), rows(c.v, c.vs)
        s = q[m] @ k.transpose(1, 2)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[..., None])
        B = (q[m].abs() @ k.abs().transpose(1, 2)).amax(-1)
        for to, x in zip(out, (p @ v, lse, p @ v.abs(), B)):
            to.append(x.reshape(c.n_q, -1).cpu().numpy())
    o, lse, A, B = (np.stack(x) for x in out)
    return o, lse[..., 0], A, B[..., 0]


def check(c, o, lse, scale=0.0, window=0, dims=None):
    """As Shared.check, with the weights' own bits: 2^-16 of a weight over bf16 pages (two bf16: what the first leaves is
    below 2^-7 of it, and half a step of that), 2^-11 over e4m3 pages.  dims: how many of q's elements are not zero."""
    ro, rl, A, B = reference(c, scale, window)
    got, got_l = O.as_f64(bits(o)).reshape(ro.shape), lse.cpu().numpy().astype(np.float64)
    bf16 = c.kv == tpx.TP_BF16
    n = np.array([min(x, window) if window else x for x in c.lens], np.float64)[:, None]
    # a score within (dims + 8) 2^-23 B (adding zeros is exact), e^x 2^-21, sums n / 16 + 300 steps of 2^-24
    ps = ((dims or c.hd) + 8) * 2.0 ** -23 * B + 2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24
    vmax = float(c.v.float().nan_to_num().abs().max()) * (1.0 if c.vs is None else float(c.vs.max()))
    e = A * (2 * ps[..., None] + (2.0 ** -16 if bf16 else 2.0 ** -11)) + (0 if bf16 else n[..., None] * 2.0 ** -25 * vmax)
    assert_within(got, ro, e + HALF * (np.abs(ro) + e), "o")
    assert_within(got_l, rl, ps + 2.0 ** -21 * (1 + np.abs(rl)), "lse")


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd,n_q", [(64, 16), (128, 32), (256, 8)])
@pytest.mark.parametrize("groups,lens", [([(1, 0)] * 6, [700, 33, 1000, 5, 129, 2500]),               # each request by itself
                                         ([(3, 2000)], [2000, 2017, 2001]),                             # few rows share
                                         ([(20, 1500), (2, 640)], [1500 + 3 * i for i in range(20)] + [700, 641])])
def test_prefix_attention_weights_keep_their_bits(dev, kv, hd, n_q, groups, lens):
    """o is off by its own rounding and what tp_paged_attn_decode's weights are off by, whether a request's positions are
    shared or its own.  One element of q is not zero, so that scores are exact and spread over some ten powers of e."""
    c = Shared(dev, 1, n_q, 2, hd, 32, groups, lens, kv, seed=hd)
    q = c.q.view(len(lens), n_q, hd)
    q[:, :, :3] = q[:, :, 4:] = 0
    q[:, :, 3] = 3.0 * q[:, :, 3].sign() * math.sqrt(hd)
    check(c, *c.launch(), dims=1)


def test_prefix_attention_begins_behind_all_work_before(dev):
    """The second and third kernel read what the call was given beside the first one, without a wait.  So the first has to
    be launched in full stream order: in a captured call its edge from the work before is an ordinary one (full completion,
    with visibility), and only the edges behind it are programmatic."""
    groups = [(4, 300)]
    c = Shared(dev, 1, 8, 2, 64, 16, groups, tails(groups, 3), seed=3)
    want, _ = c.launch()
    o, graph = torch.zeros_like(want), torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        c.q.mul_(1.0)                                                  # work that the call has to wait for
        c.call(o, None)
    f = ctypes.CDLL("libcudart.so.13").cudaGraphGetEdges
    f.argtypes = [ctypes.c_void_p] * 5
    n, handle = ctypes.c_size_t(0), ctypes.c_void_p(graph.raw_cuda_graph())
    assert f(handle, None, None, None, ctypes.byref(n)) == 0
    edges, ends = (ctypes.c_uint8 * (8 * n.value))(), [(ctypes.c_void_p * n.value)() for _ in range(2)]
    assert f(handle, *ends, edges, ctypes.byref(n)) == 0
    kinds = {ends[0][i]: (ends[1][i], edges[8 * i + 2]) for i in range(n.value)}  # node: the next one, the edge's type
    at, order = (set(ends[0]) - set(ends[1])).pop(), []
    while at in kinds:
        at, kind = kinds[at]
        order.append(kind)
    assert order == [0, 1, 1], order
    graph.instantiate()
    for _ in range(3):
        graph.replay()
    sync()
    assert torch.equal(o.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("rows", [2, 20])
def test_prefix_attention_long_sums_of_one_cta(dev, kv, rows):
    """As many tiles as CTAs, each 16384 positions long and with one key ahead of equal others, whose weight a sum of many of
    them rounds the same way every time: a chunk's sum is taken by itself, so a CTA rounds n / 128 + 34 times."""
    sms, n = torch.cuda.get_device_properties(dev).multi_processor_count, 16384
    n_kv = max(x for x in range(1, 17) if sms % x == 0)
    n_q, G = 16 * n_kv if rows == 20 else n_kv, sms // n_kv            # 320 rows: a full tile and a narrow one; or 2
    c = Shared(dev, 1, n_q, n_kv, 64, 64, [(2, n)], [n, n], kv, seed=3, poison=False, std=1.0)
    # every group names the same pages
    M = rows * G
    c.lens, c.table = [n] * M, np.repeat(c.table[:1], M, 0)
    c.cu, c.prefix = rows * np.arange(G + 1), [n] * G
    c.ws = tpx.new_prefix_attn_workspace(c.sh, M, dev)
    c.k.copy_(torch.zeros(c.k.shape, device=dev).to(c.k.dtype))
    c.k[:, int(c.table[0, 0]), :, 0, 0] = torch.ones((1, n_kv), device=dev).to(c.k.dtype)
    if kv == tpx.TP_FP8_E4M3:
        c.ks.fill_(1.0)
    q = torch.zeros((M, n_q, 64), device=dev)
    d = torch.linspace(0.05, 3.0, M * n_q, device=dev).to(torch.bfloat16)
    q[:, :, 0] = d.view(M, n_q).float()
    c.q = q.to(torch.bfloat16).view(M, -1)
    _, lse = c.launch(scale=1.0)
    x = d.double().cpu().numpy().reshape(M, n_q)
    want = x + np.log1p((n - 1) * np.exp(-x))
    # a score's product within 2^-23 of itself, e^x 2^-21, the sum's roundings, lse's own (log2 and its product: 2^-22)
    bound = 2.0 ** -23 * x + 2.0 ** -21 + (n / 128 + 34 + 10) * 2.0 ** -24 + 2.0 ** -22 * want
    over = np.abs(lse.cpu().numpy().astype(np.float64) - want) - bound
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_prefix_attention_long_runs_of_one_cta(dev, kv, hd, page):
    """Enough tiles that a CTA walks most of one, wide or narrow: dozens of chunks, page ids fetched 32 at a time, every
    group's pages its own."""
    rng = np.random.default_rng(page + hd)
    groups = [(int(n), int(p)) for n, p in zip(rng.permutation(np.arange(2, 18).tolist() * 2), rng.integers(3000, 6000, 32))]
    lens = tails(groups, page, 60)
    c = Shared(dev, 1, 64, 4, hd, page, groups, lens, kv, seed=page, poison=False)
    check(c, *c.launch())


@pytest.mark.parametrize("n", [2, 40])
def test_prefix_attention_rows_beside_an_infinite_key(dev, n):
    """A shared key of -inf weighs nothing, to the same bits as if it were not there."""
    groups = [(n, 208)]
    c = Shared(dev, 1, 8, 2, 64, 16, groups, [230] * n, seed=9, poison=False)
    c.q.fill_(1.0)
    c.k[:, int(c.table[0, 0]), :, 5] = float("-inf")
    o, lse = c.launch()
    got, got_l = O.as_f64(bits(o)).reshape(n, 8, 64), lse.cpu().numpy().astype(np.float64)
    keep = np.array([j for j in range(230) if j != 5])
    for m in (0, n - 1):
        k, v = (x[0].double()[c.table[m, keep // 16], :, keep % 16].cpu().numpy() for x in (c.k, c.v))
        for h in range(8):
            s = k[:, h // 4].sum(1) / 8
            top = s.max()
            p = np.exp(s - top)
            ref, A, rl = p @ v[:, h // 4] / p.sum(), p @ np.abs(v[:, h // 4]) / p.sum(), top + math.log(p.sum())
            ps = (64 + 8) * 2.0 ** -23 * np.abs(k[:, h // 4]).sum(1).max() / 8 + 2.0 ** -21 + 320 * 2.0 ** -24
            e = A * (2 * ps + 2.0 ** -16)
            assert_within(got[m, h], ref, e + HALF * (np.abs(ref) + e), f"o of request {m}, head {h}")
            assert abs(got_l[m, h] - rl) <= ps + 2.0 ** -21 * (1 + abs(rl))


@pytest.mark.parametrize("kv", BOTH)
def test_prefix_attention_by_what_a_row_of_the_table_can_name(dev, kv):
    """A table with room for very long requests takes three launches; with the longest one's pages given as max_pages, the
    rows as far apart as before, the call is one launch and gives the bits of a tight table.  So does one request alone."""
    def launches(c):
        before = tpx.tp_launch_count()
        out = c.launch()
        return tpx.tp_launch_count() - before, out
    groups = [(4, 300)]
    lens = tails(groups, 4)
    tight, wide, far = (Shared(dev, 1, 8, 2, 128, 16, groups, lens, kv, seed=4, small=s, stride_pad=p)
                        for s, p in ((True, 0), (False, 0), (True, 8000)))
    (n, (o, lse)), (n2, (o2, lse2)), (n3, _) = launches(tight), launches(far), launches(wide)
    assert (n, n2, n3) == (1, 1, 3)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    one = Shared(dev, 1, 8, 2, 128, 16, [(1, 300)], [317], kv, seed=5)
    n, (o, lse) = launches(one)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    pages = tpx.make_pages(16, one.n_pages, one.max_pages, kv, one.table.shape[1])
    tpx.tp_paged_attn_decode(one.sh, pages, one.q, one.k, one.v, one.table_d, one.lens_d, o2, one.ws, lse=lse2, k_scale=one.ks,
                             v_scale=one.vs)
    sync()
    assert n == 1 and torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
