"""Decode attention with shared prefixes through the C ABI against the float64 oracle, and a run of samples to one
prompt: tables, append, attention, projections, logits, sampled tokens."""
import math

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import inputs, tpx
from oracle import paged_oracle as PO
from oracle import tp_oracle as O
from tests.test_gpu_paged import HALF, Case, assert_within, dev, i32, make_qkv, sync, values  # noqa: F401
from tests.test_gpu_parity import bits

pytestmark = pytest.mark.gpu


SMALL = 96 << 20  # bytes of cache that a table can name, up to which sharing is not looked at


class Shared(Case):
    """groups: (requests, prefix) one after another; lens of all requests; rows of a group name the same pages first."""

    def __init__(self, dev, t, n_q, n_kv, hd, page, groups, lens, kv=tpx.TP_BF16, seed=0, poison=True, std=1.0, stride_pad=0,
                 small=False):
        super().__init__(dev, t, n_q, n_kv, hd, page, lens, kv, seed, poison=False, std=std, stride_pad=stride_pad)
        # Where all that M rows of the table can hold is little, the call attends to each request by itself: such a table,
        # or one with room for more.
        held = len(lens) * n_kv * hd * 2 * (2 if kv == tpx.TP_BF16 else 1) * page
        room = 0 if small else max(0, SMALL // held + 1 - self.max_pages)
        self.max_pages += room
        if room:
            self.table = np.concatenate([self.table, np.full((len(lens), room), 2 ** 31 - 1, np.int64)], 1)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in groups])])
        self.prefix = [p for _, p in groups]
        rng = np.random.default_rng(seed + 77)
        for g, (n, p) in enumerate(groups):
            whole = p // page
            if n < 2 or not 0 <= p <= self.max_pages * page:
                continue
            rows = range(int(self.cu[g]), min(int(self.cu[g + 1]), len(lens)))
            shared = max((self.table[r, :whole] for r in rows), key=lambda ids: (ids < self.n_pages).sum()).copy()
            shared[shared >= self.n_pages] = rng.integers(0, self.n_pages, (shared >= self.n_pages).sum())
            for r in rows:
                self.table[r, :whole] = shared
        if poison:  # every cache row that no request attends to holds NaN
            used = torch.zeros((self.n_pages, page), dtype=torch.bool)
            for m, n in enumerate(lens):
                for j in range(max(0, -(-n // page))):
                    if 0 <= self.table[m, j] < self.n_pages:
                        used[self.table[m, j], : max(0, min(page, n - j * page))] = True
            for x in (self.k, self.v):
                raw = x.view(torch.int16 if kv == tpx.TP_BF16 else torch.uint8)
                raw.masked_fill_(~used.to(dev)[None, :, None, :, None], 0x7FC0 if kv == tpx.TP_BF16 else 0x7F)
        self.ws = tpx.new_prefix_attn_workspace(self.sh, len(lens), dev)

    def call(self, o, lse, window=0, scale=0.0, stream=None):
        pages = tpx.make_pages(self.page, self.n_pages, self.max_pages, self.kv, self.table.shape[1])
        if not hasattr(self, "cu_d"):
            self.cu_d, self.prefix_d = i32(self.cu, self.dev), i32(self.prefix, self.dev)
        tpx.tp_prefix_attn_decode(self.sh, pages, self.q, self.k, self.v, self.table_d, self.lens_d, self.cu_d,
                                  self.prefix_d, o, self.ws, lse=lse, window=window, scale=scale, k_scale=self.ks,
                                  v_scale=self.vs, stream=stream)

    def check(self, window=0, scale=0.0):
        o, lse = self.launch(window, scale)
        M = len(self.lens)
        k, v = values(self.k), values(self.v)
        q = O.as_f64(bits(self.q)).reshape(M, self.n_q, self.hd)
        got, got_l = O.as_f64(bits(o)).reshape(q.shape), lse.cpu().numpy().astype(np.float64)
        sc = [np.ones(self.n_kv) if s is None else s.cpu().numpy().astype(np.float64) for s in (self.ks, self.vs)]
        factor = scale or 1 / math.sqrt(self.hd)
        bf16 = self.kv == tpx.TP_BF16
        for m, n in enumerate(self.lens):
            n = n if 0 <= n <= self.max_pages * self.page else 0
            ids = self.table[m][np.arange(n) // self.page]
            count = (ids >= 0) & (ids < self.n_pages)
            at, off = np.where(count, ids, 0), np.arange(n) % self.page

            def rows(x, s):
                def f(g):
                    sh, gl = divmod(g, self.n_kv // self.t)
                    return x[sh][at, gl, off] * s[g], count
                f.n_kv = self.n_kv
                return f
            ro, rl, A, B = PO.attention(q[m], rows(k, sc[0]), rows(v, sc[1]), factor, window)
            # As for tp_paged_attn_decode: a score within (hd + 8) 2^-23 B, e^x 2^-21, sums n / 16 + 300 steps of 2^-24
            # (the shared part's partial sums are joined in at most 200 steps: within the 300).  The shared weights
            # enter the product in bf16, half a step of which is 2^-8; over e4m3 pages in fp16 (2^-11, and 2^-32 of the
            # largest weight, against a sum of at least a largest weight); the others as there: 2^-25 covers both.
            ps = (self.hd + 8) * 2.0 ** -23 * B + 2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24
            pp = HALF if bf16 else 2.0 ** -11
            vmax = np.abs(v[:, at[count], :, off[count]]).max() * sc[1].max() if count.any() else 0.0
            e = A * (2 * ps[:, None] + pp) + (0 if bf16 else n * 2.0 ** -25 * vmax)
            assert_within(got[m], ro, e + HALF * (np.abs(ro) + e), f"o of request {m}, length {n}")
            fine = np.isfinite(rl)
            assert np.array_equal(np.isneginf(rl), np.isneginf(got_l[m]))
            if fine.any():
                assert_within(got_l[m][fine], rl[fine], ps[fine] + 2.0 ** -21 * (1 + np.abs(rl[fine])), f"lse of {m}")
            if not fine.any():
                assert not got[m].any()
        assert not self.ws[:4 * 1024].any()                            # the counters are left at zero
        return o, lse


def tails(groups, seed, most=200):
    """A length behind each group's prefix: none, one position, a chunk's edges among them."""
    rng = np.random.default_rng(seed)
    lens = []
    for n, p in groups:
        t = rng.integers(0, most, n)
        t[: min(n, 6)] = [1, 0, 128, 127, 16, 129][: min(n, 6)]
        lens += (max(p, 0) + t).tolist()
    return lens


BOTH = [tpx.TP_BF16, tpx.TP_FP8_E4M3]


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("t,n_q,n_kv,hd", [(1, 8, 4, 64), (2, 16, 4, 128), (4, 16, 4, 256), (2, 32, 2, 128), (1, 3, 3, 64),
                                           (1, 6, 2, 128), (1, 5, 1, 256)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prefix_attention_groups(dev, kv, t, n_q, n_kv, hd, page):
    groups = [(3, 300), (1, 200), (2, 16), (5, 128), (2, 1), (2, 0), (4, 513), (2, page), (3, 2 * page - 1)]
    Shared(dev, t, n_q, n_kv, hd, page, groups, tails(groups, page + hd), kv, seed=page + hd, stride_pad=page // 16).check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("t,n_q,n_kv,hd,page", [(1, 8, 4, 64, 16), (2, 16, 4, 128, 32), (1, 5, 1, 256, 64)])
def test_prefix_attention_small_tables(dev, kv, t, n_q, n_kv, hd, page):
    """Tables that hold little: each request by itself, the bits of tp_paged_attn_decode."""
    groups = [(3, 300), (1, 200), (5, 128)]
    c = Shared(dev, t, n_q, n_kv, hd, page, groups, tails(groups, hd), kv, seed=hd, small=True)
    o, lse = c.check()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    pages = tpx.make_pages(page, c.n_pages, c.max_pages, kv, c.table.shape[1])
    tpx.tp_paged_attn_decode(c.sh, pages, c.q, c.k, c.v, c.table_d, c.lens_d, o2, c.ws, lse=lse2, k_scale=c.ks, v_scale=c.vs)
    sync()
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("t,n_q,n_kv,hd,n", [(1, 16, 2, 128, 16), (1, 16, 2, 128, 17), (2, 16, 2, 128, 33), (1, 32, 2, 128, 40),
                                             (1, 3, 1, 128, 171), (1, 16, 1, 64, 50), (2, 8, 2, 256, 65), (1, 16, 1, 256, 24)])
def test_prefix_attention_rows_of_a_group(dev, kv, t, n_q, n_kv, hd, n):
    """Requests times heads: one tile of rows full, a little more, several, the last one ragged."""
    groups = [(n, 700), (2, 260)]
    Shared(dev, t, n_q, n_kv, hd, 32, groups, tails(groups, n, 40), kv, seed=n).check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd,n_q", [(64, 4), (128, 16), (256, 8)])
def test_prefix_attention_long_prefix(dev, kv, hd, n_q):
    """All SMs share one prefix, and the same bits come again; lse is optional."""
    groups = [(9, 20011)]
    c = Shared(dev, 1, n_q, 2, hd, 64, groups, tails(groups, 1), kv, seed=5, std=2.0)
    o, lse = c.check()
    o2, lse2 = c.launch()
    o3, _ = c.launch(with_lse=False)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    assert torch.equal(o.view(torch.int16), o3.view(torch.int16))


@pytest.mark.parametrize("M,G", [(33, 16), (289, 100), (700, 9), (600, 290)])
def test_prefix_attention_many_groups(dev, M, G):
    rng = np.random.default_rng(M)
    cuts = np.sort(rng.choice(np.arange(1, M), G - 1, replace=False))
    sizes = np.diff(np.concatenate([[0], cuts, [M]]))
    groups = [(int(n), int(p)) for n, p in zip(sizes, rng.integers(0, 300, G))]
    lens = tails(groups, M, 50)
    lens[5] = 0
    Shared(dev, 1, 4, 2, 64, 16, groups, lens, seed=M).check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("chunks", [1, 3, 4])
def test_prefix_attention_tiles_of_both_kinds_in_turn(dev, kv, hd, chunks):
    """Every CTA takes several tiles, of two blocks of rows and of one in turn, whole ones and parts: as paged attention
    of each request by itself, to within the weights' rounding and the outputs'."""
    groups = [g for _ in range(130) for g in ((9, 128 * chunks - 20), (2, 128 * chunks), (17, 64))]
    lens = tails(groups, chunks, 40)
    c = Shared(dev, 1, 64, 4, hd, 16, groups, lens, kv, seed=chunks, poison=False)
    o, lse = c.launch()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    pages = tpx.make_pages(16, c.n_pages, c.max_pages, kv, c.table.shape[1])
    tpx.tp_paged_attn_decode(c.sh, pages, c.q, c.k, c.v, c.table_d, c.lens_d, o2, c.ws, lse=lse2, k_scale=c.ks, v_scale=c.vs)
    sync()
    seen = torch.isfinite(lse2)
    assert torch.equal(seen, torch.isfinite(lse)) and float((lse - lse2)[seen].abs().max()) <= 1e-4
    a, b = o.float().view(-1, hd), o2.float().view(-1, hd)
    # row by row: half a step of the weights and of both outputs, against the row's size, with room for unlike signs
    far = (a - b).norm(dim=1) / b.norm(dim=1).clamp(min=1e-6)
    assert float(far.max()) <= 6 * HALF, int(far.argmax())


@pytest.mark.parametrize("kv", BOTH)
def test_prefix_attention_rows_by_themselves(dev, kv):
    """Shorter than the shared part, empty, negative, past the table, outside every group: as without sharing."""
    groups = [(6, 400), (3, 300), (2, 64)]
    lens = [450, 399, 0, 100, 400, 384, 20, 700, 301, 3, 64]
    c = Shared(dev, 2, 8, 4, 128, 16, groups, lens, kv, seed=6, poison=False)
    c.check()
    c.lens = [500, -5, 2 ** 31 - 1, 100, 400, 384, -(2 ** 31), 700, 301, 3, 64]
    c.check()
    c.cu_d = i32([2, 6, 6, 6], dev)                                    # rows before and behind the groups
    c.check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("window", [1, 100, 300, 470, 1000])
def test_prefix_attention_window(dev, kv, window):
    """A window that begins behind, among, and before the shared positions."""
    groups = [(5, 320), (4, 150)]
    c = Shared(dev, 1, 8, 4, 128, 32, groups, tails(groups, 3, 250), kv, seed=window, poison=False)
    c.check(window)


@pytest.mark.parametrize("cu,prefix", [([0, 4, 2, 9], [300, 300, 300]), ([0, 4, 40], [300, 300]), ([-3, 4, 9], [300, 200]),
                                       ([0, 5, 9], [-7, 2 ** 31 - 1]), ([0, 0, 9, 9], [300, 300, 300]),
                                       ([2 ** 31 - 1, -(2 ** 31), 9], [300, 300]), ([9, 9, 9], [5, 300]), ([3], [])])
def test_prefix_attention_groups_out_of_order(dev, cu, prefix):
    """Groups that break the rules count as without a prefix; the result is the requests' own in any case."""
    c = Shared(dev, 1, 8, 2, 128, 16, [(9, 304)], tails([(9, 304)], 8), seed=8, poison=False)
    c.cu_d, c.prefix_d = i32(cu, dev), i32(prefix, dev)
    c.check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prefix_attention_pages_that_are_none(dev, kv, page, hd):
    """Shared pages outside the pool are left out for all; where no other position is left, the row is zero."""
    groups = [(4, 5 * page), (3, 2 * page), (2, page)]
    c = Shared(dev, 2, 8, 2, hd, page, groups, [5 * page + 9, 5 * page, 6 * page + 1, 5 * page] + [2 * page] * 3 + [page, page + 3],
               kv, seed=7, poison=False)
    c.table[:4, [0, 3]] = [-1, c.n_pages]
    c.table[4:7, :2] = -(2 ** 31)
    c.table[7:, 0] = 2 ** 31 - 1
    c.check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prefix_attention_scale_and_peaky_scores(dev, kv, hd):
    groups = [(20, 600), (3, 130)]
    c = Shared(dev, 1, 16, 2, hd, 32, groups, tails(groups, 9), kv, seed=9, std=30.0)
    c.check()
    c.check(scale=0.003)
    c.check(scale=-0.2)
    c.q.mul_(1e-30)
    c.check()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 28, 2.0 ** 60, -(2.0 ** 32)])
@pytest.mark.parametrize("n_q", [4, 32])
def test_prefix_attention_scores_with_a_spacing_above_one(dev, kv, scale, n_q):
    """As for paged attention: q (1, 0, ..), k (1, 3 or 5, 0, ..): only the largest scores weigh, all alike."""
    groups = [(3, 2000), (2, 48)]
    c = Shared(dev, 1, n_q, 2, 64, 16, groups, [2000, 2100, 2001, 48, 60], kv, seed=31, poison=False)
    c.q.zero_()
    c.q.view(5, n_q, 64)[:, :, 0] = 1.0
    c.k.copy_(torch.zeros(c.k.shape, device=dev).to(c.k.dtype))
    if kv == tpx.TP_FP8_E4M3:
        c.ks.fill_(1.0)
    keys = np.random.default_rng(31).choice([1.0, 3.0, 5.0], size=(c.n_pages, 2, 16), p=[0.4, 0.3, 0.3])
    keys[c.table[3, :3]] = np.minimum(keys[c.table[3, :3]], 3.0)
    c.k[0, :, :, :, 0] = torch.tensor(keys, dtype=torch.float32, device=dev).to(c.k.dtype)
    o, lse = c.launch(scale=scale)
    got, got_l, v = O.as_f64(bits(o)).reshape(5, n_q, 64), lse.cpu().numpy().astype(np.float64), values(c.v)
    vs = np.ones(2) if c.vs is None else c.vs.cpu().numpy().astype(np.float64)
    for m, n in enumerate(c.lens):
        at, off = c.table[m, np.arange(n) // 16], np.arange(n) % 16
        for h in range(n_q):
            g = h // (n_q // 2)
            s = keys[at, g, off] * scale
            rows = v[0][at, g, off][s == s.max()] * vs[g]
            ref, A = rows.mean(0), np.abs(rows).mean(0)
            # equal weights: their common rounding divides out of nothing (the sum holds them unrounded): half a bf16
            e = A * (2 * (2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24) + HALF)
            if kv == tpx.TP_FP8_E4M3:
                e = e + n * 2.0 ** -25 * np.abs(rows).max()
            assert_within(got[m, h], ref, e + HALF * (np.abs(ref) + e), f"o of request {m}")
            want = s.max() + math.log(len(rows))
            assert abs(got_l[m, h] - want) <= 2.0 ** -20 * (1 + abs(want)), (m, h)


@pytest.mark.parametrize("kv", BOTH)
def test_prefix_attention_scores_near_the_lowest(dev, kv):
    """Scores of -2^126 are scores, not masks: the mean of v and lse -2^126."""
    groups = [(3, 1000)]
    c = Shared(dev, 1, 4, 2, 64, 16, groups, [1000, 1030, 1001], kv, seed=32, poison=False)
    c.q.fill_(2.0 ** 60)
    c.k.copy_(torch.full(c.k.shape, -(2.0 ** 60) if kv == tpx.TP_BF16 else -256.0, device=dev).to(c.k.dtype))
    if kv == tpx.TP_FP8_E4M3:
        c.ks.fill_(2.0 ** 52)
    o, lse = c.launch(scale=1.0)
    got, got_l, v = O.as_f64(bits(o)).reshape(3, 4, 64), lse.cpu().numpy().astype(np.float64), values(c.v)
    vs = np.ones(2) if c.vs is None else c.vs.cpu().numpy().astype(np.float64)
    for m, n in enumerate(c.lens):
        for h in range(4):
            rows = v[0][c.table[m, np.arange(n) // 16], h // 2, np.arange(n) % 16] * vs[h // 2]
            ref, A = rows.mean(0), np.abs(rows).mean(0)
            e = A * (2 * (2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24) + HALF)
            if kv == tpx.TP_FP8_E4M3:
                e = e + n * 2.0 ** -25 * np.abs(rows).max()
            assert_within(got[m, h], ref, e + HALF * (np.abs(ref) + e), f"o of request {m}")
            assert abs(got_l[m, h] + 2.0 ** 126) <= 2.0 ** (126 - 20), (m, h)


@pytest.mark.parametrize("n", [2, 40])
def test_prefix_attention_infinite_and_nan_scores(dev, n):
    """In the shared part: a key of -inf weighs nothing, a NaN one makes its group's rows NaN and no others."""
    groups = [(n, 208), (n, 208), (n, 16)]
    c = Shared(dev, 1, 8, 2, 64, 16, groups, [230] * n + [209] * n + [16] * n, seed=9, poison=False)
    c.q.fill_(1.0)
    page = lambda m, j: int(c.table[m, j // 16])
    c.k[:, page(0, 5), :, 5] = float("-inf")
    c.k[:, page(n, 20), 0, 20 % 16] = float("nan")
    c.k[:, page(2 * n, 0)] = float("-inf")                             # nothing else to attend to
    o, lse = c.launch()
    o, lse = o.view(3, n, 8, 64).float(), lse.view(3, n, 8)
    k, v = values(c.k), values(c.v)
    keep = [j for j in range(230) if j != 5]
    for h in (0, 7):
        s = np.array([k[0, page(1, j), h // 4, j % 16].sum() / 8 for j in keep])
        p = np.exp(s - s.max())
        ref = (p / p.sum()) @ np.array([v[0, page(1, j), h // 4, j % 16] for j in keep])
        assert np.allclose(o[0, 1, h].cpu().numpy(), ref, rtol=2 ** -6, atol=1e-3)
    assert torch.isfinite(o[0]).all() and torch.isnan(o[1, :, :4]).all() and torch.isfinite(o[1, :, 4:]).all()
    assert not o[2].any() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("kv", BOTH)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prefix_attention_infinite_q(dev, kv, hd):
    """An infinity in q makes its head's row NaN and leaves every other row its bits."""
    groups = [(5, 300), (2, 33)]
    c = Shared(dev, 2, 8, 4, hd, 32, groups, tails(groups, 21), kv, seed=21)
    want, want_l = c.launch()
    c.q[0, 5 * hd + 3] = float("inf")
    c.q[3, 1 * hd + 50] = float("-inf")
    o, lse = c.launch()
    hit = torch.zeros((7, 8), dtype=torch.bool, device=dev)
    hit[0, 5] = hit[3, 1] = True
    o, want = o.view(7, 8, hd), want.view(7, 8, hd)
    assert torch.isnan(o[hit].float()).all() and torch.isfinite(want.float()).all()
    assert torch.equal(o[~hit].view(torch.int16), want[~hit].view(torch.int16))
    assert torch.equal(lse[~hit], want_l[~hit]) and not torch.isfinite(lse[hit]).any()


def test_prefix_attention_small_q_and_weights(dev):
    """Over e4m3 pages: elements of q far below their head's largest, and many small weights beside a large one."""
    groups = [(3, 4096)]
    c = Shared(dev, 1, 4, 2, 128, 64, groups, [4100, 4096, 4200], tpx.TP_FP8_E4M3, seed=40)
    c.q.view(3, 4, 128)[:, :, ::2] *= 2.0 ** -12
    c.q.view(3, 4, 128)[1] *= 2.0 ** -100
    c.q.view(3, 4, 128)[2, 0] *= 2.0 ** 90
    c.q.view(3, 4, 128)[2, 0, 1::2] = 0
    c.check()
    c.q.view(3, 4, 128)[1, 1] = 0                                      # an all-zero head
    c.check()


def test_one_workspace_for_shapes_sizes_and_paged_calls(dev):
    """A workspace of the largest size serves other shapes, fewer requests and paged calls in between."""
    groups = [(30, 900), (3, 100)]
    big = Shared(dev, 1, 32, 2, 256, 16, groups, tails(groups, 2), seed=11)
    for t, n_q, n_kv, hd in ((1, 4, 4, 64), (2, 32, 2, 128), (1, 8, 1, 256)):
        g = [(4, 700), (2, 64)]
        c = Shared(dev, t, n_q, n_kv, hd, 32, g, tails(g, hd), seed=hd)
        assert c.ws.numel() <= big.ws.numel()
        c.ws = big.ws
        c.check()
        p = Case(dev, t, n_q, n_kv, hd, 32, [2500, 0, 33, 4000], seed=hd)
        p.ws = big.ws
        p.check()
    big.check()


def test_two_prefix_calls_at_once(dev):
    """Calls on two streams with a workspace each, and replays of captured ones, give the bits of calls in order."""
    ga, gb = [(40, 3000), (2, 500)], [(5, 700), (1, 30), (9, 100)]
    a = Shared(dev, 1, 32, 8, 128, 64, ga, tails(ga, 1), seed=23)
    b = Shared(dev, 1, 8, 4, 256, 16, gb, tails(gb, 2), tpx.TP_FP8_E4M3, seed=24)
    want = [x.launch()[0].clone() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for x, s, o in zip((a, b), streams, outs):
            x.call(o[i], None, stream=s)
    torch.cuda.synchronize()
    graphs = []
    for x, s, w in zip((a, b), streams, want):
        graph, o = torch.cuda.CUDAGraph(), torch.zeros_like(w)
        with torch.cuda.graph(graph, stream=s):
            x.call(o, None, stream=s)
            x.call(o, None, stream=s)
        graphs.append((graph, o))
    for _ in range(5):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    sync()
    torch.cuda.synchronize()
    for w, o, (_, g) in zip(want, outs, graphs):
        assert all(torch.equal(w.view(torch.int16), y.view(torch.int16)) for y in o + [g])


def test_prefix_attention_past_4_gib(dev):
    """Shared pages whose byte offsets pass 32 bits (a pool of 5 GiB per side)."""
    n_kv, hd, page, n_pages = 8, 128, 256, 10400
    sh = tpx.make_shape(1024, n_q=16, n_kv=n_kv, hd=hd)
    k, v = (torch.empty((1, n_pages, n_kv, page, hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    room = SMALL // (2 * n_kv * hd * 4 * page) + 4
    pages = tpx.make_pages(page, n_pages, 4 + room)
    small = tpx.make_pages(page, 5, 4 + room)
    at = [n_pages - 1, n_pages - 3, 17, n_pages - 2, 9000]
    ks, vs = (torch.empty((1, 5, n_kv, page, hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    for j, p in enumerate(at):
        for x, y, s in ((k, ks, 1), (v, vs, 2)):
            y[0, j] = x[0, p] = inputs.normal_bf16((n_kv, page, hd), 1.0, 50 + j, 90 + s, dev)
    q = inputs.normal_bf16((2, 16 * hd), 1.0, 51, 95, dev)
    o, o2 = (torch.zeros((2, 16 * hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = tpx.new_prefix_attn_workspace(sh, 2, dev)
    lens, cu, prefix = i32([1000, 900], dev), i32([0, 2], dev), i32([600], dev)
    for pg, kk, vv, table, out in ((pages, k, v, [at[:4], at[:2] + at[3:]], o), (small, ks, vs, [[0, 1, 2, 3], [0, 1, 3, 4]], o2)):
        tpx.tp_prefix_attn_decode(sh, pg, q, kk, vv, i32(np.pad(table, ((0, 0), (0, room))), dev), lens, cu, prefix, out, ws)
    sync()
    assert torch.isfinite(o.float()).all() and torch.equal(o.view(torch.int16), o2.view(torch.int16))


@pytest.mark.parametrize("kv", BOTH)
def test_samples_to_one_prompt(dev, kv):
    """As a server runs it: a prompt is appended once, n samples share its whole pages (the page that it ends in is
    written for each), and step by step: tables, QKV, append, attention, o_proj, logits, sampled tokens, their log
    probabilities, the next embeddings; captured once and replayed, nothing read by the host in between.  The steps' attention
    agrees with paged attention by itself, and the samples differ."""
    d, n_q, n_kv, hd, t, page, V, n, steps = 512, 8, 4, 64, 2, 16, 1024, 6, 12
    P = SMALL // (n * n_kv * hd * 2 * page) + 20                       # pages that a row of the table can name
    sh = tpx.make_shape(d, n_q=n_q, n_kv=n_kv, hd=hd, t=t, vocab=V)
    rnd = lambda *s, std=1.0, seed=0: inputs.normal_bf16(s, std, seed, 60, dev)
    wq, dq = tpx.tp_partition_weights(sh, tpx.TP_W_QKV, rnd(d, (n_q + 2 * n_kv) * hd, std=0.05, seed=1))
    wo, do = tpx.tp_partition_weights(sh, tpx.TP_W_O, rnd(n_q * hd, d, std=0.1, seed=2))
    wv, dv = tpx.tp_partition_weights(sh, tpx.TP_W_VOCAB, rnd(d, V, std=0.08, seed=3))
    we, de = tpx.tp_partition_weights(sh, tpx.TP_W_EMBED, rnd(V, d, seed=4))
    rope = tpx.make_rope(hd)
    prompt = np.random.default_rng(3).integers(0, V, 203)
    whole, rest = divmod(len(prompt), page)
    pages = tpx.make_pages(page, 200, P, kv)
    z = lambda *s, d_=torch.int32: torch.zeros(s, dtype=d_, device=dev)
    kp, vp = (z(t, 200, n_kv // t, page, hd, d_=torch.bfloat16 if kv == tpx.TP_BF16 else torch.float8_e4m3fn) for _ in range(2))
    order = np.random.default_rng(4).permutation(200)
    table = np.full((n, P), -1)
    table[:, :whole] = order[:whole]
    table[:, whole] = order[whole: whole + n]                          # each sample's own copy of the last page
    table_d, free = i32(table, dev), i32(order[whole + n:], dev)
    # the prompt: its whole pages once, its last positions once per sample
    x, qkv, q = (z(len(prompt), w, d_=torch.bfloat16) for w in (d, (n_q + 2 * n_kv) * hd, n_q * hd))
    tpx.tp_embed_lookup(de, we, i32(prompt, dev), x)
    tpx.tp_colpar_forward(dq, wq, x, qkv)
    pos = np.arange(len(prompt))
    for r in [0] + list(range(1, n)):
        rows = slice(0, None) if r == 0 else slice(whole * page, None)
        slots = table[r, pos[rows] // page] * page + pos[rows] % page
        tpx.tp_rope_append(sh, rope, pages, qkv[rows].contiguous(), i32(pos[rows], dev), i32(slots, dev), q[rows].clone(), kp, vp)
    s = dict(lens=[i32([len(prompt)] * n, dev), z(n)], counts=[z(3), z(3)], cu=z(n + 1), pos=z(n), slots=z(n),
             x=z(n, d, d_=torch.bfloat16), qkv=z(n, (n_q + 2 * n_kv) * hd, d_=torch.bfloat16), q=z(n, n_q * hd, d_=torch.bfloat16),
             o=z(n, n_q * hd, d_=torch.bfloat16), y=z(n, d, d_=torch.bfloat16), logits=z(n, V, d_=torch.float32),
             ids=i32([prompt[-1]] * n, dev), lp=z(n, d_=torch.float32), lp2=z(n, d_=torch.float32),
             lse=z(n, n_q, d_=torch.float32), out=z(steps, n), step=z(1), u=z(steps, n, d_=torch.float32))
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    s["u"].copy_(torch.rand((steps, n), generator=g, device=dev))
    u = z(n, d_=torch.float32)
    add, cu_g, prefix = i32([1] * n, dev), i32([0, n], dev), i32([len(prompt)], dev)
    T, top_p = torch.full((n,), 0.9, device=dev), torch.full((n,), 0.95, device=dev)
    ws = tpx.new_workspace(sh, n, dev)
    aws = tpx.new_prefix_attn_workspace(sh, n, dev)

    def attention(o, lse, lens):
        tpx.tp_prefix_attn_decode(sh, pages, s["q"], kp, vp, table_d, lens, cu_g, prefix, o, aws, lse=lse)

    def step(i):
        a, b = i % 2, 1 - i % 2
        tpx.tp_paged_tables(pages, s["lens"][a], add, free, table_d, s["lens"][b], s["cu"], s["pos"], s["slots"], s["counts"][b],
                            head=s["counts"][a])
        tpx.tp_embed_lookup(de, we, s["ids"], s["x"])
        tpx.tp_colpar_forward(dq, wq, s["x"], s["qkv"])
        tpx.tp_rope_append(sh, rope, pages, s["qkv"], s["pos"], s["slots"], s["q"], kp, vp)
        attention(s["o"], s["lse"], s["lens"][b])
        tpx.tp_rowpar_forward(do, wo, s["o"], s["x"], s["y"], ws)
        tpx.tp_lm_head_forward(dv, wv, s["y"], s["logits"])
        u.copy_(s["u"].index_select(0, s["step"].long())[0])
        tpx.tp_sample_tokens(s["logits"], u, s["ids"], temperature=T, top_p=top_p, logprob=s["lp"])
        tpx.tp_token_logprobs(s["logits"], s["ids"], s["lp2"], None, None)
        s["out"].index_copy_(0, s["step"].long(), s["ids"][None])
        s["step"].add_(1)

    for i in range(4):
        step(i)
        o2, lse2 = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
        tpx.tp_paged_attn_decode(sh, pages, s["q"], kp, vp, table_d, s["lens"][1 - i % 2], o2, aws, lse=lse2)
        sync()
        a, b = s["o"].float(), o2.float()
        assert float((a - b).norm() / b.norm()) <= 4 * HALF and float((s["lse"] - lse2).abs().max()) <= 1e-4
        # the sampled token's probability among the kept ones is at least that among all
        assert (s["lp"] >= s["lp2"] / 0.9 - 1e-4 * s["lp2"].abs() - 1.0).all() and (s["lp"] <= 0).all()
        may = [PO.sample(s["logits"][m].cpu().numpy(), float(s["u"][i, m]), float(T[m]), p=float(top_p[m]), slack=2.0 ** -26)[0]
               for m in range(n)]
        assert all(int(s["ids"][m]) in may[m] for m in range(n))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(0)
        step(1)
    for _ in range(4):
        with torch.cuda.stream(side):
            graph.replay()
    sync(), torch.cuda.synchronize()
    assert s["lens"][0].tolist() == [len(prompt) + 12] * n and int(s["step"]) == steps
    got = s["out"].cpu().numpy()
    assert ((got >= 0) & (got < V)).all() and len({tuple(got[:, m]) for m in range(n)}) == n
