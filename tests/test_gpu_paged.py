"""The paged key-value cache through the C ABI, against the float64 oracle: block tables and slots, rotary
positions and the append, decode attention over the pages, and a decode step of all of them."""
import math

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import inputs, tpx
from oracle import paged_oracle as PO
from oracle import tp_oracle as O
from tests.test_gpu_parity import bits, check_close

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8   # a bf16 rounding, relative
NAMES = {"none": tpx.TP_ROPE_NONE, "linear": tpx.TP_ROPE_LINEAR, "wavelength": tpx.TP_ROPE_WAVELENGTH,
         "yarn": tpx.TP_ROPE_YARN}


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_transformer_gb300 import build
    build.build_library()
    tpx.lib()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def sync():
    assert tpx.tp_sync(timeout_ms=20000) == tpx.TP_OK


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------------------------------ tables
def run_tables(dev, lens, add, page, max_pages, n_free, head=0, rows=None, n_pages=None, stride=None, seed=0, bad=()):
    """A pool in random order; `bad`: entries of the free list that name no page."""
    rng = np.random.default_rng(seed)
    lens, add = np.array(lens, np.int64), np.array(add, np.int64)
    held = -(-np.clip(lens, 0, max_pages * page) // page)
    n_pages = n_pages or int(held.sum()) + n_free + 3
    order = rng.permutation(n_pages)
    M, stride = len(lens), stride or max_pages
    table = np.full((M, stride), -1, np.int64)
    at = 0
    for m in range(M):
        table[m, : held[m]] = order[at: at + held[m]]
        at += held[m]
    free = order[at: at + n_free].copy()
    for j, v in bad:
        free[j] = v
    rows = int(np.clip(add, 0, None).sum()) if rows is None else rows
    want = PO.tables(lens.tolist(), add.tolist(), free.tolist(), head, table, page, max_pages, n_pages, rows)
    pages = tpx.make_pages(page, n_pages, max_pages, table_stride=stride)
    table_d = i32(table, dev)
    out = [torch.full((n + 4,), 77, dtype=torch.int32, device=dev) for n in (M, M + 1, rows, rows, 3)]
    lo, cu, pos, slots, counts = (b[:n] for b, n in zip(out, (M, M + 1, rows, rows, 3)))
    tpx.tp_paged_tables(pages, i32(lens, dev), i32(add, dev), i32(free, dev), table_d, lo, cu, pos, slots, counts,
                        head=None if head == 0 else i32([head], dev))
    sync()
    for got, ref, what in zip((table_d, lo, cu, pos, slots, counts), want, ("table", "lens", "cu", "pos", "slots", "counts")):
        assert np.array_equal(got.cpu().numpy(), ref), what
    assert all((b[-4:] == 77).all() for b in out)          # nothing behind the outputs
    return want


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_tables_ragged(dev, page):
    rng = np.random.default_rng(page)
    lens = [0, 1, page - 1, page, page + 1, 3 * page, 0] + rng.integers(0, 900, 60).tolist()
    add = [0, page, 1, 1, 0, page + 1, 2 * page] + rng.integers(0, 300, 60).tolist()
    run_tables(dev, lens, add, page, 100, 900, head=5, stride=103, rows=sum(add) + 129)


@pytest.mark.parametrize("M", [1, 2, 511, 512, 513, 2500])
def test_tables_one_token_each(dev, M):
    rng = np.random.default_rng(M)
    run_tables(dev, rng.integers(0, 200, M), np.ones(M, int), 16, 14, M)


def test_tables_long_prompts_and_many_rows(dev):
    run_tables(dev, [0, 40000, 7], [100003, 0, 30011], 64, 2000, 2200)
    run_tables(dev, [0] * 1500, [0, 1, 200] * 500, 32, 8, 3600)


def test_tables_refusals_on_the_device(dev):
    big = 2 ** 31 - 1
    # the pool runs out in the middle: later requests that need no page are still served
    w = run_tables(dev, [15, 0, 0, 3, 0, 15], [1, 40, 40, 5, 1, 1], 16, 8, 4, rows=100)
    assert w[5].tolist() == [3, 88, 2]
    run_tables(dev, [5, 5], [20, 20], 16, 8, 0)                          # nothing free
    run_tables(dev, [5, -3, 5, 5, 5], [20, 20, -7, 5, 9], 16, 8, 6)      # negative lengths
    run_tables(dev, [0, 100, 128, 0], [129, 29, 0, 128], 16, 8, 30)      # longer than a row of the table
    run_tables(dev, [0, 0, 0, 0], [10, 30, 25, 4], 16, 8, 30, rows=50)   # rows that do not fit
    run_tables(dev, [5, 6], [20, 20], 16, 8, 3, head=9)                  # head outside the list
    run_tables(dev, [5, 6], [20, 20], 16, 8, 3, head=-1)
    run_tables(dev, [4, big, 4], [3, 5, 60], 16, 8, 9, rows=300)
    run_tables(dev, [3, 3], [40, 40], 16, 8, 9, bad=[(1, -5), (3, 10 ** 6)])   # the list names no page


@pytest.mark.parametrize("head", [-1, -(2 ** 31), 4, 2 ** 31 - 1])
def test_tables_growth_within_a_page_with_no_page_left(dev, head):
    """With *head outside the free list no page is left, but a request that grows within a page it holds needs none:
    it is served and its rows have slots, whatever refused requests are before it."""
    w = run_tables(dev, [5], [1], 16, 8, 3, head=head)
    assert w[1].tolist() == [6] and w[4][0] >= 0 and w[5].tolist() == [head, 1, 0]
    w = run_tables(dev, [5, 16, 30, 0, 47, 0, 1], [3, 1, 2, 40, 1, 0, 15], 16, 8, 3, head=head, rows=70)
    assert w[5].tolist() == [head, 62, 2] and (w[4] >= 0).sum() == 21


def test_tables_sums_past_32_bits(dev):
    big = 2 ** 31 - 1
    lens, add = [0, 0, 0, 4], [big, big, big, 3]
    pages = tpx.make_pages(16, 50, 8)
    table = torch.full((4, 8), -1, dtype=torch.int32, device=dev)
    lo, cu, counts = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (4, 5, 3))
    pos, slots = (torch.zeros(64, dtype=torch.int32, device=dev) for _ in range(2))
    tpx.tp_paged_tables(pages, i32(lens, dev), i32(add, dev), i32(range(9), dev), table, lo, cu, pos, slots, counts)
    sync()
    assert lo.tolist() == lens and cu.tolist() == [0, big, big, big, big] and counts.tolist() == [0, big, 4]
    assert (slots == -1).all() and (table == -1).all() and pos.tolist() == list(range(64))


def test_tables_step_after_step_without_the_host(dev):
    """counts is the next call's head and lens_out its lens: the same as one call with all the tokens."""
    M, page, P = 40, 16, 20
    rng = np.random.default_rng(5)
    lens, free = np.zeros(M, int), rng.permutation(400)
    pages = tpx.make_pages(page, 400, P)
    table = torch.full((M, P), -1, dtype=torch.int32, device=dev)
    a = [i32(lens, dev), torch.zeros(3, dtype=torch.int32, device=dev)]
    b = [torch.zeros_like(a[0]), torch.zeros_like(a[1])]
    cu, pos, slots = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (M + 1, M, M))
    seen = []
    add, free_d = i32(np.ones(M, int), dev), i32(free, dev)
    for step in range(70):
        tpx.tp_paged_tables(pages, a[0], add, free_d, table, b[0], cu, pos, slots, b[1], head=a[1])
        a, b = b, a
        seen.append(slots.clone())
    sync()
    assert (a[0] == 70).all() and a[1].tolist() == [M * 5, M, 0]
    got = torch.stack(seen).cpu().numpy()
    t = table.cpu().numpy()
    assert np.array_equal(np.sort(t[:, :5].ravel()), np.sort(free[: M * 5])) and (t[:, 5:] == -1).all()
    for p in range(70):
        assert np.array_equal(got[p], t[:, p // page] * page + p % page)


def test_tables_a_step_without_requests_writes_nothing(dev):
    """The chain goes on from the counts written last, and every page goes out once."""
    page, P = 16, 4
    pages = tpx.make_pages(page, 40, P)
    free = i32(np.random.default_rng(6).permutation(40), dev)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    head, given = z(3), []
    for M, rows in ((2, 6), (0, 6), (3, 6), (0, 0), (1, 6)):
        counts, table = torch.full((3,), -9, dtype=torch.int32, device=dev), z(M, P) - 1
        lo, cu, pos, slots = z(M) - 9, z(M + 1) - 9, z(rows) - 9, z(rows) - 9
        tpx.tp_paged_tables(pages, z(M), i32(np.full(M, 1), dev), free, table, lo, cu, pos, slots, counts, head=head)
        sync()
        if M == 0:
            assert all((x == -9).all() for x in (counts, cu, pos, slots))
            continue
        given += table[:, 0].tolist()
        head = counts
    assert given == free[:6].tolist() and head.tolist() == [6, 1, 0]


# -------------------------------------------------------------------------------------------- rope
def make_qkv(dev, M, n_q, n_kv, hd, seed):
    return inputs.normal_bf16((M, (n_q + 2 * n_kv) * hd), 1.0, seed, 90, dev)


def rope_case(M, hd, rot, layout, scaling, seed, far=1 << 20):
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, far, M)
    pos[:: 7] = rng.integers(0, 50, len(pos[::7]))
    rope = tpx.make_rope(rot, 500000.0, tpx.TP_ROPE_HALF if layout == "half" else tpx.TP_ROPE_INTERLEAVED, NAMES[scaling],
                         factor=8.0, original_len=8192)
    f, ms = PO.rope_freqs(rot, 500000.0, scaling, 8.0, 8192)
    return pos, rope, f, ms


def turned_bound(x, rot, layout, ms):
    """|error| of a turned value in fp32.  cos and sin: the reduced angle is at most pi/4 and off by 2^-24 of it
    (its conversion to fp32), sincospi adds 2 ulp and the factor's product half of one: 2^-22 ms covers them;
    the two products and their sum add 2^-23 of the terms: (|a| + |b|) 2^-21 ms in all."""
    y = np.abs(np.array(x, np.float64))
    z = y.copy()
    r = rot // 2
    if layout == "half":
        z[..., :r] = z[..., r:rot] = y[..., :r] + y[..., r:rot]
    else:
        z[..., 0:rot:2] = z[..., 1:rot:2] = y[..., 0:rot:2] + y[..., 1:rot:2]
    z[..., rot:] = 0
    return z * ms * 2.0 ** -21


def assert_within(got, ref, bound, what):
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), f"{what}: {over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,rot,n_q,n_kv,t", [(128, 128, 8, 4, 2), (64, 32, 8, 8, 8), (256, 64, 4, 2, 1), (48, 48, 6, 2, 2),
                                               (16, 16, 3, 1, 1), (80, 32, 8, 4, 4)])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_rope_forward(dev, layout, hd, rot, n_q, n_kv, t, scaling):
    M = 37
    pos, rope, f, ms = rope_case(M, hd, rot, layout, scaling, hd + rot)
    sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=t)
    qkv = make_qkv(dev, M, n_q, n_kv, hd, 1)
    out = torch.full_like(qkv, float("nan"))
    tpx.tp_rope_forward(sh, rope, qkv, i32(pos, dev), out)
    sync()
    x = PO.split_qkv(O.as_f64(bits(qkv)), t, n_q, n_kv, hd)
    y = PO.split_qkv(O.as_f64(bits(out)), t, n_q, n_kv, hd)
    for a, b, name in zip(x[:2], y[:2], "qk"):
        ref = PO.rope(a, pos, f, ms, layout)
        e = turned_bound(a, rot, layout, ms)
        assert_within(b, ref, e + HALF * (np.abs(ref) + e) * (e > 0), name)  # unturned dims are copied
    assert np.array_equal(x[2], y[2])
    same = qkv.clone()
    tpx.tp_rope_forward(sh, rope, same, i32(pos, dev), same)            # in place: the same bits
    sync()
    assert torch.equal(same.view(torch.int16), out.view(torch.int16))


def test_rope_far_and_negative_positions(dev):
    """Every int32 position: the angle is reduced exactly, so the error does not grow with the position.  (The
    reference reduces pos * f / 2 pi in rational arithmetic on the described 64-bit steps.)"""
    from fractions import Fraction
    pos = [0, 1, -1, 12345678, -(2 ** 31), 2 ** 31 - 1, 2 ** 30 + 1]
    M, hd = len(pos), 128
    sh = tpx.make_shape(1024, n_q=2, n_kv=1, hd=hd)
    rope = tpx.make_rope(hd, 10000.0)
    qkv = make_qkv(dev, M, 2, 1, hd, 2)
    out = torch.empty_like(qkv)
    tpx.tp_rope_forward(sh, rope, qkv, i32(pos, dev), out)
    sync()
    x, y = (O.as_f64(bits(z)).reshape(M, 4, hd) for z in (qkv, out))
    for m, p in enumerate(pos):
        turn = np.array([float(Fraction(p * rope.step[i], 1 << 64) % 1) for i in range(hd // 2)])
        ref = PO.rope(x[m:m + 1, :3], [1], 2 * math.pi * turn, 1.0, "half")
        e = turned_bound(x[m:m + 1, :3], hd, "half", 1.0)
        assert_within(y[m:m + 1, :3], ref, e + HALF * (np.abs(ref) + e), f"position {p}")


def pool(dev, t, n_pages, n_kv, page, hd, kv, seed, stream):
    v = inputs.normal_bf16((t, n_pages, n_kv // t, page, hd), 1.0 if kv == tpx.TP_BF16 else 70.0, seed, stream, dev)
    return v if kv == tpx.TP_BF16 else v.float().to(torch.float8_e4m3fn)


def values(x):
    return x.float().cpu().numpy().astype(np.float64)


def scales(dev, n_kv, kv, seed):
    if kv == tpx.TP_BF16:
        return None, None
    g = np.random.default_rng(seed)
    return tuple(torch.tensor(g.uniform(0.5, 1.5, n_kv) / 70, dtype=torch.float32, device=dev) for _ in range(2))


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("layout,scaling", [("half", "wavelength"), ("interleaved", "linear")])
@pytest.mark.parametrize("hd,rot,n_q,n_kv,t,page,M", [(128, 64, 8, 4, 2, 16, 1), (64, 64, 12, 4, 4, 256, 53),
                                                     (256, 256, 4, 4, 1, 64, 300), (48, 16, 4, 2, 2, 32, 33)])
def test_rope_append(dev, kv, layout, scaling, hd, rot, n_q, n_kv, t, page, M):
    rng = np.random.default_rng(M)
    pos, rope, f, ms = rope_case(M, hd, rot, layout, scaling, M)
    sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=t)
    n_pages = -(-M // page) + 2
    pages = tpx.make_pages(page, n_pages, 4, kv)
    slots = rng.permutation(n_pages * page)[:M]
    out = [j for j in (3, 7) if j < M]
    slots[out] = [-1, n_pages * page][: len(out)]                     # rows that are not appended
    qkv = make_qkv(dev, M, n_q, n_kv, hd, 3)
    kp, vp = pool(dev, t, n_pages, n_kv, page, hd, kv, 3, 91), pool(dev, t, n_pages, n_kv, page, hd, kv, 3, 92)
    before = [values(kp), values(vp)]
    ks, vs = scales(dev, n_kv, kv, 3)
    q = torch.full((M, n_q * hd), float("nan"), dtype=torch.bfloat16, device=dev)
    tpx.tp_rope_append(sh, rope, pages, qkv, i32(pos, dev), i32(slots, dev), q, kp, vp, ks, vs)
    sync()
    x = PO.split_qkv(O.as_f64(bits(qkv)), t, n_q, n_kv, hd)
    ref = PO.rope(x[0], pos, f, ms, layout)
    e = turned_bound(x[0], rot, layout, ms)
    assert_within(O.as_f64(bits(q)).reshape(M, n_q, hd), ref, e + HALF * (np.abs(ref) + e) * (e > 0), "q")
    refs = [(PO.rope(x[1], pos, f, ms, layout), turned_bound(x[1], rot, layout, ms), ks), (x[2], 0 * x[2], vs)]
    kept = [m for m in range(M) if 0 <= slots[m] < n_pages * page]
    for got, old, (ref, e, sc) in zip((values(kp), values(vp)), before, refs):
        touched = np.zeros(got.shape[:4], bool)
        for m in kept:
            p, off = divmod(int(slots[m]), page)
            row = got[:, p, :, off].reshape(n_kv, hd)                 # shard-major: heads in order
            touched[:, p, :, off] = True
            if sc is None:
                assert_within(row, ref[m], e[m] + HALF * (np.abs(ref[m]) + e[m]) * (e[m] > 0), "appended")
            else:  # half a step of the code, 2^-10 among the subnormal ones, and the divide's rounding
                s = sc.cpu().numpy().astype(np.float64)[:, None]
                want, slack = np.clip(ref[m] / s, -448, 448), e[m] / s + np.abs(ref[m] / s) * 2.0 ** -23
                assert_within(row, want, slack + np.maximum(2.0 ** -4 * (np.abs(want) + slack), 2.0 ** -10), "code")
        assert np.array_equal(got[~touched], old[~touched])           # the rest of the pool


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("M,hd,rot,n_q,n_kv,t,layout", [(1303, 128, 128, 64, 8, 8, "half"), (701, 64, 32, 12, 4, 2, "half"),
                                                        (612, 256, 256, 3, 1, 1, "interleaved"),
                                                        (905, 16, 16, 300, 4, 4, "interleaved")])
def test_rope_many_rows_equal_few(dev, kv, M, hd, rot, n_q, n_kv, t, layout):
    """A call of many rows (two to a CTA, odd numbers of rows and heads too) gives the bits of calls of few."""
    pos, rope, _, _ = rope_case(M, hd, rot, layout, "yarn", M)
    sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=t)
    n_pages = M // 32 + 2
    pages = tpx.make_pages(32, n_pages, 4, kv)
    slots = np.random.default_rng(M).permutation(n_pages * 32)[:M]
    slots[[5, M - 1]] = -1
    qkv, pos, slots = make_qkv(dev, M, n_q, n_kv, hd, 13), i32(pos, dev), i32(slots, dev)
    ks, vs = scales(dev, n_kv, kv, 3)
    outs = []
    for step in (M, 3):
        kp, vp = (pool(dev, t, n_pages, n_kv, 32, hd, kv, 3, s) for s in (91, 92))
        q = torch.zeros((M, n_q * hd), dtype=torch.bfloat16, device=dev)
        turned = torch.zeros_like(qkv)
        for m in range(0, M, step):
            rows = slice(m, min(M, m + step))
            tpx.tp_rope_append(sh, rope, pages, qkv[rows], pos[rows].clone(), slots[rows].clone(), q[rows], kp, vp, ks, vs)
            tpx.tp_rope_forward(sh, rope, qkv[rows], pos[rows].clone(), turned[rows])
        sync()
        outs.append([x.view(torch.uint8) for x in (q, kp, vp, turned)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_append_codes_exactly_without_turning(dev):
    """rope None: bf16 pages hold the bits, e4m3 pages the nearest codes; overflow saturates, NaN stays."""
    M, n_q, n_kv, hd, page = 5, 4, 2, 64, 16
    sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=2)
    qkv = make_qkv(dev, M, n_q, n_kv, hd, 4) * 200
    qkv[1, 3 * hd - 5] = float("nan")
    qkv[2, 3 * hd - 7] = float("inf")
    qkv[3, 3 * hd: 4 * hd] = -1e30
    slots = i32([3, 40, 17, 16, 0], dev)
    for kv in (tpx.TP_BF16, tpx.TP_FP8_E4M3):
        kp = torch.zeros((2, 3, 1, page, hd), dtype=torch.bfloat16 if kv == tpx.TP_BF16 else torch.float8_e4m3fn, device=dev)
        vp = torch.zeros_like(kp)
        q = torch.empty((M, n_q * hd), dtype=torch.bfloat16, device=dev)
        tpx.tp_rope_append(sh, None, tpx.make_pages(page, 3, 3, kv), qkv, None, slots, q, kp, vp)
        sync()
        x = qkv.view(M, 2, 4, hd)
        assert torch.equal(q.view(M, 2, 2, hd).view(torch.int16), x[:, :, :2].contiguous().view(torch.int16))
        for m, s in enumerate(slots.tolist()):
            for got, want in ((kp, x[m, :, 2]), (vp, x[m, :, 3])):
                row = got[:, s // page, 0, s % page].float()
                want = want.float()
                if kv != tpx.TP_BF16:
                    want = want.clamp(-448, 448).to(torch.float8_e4m3fn).float()
                assert torch.equal(row.nan_to_num(nan=-9.0), want.nan_to_num(nan=-9.0))


# --------------------------------------------------------------------------------------- attention
class Case:
    """A paged cache with random tables; run() checks one call against the oracle."""

    def __init__(self, dev, t, n_q, n_kv, hd, page, lens, kv=tpx.TP_BF16, seed=0, poison=True, extra=2, std=1.0,
                 stride_pad=0):
        self.t, self.n_q, self.n_kv, self.hd, self.page, self.lens, self.kv = t, n_q, n_kv, hd, page, list(lens), kv
        self.dev, M = dev, len(lens)
        self.sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=t)
        held = [max(0, -(-n // page)) for n in lens]
        self.max_pages = max(held + [1]) + 1
        self.n_pages = sum(held) + extra
        rng = np.random.default_rng(seed)
        order = rng.permutation(self.n_pages)
        self.table = np.full((M, self.max_pages + stride_pad), 2 ** 31 - 1, np.int64)
        at = 0
        self.k = pool(dev, t, self.n_pages, n_kv, page, hd, kv, seed, 93)
        self.v = pool(dev, t, self.n_pages, n_kv, page, hd, kv, seed, 94)
        for m in range(M):
            self.table[m, : held[m]] = order[at: at + held[m]]
            at += held[m]
        if poison:  # every cache row that no request attends to holds NaN
            used = torch.zeros((self.n_pages, page), dtype=torch.bool)
            for m, n in enumerate(lens):
                for j in range(held[m]):
                    used[self.table[m, j], : max(0, min(page, n - j * page))] = True
            for x in (self.k, self.v):
                raw = x.view(torch.int16 if kv == tpx.TP_BF16 else torch.uint8)
                hole = ~used.to(dev)[None, :, None, :, None]
                raw.masked_fill_(hole, 0x7FC0 if kv == tpx.TP_BF16 else 0x7F)
        self.ks, self.vs = scales(dev, n_kv, kv, seed)
        self.q = inputs.normal_bf16((M, n_q * hd), std, seed, 95, dev)
        self.ws = tpx.new_paged_attn_workspace(self.sh, dev)

    def call(self, o, lse, window=0, scale=0.0, stream=None, lens=None):
        pages = tpx.make_pages(self.page, self.n_pages, self.max_pages, self.kv, self.table.shape[1])
        tpx.tp_paged_attn_decode(self.sh, pages, self.q, self.k, self.v, self.table_d, self.lens_d, o, self.ws, lse=lse,
                                 window=window, scale=scale, k_scale=self.ks, v_scale=self.vs, stream=stream)

    def launch(self, window=0, scale=0.0, with_lse=True):
        M = len(self.lens)
        self.table_d, self.lens_d = i32(self.table, self.dev), i32(self.lens, self.dev)
        buf = torch.full((M * self.n_q * self.hd + 64,), 7.0, dtype=torch.bfloat16, device=self.dev)
        o = buf[: M * self.n_q * self.hd].view(M, -1)
        lse = torch.full((M, self.n_q), 7.0, dtype=torch.float32, device=self.dev) if with_lse else None
        self.call(o, lse, window, scale)
        sync()
        assert (buf[M * self.n_q * self.hd:] == 7.0).all()
        return o, lse

    def check(self, window=0, scale=0.0):
        o, lse = self.launch(window, scale)
        k, v = values(self.k), values(self.v)
        q = O.as_f64(bits(self.q)).reshape(len(self.lens), self.n_q, self.hd)
        got, got_l = O.as_f64(bits(o)).reshape(q.shape), lse.cpu().numpy().astype(np.float64)
        sc = [np.ones(self.n_kv) if s is None else s.cpu().numpy().astype(np.float64) for s in (self.ks, self.vs)]
        factor = scale or 1 / math.sqrt(self.hd)
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
            # A score is a sum of hd exact products in fp32 (at most hd steps of 2^-23 of sum |q||k|), times a few
            # factors rounded to fp32: (hd + 8) 2^-23 B.  e^x: 2^-21 (the argument's rounding and ex2).  P enters
            # the product in two bf16 (2^-16) or in three e4m3 (2^-12, or an absolute 2^-25 each, against a sum of
            # at least 1/2: the 2^-11 and 2^-25 n below cover both); the sums over n positions, 16 at a time:
            # n / 16 + 300 steps of 2^-24.  All of it twice, in the numerator and in the sum.
            ps = (self.hd + 8) * 2.0 ** -23 * B + 2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24
            pp = 2.0 ** -16 if self.kv == tpx.TP_BF16 else 2.0 ** -11
            vmax = np.abs(v[:, at[count], :, off[count]]).max() * sc[1].max() if count.any() else 0.0
            e = A * (2 * ps[:, None] + pp) + (0 if self.kv == tpx.TP_BF16 else n * 2.0 ** -25 * vmax)
            assert_within(got[m], ro, e + HALF * (np.abs(ro) + e), f"o of request {m}, length {n}")
            fine = np.isfinite(rl)
            assert np.array_equal(np.isneginf(rl), np.isneginf(got_l[m]))
            if fine.any():
                assert_within(got_l[m][fine], rl[fine], ps[fine] + 2.0 ** -21 * (1 + np.abs(rl[fine])), "lse")
            if not fine.any():
                assert not got[m].any()
        assert not self.ws[:4 * 1024].any()                            # the counters are left at zero
        return o, lse


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("t,n_q,n_kv,hd", [(1, 8, 4, 64), (2, 16, 4, 128), (4, 16, 4, 256), (2, 32, 2, 128), (1, 3, 3, 64),
                                           (1, 6, 2, 128)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_paged_attention_lengths(dev, kv, t, n_q, n_kv, hd, page):
    Case(dev, t, n_q, n_kv, hd, page, EDGES, kv, seed=page + hd).check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("hd,page,window", [(64, 16, 1), (128, 16, 100), (128, 256, 128), (256, 32, 129), (128, 64, 1000),
                                            (64, 128, 33)])
def test_paged_attention_window(dev, kv, hd, page, window):
    """Before the window the table may name no page and the rows may hold anything."""
    c = Case(dev, 1, 8, 4, hd, page, EDGES, kv, seed=window)
    for m, n in enumerate(c.lens):
        gone = max(0, n - window)
        c.table[m, : gone // page] = -1
        if gone % page:  # the page the window begins in: NaN up to there
            p = int(c.table[m, gone // page])
            for x in (c.k, c.v):
                raw = x.view(torch.int16 if kv == tpx.TP_BF16 else torch.uint8)
                raw[:, p, :, : gone % page] = 0x7FC0 if kv == tpx.TP_BF16 else 0x7F
    # the oracle leaves out the rows before the window by itself; NaN there must not reach it either
    k, v = c.k, c.v
    o, lse = c.launch(window)
    for m, n in enumerate(c.lens):
        assert torch.isfinite(o[m]).all() and (n == 0 or torch.isfinite(lse[m]).all())
    for x in (k, v):
        x.view(torch.int16 if kv == tpx.TP_BF16 else torch.uint8)[x.float().isnan()] = 0
    c.check(window)


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
def test_paged_attention_one_long_request(dev, kv):
    """All SMs share one request: pieces joined in order, the same bits again, lse optional."""
    c = Case(dev, 2, 16, 2, 128, 64, [40001], kv, seed=5, std=2.0)
    o, lse = c.check()
    o2, lse2 = c.launch()
    o3, _ = c.launch(with_lse=False)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    assert torch.equal(o.view(torch.int16), o3.view(torch.int16))


@pytest.mark.parametrize("M", [1, 33, 289, 700])
def test_paged_attention_many_requests(dev, M):
    rng = np.random.default_rng(M)
    lens = np.where(rng.random(M) < 0.2, 0, rng.integers(1, 90, M))
    lens[rng.integers(M)] = 1500
    Case(dev, 1, 4, 2, 64, 16, lens, seed=M).check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("t,n_q,n_kv,hd,page,M", [(1, 32, 2, 128, 16, 200), (2, 8, 4, 256, 32, 90), (1, 16, 1, 256, 64, 61),
                                                  (2, 16, 2, 128, 128, 333), (1, 16, 1, 64, 16, 170)])
def test_paged_attention_many_requests_by_heads(dev, kv, t, n_q, n_kv, hd, page, M):
    """Batches whose CTAs take several items each, over both types, 4 and 8 heads a thread and every width."""
    rng = np.random.default_rng(M)
    lens = np.where(rng.random(M) < 0.1, 0, rng.integers(1, 400, M))
    lens[[3, M - 1]] = [1700, 1]
    Case(dev, t, n_q, n_kv, hd, page, lens, kv, seed=M).check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("t,n_q,n_kv,hd,page", [(1, 16, 1, 128, 32), (2, 32, 2, 256, 64), (1, 4, 1, 256, 128), (1, 2, 2, 64, 16),
                                                (1, 15, 1, 64, 256), (1, 5, 1, 128, 16)])
def test_paged_attention_pieces_joined_twice(dev, kv, t, n_q, n_kv, hd, page):
    """One or two long requests of few kv heads: more pieces than are joined at once, for every number of heads a
    thread and every width, and the same bits again."""
    c = Case(dev, t, n_q, n_kv, hd, page, [9001, 0, 6007], kv, seed=n_q, std=2.0)
    o, lse = c.check()
    o2, lse2 = c.launch()
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


def test_paged_attention_lengths_out_of_range(dev):
    """Lengths below zero or past the table's row: zero rows, and nothing is read for them."""
    c = Case(dev, 1, 8, 2, 128, 16, [40, 100, 7], seed=6)
    c.lens = [-5, 2 ** 31 - 1, 7]
    c.check()
    c.lens = [c.max_pages * 16 + 1, 100, -(2 ** 31)]
    c.check()
    c.lens = [0, 0, 0]
    c.check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("page", [16, 128])
def test_paged_attention_pages_that_are_none(dev, kv, page):
    """Ids outside the pool: their positions are left out; a request with no other page is a zero row."""
    c = Case(dev, 2, 8, 2, 128, page, [700, 300, 16, 513], kv, seed=7, stride_pad=3)
    c.table[0, [0, 2]] = [-1, c.n_pages]
    c.table[1, :] = 2 ** 31 - 1
    c.table[2, 0] = -(2 ** 31)
    c.table[3, 512 // page] = -7
    c.check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
def test_paged_attention_scale_and_peaky_scores(dev, kv):
    c = Case(dev, 1, 8, 4, 128, 32, [500, 64, 1200], kv, seed=8, std=30.0)   # one position takes nearly all
    c.check()
    c.check(scale=0.003)
    c.check(scale=-0.2)
    c.q.mul_(1e-30)                                                          # all scores zero
    c.check()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 26, 2.0 ** 28, 2.0 ** 32, 2.0 ** 60, -(2.0 ** 28), -(2.0 ** 32)])
@pytest.mark.parametrize("n_q", [4, 32])
def test_paged_attention_scores_with_a_spacing_above_one(dev, kv, scale, n_q):
    """Scores whose neighbouring fp32 values are far apart: q is (1, 0, ..), k (1, 3 or 5, 0, ..), so the scores are
    exact, equal ones are equal in any rounding, and only the largest weigh: o is the mean of their v, lse their score
    and the logarithm of their number."""
    c = Case(dev, 1, n_q, 2, 64, 16, [40, 3000, 17, 1], kv, seed=31, poison=False)
    c.q.zero_()
    c.q.view(4, n_q, 64)[:, :, 0] = 1.0
    c.k.copy_(torch.zeros(c.k.shape, device=dev).to(c.k.dtype))
    if kv == tpx.TP_FP8_E4M3:
        c.ks.fill_(1.0)
    rng = np.random.default_rng(31)
    keys = rng.choice([1.0, 3.0, 5.0], size=(c.n_pages, 2, 16), p=[0.4, 0.3, 0.3])
    keys[c.table[0, :3]] = np.minimum(keys[c.table[0, :3]], 3.0)         # the first request's largest score is another
    c.k[0, :, :, :, 0] = torch.tensor(keys, dtype=torch.float32, device=dev).to(c.k.dtype)
    o, lse = c.launch(scale=scale)
    got, got_l, v = O.as_f64(bits(o)).reshape(4, n_q, 64), lse.cpu().numpy().astype(np.float64), values(c.v)
    vs = np.ones(2) if c.vs is None else c.vs.cpu().numpy().astype(np.float64)
    for m, n in enumerate(c.lens):
        at, off = c.table[m, np.arange(n) // 16], np.arange(n) % 16
        for h in range(n_q):
            g = h // (n_q // 2)
            s = keys[at, g, off] * scale
            rows = v[0][at, g, off][s == s.max()] * vs[g]
            ref, A = rows.mean(0), np.abs(rows).mean(0)
            # the weights of equal scores are equal; ex2 of them and the sums as in Case.check, without the scores' error
            e = A * (2 * (2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24) + 2.0 ** -11)
            if kv == tpx.TP_FP8_E4M3:
                e = e + n * 2.0 ** -25 * np.abs(rows).max()
            assert_within(got[m, h], ref, e + HALF * (np.abs(ref) + e), f"o of request {m}")
            want = s.max() + math.log(len(rows))
            assert abs(got_l[m, h] - want) <= 2.0 ** -20 * (1 + abs(want)), (m, h)


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
@pytest.mark.parametrize("n_q", [4, 32])
def test_paged_attention_scores_near_the_lowest(dev, kv, n_q):
    """Scores near fp32's lowest value are scores, not masks: -2^126 everywhere (times log2 e it is below -1e38) gives
    the mean of v and lse -2^126."""
    c = Case(dev, 1, n_q, 2, 64, 16, [40, 3000, 0, 1], kv, seed=32, poison=False)
    c.q.fill_(2.0 ** 60)
    c.k.copy_(torch.full(c.k.shape, -(2.0 ** 60) if kv == tpx.TP_BF16 else -256.0, device=dev).to(c.k.dtype))
    if kv == tpx.TP_FP8_E4M3:
        c.ks.fill_(2.0 ** 52)
    o, lse = c.launch(scale=1.0)
    got, got_l, v = O.as_f64(bits(o)).reshape(4, n_q, 64), lse.cpu().numpy().astype(np.float64), values(c.v)
    vs = np.ones(2) if c.vs is None else c.vs.cpu().numpy().astype(np.float64)
    for m, n in enumerate(c.lens):
        for h in range(n_q):
            g = h // (n_q // 2)
            if n == 0:
                assert not got[m, h].any() and np.isneginf(got_l[m, h])
                continue
            rows = v[0][c.table[m, np.arange(n) // 16], g, np.arange(n) % 16] * vs[g]
            ref, A = rows.mean(0), np.abs(rows).mean(0)
            e = A * (2 * (2.0 ** -21 + (n / 16 + 300) * 2.0 ** -24) + 2.0 ** -11)   # as for scores far apart
            if kv == tpx.TP_FP8_E4M3:
                e = e + n * 2.0 ** -25 * np.abs(rows).max()
            assert_within(got[m, h], ref, e + HALF * (np.abs(ref) + e), f"o of request {m}")
            assert abs(got_l[m, h] + 2.0 ** 126) <= 2.0 ** (126 - 20), (m, h)


def test_paged_attention_infinite_scores(dev):
    """A key of -inf in the scores weighs nothing; where all do, or one is +inf or NaN, the row says so."""
    c = Case(dev, 1, 2, 2, 64, 16, [40, 40, 40, 1], seed=9, poison=False)
    c.q.fill_(1.0)
    page = lambda m, j: int(c.table[m, j // 16])
    c.k[:, page(0, 5), :, 5] = float("-inf")
    c.k[:, page(1, 20), :, 20 % 16] = float("nan")
    c.k[:, page(2, 3), 0, 3] = float("inf")
    c.k[:, page(3, 0), :, 0] = float("-inf")
    o, lse = c.launch()
    q, k, v = (values(x) for x in (c.q, c.k, c.v))
    at = [page(0, j) for j in range(40)]
    keep = [j for j in range(40) if j != 5]
    for h in range(2):
        s = np.array([k[0, at[j], h, j % 16].sum() / 8 for j in keep])
        p = np.exp(s - s.max())
        ref = (p / p.sum()) @ np.array([v[0, at[j], h, j % 16] for j in keep])
        assert np.allclose(O.as_f64(bits(o))[0, h * 64:(h + 1) * 64], ref, rtol=2 ** -7, atol=1e-4)
    assert torch.isnan(o[1].float()).all() and torch.isnan(o[2, :64].float()).all()
    assert torch.isfinite(o[2, 64:].float()).all()
    assert not o[3].float().any() and torch.isneginf(lse[3]).all()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
def test_paged_attention_infinite_q(dev, kv):
    """An infinity in q makes its head's row NaN over pages of either type, and no other row another one."""
    c = Case(dev, 2, 8, 4, 128, 32, [200, 77, 1500], kv, seed=21)
    want, want_l = c.launch()
    c.q[0, 5 * 128 + 3] = float("inf")
    c.q[2, 1 * 128 + 100] = float("-inf")
    o, lse = c.launch()
    hit = torch.zeros((3, 8), dtype=torch.bool, device=dev)
    hit[0, 5] = hit[2, 1] = True
    o, want = o.view(3, 8, 128), want.view(3, 8, 128)
    assert torch.isnan(o[hit].float()).all() and torch.isfinite(want.float()).all()
    assert torch.equal(o[~hit].view(torch.int16), want[~hit].view(torch.int16))
    assert torch.equal(lse[~hit], want_l[~hit]) and not torch.isfinite(lse[hit]).any()


@pytest.mark.parametrize("kv", [tpx.TP_BF16, tpx.TP_FP8_E4M3])
def test_paged_attention_requests_that_share_pages(dev, kv):
    """Requests with a common beginning name the same pages, one of them a page twice."""
    c = Case(dev, 1, 8, 2, 64, 16, [400, 333, 96, 400], kv, seed=22, poison=False)
    c.table[1, :20] = c.table[0, :20]
    c.table[2, :6] = c.table[0, :6]
    c.table[3, 7:9] = c.table[3, 3]
    c.check()
    c.check(window=90)


def test_two_attention_calls_at_once(dev):
    """Calls on two streams with a workspace each, over the same pages and in any overlap, give the bits of
    calls one after the other."""
    a = Case(dev, 1, 32, 8, 128, 64, [9000, 1, 777], seed=23)
    b = Case(dev, 1, 8, 4, 256, 16, [50, 0, 3100, 640, 12], seed=24)
    want = [x.launch()[0].clone() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for x, s, o in zip((a, b), streams, outs):
            x.call(o[i], None, stream=s)
    sync()
    for w, o in zip(want, outs):
        assert all(torch.equal(w.view(torch.int16), y.view(torch.int16)) for y in o)


def test_paged_attention_and_append_past_4_gib(dev):
    """Pages whose byte offsets pass 32 bits (a pool of 5 GiB per side)."""
    n_kv, hd, page, n_pages = 8, 128, 256, 10400
    sh = tpx.make_shape(1024, n_q=16, n_kv=n_kv, hd=hd)
    k, v = (torch.empty((1, n_pages, n_kv, page, hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    n = 700
    ids = [10399, 4, 9001]
    qkv = inputs.normal_bf16((n, 32 * hd), 1.0, 10, 96, dev)
    j = np.arange(n)
    slots = np.array(ids)[j // page] * page + j % page
    pages = tpx.make_pages(page, n_pages, 3)
    q = torch.empty((n, 16 * hd), dtype=torch.bfloat16, device=dev)
    tpx.tp_rope_append(sh, None, pages, qkv, None, i32(slots, dev), q, k, v)
    o = torch.empty((1, 16 * hd), dtype=torch.bfloat16, device=dev)
    tpx.tp_paged_attn_decode(sh, pages, q[-1:], k, v, i32([ids], dev), i32([n], dev), o,
                             tpx.new_paged_attn_workspace(sh, dev))
    sync()
    x = PO.split_qkv(O.as_f64(bits(qkv)), 1, 16, n_kv, hd)

    def rows(y):
        def f(g):
            return y[:, g], np.ones(n, bool)
        f.n_kv = n_kv
        return f
    ref, _, A, B = PO.attention(x[0][-1], rows(x[1]), rows(x[2]), 1 / math.sqrt(hd))
    e = A * (2 * (136 * 2.0 ** -23 * B[:, None] + 2.0 ** -20 + 350 * 2.0 ** -24) + 2.0 ** -16)
    assert_within(O.as_f64(bits(o)).reshape(16, hd), ref, e + HALF * (np.abs(ref) + e), "o")


def test_one_workspace_for_many_shapes_and_streams_in_order(dev):
    """A workspace of the largest size serves every shape; work on a side stream waits for nothing else."""
    big = Case(dev, 1, 32, 2, 256, 16, [3000, 5], seed=11)
    for t, n_q, n_kv, hd in ((1, 4, 4, 64), (2, 32, 2, 128), (1, 8, 1, 256)):
        c = Case(dev, t, n_q, n_kv, hd, 32, [2500, 0, 33, 4000], seed=hd)
        assert tpx.tp_paged_attn_workspace_bytes(c.sh) <= big.ws.numel()
        c.ws = big.ws
        c.check()
    big.check()


def test_captured_step_on_a_side_stream(dev):
    """tables -> append -> attention captured on a side stream and replayed: each replay continues from the
    last one's lengths, as eager calls do."""
    M, n_q, n_kv, hd, page, P = 6, 8, 2, 64, 16, 12
    sh = tpx.make_shape(512, n_q=n_q, n_kv=n_kv, hd=hd, t=2)
    pages = tpx.make_pages(page, M * P, P)
    rope = tpx.make_rope(hd)
    free = i32(np.random.default_rng(1).permutation(M * P), dev)
    qkv = make_qkv(dev, M, n_q, n_kv, hd, 12)
    add = i32([1, 2, 0, 1, 1, 1], dev)

    def state():
        z = lambda *s, d=torch.int32: torch.zeros(s, dtype=d, device=dev)
        return dict(table=z(M, P) - 1, lens=[z(M), z(M)], counts=[z(3), z(3)], cu=z(M + 1), pos=z(8), slots=z(8),
                    k=z(2, M * P, 1, page, hd, d=torch.bfloat16), v=z(2, M * P, 1, page, hd, d=torch.bfloat16),
                    q=z(8, n_q * hd, d=torch.bfloat16), o=z(M, n_q * hd, d=torch.bfloat16),
                    ws=tpx.new_paged_attn_workspace(sh, dev))
    rows = torch.cat([qkv, qkv[:2]])                                    # 8 rows, two of them padding

    def step(s, i, stream=None):
        a, b = i % 2, 1 - i % 2
        tpx.tp_paged_tables(pages, s["lens"][a], add, free, s["table"], s["lens"][b], s["cu"], s["pos"], s["slots"],
                            s["counts"][b], head=s["counts"][a], stream=stream)
        tpx.tp_rope_append(sh, rope, pages, rows, s["pos"], s["slots"], s["q"], s["k"], s["v"], stream=stream)
        tpx.tp_paged_attn_decode(sh, pages, s["q"][:M], s["k"], s["v"], s["table"], s["lens"][b], s["o"], s["ws"],
                                 stream=stream)
    eager, graphed = state(), state()
    outs = []
    for i in range(40):
        step(eager, i)
        outs.append(eager["o"].clone())
    sync()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(graphed, 0, side)
            step(graphed, 1, side)
        for i in range(0, 40, 2):
            graph.replay()
            assert torch.equal(graphed["o"].view(torch.int16), outs[i + 1].view(torch.int16)), i
    sync()
    for key in ("table", "k", "v", "q", "slots"):
        assert torch.equal(eager[key].view(torch.uint8), graphed[key].view(torch.uint8)), key
    assert eager["lens"][0].tolist() == [40, 80, 0, 40, 40, 40]


def test_paged_equals_contiguous_attention(dev):
    """The same tokens in a contiguous and in a paged cache, rotated by tp_rope_forward and by tp_rope_append:
    the caches hold the same bits and the attention outputs agree within both roundings."""
    M, n_q, n_kv, hd, page, L, t = 4, 16, 4, 128, 16, 300, 2
    sh = tpx.make_shape(1024, n_q=n_q, n_kv=n_kv, hd=hd, t=t)
    rope = tpx.make_rope(hd, 500000.0)
    P = -(-L // page)
    pages = tpx.make_pages(page, M * P, P)
    table = np.random.default_rng(2).permutation(M * P).reshape(M, P)
    kc, vc = (torch.zeros((t, M, n_kv // t, L, hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    kp, vp = (torch.zeros((t, M * P, n_kv // t, page, hd), dtype=torch.bfloat16, device=dev) for _ in range(2))
    aws = torch.empty(tpx.tp_attn_workspace_bytes(sh, M, L), dtype=torch.uint8, device=dev)
    ws = tpx.new_paged_attn_workspace(sh, dev)
    oc, op, q = (torch.empty((M, n_q * hd), dtype=torch.bfloat16, device=dev) for _ in range(3))
    for step in range(150):
        qkv = make_qkv(dev, M, n_q, n_kv, hd, 100 + step)
        pos = i32([step] * M, dev)
        turned = torch.empty_like(qkv)
        tpx.tp_rope_forward(sh, rope, qkv, pos, turned)
        tpx.tp_attn_decode(sh, turned, kc, vc, pos, oc, aws)
        slots = i32([table[m, step // page] * page + step % page for m in range(M)], dev)
        tpx.tp_rope_append(sh, rope, pages, qkv, pos, slots, q, kp, vp)
        tpx.tp_paged_attn_decode(sh, pages, q, kp, vp, i32(table, dev), pos + 1, op, ws)
    sync()
    for m in range(M):
        for c, p in ((kc, kp), (vc, vp)):
            flat = p[:, table[m]].transpose(1, 2).reshape(t, n_kv // t, P * page, hd)[:, :, :150]
            assert torch.equal(flat.contiguous().view(torch.int16), c[:, m, :, :150].contiguous().view(torch.int16))
    a, b = O.as_f64(bits(oc)), O.as_f64(bits(op))
    assert O.rel_frobenius(bits(op), a) <= 5e-3 and np.abs(a - b).max() <= 2e-2 * np.sqrt((a * a).mean())


@pytest.mark.parametrize("wtype,kv", [(tpx.TP_BF16, tpx.TP_BF16), (tpx.TP_FP8_E4M3, tpx.TP_FP8_E4M3),
                                      (tpx.TP_BF16, tpx.TP_FP8_E4M3)])
@pytest.mark.parametrize("M", [1, 5, 70])
def test_paged_attention_block_decode_steps(dev, wtype, kv, M):
    """Decode steps as a server makes them: tables, the block in one call, the lm_head and the log probabilities.
    The block equals its four calls bit for bit, and the last step's y equals the oracle on the cache it left."""
    d, n_q, n_kv, hd, t, page, P, V = 1024, 8, 4, 128, 2, 16, 6, 1000
    x, wqkv, wo = inputs.proj_inputs(d, n_q, n_kv, hd, M, seed=13, device=dev)
    sh = tpx.make_shape(d, n_q=n_q, n_kv=n_kv, hd=hd, t=t, wtype=wtype)
    q_w, qd = tpx.tp_partition_weights(sh, tpx.TP_W_QKV, wqkv)
    o_w, od = tpx.tp_partition_weights(sh, tpx.TP_W_O, wo)
    vsh = tpx.make_shape(d, t=t, vocab=V)
    v_w, vd = tpx.tp_partition_weights(vsh, tpx.TP_W_VOCAB, inputs.normal_bf16((d, V), 0.02, 13, 98, dev))
    pages, rope = tpx.make_pages(page, M * P, P, kv), tpx.make_rope(64, 500000.0)
    ks, vs = scales(dev, n_kv, kv, 13)
    free = i32(np.random.default_rng(13).permutation(M * P), dev)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=dev)
    b16 = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev)
    raw = torch.bfloat16 if kv == tpx.TP_BF16 else torch.float8_e4m3fn
    caches = [[z(t, M * P, n_kv // t, page, hd, dt=raw) for _ in range(2)] for _ in range(2)]
    table, lens, counts = z(M, P) - 1, [z(M), z(M)], [z(3), z(3)]
    cu, pos, slots, add = z(M + 1), z(M), z(M), i32(np.ones(M), dev)
    ws, ws2 = tpx.new_paged_attn_block_workspace(sh, M, dev), tpx.new_workspace(sh, M, dev)
    aws = tpx.new_paged_attn_workspace(sh, dev)
    Q = (n_q + 2 * n_kv) * hd
    out = [dict(y=b16(M, d), qkv=b16(M, Q), q=b16(M, n_q * hd), o=b16(M, n_q * hd)) for _ in range(2)]
    for step in range(35):
        xs = inputs.normal_bf16((M, d), 1.0, 14 + step, 99, dev)
        tpx.tp_paged_tables(pages, lens[0], add, free, table, lens[1], cu, pos, slots, counts[1], head=counts[0])
        a, b = out
        tpx.tp_paged_attn_block_forward(qd, q_w, od, o_w, xs, xs, rope, pages, pos, slots, *caches[0], table, lens[1],
                                        a["y"], a["qkv"], a["q"], a["o"], ws, window=20, k_scale=ks, v_scale=vs)
        tpx.tp_colpar_forward(qd, q_w, xs, b["qkv"], ws=ws2)
        tpx.tp_rope_append(sh, rope, pages, b["qkv"], pos, slots, b["q"], *caches[1], ks, vs)
        tpx.tp_paged_attn_decode(sh, pages, b["q"], *caches[1], table, lens[1], b["o"], aws, window=20, k_scale=ks,
                                 v_scale=vs)
        tpx.tp_rowpar_forward(od, o_w, b["o"], xs, b["y"], ws2)
        lens.reverse()
        counts.reverse()
    sync()
    for key in out[0]:
        assert torch.equal(out[0][key].view(torch.int16), out[1][key].view(torch.int16)), key
    for u, v in zip(*caches):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    assert lens[0].tolist() == [35] * M and counts[0].tolist() == [M * 3, M, 0]
    wo_ref = O.as_f64(bits(wo))
    if wtype == tpx.TP_FP8_E4M3:
        wo_ref = O.dequantize_fp8(*O.quantize_fp8_per_channel(wo_ref))
    y_ref = O.as_f64(bits(out[0]["o"])) @ wo_ref + O.as_f64(bits(xs))
    check_close(bits(out[0]["y"]), y_ref, what="y of the last step")
    logits = torch.empty((M, V), dtype=torch.float32, device=dev)
    tpx.tp_lm_head_forward(vd, v_w, out[0]["y"], logits)
    lp, ent, rank = (torch.zeros(M, dtype=dt, device=dev) for dt in (torch.float32, torch.float32, torch.int32))
    tl, ti = torch.zeros((M, 3), device=dev), z(M, 3)
    tpx.tp_token_logprobs(logits, logits.argmax(1).to(torch.int32), lp, ent, rank, tl, ti)
    sync()
    assert (rank == 1).all() and torch.equal(lp, tl[:, 0]) and torch.equal(ti[:, 0].long(), logits.argmax(1))


@pytest.mark.parametrize("wtype,kv", [(tpx.TP_BF16, tpx.TP_BF16), (tpx.TP_FP8_E4M3, tpx.TP_FP8_E4M3)])
def test_paged_attention_block_shares_a_workspace_over_m(dev, wtype, kv):
    """One workspace of the largest M, zero-filled once, serves steps of any M in any order, with the shape's other
    calls between them: the bits of the four calls, whose attention has a workspace of its own.  The requests are
    long enough to be split over CTAs, so each step counts pieces."""
    d, n_q, n_kv, hd, t, page, L = 1024, 8, 4, 128, 2, 16, 2600
    big = 70
    _, wqkv, wo = inputs.proj_inputs(d, n_q, n_kv, hd, 1, seed=15, device=dev)
    sh = tpx.make_shape(d, n_q=n_q, n_kv=n_kv, hd=hd, t=t, wtype=wtype)
    q_w, qd = tpx.tp_partition_weights(sh, tpx.TP_W_QKV, wqkv)
    o_w, od = tpx.tp_partition_weights(sh, tpx.TP_W_O, wo)
    held = L // page + 1
    n_pages = 3 * held
    pages, rope = tpx.make_pages(page, n_pages, held, kv), tpx.make_rope(hd, 500000.0)
    ks, vs = scales(dev, n_kv, kv, 15)
    cache = [pool(dev, t, n_pages, n_kv, page, hd, kv, 15, s) for s in (101, 102)]
    order = np.random.default_rng(15).permutation(n_pages).reshape(3, held)
    table = i32([order[m % 3] for m in range(big)], dev)                # requests share pages; none is appended to
    slots = i32([-1] * big, dev)
    lens = i32([L - 37 * m if m % 5 else 0 for m in range(1, big + 1)], dev)
    pos = lens - 1
    xs = inputs.normal_bf16((big, d), 1.0, 16, 99, dev)
    ws, ws2 = tpx.new_paged_attn_block_workspace(sh, big, dev), tpx.new_workspace(sh, big, dev)
    aws = tpx.new_paged_attn_workspace(sh, dev)
    b16 = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev)
    for M in (70, 32, 31, 1, 8, 64, 4, 5, 1, 33, 70, 2):
        a, b = [dict(y=b16(M, d), qkv=b16(M, (n_q + 2 * n_kv) * hd), q=b16(M, n_q * hd), o=b16(M, n_q * hd))
                for _ in range(2)]
        x = xs[:M]
        tpx.tp_paged_attn_block_forward(qd, q_w, od, o_w, x, x, rope, pages, pos, slots, *cache, table, lens, a["y"],
                                        a["qkv"], a["q"], a["o"], ws, k_scale=ks, v_scale=vs)
        tpx.tp_colpar_forward(qd, q_w, x, b["qkv"], ws=ws2)
        tpx.tp_rope_append(sh, rope, pages, b["qkv"], pos, slots, b["q"], *cache, ks, vs)
        tpx.tp_paged_attn_decode(sh, pages, b["q"], *cache, table, lens, b["o"], aws, k_scale=ks, v_scale=vs)
        tpx.tp_rowpar_forward(od, o_w, b["o"], x, b["y"], ws2)
        sync()
        for key in a:
            assert torch.equal(a[key].view(torch.int16), b[key].view(torch.int16)), (M, key)
        tpx.tp_rowpar_forward(od, o_w, xs[:, :n_q * hd].contiguous(), None, b16(big, d), ws)  # scratch over the counters
    # steps captured into a graph per M, as a server keeps them, replayed in turn over the one workspace
    graphs, side = {}, torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for M in (8, 33, 70):
        out = dict(y=b16(M, d), qkv=b16(M, (n_q + 2 * n_kv) * hd), q=b16(M, n_q * hd), o=b16(M, n_q * hd))
        g = torch.cuda.CUDAGraph()
        step = lambda st: tpx.tp_paged_attn_block_forward(qd, q_w, od, o_w, xs[:M], xs[:M], rope, pages, pos, slots, *cache,
                                                          table, lens, out["y"], out["qkv"], out["q"], out["o"], ws,
                                                          k_scale=ks, v_scale=vs, stream=st)
        step(torch.cuda.current_stream())
        sync()
        want = out["y"].clone()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            step(side)
        graphs[M] = (g, out, want)                                      # the graph's buffers live as long as it does
    for M in (70, 8, 33, 8, 70, 33):
        g, out, want = graphs[M]
        out["y"].fill_(float("nan"))
        g.replay()
        sync()
        assert torch.equal(out["y"].view(torch.int16), want.view(torch.int16)), M
