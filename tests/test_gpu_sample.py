"""Sampled tokens through the C ABI against the float64 oracle: the id exactly (or, where a sum lies within the
weights' error of its border, one of the two beside it), logprob within its rounding."""
import math

import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import inputs, tpx
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

# Weights are good to 2^-29 of themselves, one below 2^-44 may be missing: 2^19 of those are 2^-25 of the largest at
# most, 2^17 and fewer (these tests') 2^-27.  A sum against its border: both are off by that.
SLACK = 2.0 ** -26


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_transformer_gb300 import build
    build.build_library()
    tpx.lib()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def run(dev, x, u, T=None, k=None, p=None, q=None, pad=0, lead=0, logprob=True, stream=None):
    """x: fp32 array [M, V]; rows V + pad apart from element `lead` of the buffer on, NaN between them."""
    M, V = x.shape
    buf = torch.full((lead + M * (V + pad),), float("nan"), dtype=torch.float32, device=dev)
    rows = buf[lead:].view(M, V + pad)[:, :V]
    rows.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    f = lambda v: None if v is None else torch.tensor(np.broadcast_to(np.asarray(v, np.float32), M).copy(), device=dev)
    n = lambda v: None if v is None else torch.tensor(np.broadcast_to(np.asarray(v, np.int32), M).copy(), device=dev)
    ids = torch.full((M + 1,), 77, dtype=torch.int32, device=dev)
    lp = torch.full((M + 1,), 77.0, dtype=torch.float32, device=dev)
    tpx.tp_sample_tokens(rows, f(u), ids[:M], f(T), n(k), f(p), f(q), lp[:M] if logprob else None, stream=stream)
    assert tpx.tp_sync(stream, timeout_ms=10000) == tpx.TP_OK
    assert ids[M] == 77 and lp[M] == 77.0                              # nothing behind the outputs
    return ids[:M].cpu().numpy(), lp[:M].cpu().numpy()


def check(dev, x, u, T=1.0, k=0, p=1.0, q=0.0, sharp=True, **kw):
    x = np.asarray(x, np.float32)
    M = len(x)
    ids, lp = run(dev, x, u, T, k, p, q, **kw)
    f = lambda v: np.broadcast_to(np.asarray(v, np.float32), M).astype(np.float64)
    u, T, p, q, k = f(u), f(T), f(p), f(q), np.broadcast_to(np.asarray(k), M)
    sure = 0
    for m in range(M):
        may, want = PO.sample(x[m], u[m], T[m], int(k[m]), p[m], q[m], SLACK)
        assert ids[m] in may, (m, ids[m], may)
        sure += len(set(may)) == 1
        refs = [y for i, y in zip(may, want) if i == ids[m]]
        # the sum's error (2^-28), one rounding to fp32
        near = lambda y: abs(float(lp[m]) - y) <= 2.0 ** -24 * abs(y) + 2.0 ** -24
        assert not kw.get("logprob", True) or any(np.isnan(lp[m]) if np.isnan(y) else near(y) for y in refs), (m, lp[m], refs)
    assert sure >= 0.95 * M - 1 or not sharp                           # the borders are the exception
    return ids, lp


def normal(M, V, seed, std=3.0):
    rng = np.random.default_rng(seed)
    return inputs.normal_bf16((M, V), std, seed, 98).float().numpy() + rng.uniform(-0.01, 0.01, (M, V)).astype(np.float32)


def us(M, seed):
    return (np.random.default_rng(seed + 1000).integers(0, 1 << 24, M) / float(1 << 24)).astype(np.float32)


SETTINGS = [dict(), dict(T=0.7), dict(T=0.0), dict(k=1), dict(k=7, T=1.3), dict(k=300), dict(p=0.9), dict(p=0.3, T=0.5),
            dict(p=0.999, T=2.0), dict(q=0.05), dict(q=0.5, T=3.0), dict(k=40, p=0.8, q=0.02, T=0.8), dict(k=3, p=0.99)]


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 33, 1000, 4099, 17001, 128256])
@pytest.mark.parametrize("s", range(len(SETTINGS)))
def test_sample_sizes(dev, V, s):
    M = 3 if V > 20000 else 6
    check(dev, normal(M, V, V + s), us(M, V + s), **SETTINGS[s])


@pytest.mark.parametrize("M", [1, 2, 18, 19, 37, 75, 151, 300])
def test_sample_rows_with_their_own_settings(dev, M):
    """Batches of every way to share a row among CTAs; each row brings its settings."""
    rng = np.random.default_rng(M)
    T = rng.choice([0.0, 0.3, 0.7, 1.0, 1.5], M)
    check(dev, normal(M, 20011, M), us(M, M), T, rng.choice([0, 1, 20, 500, 30000], M), rng.choice([0.0, 0.5, 0.95, 1.0], M),
          rng.choice([0.0, 0.02, 0.9, 1.0], M))


def test_sample_largest_vocabulary(dev):
    V = 1 << 19
    check(dev, normal(2, V, 5), [0.3, 0.9], p=[0.9, 1.0])
    ids, _ = run(dev, np.zeros((2, V), np.float32), [0.25, 1 - 2.0 ** -24], p=[1.0, 0.5])
    assert ids.tolist() == [V // 4, V // 2 - 1]                        # exact: on the border itself


@pytest.mark.parametrize("V,pad,lead", [(1000, 1, 0), (1000, 2, 1), (999, 0, 3), (6, 1, 1), (2, 3, 3), (20001, 6, 2), (1, 5, 1)])
def test_sample_strides_and_alignment(dev, V, pad, lead):
    for s in (SETTINGS[0], SETTINGS[2], SETTINGS[6], SETTINGS[11]):
        check(dev, normal(5, V, V), us(5, V), pad=pad, lead=lead, **s)


def test_sample_equal_logits_by_id(dev):
    """All equal: every id weighs the same, so the choice is floor(u n) exactly, and top-k and top-p keep the lowest."""
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.1], np.float32)
    for V in (8, 1000, 40000):
        x = np.full((6, V), -3.25, np.float32)
        x[1, :] = np.where(np.arange(V) % 3 == 0, 0.0, -0.0)           # zeros of both signs are equal
        for n, kw in ((V, {}), (5, dict(k=5)), (V // 2, dict(p=0.5)), (V, dict(q=1.0)), (4, dict(k=8, p=0.5)), (1, dict(T=0.0)),
                      (V, dict(T=1e-30)), (V, dict(T=1e30)), (1, dict(p=0.0)), (1, dict(p=-1.0)), (V, dict(k=-3)), (V, dict(k=2 ** 31 - 1))):
            ids, lp = run(dev, x, u, **kw)
            assert np.array_equal(ids, np.floor(u.astype(np.float64) * n).astype(int)), (V, kw)
            assert np.abs(lp + np.log(n)).max() <= 2.0 ** -24 * (1 + np.log(n)), (V, kw)


def test_sample_many_ties(dev):
    """A few values many times: the border of top-k and of top-p lies among equal logits."""
    rng = np.random.default_rng(2)
    for V in (60, 5000, 40000):
        x = rng.choice([-4.0, -1.0, 0.5, 2.0], (12, V), p=[0.3, 0.3, 0.3, 0.1]).astype(np.float32)
        check(dev, x, us(12, V), k=rng.integers(1, V, 12))
        check(dev, x, us(12, V), p=rng.uniform(0.05, 0.99, 12), k=rng.choice([0, V // 2], 12))


def test_sample_every_u_gives_its_share(dev):
    """One row, a grid of random numbers: the ids ascend with u and each token is chosen in its share of them."""
    M = 1024
    x = np.repeat(normal(1, 3001, 9, 2.0), M, 0)
    u = ((np.arange(M) + 0.5) / M).astype(np.float32)
    ids, lp = check(dev, x, u, p=0.97)
    assert np.all(np.diff(ids) >= 0)
    for t in np.unique(ids):
        assert abs((ids == t).sum() - M * np.exp(lp[ids == t][0])) <= 1 + 1e-3


def test_sample_masked_rows(dev):
    x = normal(8, 9000, 3)
    rng = np.random.default_rng(3)
    x[0, rng.random(9000) < 0.999] = -np.inf
    x[1, :] = -np.inf
    x[1, 8000] = 2.0                                                   # one token left: logprob 0
    x[2, :] = -np.inf                                                  # none left
    x[3, 17] = np.nan
    x[4, 8999] = np.inf
    x[5, :] = np.finfo(np.float32).min                                 # the type's lowest value is a number
    x[6, :] = np.finfo(np.float32).min
    x[6, 4000:4004] = np.finfo(np.float32).max                         # differences past the type's range weigh nothing
    x[7, 0] = -np.inf
    for kw in (dict(), dict(k=6), dict(p=0.8), dict(T=0.0), dict(q=0.1, p=0.9, k=50)):
        ids, lp = check(dev, x, us(8, 4), **kw)
        assert ids[1] == 8000 and lp[1] == 0.0 and ids[2] == ids[3] == ids[4] == -1
        assert 4000 <= ids[6] < 4004
    nan_u, nan_t = np.full(8, np.nan), np.full(8, np.nan)
    for kw in (dict(u=nan_u), dict(T=nan_t), dict(p=nan_t), dict(q=nan_t)):
        ids, lp = run(dev, x, **{"u": us(8, 4), **kw})
        assert (ids == -1).all() and np.isnan(lp).all()


def test_sample_u_outside(dev):
    """u below 0 takes the first kept token, from 1 on the last one that has a weight."""
    x = normal(4, 5000, 8)
    x[:, 4990:] = -200.0                                               # kept without top-p, but without weight
    check(dev, x, [-0.5, 1.0, 7.0, -np.inf])
    check(dev, x, [np.inf, 1.0, 0.0, 2.0 ** -30], p=0.9)


@pytest.mark.parametrize("T", [2.0 ** -140, 2.0 ** -100, 1e-6, 1e-3, 50.0, 1e9, 3e38])
def test_sample_temperatures(dev, T):
    check(dev, normal(6, 7001, 11, 20.0), us(6, 11), T=T, p=[1.0, 1.0, 0.7, 0.7, 0.1, 0.999])


@pytest.mark.parametrize("V", [3001, 120011])
def test_sample_borders_among_light_tokens(dev, V):
    """One token ahead of all others, far enough that the borders of top-p and top-k lie among weights of 2^-20 to 2^-40,
    spread, nearly alike, and alike."""
    rng = np.random.default_rng(V)
    x = np.stack([-rng.uniform(11, 28, V), -rng.uniform(14.0, 14.02, V), np.full(V, -15.5), -rng.uniform(10, 30, V)]).astype(np.float32)
    x[:, V // 3] = 0.0
    rest = np.exp(x.astype(np.float64)).sum(1) - 1
    for share in (0.1, 0.5, 0.93):
        check(dev, x, us(4, V), p=(1 + share * rest) / (1 + rest), sharp=False)  # a weight is as small as the slack
    check(dev, x, [1 - 2.0 ** -24] * 4, p=(1 + 0.7 * rest) / (1 + rest), sharp=False)
    check(dev, x, [1 - 2.0 ** -24] * 4, k=[V // 2, V // 2, 1000, V - 1], p=[1.0, 1.0, 1.0, 0.9999999], sharp=False)


def test_sample_far_logits(dev):
    """Large logits a little apart, tiny ones, and ones around zero: the differences count to their last bit."""
    rng = np.random.default_rng(12)
    base = (3e4 + rng.integers(0, 4000, (4, 6000)) * 2.0 ** -9).astype(np.float32)
    check(dev, base, us(4, 12), T=0.9, p=0.9)
    check(dev, (rng.normal(size=(4, 6000)) * 1e-30).astype(np.float32), us(4, 13), T=[1e-30, 1e-30, 1.0, 1e-31], p=[0.9, 1, 0.5, 1])
    check(dev, (rng.normal(size=(4, 6000)) * 1e30).astype(np.float32), us(4, 14), T=1e29)


def test_sample_without_settings(dev):
    x = normal(5, 3000, 15)
    ids, _ = run(dev, x, us(5, 15), logprob=False)
    want, lp = run(dev, x, us(5, 15), 1.0, 0, 1.0, 0.0)
    assert np.array_equal(ids, want) and np.isfinite(lp).all()


def test_sample_repeats_and_streams(dev):
    """Captured, replayed, on two streams at once: the same ids and bits."""
    V = 128256
    big, few = (torch.from_numpy(normal(M, V, M)).to(dev) for M in (40, 3))
    st = {}
    for x in (big, few):
        M = x.shape[0]
        g = np.random.default_rng(M)
        st[M] = [torch.tensor(v, device=dev) for v in (us(M, 3), g.uniform(0.5, 1.2, M).astype(np.float32),
                                                       g.choice([0, 50], M).astype(np.int32), g.uniform(0.5, 1.01, M).astype(np.float32))]
    def call(x, out, lp, stream=None):
        u, T, k, p = st[x.shape[0]]
        tpx.tp_sample_tokens(x, u, out, T, k, p, None, lp, stream=stream)
    new = lambda x: (torch.zeros(x.shape[0], dtype=torch.int32, device=dev), torch.zeros(x.shape[0], device=dev))
    want = {}
    for x in (big, few):
        want[x] = new(x)
        call(x, *want[x])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = {x: [new(x) for _ in range(20)] for x in (big, few)}
    torch.cuda.synchronize()
    for i in range(20):
        for x, s in zip((big, few), streams):
            call(x, *outs[x][i], stream=s)
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), new(big)
    with torch.cuda.graph(graph, stream=streams[0]):
        call(big, *got, stream=streams[0])
    for _ in range(3):
        got[0].fill_(-9)
        graph.replay()
        outs[big].append(tuple(t.clone() for t in got))
    torch.cuda.synchronize()
    for x in (big, few):
        for ids, lp in outs[x]:
            assert torch.equal(ids, want[x][0]) and torch.equal(lp, want[x][1])


@pytest.mark.parametrize("low,high", [(14.9, 15.1), (15.0, 19.0), (22.0, 31.0), (29.9, 30.1), (30.0, 33.0), (40.0, 47.0)])
@pytest.mark.parametrize("kind", ["k", "p", "both"])
def test_sample_border_many_octaves_down(dev, low, high, kind):
    """A few heavy tokens and very many that weigh 2^-low to 2^-high: the border lies among these, and u chooses there."""
    V, M = 100003, 8
    rng = np.random.default_rng(int(low * 10))
    E = np.sort(rng.uniform(low, high, (M, V)), axis=1)
    E[:, :3] = (0.0, 1.0, 2.5)
    x = (-E * np.log(2.0)).astype(np.float32)
    tail = 2.0 ** -np.float64(E[:, 3:]).mean(1) * (V - 3)
    whole = 1.0 + 0.5 + 2.0 ** -2.5 + tail
    k = np.array([4, 5, 100, V // 3, V // 2, V - 2, V - 1, V]) if kind != "p" else 0
    p = np.float32(1.0 - tail / whole * np.linspace(0.02, 0.98, M)) if kind != "k" else 1.0
    u = np.float32(1.0 - tail / whole * np.linspace(0.9, 0.1, M))
    u = np.minimum(u, np.float32(1.0 - 2.0 ** -24))
    ids, lp = run(dev, x, u, 1.0, k, p)
    k, p = np.broadcast_to(k, M), np.broadcast_to(np.float64(p), M)
    for m in range(M):
        # Tokens here are lighter than the slack of a sum: the oracle names those at its two ends, and each one between
        # them is as near to the border, since the sum of the kept weights grows with the id.
        may, want = PO.sample(x[m], np.float64(u[m]), 1.0, int(k[m]), p[m], 0.0, SLACK)
        assert min(may) <= ids[m] <= max(may), (m, ids[m], may)
        ref = want[0] + np.float64(x[m, ids[m]]) - np.float64(x[m, may[0]])
        assert abs(float(lp[m]) - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -24, (m, lp[m], ref)


@pytest.mark.parametrize("V", [129, 257, 1001, 40003, 128256])
def test_sample_few_and_many_of_top_k(dev, V):
    """Top-k's tokens are taken from a list up to some number: on both sides of it, with the other filters and with ties."""
    ks = [1, 2, 31, 32, 33, 100, 128, 129, 200, 255, 256, 257, 300]
    settings = [dict(), dict(p=0.9), dict(p=0.4, q=0.03), dict(q=0.2), dict(p=0.0), dict(q=1.0), dict(p=0.7, T=2.0), dict(T=0.0)]
    rows = [(k, s) for k in ks for s in settings]
    x = normal(len(rows), V, V + 5)
    x[::3] = np.round(x[::3] * 2.0) / 2.0                              # ties across the border
    x[1::5] = np.where(np.random.default_rng(V).random(x[1::5].shape) < 0.3, -np.inf, x[1::5])
    x[1::5, 5] = 1.0
    f = lambda key, d: np.array([s.get(key, d) for _, s in rows], np.float32)
    check(dev, x, us(len(rows), V), T=f("T", 1.0), k=np.array([k for k, _ in rows]), p=f("p", 1.0), q=f("q", 0.0), sharp=False)


@pytest.mark.parametrize("kw", [dict(q=1.0), dict(q=0.5), dict(), dict(p=0.3), dict(k=700, p=0.9, q=1.0), dict(k=40, p=0.6, q=1.0)])
def test_sample_infinite_temperature(dev, kw):
    """Every token that is not masked weighs the same, min_p of 1 and less leaves all of them."""
    V = 5003
    x = normal(6, V, 17)
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.1], np.float32)
    check(dev, x, u, T=np.inf, sharp=False, **kw)                      # (u n is a whole number, a border, for some n and u)
    x[:, 1000:1400] = -np.inf
    x[3, 1:] = -np.inf
    x[4, 7], x[4, 8] = 3e38, -3e38                                     # every difference to the largest but this one is finite
    ids, lp = check(dev, x, u, T=np.inf, sharp=False, **kw)
    assert ids[3] == 0 and lp[3] == 0.0 and not ((1000 <= ids) & (ids < 1400)).any() and ids[4] != 8
    ids, _ = run(dev, np.where(np.arange(V) % 2 == 0, x[:1], -np.inf).repeat(6, 0), u, np.inf, 0, 1.0, 1.0)
    n = (V + 1) // 2 - 200                                             # even ids, but for 1000 .. 1398
    nth = np.floor(u.astype(np.float64) * n).astype(int)
    assert np.array_equal(ids, np.where(nth < 500, 2 * nth, 2 * nth + 400))


@pytest.mark.parametrize("q", [1.0 + 2.0 ** -23, 1.5, 3e38, np.inf])
def test_sample_min_p_above_one(dev, q):
    """No weight reaches it, so the first rank alone is left: of equal largest logits the lowest id."""
    x = normal(8, 3001, 18)
    x[::2, [2000, 50, 700]] = 40.0
    for kw in (dict(), dict(T=0.3), dict(T=np.inf), dict(k=5), dict(k=1000, p=0.99), dict(p=0.2)):
        ids, lp = check(dev, x, us(8, 18), q=q, **kw)
        assert np.array_equal(ids, x.argmax(1)) and (lp == 0).all()
    ids, lp = check(dev, x, us(8, 18), q=1.0)                          # reached by the equal ones
    assert set(ids[::2]) <= {50, 700, 2000} and len(set(ids[::2])) > 1 and np.abs(lp[::2] + np.log(3)).max() < 1e-6


def timed(dev, x, p, M):
    """Microseconds of a call over M rows x, the median of seven; and its ids."""
    rows = torch.from_numpy(x).to(dev).expand(M, -1).contiguous()
    u = torch.full((M,), 0.5, device=dev)
    p = torch.tensor(np.broadcast_to(np.float32(p), M).copy(), device=dev)
    ids, lp = torch.zeros(M, dtype=torch.int32, device=dev), torch.zeros(M, device=dev)
    times = []
    for _ in range(7):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        tpx.tp_sample_tokens(rows, u, ids, None, None, p, None, lp)
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]) * 1e3)
    return sorted(times)[3], ids.cpu().numpy(), lp.cpu().numpy()


@pytest.mark.parametrize("share,low,high", [(0.5, 17.0, 17.0), (0.99, 24.0, 40.0), (1 - 2.0 ** -20, 36.0, 45.0)])
def test_sample_border_at_the_heavy_tokens_end(dev, share, low, high):
    """One token with nearly `share` of the weight, then many light ones octaves below; top-p on both sides of that share, to
    the last bits.  Sums in fp32 cannot tell which side it is on; a row takes a few passes more for it, not a thousand."""
    V, M = 128256, 64
    rng = np.random.default_rng(int(low))
    E = rng.uniform(low, high, V) if high > low else np.full(V, low)
    x = (-E * np.log(2.0)).astype(np.float32)
    rest = np.exp(x.astype(np.float64)).sum() - math.exp(x[777])
    x[777] = math.log(share / (1 - share) * rest)
    w = np.exp(x.astype(np.float64) - x[777])
    own = 1 / w.sum()                                                  # the heavy token's share
    step = np.spacing(np.float32(own))
    p = np.minimum(np.float32(own) + step * np.arange(-M // 2, M // 2), 1 - 2.0 ** -24).astype(np.float32)
    usual, _, _ = timed(dev, x[None], 0.7 * own, M)                    # far from the border: the heavy token alone is left
    took, ids, lp = timed(dev, x[None], p, M)
    for m in range(M):
        may, _ = PO.sample(x, 0.5, 1.0, 0, np.float64(p[m]), 0.0, SLACK)
        assert min(may) <= ids[m] <= max(may), (m, ids[m], may)
    assert took <= 4 * usual + 40, (took, usual)
