"""Token log probabilities through the C ABI against the float64 oracle: ids and ranks exactly, values within
the bound of their fp32 sums."""
import numpy as np
import pytest
import torch

from megatron_tensor_transformer_gb300 import inputs, tpx
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from megatron_tensor_transformer_gb300 import build
    build.build_library()
    tpx.lib()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def run(dev, x, ids, k, pad=0, lead=0, skip=()):
    """x: fp32 array [M, V]; rows V + pad apart from element `lead` of the buffer on."""
    M, V = x.shape
    buf = torch.full((lead + M * (V + pad),), float("nan"), dtype=torch.float32, device=dev)
    rows = buf[lead:].view(M, V + pad)[:, :V]
    rows.copy_(torch.from_numpy(x))
    f = lambda *s: torch.full(s, 5.0, dtype=torch.float32, device=dev)
    n = lambda *s: torch.full(s, 5, dtype=torch.int32, device=dev)
    out = dict(logprob=f(M + 1), rank=n(M + 1), entropy=f(M + 1), tl=f(M + 1, max(k, 1)), ti=n(M + 1, max(k, 1)))
    use = {key: None if key in skip else v[:M] for key, v in out.items()}
    ids_d = None if "ids" in skip else torch.tensor(np.asarray(ids), dtype=torch.int32, device=dev)
    tpx.tp_token_logprobs(rows, ids_d, use["logprob"], use["entropy"], use["rank"], use["tl"] if k else None,
                          use["ti"] if k else None)
    assert tpx.tp_sync(timeout_ms=10000) == tpx.TP_OK
    for key, v in out.items():
        assert (v[M] == 5).all(), key                                  # nothing behind the outputs
    return {key: v[:M].cpu().numpy() for key, v in out.items()}


def check(dev, x, ids, k, **kw):
    x = np.asarray(x, np.float32)
    got = run(dev, x, ids, k, **kw)
    lp, rank, ent, tl, ti = PO.logprobs(x.astype(np.float64), ids, k)
    assert np.array_equal(got["rank"], rank)
    V = x.shape[1]
    # S: e^d with d = x - m rounded to fp32 (2^-24 |d|, and d e^d stays below 1), the product with log2 e (2^-24
    # |d| again) and ex2 (2^-22): 2^-21 of S; a thread sums V / 512 values, then the threads: V / 512 + 64 steps of
    # 2^-24.  ln P adds the roundings of x - m, of ln S and of their difference: 2^-22 of |ln P| + |ln S| < |ln P| + 12.
    s = 2.0 ** -21 + (V / 512 + 64) * 2.0 ** -24
    near = lambda a, b, extra: np.testing.assert_array_less(
        np.where(np.isfinite(b), np.abs(a - np.where(np.isfinite(b), b, 0)), 0), s + 2.0 ** -22 * (12 + np.abs(
            np.where(np.isfinite(b), b, 0))) + extra)
    same = lambda a, b: np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
    assert same(got["logprob"], lp) and same(got["entropy"], ent)
    near(got["logprob"], lp, 0)
    near(got["entropy"], ent, 4 * s * (1 + np.abs(np.nan_to_num(ent))))  # T / S: both sums, and d e^d in T
    if k:
        assert np.array_equal(got["ti"], ti) and same(got["tl"], tl)
        near(got["tl"], tl, 0)
    return got


def normal(M, V, seed, std=3.0):
    return inputs.normal_bf16((M, V), std, seed, 97).float().numpy() + np.random.default_rng(seed).uniform(
        -0.01, 0.01, (M, V)).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 33, 1000, 4099, 17001, 128256])
@pytest.mark.parametrize("M,k", [(1, 1), (7, 5), (3, 32), (2, 0)])
def test_logprobs_sizes(dev, V, M, k):
    ids = np.random.default_rng(V).integers(0, V, M)
    check(dev, normal(M, V, V + M), ids, min(k, V))


@pytest.mark.parametrize("M", [20, 90, 200, 700])
def test_logprobs_rows_per_cluster(dev, M):
    check(dev, normal(M, 20000, M), np.random.default_rng(M).integers(0, 20000, M), 6)


@pytest.mark.parametrize("V,pad,lead", [(1000, 1, 0), (1000, 2, 1), (999, 0, 3), (6, 1, 1), (2, 3, 3), (20001, 6, 2)])
def test_logprobs_strides_and_alignment(dev, V, pad, lead):
    check(dev, normal(5, V, V), [0, V - 1, V // 2, 1, 0], min(V, 7), pad=pad, lead=lead)


def test_logprobs_ties_go_to_the_lower_id(dev):
    rng = np.random.default_rng(1)
    for V in (40, 5000, 40000):
        x = rng.integers(-2, 3, (6, V)).astype(np.float32)
        x[1] = 0.5                                       # all equal
        x[2] = np.where(rng.random(V) < 0.5, 0.0, -0.0)  # zeros of both signs are equal
        check(dev, x, rng.integers(0, V, 6), 32)


def test_logprobs_sorted_rows(dev):
    """Ascending logits: every value passes the bar (the slowest case for the top list)."""
    V = 30000
    x = np.stack([np.linspace(-9, 9, V), np.linspace(9, -9, V), np.arange(V) * 1e-3]).astype(np.float32)
    check(dev, x, [0, V - 1, 17], 32)


def test_logprobs_masked_rows(dev):
    x = normal(8, 9000, 3)
    rng = np.random.default_rng(3)
    x[0, rng.random(9000) < 0.999] = -np.inf
    x[1, :] = -np.inf
    x[1, 8000] = 2.0                                     # one id left: ln P = 0, entropy 0
    x[2, :] = -np.inf                                    # none left
    x[3, 5] = np.nan
    x[4, 8999] = np.inf
    x[5, :4500] = np.finfo(np.float32).min               # masks of the type's lowest value
    x[6, :] = np.finfo(np.float32).min
    x[7, :] = np.finfo(np.float32).max
    got = check(dev, x, [1, 8000, 3, 7, 8, 2, 2, 2], 10)
    assert got["logprob"][1] == 0 and got["entropy"][1] == 0 and got["rank"][1] == 1
    assert got["ti"][2].tolist() == [-1] * 10 and got["rank"][3] == 0


@pytest.mark.parametrize("V", [20, 40, 130, 511, 1000, 2047, 8001])
@pytest.mark.parametrize("kept", [0.02, 0.3, 1.0])
def test_logprobs_short_masked_rows(dev, V, kept):
    """Rows with fewer vectors than groups of threads, most of them masked: fewer groups hold a value than there are
    alternatives, which then go on into the masked ids, the lowest first."""
    M, rng = 6, np.random.default_rng(V)
    x = normal(M, V, V)
    x[rng.random((M, V)) >= kept] = -np.inf
    x[np.arange(M), rng.integers(0, V, M)] = 1.0            # none is masked altogether
    for k in (1, min(V, 20), min(V, 24), min(V, 25), min(V, 32)):
        check(dev, x, rng.integers(0, V, M), k, pad=V % 3, lead=V % 4)


@pytest.mark.parametrize("left", [1, 7, 40])
def test_logprobs_few_ids_left_of_a_large_vocabulary(dev, left):
    """A vocabulary masked down to a few ids that lie far apart, over one CTA a row and several."""
    V, rng = 128256, np.random.default_rng(left)
    for M in (3, 160):
        x = np.full((M, V), -np.inf, np.float32)
        for m in range(M):
            x[m, rng.choice(V, left, replace=False)] = rng.normal(size=left)
        check(dev, x, [int(np.argmax(r)) for r in x], 20)


def test_logprobs_ids_that_ask_for_nothing(dev):
    x = normal(5, 700, 4)
    x[4, 3] = np.nan
    got = check(dev, x, [-1, 700, 2 ** 31 - 1, -(2 ** 31), -100], 3)
    assert not got["logprob"].any() and not got["rank"].any()


def test_logprobs_large_and_peaky(dev):
    x = normal(4, 5000, 5, std=1.0)
    x[0] *= 1e4
    x[1] += 1e6                                          # a common offset
    x[2, 77] = 90.0                                      # e^-90 elsewhere
    x[3] *= 1e-30
    check(dev, x, [3, 4, 78, 5], 8)


@pytest.mark.parametrize("skip", [("ids", "logprob", "rank"), ("entropy",), ("rank",), ("logprob",)])
def test_logprobs_without_some_outputs(dev, skip):
    x = normal(3, 3001, 6)
    got, all_ = run(dev, x, [1, 2, 3], 4, skip=skip), run(dev, x, [1, 2, 3], 4)
    for key in got:
        if key not in skip:
            assert np.array_equal(got[key], all_[key])


def test_logprobs_captured_and_repeated(dev):
    """The same bits on every run, eager and replayed from a graph with new logits in the same buffer."""
    M, V, k = 9, 50001, 5
    x = torch.from_numpy(normal(M, V, 7)).to(dev)
    ids = torch.arange(M, dtype=torch.int32, device=dev)
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device=dev)
    n = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    def outs():
        return f(M), f(M), n(M), f(M, k), n(M, k)
    a, b = outs(), outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        tpx.tp_token_logprobs(x, ids, *b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        x += 0.01 * step * torch.randn_like(x)
        tpx.tp_token_logprobs(x, ids, *a)
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(a, b):
            assert torch.equal(u, v)
