"""Sampling against the fp64 oracle on a B200."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from confidence_gated_kv_logit_b200 import build, load_library, sample
from oracle import sampling as oracle

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def dev(v, dtype=torch.float32):
    return None if v is None else torch.tensor(v, dtype=dtype, device="cuda")


def run(logits, u, **kw):
    R = logits.shape[0]
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((R,), -7.0, device="cuda")
    kw = {k: dev(v, torch.int32 if k == "top_k" else torch.float32) for k, v in kw.items()}
    sample(logits, dev(u), token, prob_out=prob, **kw)
    return token.cpu().numpy(), prob.cpu().numpy()


def check(logits, u, near_ok=None, **kw):
    """Tokens equal to the oracle's, except where u falls within 2e-7 of a step
    of the running weight: weights carry fp32 rounding (2^-23 of a weight, whose
    errors in a running sum and its total partly cancel). The share carries that
    of one weight and of the total."""
    token, prob = run(logits, u, **kw)
    x = logits.float().cpu().numpy()
    near = 0
    for r in range(x.shape[0]):
        p = {k: (np.float32(v[r]) if k != "top_k" else v[r]) for k, v in kw.items() if v is not None}
        t, share, margin = oracle.sample(x[r], np.float32(u[r]), **p)
        if margin < 2e-7 and t >= 0:
            near += 1
            assert token[r] >= 0
            continue
        assert token[r] == t, (r, token[r], t, margin)
        assert abs(prob[r] - share) <= 1e-6 * share + 1e-12, (r, prob[r], share)
    assert near <= (max(1, x.shape[0] // 8) if near_ok is None else near_ok)
    return token


def logits_of(rows, vocab, seed, dtype=torch.float32, scale=None, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = torch.where(torch.rand((rows, 1), generator=g, device="cuda") < 0.7, 8.0, 0.5) if scale is None else scale
    return (torch.randn((rows, vocab + pad), generator=g, device="cuda") * s).to(dtype)[:, :vocab]


FILTERS = [dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=1000, top_p=0.95, min_p=0.02),
           dict(temperature=0.7), dict(temperature=1.8, top_p=0.5), dict(top_k=3, top_p=0.999)]


@pytest.mark.parametrize("kw", FILTERS, ids=lambda k: "-".join(k) or "plain")
@pytest.mark.parametrize("vocab", [1, 2, 7, 500, 2049, 8191, 8193, 50257, 128256])
def test_filters_and_sizes(vocab, kw):
    R = 6
    x = logits_of(R, vocab, vocab)
    u = np.random.RandomState(vocab).rand(R).astype(np.float32)
    check(x, u, **{k: [v] * R for k, v in kw.items()})


@pytest.mark.parametrize("vocab", [400001, 1 << 20])
def test_rows_too_wide_for_shared_memory(vocab):
    x = logits_of(2, vocab, 9)
    check(x, [0.3, 0.8], top_p=[0.9, 0.3], temperature=[1.0, 0.9])
    check(x, [0.3, 0.8], top_k=[5000, 1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 1, 64])
def test_types_and_padded_rows(dtype, pad):
    # 16-bit logits tie at most cuts
    x = logits_of(5, 20011, 11, dtype, pad=pad)
    u = [0.01, 0.2, 0.5, 0.77, 0.999]
    check(x, u, top_k=[40, 300, 5000, 19000, 2], top_p=[1.0, 0.8, 0.9, 0.95, 0.5])
    check(x, u, min_p=[0.1, 0.01, 0.5, 1.0, 2.0])


def test_rows_have_their_own_parameters():
    R = 9
    x = logits_of(R, 3001, 13)
    check(x, np.linspace(0, 0.99, R), temperature=[0.0, 0.5, 1, 2, 1e-30, 1e-3, 50, 1, 1],
          top_k=[0, 1, 5, -3, 10, 10 ** 9, 2999, 3000, 3001], top_p=[0.5, 0.9, 1.0, 2.0, 0.5, 0.9, 0.0, -1.0, 0.999],
          min_p=[0, 0, 0.1, 0, 0, 0, 0.5, 0.9, -1.0])


def test_many_equal_logits():
    """Cuts inside long runs of equal logits: the lower indices stay."""
    V = 30011
    flat = torch.zeros((4, V), device="cuda")
    check(flat, [0.0, 0.25013, 0.50027, 0.9999], top_k=[10, 5000, 2048, 30010])
    steps = (torch.arange(V, device="cuda") % 3).float().repeat(4, 1)
    check(steps, [0.1, 0.3, 0.6, 0.9], top_k=[9000, 10004, 15000, 25000])
    # equal fp32 weights: a border that falls exactly between two tokens keeps the tokens before it
    tokens = run(torch.zeros((1, 4096), device="cuda"), [0.99999], top_p=[0.5])[0]
    assert tokens[0] == 2047
    tokens = run(torch.full((1, 100000), -3.402823466e38, device="cuda"), [0.99999], top_k=[70000])[0]
    assert tokens[0] == int(0.99999 * 70000)


def test_cuts_by_every_digit():
    """A million equal logits: both cuts go down to the last bits of the index."""
    V = 1 << 20
    x = torch.zeros((2, V), device="cuda")
    x[1, ::2] = -1.0
    # the last token kept is drawn by u just below 1: of 700001 tokens, those before which less than half the weight lies
    t, p = run(x, [0.9999999, 0.9999999], top_k=[700001, 400001], top_p=[0.5, 0.75])
    assert list(t) == [350000, 2 * 300000 + 1]
    assert abs(p[0] * 350001 - 1) < 1e-6 and abs(p[1] * 300001 - 1) < 1e-6
    t, _ = run(x, [0.9999999, 0.9999999], top_k=[700001, 524289])
    assert list(t) == [700000, V - 1]


def test_close_logits_in_one_bin():
    """Thousands of distinct logits within one histogram bin."""
    V = 60000
    x = (1.0 + torch.randperm(V, device="cuda").float() * 2.0 ** -23)[None].repeat(3, 1)
    x[:, 17] = 9.0
    check(x, [0.2, 0.5, 0.8], top_k=[100, 30000, 59990])
    # nearly equal weights: the cut by weight is decided below fp32, so only the counts are pinned
    t, p = run(x, [0.9999, 0.9999, 0.9999], top_p=[0.9, 0.99, 0.5])
    assert (t >= 0).all()


def test_masked_rows():
    V = 5003
    x = logits_of(6, V, 21)
    x[0, 1:] = -INF
    x[1, :-1] = -INF
    x[2] = -INF
    x[3, ::2] = -INF
    x[4, 100:] = torch.finfo(torch.float32).min
    x[5, :] = torch.finfo(torch.float32).min
    u = [0.9, 0.1, 0.5, 0.7, 0.999, 0.6]
    t = check(x, u)
    assert (t[0], t[1], t[2]) == (0, V - 1, -1)
    check(x, u, top_k=[5] * 6, top_p=[0.9] * 6, min_p=[0.1] * 6)
    check(x, u, top_k=[5002] * 6)
    huge = torch.tensor([[3e38, -3e38, -INF, 3e38]], device="cuda")
    assert run(huge, [0.75])[0][0] == 3


def test_bad_rows_get_minus_one_and_leave_the_others():
    x = logits_of(8, 10000, 23)
    x[1, 5000] = math.nan
    x[2, 9999] = INF
    kw = dict(temperature=[1, 1, 1, -1.0, math.nan, 1, 1, INF], top_p=[0.9, 1, 1, 1, 1, math.nan, 1, 1],
              min_p=[0, 0, 0, 0, 0, 0, math.nan, 0])
    t, p = run(x, [0.5] * 8, **kw)
    assert t[0] >= 0 and (t[1:] == -1).all() and (p[1:] == 0).all()
    t, p = run(x[:1].repeat(4, 1), [1.0, -0.1, math.nan, 0.0])
    assert list(t[:3]) == [-1, -1, -1] and t[3] >= 0


def test_ends_of_the_unit_interval():
    x = logits_of(2, 50257, 25)
    # both ends are within 2e-7 of a step: the first logit of row 0 lies 25 or more below the largest (a share
    # under e^-25), and 1 - u is 2^-24
    check(x, [0.0, np.nextafter(np.float32(1), np.float32(0))], near_ok=2)
    only = torch.full((1, 9001), -INF, device="cuda")
    only[0, [77, 9000]] = 0.0
    assert run(only, [0.0])[0][0] == 77 and run(only, [0.5])[0][0] == 9000 and run(only, [0.499999])[0][0] == 77


def test_same_answers_twice_on_a_stream_and_captured():
    x = logits_of(16, 128256, 27)
    u = torch.rand(16, device="cuda")
    kw = dict(top_k=torch.full((16,), 900, dtype=torch.int32, device="cuda"), top_p=torch.full((16,), 0.9, device="cuda"))
    out = [torch.empty(16, dtype=torch.int32, device="cuda") for _ in range(3)]
    pr = [torch.empty(16, device="cuda") for _ in range(3)]
    sample(x, u, out[0], prob_out=pr[0], **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    sample(x, u, out[1], prob_out=pr[1], stream=st, **kw)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sample(x, u, out[2], prob_out=pr[2], **kw)
    graph.replay()
    torch.cuda.synchronize()
    for k in (1, 2):
        assert torch.equal(out[0], out[k]) and torch.equal(pr[0], pr[k])
    u.copy_(torch.rand(16, device="cuda"))
    graph.replay()
    sample(x, u, out[0], prob_out=pr[0], **kw)
    assert torch.equal(out[0], out[2]) and torch.equal(pr[0], pr[2])


def test_refusals():
    x = torch.zeros((2, 10), device="cuda")
    u, t = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    sample(x[:0], u[:0], t[:0])
    with pytest.raises(TypeError):
        sample(x, u, t.long())
    with pytest.raises(TypeError):
        sample(x, None, t)
    with pytest.raises(ValueError):
        sample(x, u[:1], t)
    with pytest.raises(TypeError):
        sample(x.double(), u, t)
    with pytest.raises(ValueError):
        sample(x.t(), torch.zeros(10, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        sample(x, u, t, top_k=u)
    with pytest.raises(TypeError):
        sample(x.cpu(), u, t)


@pytest.mark.parametrize("vocab", [3001, 128256])
def test_top_k_far_below_the_maximum(vocab):
    """The k-th token lies past the bins (2^-32 of the largest weight), past the wider ones, and below tokens
    masked with the type's lowest value."""
    x = logits_of(5, vocab, 21, scale=8.0)
    k = vocab // 3
    check(x, [0.1, 0.5, 0.9, 0.99, 0.0], temperature=[0.6, 0.1, 0.02, 0.3, 1.0], top_k=[k, k, k, vocab - 1, 1500],
          top_p=[1.0, 0.9, 0.9, 1.0, 0.95])
    x[:, ::2] = -3.402823466e38
    check(x, [0.1, 0.5, 0.9, 0.99, 0.3], temperature=[0.6, 0.1, 1.5, 1.0, 1.0], top_k=[k, k, vocab - 2, 40, 1500],
          top_p=[1.0, 0.9, 0.9, 1.0, 0.5])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.01, 0.5, 3.0])
def test_lists_of_hundreds(dtype, scale):
    """Cuts and draws over some hundreds of tokens, as many as one CTA finishes and one more, with ties and without."""
    ks = [127, 128, 129, 500, 1111, 2046, 2047, 2048, 2049]
    R = len(ks)
    x = logits_of(R, 50257, 23, dtype, scale=scale)
    u = np.random.RandomState(5).rand(R).astype(np.float32)
    check(x, u, top_k=ks)
    check(x, u, top_k=ks, top_p=np.linspace(0.05, 0.99, R), min_p=[0.0, 0.3, 0.01] * 3)
    check(x, u, top_p=[0.001, 0.01, 0.02, 0.03, 0.04, 0.05, 0.2, 0.5, 0.999], temperature=np.linspace(0.3, 2, R))


def test_finished_rows_repeat_bit_for_bit():
    x = logits_of(33, 50257, 25)
    u = np.random.RandomState(6).rand(33).astype(np.float32)
    kw = dict(top_k=[700 + r for r in range(33)], top_p=[0.97] * 33)
    first = run(x, u, **kw)
    for _ in range(20):
        again = run(x, u, **kw)
        assert (again[0] == first[0]).all() and (again[1] == first[1]).all()


def test_digits_with_more_ties_than_a_list_holds():
    """Cuts and draws among 1600 equal logits side by side: every selection is split by the keys' bits, by 128 and
    more keys a digit, in each of the three selections of a row, again and again."""
    R, V, n = 96, 262144, 1600
    at = np.random.RandomState(8).randint(0, V - n, R)
    x = torch.full((R, V), -30.0, device="cuda")
    for r in range(R):
        x[r, at[r]:at[r] + n] = 2.0
    u = ((np.arange(R) + 0.5) / R).astype(np.float32)
    k = np.array([(200, 1000, 1599)[r % 3] for r in range(R)])
    # the weights are equal: of k tokens those before which less than top_p of the weight lies (the products
    # below are not whole numbers), of m kept tokens the one at floor(u m)
    for kw, m in ((dict(top_k=k), k), (dict(top_k=k, top_p=[0.6137] * R), np.ceil(np.float32(0.6137).astype(np.float64) * k))):
        want = at + np.floor(u.astype(np.float64) * m).astype(np.int64)
        for _ in range(10):
            token, prob = run(x, u, **kw)
            assert np.array_equal(token, want)
            assert np.abs(prob * m - 1).max() <= 1e-6


class Job(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("u", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("token", ctypes.c_void_p), ("stream", ctypes.c_void_p),
                ("calls", ctypes.c_int32), ("failed", ctypes.c_int32), ("sample", ctypes.c_void_p)]


def test_threads_with_rows_of_different_sizes(tmp_path):
    """Calls of one kernel from several threads, whose rows take different amounts of shared memory."""
    here = os.path.dirname(os.path.abspath(__file__))
    helper = tmp_path / "sample_threads.so"
    subprocess.run(["gcc", "-std=c99", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-pthread", "-I",
                    os.path.join(here, "..", "include"), os.path.join(here, "sample_threads.c"), "-o", str(helper)], check=True)
    fn = ctypes.cast(load_library().confkv_sample, ctypes.c_void_p).value
    work, jobs = [], (Job * 4)()
    for i, (R, V) in enumerate([(2, 128256), (2, 50257), (40, 60001), (1, 9000)]):
        x, u, top_p = logits_of(R, V, 40 + i).contiguous(), torch.rand(R, device="cuda"), torch.full((R,), 0.8, device="cuda")
        want, got, stream = torch.empty(R, dtype=torch.int32, device="cuda"), torch.zeros(R, device="cuda").int(), torch.cuda.Stream()
        sample(x, u, want, top_p=top_p)
        work.append((x, u, top_p, want, got, stream))
        jobs[i] = Job(x.data_ptr(), R, V, u.data_ptr(), top_p.data_ptr(), got.data_ptr(), stream.cuda_stream, 3000, 0, fn)
    torch.cuda.synchronize()
    assert ctypes.CDLL(str(helper)).run_threads(jobs, 4) == 0
    torch.cuda.synchronize()
    assert [j.failed for j in jobs] == [0] * 4
    for _, _, _, want, got, _ in work:
        assert torch.equal(want, got)


@pytest.mark.parametrize("V", [2000, 50257, 128256, 400001])
@pytest.mark.parametrize("tail", [-19.0, -21.4, -21.6, -24.5])
@pytest.mark.parametrize("p", [0.5, 0.9999, 0.99995, 0.99998, 0.9999995])
def test_long_light_tails(V, tail, p):
    """One token over a tail that weighs 6e-9 to 2e-11 of it a token: top_p cuts by the tail's sum."""
    x = torch.full((1, V), tail, device="cuda")
    x[0, 0] = 0.0
    u, w1 = np.nextafter(np.float32(1), np.float32(0)), math.exp(tail)
    idx, w = oracle.kept_set(x[0].cpu().numpy(), top_p=np.float32(p))
    (token,), (prob,) = run(x, [0.0], top_p=[p])
    (far,), _ = run(x, [u], top_p=[p])
    # What may move the border, as a share of the largest weight: half a unit of 2^-40 a token of the row, in the
    # cut and again in the draw; 2^-22 of the tail's sum, for fp32 weights. Then, in tokens: four weights that are
    # added in fp32 before fp64 takes them, where the largest swallows the other three; one for a border's two sides.
    off = 2 * V * 2.0 ** -41 + V * w1 * 2.0 ** -22
    if len(idx) == 1:
        # (no border near: what is missing to the first token's weight is more than that)
        assert 1 - float(np.float32(p)) * (1 + (V - 1) * w1) > off + 2.0 ** -23
        assert far == 0 and prob == 1
        return
    # the last kept token but those that weigh 1 - u of the total together
    want = len(idx) - 1 - int((1 - float(u)) * w.sum() / w1)
    assert abs(far - max(want, 0)) <= off / w1 + 5
    # the largest token's share is one over the sum of the kept weights (and an fp32 number below 1)
    assert token == 0 and abs(1 / float(prob) - w.sum()) <= off + 5 * w1 + 2.0 ** -24
