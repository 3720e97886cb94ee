"""Rotary positions and per-head norms against the fp64 oracle on a B200."""
import numpy as np
import pytest
import torch

from confidence_gated_kv_logit_b200 import ConfKVError, Rope, build
from oracle.rope import frequencies

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def oracle(x, positions, rope_kw, rd, layout, weight, eps):
    """oracle.rope.rotate_row for every row at once (fp64); also the length of each value's pair."""
    f, mag = frequencies(rd, **rope_kw) if rd else (np.zeros(0), 1.0)
    x = x.double().cpu().numpy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.double().cpu().numpy()
    ang = positions.cpu().numpy().astype(np.float64)[:, :, None, None] * f
    c, s = np.cos(ang) * mag, np.sin(ang) * mag
    n = rd // 2
    ia = np.arange(n) if layout == "half" else 2 * np.arange(n)
    ib = ia + n if layout == "half" else ia + 1
    y, size = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.hypot(a, b) * mag
    return y, size


def check(got, want, size, dtype):
    # Rounding to the output type: half a step relative, half the smallest step
    # absolute. fp32 arithmetic: the angle's fraction (2^-25 pi), sincospif (2
    # steps), three products and the norm's sum, root and scaling (under 20
    # roundings) stay below 2e-6 of the pair's length.
    info = torch.finfo(dtype)
    tol = info.eps / 2 * np.abs(want) + info.smallest_normal * info.eps / 2 + 2e-6 * size
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


def make(B, T, H, D, dtype, g, pad=0):
    base = torch.randn((B, T, H, D + pad), generator=g, device="cuda").to(dtype)
    return base[..., :D]


@pytest.mark.parametrize("D,rd", [(128, 128), (64, 64), (256, 256), (32, 32), (128, 96), (128, 32), (128, 0),
                                  (64, 2), (80, 80), (96, 50), (2, 2), (254, 128), (128, 120)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("x,y", [("fp16", "fp16"), ("bf16", "fp16"), ("fp32", "fp32")])
def test_shapes_and_types(D, rd, layout, x, y):
    g = torch.Generator(device="cuda").manual_seed(1)
    B, T, Hq, Hk = 2, 5, 6, 3
    r = Rope(D, rotary_dim=rd, layout=layout, theta=5000.0)
    q, k = make(B, T, Hq, D, TYPES[x], g), make(B, T, Hk, D, TYPES[x], g)
    pos = torch.randint(0, 100000, (B, T), generator=g, device="cuda", dtype=torch.int32)
    qw = torch.randn(D, generator=g, device="cuda")
    for weights in ((None, None), (qw, qw * 2), (None, qw)):
        qo = torch.full((B, T, Hq, D), 7.0, dtype=TYPES[y], device="cuda")
        ko = torch.full((B, T, Hk, D), 7.0, dtype=TYPES[y], device="cuda")
        r.apply(q, k, pos, qo, ko, q_weight=weights[0], k_weight=weights[1], eps=1e-5)
        for src, out, w in ((q, qo, weights[0]), (k, ko, weights[1])):
            want, size = oracle(src, pos, dict(theta=5000.0), rd, layout, w, 1e-5)
            check(out, want, size, TYPES[y])


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (16, 1, 32, 8), (3, 7, 5, 1), (1, 1500, 8, 2), (1, 1, 64, 0),
                                       (700, 3, 7, 7)])
@pytest.mark.parametrize("norm", [False, True])
def test_batches(B, T, Hq, Hk, norm):
    g = torch.Generator(device="cuda").manual_seed(2)
    D = 128
    r = Rope(D)
    q = make(B, T, Hq, D, torch.float16, g)
    k = make(B, T, Hk, D, torch.float16, g) if Hk else None
    pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
    w = torch.rand(D, generator=g, device="cuda") if norm else None
    qo, ko = torch.empty_like(q), (torch.empty_like(k) if Hk else None)
    r.apply(q, k, pos, qo, ko, q_weight=w, k_weight=w if Hk else None)
    for src, out in ((q, qo),) + (((k, ko),) if Hk else ()):
        check(out, *oracle(src, pos, {}, D, "half", w, 1e-6), torch.float16)


@pytest.mark.parametrize("kw", [dict(theta=1e6, scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(theta=5e5, scaling="banded", factor=8.0, original_length=8192),
                                dict(theta=1e6, scaling="yarn", factor=4.0, original_length=32768),
                                dict(scaling="yarn", factor=2.0, magnitude=1.0)])
def test_far_positions_of_every_scaling(kw):
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.tensor([[0, 1, 131071, 1048575, 2 ** 31 - 1, -1, -2 ** 31]], dtype=torch.int32, device="cuda")
    q = make(1, 7, 4, 128, torch.float32, g)
    out = torch.empty_like(q)
    Rope(128, **kw).apply(q, None, pos, out)
    # a 53-bit frequency times 2^31 leaves the oracle's own angle off by 2^31 * 2^-53 * 2 pi < 2e-6
    want, size = oracle(q, pos, kw, 128, "half", None, 0.0)
    check(out, want, 2 * size, torch.float32)


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_strides(pad):
    """Packed projections, the cache's own key layout, padded and odd rows, in place."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, T, Hq, Hk, D = 2, 9, 4, 2, 64
    r = Rope(D)
    qkv = torch.randn((B, T, Hq + 2 * Hk, D + pad), generator=g, device="cuda").half()[..., :D]
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    pos = torch.randint(0, 5000, (B, T), generator=g, device="cuda", dtype=torch.int32)
    keep = qkv.clone()
    ko = torch.zeros((B, Hk, T, D), dtype=torch.float16, device="cuda")
    qo = torch.zeros((T, B, Hq, D + pad), dtype=torch.float16, device="cuda")[..., :D].transpose(0, 1)
    r.apply(q, k, pos, qo, ko.transpose(1, 2))
    assert torch.equal(qkv, keep)
    check(qo, *oracle(q, pos, {}, D, "half", None, 0), torch.float16)
    check(ko.transpose(1, 2), *oracle(k, pos, {}, D, "half", None, 0), torch.float16)
    want_q, want_k = qo.clone(), ko.transpose(1, 2).clone()
    r.apply(q, k, pos, q, k)                               # in place
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(qkv[:, :, Hq + Hk:], keep[:, :, Hq + Hk:])     # the values are left as they were


def test_inverse_and_special_values():
    q = torch.randn((1, 3, 2, 128), device="cuda")
    pos = torch.tensor([[5, 70000, 3]], dtype=torch.int32, device="cuda")
    r = Rope(128)
    a, b = torch.empty_like(q), torch.empty_like(q)
    r.apply(q, None, pos, a)
    r.apply(a, None, -pos, b)
    assert (b - q).abs().max().item() <= 4e-6 * q.abs().max().item()
    w = torch.ones(128, device="cuda")
    z = torch.zeros_like(q)
    r.apply(z, None, pos, a, q_weight=w)
    assert (a == 0).all()
    z[0, 1, 1, 5] = float("nan")
    z[0, 2, 0, 5] = float("inf")
    r.apply(z, None, pos, a)
    # only the pair of a special value is touched by it
    bad = torch.zeros_like(z, dtype=torch.bool)
    bad[0, 1, 1, [5, 69]] = True
    bad[0, 2, 0, [5, 69]] = True
    assert torch.equal(~torch.isfinite(a), bad)


def test_empty_calls_and_refusals():
    r = Rope(64)
    q = torch.zeros((0, 4, 2, 64), dtype=torch.float16, device="cuda")
    r.apply(q, None, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), q)
    q = torch.zeros((2, 4, 2, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        r.apply(q[..., :32], None, pos, q[..., :32])
    with pytest.raises(ValueError):
        r.apply(q, None, pos[:1], q)
    with pytest.raises(TypeError):
        r.apply(q, None, pos.long(), q)
    with pytest.raises(TypeError):
        r.apply(q, q, pos, q)
    with pytest.raises(TypeError):
        r.apply(q.double(), None, pos, q)
    with pytest.raises(TypeError):
        r.apply(q, q.float(), pos, q, q)
    with pytest.raises(TypeError):
        r.apply(q.cpu(), None, pos, q)
    with pytest.raises(ValueError):
        r.apply(q.transpose(2, 3).contiguous().transpose(2, 3), None, pos, q)
    with pytest.raises(ValueError):
        r.apply(q, None, pos, q, q_weight=torch.ones(32, device="cuda"))


def test_captured_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(5)
    q = make(4, 2, 8, 128, torch.float16, g)
    pos = torch.randint(0, 5000, (4, 2), generator=g, device="cuda", dtype=torch.int32)
    r = Rope(128)
    want, got = torch.empty_like(q), torch.zeros_like(q)
    r.apply(q, None, pos, want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    r.apply(q, None, pos, got, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.apply(q, None, pos, got)
    pos.add_(1)
    graph.replay()
    r.apply(q, None, pos, want)
    assert torch.equal(got, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rd", [(128, 100), (128, 102), (128, 2), (64, 10), (256, 250)])
def test_odd_parts_of_many_heads(D, rd, layout):
    """Rotated parts that end inside a lane's values, heads of two sides that a warp takes in turn, in place, with
    values in the plain part that a product with zero would not leave alone."""
    g = torch.Generator(device="cuda").manual_seed(8)
    B, T, Hq, Hk = 3, 300, 9, 4
    qkv = make(B, T, Hq + Hk, D, torch.float16, g)
    if rd < D - 1:
        qkv[..., -1] = float("inf")
    x = qkv.clone()
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:]
    pos = torch.randint(0, 100000, (B, T), generator=g, device="cuda", dtype=torch.int32)
    Rope(D, rotary_dim=rd, layout=layout).apply(q, k, pos, q, k)
    assert torch.equal(qkv[..., rd:], x[..., rd:])
    want, size = oracle(x[..., :rd], pos, {}, rd, layout, None, 0.0)
    check(qkv[..., :rd], want, size, torch.float16)


def test_outputs_whose_rows_overlap_are_refused():
    """Every row of an output has a place of its own, whichever way its strides go."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, T, H, D = 2, 4, 3, 64
    q = make(B, T, H, D, torch.float16, g)
    pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
    r = Rope(D)
    room = torch.zeros(B * T * H * D * 4, dtype=torch.float16, device="cuda")
    for strides in ((T * H * D, D, D), (T * D, H * D, D), (D, B * D, D), (T * H * D, H * D, D - 1), (8 * D, 2 * D, 3 * D)):
        with pytest.raises(ConfKVError) as e:
            r.apply(q, None, pos, room.as_strided(q.shape, strides + (1,)))
        assert e.value.status == 1
    with pytest.raises(ConfKVError) as e:      # one output for both sides
        r.apply(q, q, pos, room.as_strided(q.shape, q.stride()), room.as_strided(q.shape, q.stride()))
    assert e.value.status == 1
    assert (room == 0).all()
    # rows apart from one another, in every order of the dimensions and padded
    for strides in ((T * H * D, H * D, D), (D, B * H * D, B * D), (H * D, B * H * D, D), (T * D, D, B * T * D),
                    (T * H * 80, H * 80, 80)):
        out = room.as_strided(q.shape, strides + (1,))
        r.apply(q, None, pos, out)
        check(out, *oracle(q, pos, {}, D, "half", None, 0), torch.float16)


def test_dimensions_of_one_have_no_stride():
    """Whatever stride a dimension of size 1 reports, the rows are the same: in place, and as an output."""
    g = torch.Generator(device="cuda").manual_seed(10)
    D, T = 64, 5
    pos = torch.arange(T, device="cuda", dtype=torch.int32)[None]
    r = Rope(D)
    q = make(1, T, 1, D, torch.float16, g)
    want = torch.empty_like(q)
    r.apply(q, None, pos, want)
    out = torch.zeros_like(q)
    r.apply(q.as_strided(q.shape, (7, D, 3, 1)), None, pos, out.as_strided(q.shape, (0, D, 1, 1)))
    assert torch.equal(out, want)
    r.apply(q.as_strided(q.shape, (7, D, 3, 1)), None, pos, q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("y", list(TYPES))
@pytest.mark.parametrize("D,rd,layout", [(128, 128, "half"), (64, 64, "interleaved"), (128, 102, "half"), (96, 96, "interleaved")])
def test_every_pair_of_types(x, y, D, rd, layout):
    g = torch.Generator(device="cuda").manual_seed(11)
    B, T, Hq, Hk = 2, 3, 5, 2
    q, k = make(B, T, Hq, D, TYPES[x], g), make(B, T, Hk, D, TYPES[x], g)
    pos = torch.randint(0, 100000, (B, T), generator=g, device="cuda", dtype=torch.int32)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    r = Rope(D, rotary_dim=rd, layout=layout)
    for qw in (None, w):
        qo = torch.full((B, T, Hq, D), 7.0, dtype=TYPES[y], device="cuda")
        ko = torch.full((B, Hk, T, D), 7.0, dtype=TYPES[y], device="cuda")
        r.apply(q, k, pos, qo, ko.transpose(1, 2), q_weight=qw, k_weight=w)
        check(qo, *oracle(q, pos, {}, rd, layout, qw, 1e-6), TYPES[y])
        check(ko.transpose(1, 2), *oracle(k, pos, {}, rd, layout, w, 1e-6), TYPES[y])
