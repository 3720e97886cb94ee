"""Attention of drafted nodes over the cache, and the append of accepted ones,
against the fp64 oracle on a B200."""
import math

import numpy as np
import pytest
import torch

from confidence_gated_kv_logit_b200 import ALL_LAYERS, ConfKV, ConfKVError, Rope, build, logical_segment, sample, synth
from oracle.policy import ema_update
from oracle.segment import Params, append_rows, evict_compact_segment, prefill_segment
from oracle.tree import attend_nodes
from parity_util import ATOL_EMA, RTOL_EMA, c_params

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def dev_mask(mask):
    return torch.from_numpy(np.asarray(mask, np.uint64).view(np.int64)).cuda()


def tree_masks(B, N, rng, kind="tree"):
    m = np.zeros((B, N), np.uint64)
    for b in range(B):
        for i in range(N):
            bit = 1 << i
            if kind == "tree":
                m[b, i] = bit if i == 0 else int(m[b, rng.randint(max(0, i - 4), i)]) | bit
            elif kind == "chain":
                m[b, i] = 2 * bit - 1
            elif kind == "any":       # no tree at all: any bits, rows of none among them
                m[b, i] = int(rng.randint(0, 2 ** 31)) | int(rng.randint(0, 2 ** 31)) << 33 if i % 3 else 0
            else:
                m[b, i] = 2 ** 64 - 1
    return m


def drafts(lead, N, Hq, Hkv, D, g):
    q = synth.normal_fp16(tuple(lead) + (N, Hq, D), g, "cuda")
    k = synth.keys_with_heavy_hitters(tuple(lead) + (N, Hkv, D), g, "cuda")
    v = synth.normal_fp16(tuple(lead) + (N, Hkv, D), g, "cuda")
    return q, k, v


def cached(h, l, b, kv):
    """Rows the handle holds, as fp32 (codes times scale, or fp16 widened)."""
    s = logical_segment(h.export_segment(l, b, kv))
    k, v = s["k16"].astype(np.float32), s["v16"].astype(np.float32)
    i8 = ~s["is_fp16"]
    k[i8] = s["k8"][i8].astype(np.float32) * s["ks"][i8, None]
    v[i8] = s["v8"][i8].astype(np.float32) * s["vs"][i8, None]
    return k, v


def check_segment(h, out, lse, q, kd, vd, masks, counts, l, b, kv, batch_out=None):
    """One (layer, sequence, KV head) of a call over `lead` = (B,) against the oracle."""
    G, n = h.G, counts[b]
    k, v = cached(h, l, b, kv)
    m = [int(x) & ((1 << n) - 1) for x in masks[b][:n]]
    qh = q[b, :n, kv * G:kv * G + G].cpu().numpy()
    want, wl, spread, reach = attend_nodes(qh, k, v, kd[b, :n, kv].cpu().numpy(), vd[b, :n, kv].cpu().numpy(), m)
    got = out[b, :n, kv * G:kv * G + G].double().cpu().numpy()
    gl = lse[b, :n, kv * G:kv * G + G].double().cpu().numpy()
    # scores: 8 k-steps of 16 fp32 products each and the scaling, 24 roundings of the sum of magnitudes
    delta = 24 * 2.0 ** -23 * reach
    # weights: 22 bits (2^-21 allowed here), plus what an error of the score makes of them (and of their sum);
    # weights below fp16's normal range: 2^-31 of the largest value each; output: half an fp16 step
    big = float(np.abs(v).max()) if len(v) else 0.0
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -21 * spread + 2 * delta[..., None] * spread + \
        len(v) * 2.0 ** -31 * max(big, 1.0) + 2.0 ** -25
    bad = np.abs(got - want) > tol
    assert not bad.any(), (l, b, kv, float((np.abs(got - want) / tol).max()))
    fin = np.isfinite(wl)
    assert np.array_equal(fin, np.isfinite(gl))
    assert (np.abs(gl[fin] - wl[fin]) <= delta[fin] + 4e-6 + np.abs(wl[fin]) * 2.0 ** -22).all()
    assert (gl[~fin] == -np.inf).all()


def build_handle(Hkv, Hq, D, lens, g, L=1, decode=0, W=32, **kw):
    kw = dict(dict(n_low=48, n_high=96, protect_last=16, fp16_window=W, max_batch=len(lens),
                   max_prefill=max(max(lens), 1) + 80), **kw)
    h = ConfKV(L, Hkv, Hq, D, **kw)
    T = max(max(lens), 1)
    fixed = kw.get("mode") == 1
    for l in range(L):
        k, v = synth.prefill_kv(len(lens), Hkv, T, D, g, "cuda")
        pr = synth.priorities((len(lens), Hkv, T), g, "cuda") if fixed else None
        h.prefill(k, v, lens, layer=l, priority=pr)
    for _ in range(decode):
        q, kn, vn = synth.step_qkv((L, len(lens)), Hq, Hkv, D, g, "cuda")
        pn = synth.priorities((L, len(lens), Hkv), g, "cuda") if fixed else None
        h.decode_attn(q, kn, vn, torch.empty((L, len(lens), Hq, D), device="cuda"), prio_new=pn)
        h.evict_compact()
    return h


def run_tree(h, N, lens, g, kind="tree", counts=None, layer=0, seed=0, **kw):
    B = len(lens)
    q, kd, vd = drafts((B,), N, h.Hq, h.Hkv, h.D, g)
    masks = tree_masks(B, N, np.random.RandomState(seed), kind)
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, N, h.Hq), 7.0, device="cuda")
    ct = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    h.tree_attn(q, kd, vd, dev_mask(masks), out, layer=layer, counts=ct, lse_out=lse, **kw)
    counts = counts or [N] * B
    for b in range(B):
        assert (out[b, counts[b]:] == 7.0).all() and (lse[b, counts[b]:] == 7.0).all()
    return out, lse, q, kd, vd, masks, counts


@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 64), (2, 4, 128), (12, 1, 64), (2, 5, 128), (1, 8, 128), (3, 7, 64), (2, 2, 128)])
@pytest.mark.parametrize("N", [1, 2, 13, 16, 33, 64])
def test_shapes(Hkv, G, D, N):
    g = synth.generator(N * 100 + G, "cuda")
    lens = [300, 1, 129]
    h = build_handle(Hkv, Hkv * G, D, lens, g)
    r = run_tree(h, N, lens, g)
    for b in range(len(lens)):
        for kv in range(Hkv):
            check_segment(h, *r, 0, b, kv)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("kind", ["tree", "chain", "any", "all"])
@pytest.mark.parametrize("lens", [[0, 0], [1, 0], [31, 32], [33, 63], [64, 65], [127, 128], [159, 160], [161, 700]])
def test_lengths_and_masks(lens, kind):
    g = synth.generator(sum(lens) + len(kind), "cuda")
    h = build_handle(2, 4, 128, lens, g)
    r = run_tree(h, 9, lens, g, kind, counts=[9, 5])
    for b in range(2):
        for kv in range(2):
            check_segment(h, *r, 0, b, kv)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("kw", [dict(W=1), dict(W=200), dict(W=64), dict(int8_enable=0), dict(compact=1), dict(compact=2),
                                dict(mode=1, fixed_budget=100, n_sink=4, protect_last=20, int8_enable=0),
                                dict(mode=1, fixed_budget=200, protect_last=40)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("D", [64, 128])
def test_layouts_after_evictions(kw, D):
    """Caches as decoding leaves them: compacted, with a ring that has wrapped."""
    g = synth.generator(7, "cuda")
    lens = [260, 140, 5]
    h = build_handle(2, 8, D, lens, g, L=2, decode=45, **kw)
    for layer in range(2):
        r = run_tree(h, 11, lens, g, layer=layer)
        for b in range(3):
            for kv in range(2):
                check_segment(h, *r, layer, b, kv)
    assert h.last_error() == 0
    h.close()


def test_every_layer_in_one_call():
    g = synth.generator(8, "cuda")
    L, B, N, Hkv, Hq, D = 40, 2, 6, 2, 4, 64     # more segments than SMs: no split
    h = build_handle(Hkv, Hq, D, [200, 90], g, L=L)
    q, kd, vd = drafts((L, B), N, Hq, Hkv, D, g)
    masks = tree_masks(B, N, np.random.RandomState(1))
    out, lse = torch.zeros_like(q), torch.zeros((L, B, N, Hq), device="cuda")
    h.tree_attn(q, kd, vd, dev_mask(masks), out, ALL_LAYERS, lse_out=lse)
    one = torch.zeros_like(q[0])
    for l in (0, 17, 39):
        for b in range(B):
            for kv in range(Hkv):
                check_segment(h, out[l], lse[l], q[l], kd[l], vd[l], masks, [N] * B, l, b, kv)
    assert h.last_error() == 0
    h.close()


def test_long_cache_and_widest_tree():
    g = synth.generator(9, "cuda")
    lens = [9000, 4001]
    h = build_handle(1, 8, 128, lens, g, W=256)
    r = run_tree(h, 64, lens, g, counts=[64, 63])
    for b in range(2):
        check_segment(h, *r, 0, b, 0)
    h.close()


def test_extreme_scales():
    """Values from fp16's largest to its smallest next to one another, zero rows, large scores."""
    g = synth.generator(10, "cuda")
    D, T = 128, 500
    h = ConfKV(1, 1, 4, D, max_batch=1, max_prefill=T, fp16_window=16)
    k = synth.normal_fp16((1, 1, T, D), g, "cuda")
    v = synth.normal_fp16((1, 1, T, D), g, "cuda")
    v[0, 0, 10] = 0.0
    k[0, 0, 20] = 0.0
    v[0, 0, 30:60] *= 1e-3
    v[0, 0, 60:80] *= 2.0 ** -20
    v[0, 0, 200:210] *= 3000.0
    k[0, 0, 300] *= 30.0
    h.prefill(k, v, [T], layer=0)
    r = run_tree(h, 12, [T], g)
    check_segment(h, *r, 0, 0, 0)
    h.close()


def test_values_of_unseen_nodes_stay_out():
    g = synth.generator(11, "cuda")
    h = build_handle(2, 4, 128, [100, 3], g)
    N = 8
    q, kd, vd = drafts((2,), N, 4, 2, 128, g)
    masks = tree_masks(2, N, np.random.RandomState(3))
    masks[:] = [[1, 3, 5, 9, 1 | 16, 1 | 32, 1 | 64, 129]] * 2       # a root and its children
    ct = torch.tensor([8, 5], dtype=torch.int32, device="cuda")
    clean = torch.zeros_like(q)
    h.tree_attn(q, kd, vd, dev_mask(masks), clean, 0, counts=ct)
    kd2, vd2 = kd.clone(), vd.clone()
    vd2[0, 3] = math.inf
    vd2[0, 5, :, 7] = math.nan
    kd2[0, 6] = math.nan
    kd2[1, 5:] = math.nan                                            # past the count
    vd2[1, 5:] = -math.inf
    out = torch.zeros_like(q)
    h.tree_attn(q, kd2, vd2, dev_mask(masks), out, 0, counts=ct)
    for i in (0, 1, 2, 4, 7):
        assert torch.equal(out[0, i], clean[0, i]), i
    assert torch.equal(out[1], clean[1])
    assert torch.isinf(out[0, 3]).all()
    assert torch.isnan(out[0, 5, :, 7]).all() and torch.equal(out[0, 5, :, :7], clean[0, 5, :, :7])
    assert torch.isnan(out[0, 6]).all()
    h.close()


def test_agrees_with_decode_attention():
    g = synth.generator(12, "cuda")
    B, Hkv, Hq, D = 3, 2, 8, 128
    h = build_handle(Hkv, Hq, D, [400, 77, 1], g)
    q, kn, vn = synth.step_qkv((1, B), Hq, Hkv, D, g, "cuda")
    tree = torch.zeros((B, 1, Hq, D), dtype=torch.float16, device="cuda")
    h.tree_attn(q[0][:, None], kn[0][:, None], vn[0][:, None], torch.ones((B, 1), dtype=torch.int64, device="cuda"), tree, 0)
    out = torch.zeros((1, B, Hq, D), device="cuda")
    h.decode_attn(q, kn, vn, out)
    # two roundings of 2^-11 (weights, output) of values of order 1, and decode attention's own 2e-3 bound
    assert (tree[:, 0].float() - out[0]).abs().max().item() <= 2e-3 + 2 * 2.0 ** -11 * 4
    h.close()


@pytest.mark.parametrize("single", [0, 1])
@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("B,L", [(3, 1), (2, 90)])
def test_root_attention_updates_the_ema(single, score, B, L):
    """The root's attention mass equals that of decode attention with the same token."""
    Hkv, Hq, D, lens = 2, 8, 128, [300, 41, 0][:B]
    kw = dict(single_stream=single, score_source=score, seed=5)
    ha = build_handle(Hkv, Hq, D, lens, synth.generator(13, "cuda"), L=L, decode=5, **kw)
    hb = build_handle(Hkv, Hq, D, lens, synth.generator(13, "cuda"), L=L, decode=5, **kw)
    g = synth.generator(14, "cuda")
    q, kd, vd = drafts((L, B), 5, Hq, Hkv, D, g)
    masks = tree_masks(B, 5, np.random.RandomState(4))
    ha.decode_attn(q[:, :, 0].contiguous(), kd[:, :, 0].contiguous(), vd[:, :, 0].contiguous(),
                   torch.empty((L, B, Hq, D), device="cuda"))
    hb.tree_attn(q, kd, vd, dev_mask(masks), torch.empty_like(q), track=True)
    hb.append(kd, vd, index=torch.zeros((B, 1), dtype=torch.int32, device="cuda"))
    for l in (0, L - 1):
        for b in range(B):
            for kv in range(Hkv):
                a, t = (logical_segment(h.export_segment(l, b, kv)) for h in (ha, hb))
                for key in ("pos", "is_fp16", "k8", "v8", "ks", "vs", "k16", "v16", "next_pos"):
                    assert np.array_equal(a[key], t[key]), key
                # the new token: decode attention counts its own mass, an appended one starts at its initial score
                np.testing.assert_allclose(t["score_src"][:-1], a["score_src"][:-1], rtol=2 * RTOL_EMA, atol=ATOL_EMA)
    assert ha.last_error() == 0 and hb.last_error() == 0
    ha.close()
    hb.close()


def test_a_sequence_without_nodes_gives_mass_zero():
    g = synth.generator(15, "cuda")
    h = build_handle(1, 4, 64, [90, 90], g, decode=3)
    before = [logical_segment(h.export_segment(0, b, 0))["score_src"] for b in range(2)]
    q, kd, vd = drafts((1, 2), 3, 4, 1, 64, g)
    out = torch.full_like(q, 7.0)
    h.tree_attn(q, kd, vd, dev_mask([[1, 3, 7]] * 2), out, counts=torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                track=True)
    after = [logical_segment(h.export_segment(0, b, 0))["score_src"] for b in range(2)]
    np.testing.assert_array_equal(after[0], (np.float32(0.9) * before[0]).astype(np.float32))
    assert not np.array_equal(after[1], (np.float32(0.9) * before[1]).astype(np.float32))
    assert (out[0, 0] == 7.0).all()
    h.close()


MODES = [dict(), dict(fp16_window=1), dict(fp16_window=3), dict(int8=False), dict(score_source="random", seed=9),
         dict(mode="fixed", fixed_budget=500, protect_last=20, n_sink=2)]


@pytest.mark.parametrize("pkw", MODES, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "default")
@pytest.mark.parametrize("compact", ["hole-fill", "linear"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_matches_the_oracle(pkw, compact, D):
    p = Params(**dict(dict(n_low=40, n_high=80, protect_last=10, fp16_window=16), **pkw))
    if compact == "linear" and (p.mode == "fixed" or not p.int8):
        pytest.skip("the linear window needs confidence mode and INT8")
    g = synth.generator(16, "cuda")
    lens, Hkv, rows, fixed = [60, 7, 0], 2, 24, p.mode == "fixed"
    h = ConfKV(1, Hkv, 4, D, **c_params(p, 3, 200, compact=compact))
    k, v = synth.prefill_kv(3, Hkv, 60, D, g, "cuda")
    pr = synth.priorities((3, Hkv, 60), g, "cuda") if fixed else None
    h.prefill(k, v, lens, layer=0, priority=pr)
    segs = {(b, kv): prefill_segment(k[b, kv, :n].cpu().numpy(), v[b, kv, :n].cpu().numpy(),
                                     pr[b, kv, :n].cpu().numpy() if fixed else None, p, (0, b, kv))
            for b, n in enumerate(lens) for kv in range(Hkv)}
    rng = np.random.RandomState(5)
    for step in range(4):
        _, kd, vd = drafts((3,), rows, 4, Hkv, D, g)
        pn = synth.priorities((3, rows, Hkv), g, "cuda") if fixed else None
        if step == 0:      # every row, in order
            index, counts = None, [rows] * 3
            h.append(kd, vd, layer=0, prio=pn)
        else:              # a list with repeats, and counts of its own
            index = rng.randint(0, rows, (3, 20)).astype(np.int32)
            counts = [20, 0, int(rng.randint(1, 20))]
            h.append(kd, vd, layer=0, index=torch.from_numpy(index).cuda(), prio=pn,
                     counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
        for b in range(3):
            at = np.arange(rows) if index is None else index[b, :counts[b]]
            for kv in range(Hkv):
                append_rows(segs[b, kv], kd[b, :, kv].cpu().numpy()[at], vd[b, :, kv].cpu().numpy()[at],
                            pn[b, :, kv].cpu().numpy()[at] if fixed else None, p)
                got, want = logical_segment(h.export_segment(0, b, kv)), segs[b, kv]
                assert np.array_equal(got["pos"], want.pos) and got["next_pos"] == want.next_pos
                for key in ("is_fp16", "k8", "v8", "ks", "vs", "k16", "v16"):
                    assert np.array_equal(got[key], getattr(want, key)), (step, b, kv, key)
                assert np.array_equal(got["score_src"], want.score_src)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("pkw,compact", [(dict(), "hole-fill"), (dict(), "stable"), (dict(), "linear"),
                                         (dict(int8=False), "hole-fill"),
                                         (dict(mode="fixed", fixed_budget=100, protect_last=20, n_sink=3), "hole-fill")])
def test_eviction_after_many_appended_tokens(pkw, compact):
    """More victims at once than a step's, with no attention in between: kept sets equal the oracle's."""
    p = Params(**dict(dict(n_low=60, n_high=60, protect_last=10, fp16_window=16), **pkw))
    g = synth.generator(30, "cuda")
    lens, Hkv, D, fixed = [90, 31], 2, 64, p.mode == "fixed"
    h = ConfKV(1, Hkv, 2, D, **c_params(p, 2, 200, compact=compact))
    k, v = synth.prefill_kv(2, Hkv, 90, D, g, "cuda")
    pr = synth.priorities((2, Hkv, 90), g, "cuda") if fixed else None
    h.prefill(k, v, lens, layer=0, priority=pr)
    segs = {(b, kv): prefill_segment(k[b, kv, :n].cpu().numpy(), v[b, kv, :n].cpu().numpy(),
                                     pr[b, kv, :n].cpu().numpy() if fixed else None, p, (0, b, kv))
            for b, n in enumerate(lens) for kv in range(Hkv)}
    for rows in (3, 25, 1, 40 if not fixed else 20):
        _, kd, vd = drafts((2,), rows, 2, Hkv, D, g)
        pn = synth.priorities((2, rows, Hkv), g, "cuda") if fixed else None
        h.append(kd, vd, layer=0, prio=pn)
        h.evict_compact()
        for (b, kv), seg in segs.items():
            append_rows(seg, kd[b, :, kv].cpu().numpy(), vd[b, :, kv].cpu().numpy(),
                        pn[b, :, kv].cpu().numpy() if fixed else None, p)
            segs[b, kv] = seg = evict_compact_segment(seg, 60, p)
            got = logical_segment(h.export_segment(0, b, kv))
            for key in ("pos", "is_fp16", "k8", "v8", "ks", "vs", "k16", "v16", "score_src", "next_pos"):
                assert np.array_equal(got[key], getattr(seg, key)), (rows, b, kv, key)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("compact", ["hole-fill", "stable", "linear"])
def test_drafted_steps_match_the_oracle(compact):
    """The whole step with drafts: norm and rotation, tree attention with the
    root tracked, sampling at the nodes, append of the accepted path, confidence
    and eviction; kept sets and contents equal the oracle's, step by step."""
    g = synth.generator(17, "cuda")
    B, Hkv, Hq, D, N, V = 2, 2, 8, 128, 6, 3001
    p = Params(n_low=60, n_high=120, protect_last=12, fp16_window=20)
    lens = [150, 64]
    h = ConfKV(1, Hkv, Hq, D, **c_params(p, B, 220, compact=compact))
    k, v = synth.prefill_kv(B, Hkv, 150, D, g, "cuda")
    h.prefill(k, v, lens, layer=0)
    segs = {(b, kv): prefill_segment(k[b, kv, :n].cpu().numpy(), v[b, kv, :n].cpu().numpy(), None, p, (0, b, kv))
            for b, n in enumerate(lens) for kv in range(Hkv)}
    rope = Rope(D, theta=10000.0)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    chain = [[(2 << i) - 1 for i in range(N)]] * B
    mask = dev_mask(chain)
    index = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1)
    out_len = torch.tensor(lens, device="cuda", dtype=torch.int32)
    for step in range(12):
        raw_q, raw_k, vd = drafts((B,), N, Hq, Hkv, D, g)
        q, kd = torch.empty_like(raw_q), torch.empty_like(raw_k)
        pos = out_len[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)[None]
        rope.apply(raw_q, raw_k, pos, q, kd, q_weight=w, k_weight=w)
        out = torch.empty_like(q)
        lse = torch.empty((B, N, Hq), device="cuda")
        h.tree_attn(q, kd, vd, mask, out, layer=0, lse_out=lse, track=True)
        logits = synth.bursty_logits(B * N, V, g, "cuda")
        token = torch.empty(B * N, dtype=torch.int32, device="cuda")
        sample(logits, torch.rand(B * N, generator=g, device="cuda"), token,
               top_k=torch.full((B * N,), 40, dtype=torch.int32, device="cuda"))
        assert ((token >= 0) & (token < V)).all()
        taken = (1 + token.view(B, N)[:, 0] % N).int()       # how far this draft is accepted
        h.append(kd, vd, layer=0, index=index, counts=taken)
        budget = torch.empty((B, 1), dtype=torch.int32, device="cuda")
        h.confidence(logits.view(B, N, V)[:, 0].contiguous(), budget_out=budget)
        for b in range(B):
            n = int(taken[b])
            for kv in range(Hkv):
                seg = segs[b, kv]
                kh, vh = seg.rows_hat()
                want, wl, spread, reach = attend_nodes(
                    q[b, :, kv * 4:kv * 4 + 4].cpu().numpy(), kh, vh, kd[b, :, kv].cpu().numpy(),
                    vd[b, :, kv].cpu().numpy(), chain[b])
                got = out[b, :, kv * 4:kv * 4 + 4].double().cpu().numpy()
                delta = 24 * 2.0 ** -23 * reach[..., None]
                assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -21 * spread + 2 * delta * spread + 1e-6).all()
                append_rows(seg, kd[b, :n, kv].cpu().numpy(), vd[b, :n, kv].cpu().numpy(), None, p)
                got = logical_segment(h.export_segment(0, b, kv))
                # the root's mass, against the GPU's own (step-synchronised from here on)
                m = np.exp(np.einsum("gd,td->gt", q[b, 0, kv * 4:kv * 4 + 4].double().cpu().numpy(), kh.astype(np.float64)) /
                           math.sqrt(D) - wl[0][:, None]).mean(0)
                np.testing.assert_allclose(got["score_src"][:len(kh)],
                                           0.9 * seg.score_src[:len(kh)].astype(np.float64) + 0.1 * m,
                                           rtol=RTOL_EMA, atol=ATOL_EMA)
                assert np.array_equal(got["pos"], seg.pos)
                seg.score_src = got["score_src"].copy()
        h.evict_compact()
        for b in range(B):
            for kv in range(Hkv):
                segs[b, kv] = evict_compact_segment(segs[b, kv], int(budget[b, 0]), p)
                got, want = logical_segment(h.export_segment(0, b, kv)), segs[b, kv]
                assert np.array_equal(got["pos"], want.pos), (step, b, kv)
                for key in ("is_fp16", "k8", "v8", "ks", "vs", "k16", "v16", "score_src"):
                    assert np.array_equal(got[key], getattr(want, key)), (step, b, kv, key)
        out_len = out_len + taken
    assert h.last_error() == 0
    h.close()


def test_a_deferred_pass_is_applied_first():
    """Decode attention's deferred EMA pass and a tree call after it, whichever scratch the tree uses."""
    for track in (False, True):
        segs = []
        for tree in (False, True):
            g = synth.generator(18, "cuda")
            h = build_handle(2, 4, 64, [200], g, L=2, decode=2)
            q, kn, vn = synth.step_qkv((2, 1), 4, 2, 64, g, "cuda")
            h.decode_attn(q, kn, vn, torch.empty((2, 1, 4, 64), device="cuda"))
            if tree:
                qd, kd, vd = drafts((1,), 4, 4, 2, 64, g)
                h.tree_attn(qd, kd, vd, dev_mask([[1, 3, 7, 15]]), torch.empty_like(qd), layer=0, track=track)
            segs.append([logical_segment(h.export_segment(l, 0, kv))["score_src"] for l in range(2) for kv in range(2)])
            h.close()
        for i, (a, b) in enumerate(zip(*segs)):
            if track and i < 2:
                assert not np.array_equal(a, b)
            else:
                assert np.array_equal(a, b)


def test_captured_steps_replay():
    """Tree attention with tracking and append inside one graph, and a second graph of the same handle."""
    g = synth.generator(19, "cuda")
    kw = dict(single_stream=1)
    hs = [build_handle(2, 8, 128, [200, 90], synth.generator(20, "cuda"), **kw) for _ in range(2)]
    B, N = 2, 4
    q, kd, vd = drafts((B,), N, 8, 2, 128, g)
    mask = dev_mask([[1, 3, 7, 15]] * 2)
    idx = torch.tensor([[0, 1], [0, 2]], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def step(h, out):
        h.tree_attn(q, kd, vd, mask, out, layer=0, track=True)
        h.append(kd, vd, layer=0, index=idx)
        h.evict_compact()

    step(hs[1], outs[1])
    step(hs[0], outs[0])
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(hs[0], outs[0])
        graphs.append(gr)
    for k in range(4):
        q.copy_(synth.normal_fp16(q.shape, g, "cuda"))
        graphs[k % 2].replay()
        step(hs[1], outs[1])
        assert torch.equal(outs[0], outs[1]), k
    torch.cuda.synchronize()
    for b in range(2):
        for kv in range(2):
            ea, eb = (logical_segment(h.export_segment(0, b, kv)) for h in hs)
            assert all(np.array_equal(ea[key], eb[key]) for key in ("pos", "score_src", "k8", "v8", "k16", "v16"))
    assert hs[0].last_error() == 0
    del graphs
    for h in hs:
        h.close()


def test_another_stream_and_the_same_bits_twice():
    g = synth.generator(21, "cuda")
    h = build_handle(2, 8, 128, [900], g)
    a = run_tree(h, 7, [900], synth.generator(22, "cuda"))
    out, mask = [torch.zeros_like(a[0]) for _ in range(2)], dev_mask(a[5])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    h.tree_attn(a[2], a[3], a[4], mask, out[0], 0, stream=st)
    st.synchronize()
    h.tree_attn(a[2], a[3], a[4], mask, out[1], 0)
    assert torch.equal(a[0], out[0]) and torch.equal(a[0], out[1])
    h.close()


def test_split_partials_in_the_score_area():
    """Long caches of many heads keep the splits' partials where decode attention
    keeps its scores; a deferred EMA pass has read those first."""
    g = synth.generator(24, "cuda")
    B, Hkv, Hq, D, lens = 8, 8, 32, 128, [9000, 8000, 10, 5000, 9000, 1, 0, 300]
    hs = [build_handle(Hkv, Hq, D, lens, synth.generator(25, "cuda")) for _ in range(2)]
    q, kn, vn = synth.step_qkv((1, B), Hq, Hkv, D, g, "cuda")
    for h in hs:
        h.decode_attn(q, kn, vn, torch.empty((1, B, Hq, D), device="cuda"))
    r = run_tree(hs[0], 16, lens, g)
    for b, kv in ((0, 0), (3, 7), (5, 1), (6, 2)):
        check_segment(hs[0], *r, 0, b, kv)
        a, t = (logical_segment(h.export_segment(0, b, kv)) for h in hs)
        assert np.array_equal(a["score_src"], t["score_src"])
    assert hs[0].last_error() == 0
    for h in hs:
        h.close()


def test_refusals():
    g = synth.generator(23, "cuda")
    D, B = 64, 2
    h = ConfKV(2, 2, 4, D, max_batch=B, max_prefill=100, n_low=32, n_high=64)
    q, kd, vd = drafts((B,), 4, 4, 2, D, g)
    mask, out = dev_mask([[1, 3, 7, 15]] * 2), torch.empty_like(q)

    def refused(status, f, *args, **kw):
        with pytest.raises(ConfKVError) as e:
            f(*args, **kw)
        assert e.value.status == status

    h.batch = B
    refused(3, h.tree_attn, q, kd, vd, mask, out, layer=0)            # before prefill
    refused(3, h.append, kd, vd, layer=0)
    k, v = synth.prefill_kv(B, 2, 100, D, g, "cuda")
    h.prefill(k, v, [100, 100], layer=0)
    refused(3, h.tree_attn, q, kd, vd, mask, out, layer=1)
    refused(1, h.tree_attn, q, kd, vd, mask, out, layer=2)
    big = drafts((B,), 65, 4, 2, D, g)
    refused(1, h.tree_attn, *big, torch.zeros((B, 65), dtype=torch.int64, device="cuda"), torch.empty_like(big[0]), layer=0)
    refused(1, h.append, kd, vd, layer=0, prio=torch.zeros((B, 4, 2), device="cuda"))
    refused(2, h.append, *big[1:], layer=0)                           # 165 tokens in a cache of 128 rows
    for bad in (dict(q=q.float()), dict(k=kd[:, :3].contiguous()), dict(v=None), dict(mask=mask[:1]), dict(mask=mask.int()),
                dict(out=out.float()), dict(counts=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(q=q.transpose(1, 2)),
                dict(lse_out=torch.zeros((B, 4, 2), device="cuda")), dict(q=q.cpu())):
        args = dict(dict(q=q, k=kd, v=vd, mask=mask, out=out), **bad)
        with pytest.raises((TypeError, ValueError)):
            h.tree_attn(layer=0, **args)
    assert h.last_error() == 0
    before = [logical_segment(h.export_segment(0, b, kv)) for b in range(B) for kv in range(2)]
    # what only the device sees: counts and rows out of range leave their sequence as it was
    out.fill_(7.0)
    h.tree_attn(q, kd, vd, mask, out, layer=0, counts=torch.tensor([5, 4], dtype=torch.int32, device="cuda"))
    assert h.last_error_detail()[:2] == (7, 207) and h.last_error(clear=True) == 7
    assert (out[0] == 7.0).all() and torch.isfinite(out[1]).all() and not (out[1] == 7.0).all()
    h.append(kd, vd, layer=0, index=torch.tensor([[0, 4], [0, -1]], dtype=torch.int32, device="cuda"))
    assert h.last_error_detail()[:2] == (7, 104) and h.last_error(clear=True) == 7
    h.append(kd, vd, layer=0, counts=torch.tensor([-1, 5], dtype=torch.int32, device="cuda"))
    assert h.last_error_detail()[:2] == (7, 103) and h.last_error(clear=True) == 7
    for want, (b, kv) in zip(before, [(b, kv) for b in range(B) for kv in range(2)]):
        got = logical_segment(h.export_segment(0, b, kv))
        assert all(np.array_equal(want[key], got[key]) for key in ("pos", "k8", "k16", "score_src", "next_pos"))
    h.close()
    hf = ConfKV(1, 2, 4, D, max_batch=1, max_prefill=64, mode=1, fixed_budget=40, protect_last=8)
    k, v = synth.prefill_kv(1, 2, 64, D, g, "cuda")
    hf.prefill(k, v, [64], layer=0, priority=synth.priorities((1, 2, 64), g, "cuda"))
    refused(1, hf.tree_attn, q[:1], kd[:1], vd[:1], mask[:1], out[:1], layer=0, track=True)
    refused(1, hf.append, kd[:1], vd[:1], layer=0)
    hf.close()


@pytest.mark.parametrize("budget", [62, 100, 126, 1022])
@pytest.mark.parametrize("int8", [0, 1])
def test_fixed_budgets_have_room_for_the_widest_draft(budget, int8):
    """Fixed mode: a cache at its budget takes CONFKV_MAX_NODES tokens, and eviction brings it back."""
    p = Params(mode="fixed", fixed_budget=budget, protect_last=20, n_sink=3, fp16_window=16, int8=bool(int8))
    g = synth.generator(40, "cuda")
    Hkv, D, T, N = 2, 64, budget + 30, 64
    h = ConfKV(1, Hkv, 2, D, **c_params(p, 2, T))
    k, v = synth.prefill_kv(2, Hkv, T, D, g, "cuda")
    pr = synth.priorities((2, Hkv, T), g, "cuda")
    h.prefill(k, v, [T, T], layer=0, priority=pr)
    segs = {(b, kv): prefill_segment(k[b, kv].cpu().numpy(), v[b, kv].cpu().numpy(), pr[b, kv].cpu().numpy(), p, (0, b, kv))
            for b in range(2) for kv in range(Hkv)}
    for counts in ([N, N], [1, 33]):
        _, kd, vd = drafts((2,), N, 2, Hkv, D, g)
        pn = synth.priorities((2, N, Hkv), g, "cuda")
        h.append(kd, vd, layer=0, prio=pn, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
        h.evict_compact()
        for (b, kv), seg in segs.items():
            n = counts[b]
            append_rows(seg, kd[b, :n, kv].cpu().numpy(), vd[b, :n, kv].cpu().numpy(), pn[b, :n, kv].cpu().numpy(), p)
            segs[b, kv] = seg = evict_compact_segment(seg, budget, p)
            got = logical_segment(h.export_segment(0, b, kv))
            for key in ("pos", "is_fp16", "k8", "v8", "ks", "vs", "k16", "v16", "score_src", "next_pos"):
                assert np.array_equal(got[key], getattr(seg, key)), (counts, b, kv, key)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("single", [0, 1])
@pytest.mark.parametrize("Hq,N,lens", [(8, 8, [300, 41, 0]),          # 32 rows per KV head: the last of the small kernel
                                       (8, 9, [300, 41, 0]),          # 36 rows: the first of the other
                                       (8, 40, [300, 41, 700]),       # 160: each softmax group has rows of its own
                                       (16, 64, [90, 500, 1]),        # 512: two row tiles
                                       (2, 64, [9000, 20, 4100])])    # 64, over many splits
def test_tracked_roots_of_wide_trees(single, Hq, N, lens):
    """The root's mass on both sides of the kernels' border, for counts from 0 to all, against decode attention."""
    Hkv, D, B = 2, 128, 3
    for counts in ([N, 1, max(2, N - 3)], [0, N, 1]):
        ha, hb = (build_handle(Hkv, Hq, D, lens, synth.generator(41, "cuda"), decode=5, single_stream=single) for _ in range(2))
        g = synth.generator(42, "cuda")
        before = [logical_segment(hb.export_segment(0, 0, kv))["score_src"] for kv in range(Hkv)]
        q, kd, vd = drafts((1, B), N, Hq, Hkv, D, g)
        masks = tree_masks(B, N, np.random.RandomState(4))
        out, lse = torch.full_like(q, 7.0), torch.full((1, B, N, Hq), 7.0, device="cuda")
        rows = [[cached(hb, 0, b, kv) for kv in range(Hkv)] for b in range(B)]
        ct = torch.tensor(counts, dtype=torch.int32, device="cuda")
        hb.tree_attn(q, kd, vd, dev_mask(masks), out, counts=ct, lse_out=lse, track=True)
        for b in range(B):
            if counts[b] == 0:
                continue
            for kv in range(Hkv):
                G, (k, v) = Hq // Hkv, rows[b][kv]
                want, wl, spread, reach = attend_nodes(
                    q[0, b, :1, kv * G:kv * G + G].cpu().numpy(), k, v, kd[0, b, :1, kv].cpu().numpy(),
                    vd[0, b, :1, kv].cpu().numpy(), [1])
                got = out[0, b, 0, kv * G:kv * G + G].double().cpu().numpy()
                delta = 24 * 2.0 ** -23 * reach[0][:, None]       # as in check_segment
                big = float(np.abs(v).max()) if len(v) else 0.0
                tol = 2.0 ** -11 * np.abs(want[0]) + 2.0 ** -21 * spread[0] + 2 * delta * spread[0] + \
                    len(v) * 2.0 ** -31 * max(big, 1.0) + 2.0 ** -25
                assert (np.abs(got - want[0]) <= tol).all()
        for b in range(B):
            assert (out[0, b, counts[b]:] == 7.0).all() and (lse[0, b, counts[b]:] == 7.0).all()
        ha.decode_attn(q[:, :, 0].contiguous(), kd[:, :, 0].contiguous(), vd[:, :, 0].contiguous(),
                       torch.empty((1, B, Hq, D), device="cuda"))
        hb.append(kd, vd, index=torch.zeros((B, 1), dtype=torch.int32, device="cuda"))
        for b in range(B):
            for kv in range(Hkv):
                a, t = (logical_segment(h.export_segment(0, b, kv)) for h in (ha, hb))
                assert np.array_equal(a["pos"], t["pos"])
                if counts[b]:
                    np.testing.assert_allclose(t["score_src"][:-1], a["score_src"][:-1], rtol=2 * RTOL_EMA, atol=ATOL_EMA)
                else:          # no node, no mass
                    np.testing.assert_array_equal(t["score_src"][:-1], (np.float32(0.9) * before[kv]).astype(np.float32))
        assert ha.last_error() == 0 and hb.last_error() == 0
        ha.close()
        hb.close()


@pytest.mark.parametrize("N,G,kw", [(8, 4, {}), (9, 4, {}), (33, 2, {}), (33, 8, {}), (64, 8, {}), (12, 8, dict(int8_enable=0)),
                                    (40, 4, dict(int8_enable=0)), (4, 4, dict(int8_enable=0))])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_unseen_nodes_stay_out_of_every_kernel(N, G, kw, D):
    """NaN and inf of a node's key and value, and of rows past the count, on both sides of the kernels' border and
    in the second tile of rows; a count out of range beside it."""
    g = synth.generator(43, "cuda")
    h = build_handle(2, 2 * G, D, [300, 3, 40], g, **kw)
    q, kd, vd = drafts((3,), N, 2 * G, 2, D, g)
    masks = np.zeros((3, N), np.uint64)
    for i in range(N):
        masks[:, i] = 1 | 1 << i                                     # a root and its children
    ct = torch.tensor([N, N - 2, N], dtype=torch.int32, device="cuda")
    clean = torch.full_like(q, 7.0)
    h.tree_attn(q, kd, vd, dev_mask(masks), clean, 0, counts=ct)
    assert torch.isfinite(clean).all()
    kd2, vd2 = kd.clone(), vd.clone()
    vd2[0, 1] = math.inf
    vd2[0, 2, :, 7] = math.nan
    kd2[0, N - 1] = math.nan
    vd2[0, 3, :, 5] = -math.inf
    kd2[1, N - 2:] = math.nan                                        # past the count
    vd2[1, N - 2:] = -math.inf
    out, lse = torch.full_like(q, 7.0), torch.full((3, N, 2 * G), 7.0, device="cuda")
    ct[2] = N + 1
    h.tree_attn(q, kd2, vd2, dev_mask(masks), out, 0, counts=ct, lse_out=lse)
    for i in range(N):
        if i not in (1, 2, 3, N - 1):
            assert torch.equal(out[0, i], clean[0, i]), i
    assert torch.equal(out[1], clean[1])
    assert (out[0, 1] == math.inf).all()
    assert torch.isnan(out[0, 2, :, 7]).all() and torch.equal(out[0, 2, :, :7], clean[0, 2, :, :7])
    if N > 4:                                                        # (else node 3 is the one whose key is NaN)
        assert (out[0, 3, :, 5] == -math.inf).all() and torch.equal(out[0, 3, :, 6:], clean[0, 3, :, 6:])
    assert torch.isnan(out[0, N - 1]).all() and torch.isnan(lse[0, N - 1]).all()
    assert torch.isfinite(lse[0, :N - 1]).all()
    assert (out[2] == 7.0).all() and (lse[2] == 7.0).all()
    assert h.last_error_detail()[:2] == (7, 207) and h.last_error(clear=True) == 7
    h.close()


@pytest.mark.parametrize("kw", [dict(W=1), dict(W=200), dict(W=64), dict(int8_enable=0), dict(compact=1), dict(compact=2),
                                dict(mode=1, fixed_budget=100, n_sink=4, protect_last=20, int8_enable=0),
                                dict(mode=1, fixed_budget=200, protect_last=40)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N", [3, 8, 80])
def test_layouts_after_evictions_of_every_width(kw, D, N):
    """Caches as decoding leaves them: few rows per KV head, as many as the small kernel takes, and both row tiles."""
    g = synth.generator(44, "cuda")
    lens, Hq = [260, 140, 5], 8
    if N == 80:
        N, Hq = 40, 16
    h = build_handle(2, Hq, D, lens, g, decode=45, **kw)
    r = run_tree(h, N, lens, g, counts=[N, N - 1, 1])
    for b in range(3):
        for kv in range(2):
            check_segment(h, *r, 0, b, kv)
    assert h.last_error() == 0
    h.close()


@pytest.mark.parametrize("single", [0, 1])
@pytest.mark.parametrize("compact", [0, 1, 2])
@pytest.mark.parametrize("N", [4, 20])
def test_eviction_right_after_a_tracked_tree(single, compact, N):
    """A draft of which nothing is accepted: the deferred pass goes into the eviction, or runs before it."""
    kw = dict(single_stream=single, compact=compact, n_low=40, n_high=40, protect_last=8)
    hs = [build_handle(2, 8, 64, [300, 45], synth.generator(45, "cuda"), **kw) for _ in range(2)]
    for step in range(3):
        g = synth.generator(46 + step, "cuda")
        q, kd, vd = drafts((1, 2), N, 8, 2, 64, g)
        mask = dev_mask(tree_masks(2, N, np.random.RandomState(step)))
        for i, h in enumerate(hs):
            h.tree_attn(q, kd, vd, mask, torch.empty_like(q), track=True)
            if i:
                h.query()                                            # applies the deferred pass on its own
            if step:
                h.append(kd, vd, index=torch.zeros((2, 1), dtype=torch.int32, device="cuda"),
                         counts=torch.zeros(2, dtype=torch.int32, device="cuda"))
            h.evict_compact()
        for b in range(2):
            for kv in range(2):
                x, y = (logical_segment(h.export_segment(0, b, kv)) for h in hs)
                for key in ("pos", "is_fp16", "k8", "v8", "ks", "vs", "k16", "v16", "score_src", "next_pos"):
                    assert np.array_equal(x[key], y[key]), (step, b, kv, key)
        assert len(x["pos"]) == 40
    assert all(h.last_error() == 0 for h in hs)
    for h in hs:
        h.close()


@pytest.mark.parametrize("D,G", [(64, 1), (128, 1), (128, 8)])
def test_a_small_handle_stays_small(D, G):
    """Tree attention's partials share decode attention's buffer, and a handle whose caches need few holds few."""
    h = ConfKV(1, 1, G, D, n_low=32, n_high=64, max_prefill=60)
    # decode attention's 4096 units; the cache, its scratch and its metadata are below 4 MB
    assert h.query()["bytes_capacity"] <= 4096 * G * (D + 2) * 4 + (4 << 20)
    h.close()


@pytest.mark.parametrize("kw", [dict(), dict(compact=2), dict(int8_enable=0), dict(W=1), dict(W=30)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "default")
def test_a_full_cache_takes_none_of_a_list(kw):
    """Replays of a captured append go on past the host's bound: a sequence whose list no longer fits gets none of
    it (not the part that would), sets the device word, and the other goes on."""
    g = synth.generator(47, "cuda")
    n = 20
    h = build_handle(2, 4, 64, [100, 10], g, **dict(dict(W=16, single_stream=1, n_low=32, n_high=32, max_prefill=100), **kw))
    W = 0 if kw.get("int8_enable") == 0 else kw.get("W", 16)
    _, kd, vd = drafts((2,), n, 4, 2, 64, g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.append(kd, vd, layer=0)
    lens, cap, refused = [100, 10], 128, 0
    for _ in range(4):
        before = [logical_segment(h.export_segment(0, b, kv)) for b in range(2) for kv in range(2)]
        graph.replay()
        torch.cuda.synchronize()
        fits = [x + n - W <= cap for x in lens]       # rows outside the window
        refused += not all(fits)
        assert h.last_error(clear=True) == (0 if all(fits) else 7)
        lens = [x + n if f else x for x, f in zip(lens, fits)]
        for i, was in enumerate(before):
            now = logical_segment(h.export_segment(0, i // 2, i % 2))
            assert len(now["pos"]) == now["next_pos"] == lens[i // 2]
            if not fits[i // 2]:
                assert all(np.array_equal(was[key], now[key]) for key in was)
    assert refused
    h.close()


@pytest.mark.parametrize("N,Hq", [(3, 4), (40, 8)])
def test_fewer_sequences_than_the_handle_is_sized_for(N, Hq):
    """Three sequences in a handle of five, every layer in one call: drafts, roots and appends as in a handle of three."""
    L, B, Hkv, D, lens = 2, 3, 2, 64, [200, 31, 90]
    hs = [build_handle(Hkv, Hq, D, lens, synth.generator(50, "cuda"), L=L, decode=3, max_batch=m) for m in (3, 5)]
    g = synth.generator(51, "cuda")
    q, kd, vd = drafts((L, B), N, Hq, Hkv, D, g)
    mask = dev_mask(tree_masks(B, N, np.random.RandomState(6)))
    counts = torch.tensor([N, 1, N - 1], dtype=torch.int32, device="cuda")
    index = torch.tensor([[0, N - 1], [0, 0], [1, 0]], dtype=torch.int32, device="cuda")
    outs = []
    for h in hs:
        outs.append((torch.full_like(q, 7.0), torch.full((L, B, N, Hq), 7.0, device="cuda")))
        h.tree_attn(q, kd, vd, mask, outs[-1][0], counts=counts, lse_out=outs[-1][1], track=True)
        h.append(kd, vd, index=index, counts=torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"))
        h.evict_compact()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    for l in range(L):
        for b in range(B):
            for kv in range(Hkv):
                x, y = (logical_segment(h.export_segment(l, b, kv)) for h in hs)
                assert all(np.array_equal(x[key], y[key]) for key in x)
    assert all(h.last_error() == 0 for h in hs)
    for h in hs:
        h.close()


@pytest.mark.parametrize("N,Hq", [(6, 8), (20, 8), (64, 16)])
def test_queries_that_are_not_finite_stay_in_their_rows(N, Hq):
    g = synth.generator(52, "cuda")
    lens = [300, 20]
    h = build_handle(2, Hq, 128, lens, g)
    q, kd, vd = drafts((2,), N, Hq, 2, 128, g)
    masks = tree_masks(2, N, np.random.RandomState(7))
    q2 = q.clone()
    q2[0, 1, 0] = math.nan
    q2[1, 4, Hq - 1, 3] = math.inf
    out, lse = torch.full_like(q, 7.0), torch.full((2, N, Hq), 7.0, device="cuda")
    h.tree_attn(q2, kd, vd, dev_mask(masks), out, 0, lse_out=lse)
    assert torch.isnan(out[0, 1, 0]).all() and torch.isnan(lse[0, 1, 0])
    assert torch.isnan(out[1, 4, Hq - 1]).all()
    # the others, by the rows of the same call with zeros in those two places
    q2[0, 1, 0] = 0
    q2[1, 4, Hq - 1, 3] = 0
    clean, clean_lse = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
    h.tree_attn(q2, kd, vd, dev_mask(masks), clean, 0, lse_out=clean_lse)
    for b in range(2):
        for kv in range(2):
            check_segment(h, clean, clean_lse, q2, kd, vd, masks, [N, N], 0, b, kv)
    out[0, 1, 0], lse[0, 1, 0] = clean[0, 1, 0], clean_lse[0, 1, 0]
    out[1, 4, Hq - 1], lse[1, 4, Hq - 1] = clean[1, 4, Hq - 1], clean_lse[1, 4, Hq - 1]
    for b in range(2):
        for kv in range(2):
            check_segment(h, out, lse, q2, kd, vd, masks, [N, N], 0, b, kv)
    h.close()
