"""The router with groups of experts against the fp64 definition: group counts, both merits, ties,
NaN experts and tokens, masks by a bias of -inf, lengths on both sides of the one-launch form.
The ids are exact (inputs whose near ties fp64 does not resolve are left out by assertion); the
weights are fp64 values rounded to fp32, 2^-23 taken."""
import itertools

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.test_gpu_router import SCORES, check, host, make, say, scores_ref

pytestmark = pytest.mark.gpu


def merits(key, n, by):
    size = key.shape[1] // n
    k = -np.sort(-key.reshape(-1, n, size), axis=2)
    return k[:, :, :2].sum(axis=2) if by == "top2" and size > 1 else k[:, :, 0]


def groups_ref(x, w, K, kind, norm, scale, bias, n, top, by):
    with np.errstate(all="ignore"):
        s = scores_ref(x.astype(np.float64) @ w.astype(np.float64).T, kind)
    key = s if bias is None else s + bias.astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    m = merits(key, n, by)
    kept = np.argsort(-m, axis=1, kind="stable")[:, :top]
    out = np.ones((x.shape[0], n), bool)
    np.put_along_axis(out, kept, False, axis=1)
    out = np.repeat(out, key.shape[1] // n, axis=1)
    # outside the kept groups: behind everything, -inf and NaN inside them included
    ids = np.array([sorted(np.nonzero(~o)[0], key=lambda e: (-k[e], e))[:K] for k, o in zip(key, out)])
    rw = np.take_along_axis(s, ids, 1)
    if norm:
        with np.errstate(invalid="ignore"):
            tot = rw.sum(axis=1, keepdims=True)
            rw = np.where(tot == 0, 0.0, rw / np.where(tot == 0, 1.0, tot))
    return ids, rw * scale, (key, m)


def clear(ref, T):
    """Tokens whose merits and keys lie apart by more than fp64's own errors."""
    key, m = ref[2]
    with np.errstate(invalid="ignore"):
        gm = np.abs(np.diff(np.sort(m, axis=1), axis=1)).min(axis=1, initial=1.0)
        gk = np.abs(np.diff(np.sort(key, axis=1), axis=1)).min(axis=1, initial=1.0)
    return (gm > 1e-12) & (gk > 1e-13)


CASES = [  # T, H, E, K, groups, kept
    (1, 4096, 256, 6, 8, 4), (3, 1024, 64, 4, 2, 1), (2, 24, 12, 4, 3, 2), (7, 512, 60, 8, 4, 1), (16, 2048, 1024, 16, 16, 5),
    (9, 256, 64, 3, 64, 7), (64, 4096, 256, 8, 8, 3), (65, 1032, 180, 6, 5, 2), (300, 768, 390, 7, 13, 4), (130, 512, 992, 8, 31, 9),
    (5, 64, 48, 2, 16, 2), (200, 128, 40, 5, 40, 5), (70, 64, 8, 8, 2, 1 + 1),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("kind,by", list(itertools.product(SCORES, ("top2", "max"))))
def test_groups(case, kind, by):
    T, H, E, K, n, top = case
    say("groups", case, kind, by)
    bias, norm = (T + E + len(by)) % 2 == 0, (T + K) % 2 == 0
    x, w, b = make(T, H, E, T * 11 + E, bias)
    r = mq.Router(w, K, scoring=kind, normalize=norm, scale=2.5, bias=b, n_groups=n, top_groups=top, group_score=by)
    ids, rw = mq.router_topk(r, x)
    ref = groups_ref(host(x), host(w), K, kind, norm, 2.5, host(b), n, top, by)
    ok = clear(ref, T)
    assert ok.mean() > 0.9
    check(ids[torch.from_numpy(ok).cuda()], rw[torch.from_numpy(ok).cuda()], [a[ok] for a in ref[:2]] + [None])
    chosen = ids.cpu().numpy()
    assert all(len(set(c)) == K and len(set(c // (E // n))) <= top for c in chosen)


@pytest.mark.parametrize("T", [4, 100])
@pytest.mark.parametrize("by", ["top2", "max"])
def test_equal_experts_and_equal_groups(T, by):
    """All groups equal: the lowest are kept. All experts equal: the lowest ids."""
    say("groups ties", T, by)
    x, w, _ = make(T, 256, 8, 1)
    same = w.repeat(4, 1)  # four equal groups of eight
    for kind in SCORES:
        r = mq.Router(same, 4, scoring=kind, n_groups=4, top_groups=2, group_score=by)
        ids = mq.router_topk(r, x)[0].cpu().numpy()
        ref = groups_ref(host(x), host(same), 4, kind, False, 1.0, None, 4, 2, by)
        assert np.array_equal(ids, ref[0]) and ids.max() < 16
        flat = mq.Router(w[:1].repeat(32, 1), 5, scoring=kind, n_groups=8, top_groups=3, group_score=by)
        assert mq.router_topk(flat, x)[0].cpu().tolist() == [[0, 1, 2, 3, 4]] * T


@pytest.mark.parametrize("T", [2, 90])
def test_near_ties_of_merits_are_decided_in_64_bits(T):
    """Groups whose merits differ by a few parts in 1e8."""
    say("groups near ties", T)
    x, w, _ = make(T, 1024, 64, 5)
    w[32:] = w[:32]  # groups 4..7 are 0..3 but for one weight that moves by one step or stays
    w[32:, 100] = (w[:32, 100].float() * (1 + 2.0 ** -8)).to(torch.bfloat16)
    x[:, 100] = 2.0 ** -14
    r = mq.Router(w, 6, scoring="sigmoid", normalize=True, n_groups=8, top_groups=3)
    ref = groups_ref(host(x), host(w), 6, "sigmoid", True, 1.0, None, 8, 3, "top2")
    m = -np.sort(-ref[2][1], axis=1)
    k = -np.sort(-ref[2][0], axis=1)
    # (a step that bf16 rounds away leaves two experts equal, which the ids decide)
    dm, dk = np.abs(np.diff(m, axis=1)), np.abs(np.diff(k, axis=1))
    apart = ((dm == 0) | (dm > 1e-12)).all(axis=1) & ((dk == 0) | (dk > 1e-13)).all(axis=1)
    assert apart.any()
    assert (np.where(dm == 0, 1.0, dm).min(axis=1)[apart] < 1e-6).any()
    ids = mq.router_topk(r, x)[0].cpu().numpy()
    assert np.array_equal(ids[apart], ref[0][apart])


@pytest.mark.parametrize("T", [3, 80])
@pytest.mark.parametrize("by", ["top2", "max"])
def test_masks_and_numbers_that_are_not_finite(T, by):
    """Experts masked by a bias of -inf (whole groups among them), NaN experts, a NaN token."""
    say("groups masks", T, by)
    x, w, b = make(T, 512, 48, 7)
    b[:8], b[8:15], b[20], b[24:] = -np.inf, -np.inf, np.nan, b[24:]  # group 0 masked, 1 but for one, one NaN in 2
    w[30, 3] = float("nan")
    x[T - 1, 9] = float("nan")
    for kind in ("sigmoid", "sqrtsoftplus"):
        r = mq.Router(w, 6, scoring=kind, normalize=False, bias=b, n_groups=6, top_groups=2, group_score=by)
        ids, rw = mq.router_topk(r, x)
        ref = groups_ref(host(x), host(w), 6, kind, False, 1.0, host(b), 6, 2, by)
        assert np.array_equal(ids.cpu().numpy(), ref[0])
        assert np.allclose(rw.cpu().numpy(), ref[1], rtol=2.0 ** -23, atol=0, equal_nan=True)
    all_masked = torch.full_like(b, -np.inf)
    r = mq.Router(w, 6, scoring="sigmoid", bias=all_masked, n_groups=6, top_groups=2, group_score=by)
    assert mq.router_topk(r, x)[0].cpu().tolist() == [[0, 1, 2, 3, 4, 5]] * T


def test_all_groups_kept_is_the_router_without_groups():
    say("groups all")
    for T in (5, 120):
        x, w, b = make(T, 512, 64, 8)
        plain = mq.router_topk(mq.Router(w, 6, scoring="sigmoid", bias=b), x)
        for n in (1, 4, 8):
            got = mq.router_topk(mq.Router(w, 6, scoring="sigmoid", bias=b, n_groups=n, top_groups=n), x)
            assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


MANY = [  # 2^30 products and more: logits with bounds, and exact ones of those that matter
    (2100, 2048, 256, 6, 8, 4), (1100, 4096, 240, 8, 5, 2), (280, 4104, 960, 16, 30, 7), (700, 4096, 400, 6, 50, 9),
    (4200, 4096, 64, 3, 64, 7), (9000, 520, 240, 4, 3, 1), (140, 8200, 1000, 8, 8, 3),
]


@pytest.mark.parametrize("case", MANY)
@pytest.mark.parametrize("kind,by", list(itertools.product(("sigmoid", "sqrtsoftplus"), ("top2", "max"))))
def test_groups_of_many_logits(case, kind, by):
    test_groups(case, kind, by)


@pytest.mark.parametrize("by", ["top2", "max"])
def test_ties_among_many_logits(by):
    """Equal groups, equal experts, tokens of zeros, and merits that differ by a few parts in 1e8."""
    say("groups many ties", by)
    T, H = 4200, 4096
    x, w, _ = make(T, H, 16, 1)
    x[::3] = 0
    same = w.repeat(4, 1)
    for kind in ("sigmoid", "sqrtsoftplus"):
        r = mq.Router(same, 4, scoring=kind, n_groups=4, top_groups=2, group_score=by)
        ids = mq.router_topk(r, x)[0].cpu().numpy()
        assert np.array_equal(ids, groups_ref(host(x), host(same), 4, kind, False, 1.0, None, 4, 2, by)[0]) and ids.max() < 32
        flat = mq.Router(w[:1].repeat(64, 1), 5, scoring=kind, n_groups=8, top_groups=3, group_score=by)
        assert mq.router_topk(flat, x)[0].cpu().tolist() == [[0, 1, 2, 3, 4]] * T
    x, w, _ = make(T, H, 64, 5)
    w[32:] = w[:32]
    w[32:, 100] = (w[:32, 100].float() * (1 + 2.0 ** -8)).to(torch.bfloat16)
    x[:, 100] = 2.0 ** -14
    ref = groups_ref(host(x), host(w), 6, "sigmoid", True, 1.0, None, 8, 3, by)
    dm, dk = (np.abs(np.diff(np.sort(a, axis=1), axis=1)) for a in (ref[2][1], ref[2][0]))
    apart = ((dm == 0) | (dm > 1e-12)).all(axis=1) & ((dk == 0) | (dk > 1e-13)).all(axis=1)
    assert apart.any() and (np.where(dm == 0, 1.0, dm).min(axis=1)[apart] < 1e-6).any()
    r = mq.Router(w, 6, scoring="sigmoid", normalize=True, n_groups=8, top_groups=3, group_score=by)
    assert np.array_equal(mq.router_topk(r, x)[0].cpu().numpy()[apart], ref[0][apart])


@pytest.mark.parametrize("by", ["top2", "max"])
def test_masks_among_many_logits(by):
    say("groups many masks", by)
    T, H = 5600, 4096
    x, w, b = make(T, H, 48, 7)
    b[:8], b[8:15], b[20] = -np.inf, -np.inf, np.nan
    w[30, 3] = float("nan")
    w[33] = 0
    w[40, 5] = float("inf")
    x[T - 1, 9] = float("nan")
    x[7] = 0
    for kind in ("sigmoid", "sqrtsoftplus"):
        r = mq.Router(w, 6, scoring=kind, bias=b, n_groups=6, top_groups=2, group_score=by)
        ids, rw = mq.router_topk(r, x)
        ref = groups_ref(host(x), host(w), 6, kind, False, 1.0, host(b), 6, 2, by)
        ok = clear((None, None, tuple(np.where(np.isfinite(a), a, 1e3 * np.arange(1, a.shape[1] + 1)) for a in ref[2])), T)
        assert ok.mean() > 0.9
        assert np.array_equal(ids.cpu().numpy()[ok], ref[0][ok])
        assert np.allclose(rw.cpu().numpy()[ok], ref[1][ok], rtol=2.0 ** -23, atol=0, equal_nan=True)


@pytest.mark.parametrize("T", [2, 64, 150])
def test_graph_and_streams(T):
    say("groups graph", T)
    x, w, b = make(T, 1024, 128, 9)
    r = mq.Router(w, 6, scoring="softmax", normalize=True, bias=b, n_groups=8, top_groups=3, group_score="max")
    ids = torch.empty((T, 6), dtype=torch.int32, device="cuda")
    rw = torch.empty((T, 6), device="cuda")
    ws = r.workspace(T)
    mq.router_topk(r, x, ids=ids, rw=rw, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        mq.router_topk(r, x, ids=ids, rw=rw, ws=ws)
    for i in range(4):
        x.copy_(make(T, 1024, 128, 50 + i)[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = mq.router_topk(r, x)
        side.synchronize()
        ids.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(rw, want[1])
