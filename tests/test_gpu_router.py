"""Router with scores and its gradient against oracle/router.py: ids and the whole
permutation exactly, weights and scores within the one rounding to float32,
gradients within the bound of float32 arithmetic."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_permute_amd as m
from oracle import moe as OM
from oracle import router as R
from oracle.experts16 import TINY, U
from tests.gpu_common import DEV, up

pytestmark = pytest.mark.gpu

F = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KIND = {"softmax": m.SCORE_SOFTMAX, "sigmoid": m.SCORE_SIGMOID}
INF, NAN = np.inf, np.nan

# T, E, k, kind, bias, (n_group, topk_group, group_top), renormalize, dtype
CASES = [
    (1, 1, 1, "softmax", False, (1, 1, 1), True, "f32"),
    (1, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),
    (3, 7, 2, "sigmoid", True, (1, 1, 1), False, "bf16"),
    (16, 256, 16, "softmax", True, (16, 3, 1), False, "f16"),       # 256 rows: the last of the single launch
    (16, 512, 8, "sigmoid", False, (4, 2, 2), True, "f32"),
    (16, 60, 3, "sigmoid", True, (6, 2, 2), True, "f32"),           # groups of 10: by way of LDS, in the single launch
    (17, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),          # the first past it
    (5, 300, 32, "softmax", False, (1, 1, 1), True, "f32"),
    (33, 513, 9, "sigmoid", True, (3, 2, 2), True, "bf16"),
    (9, 1024, 32, "softmax", True, (32, 8, 1), False, "f32"),
    (6, 1025, 31, "sigmoid", False, (1, 1, 1), True, "f16"),
    (7, 4096, 32, "sigmoid", True, (64, 5, 2), True, "f32"),
    (4, 4095, 7, "softmax", True, (9, 2, 2), True, "f32"),
    (2047, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),        # the last on 64 lanes a token
    (2051, 256, 8, "sigmoid", True, (8, 4, 2), True, "f32"),        # 16 lanes a token from here
    (2049, 256, 16, "softmax", False, (1, 1, 1), False, "bf16"),
    (2050, 64, 8, "sigmoid", False, (8, 2, 2), True, "bf16"),
    (2053, 61, 5, "softmax", True, (1, 1, 1), True, "f16"),
    (2055, 96, 6, "sigmoid", True, (12, 4, 2), False, "f32"),       # groups of 8, 16 experts a lane: by way of LDS
    (2048, 250, 8, "softmax", True, (5, 3, 1), True, "f32"),
    (2048, 256, 17, "softmax", True, (2, 1, 2), True, "f32"),
]
IDS = ["-".join(str(x) for x in c) for c in CASES]


def _logits(c, seed=0):
    T, E, dtype = c[0], c[1], c[7]
    r = np.random.default_rng([T, E, seed])
    l = r.standard_normal((T, E)).astype(np.float32) * 1.5
    bias = (r.standard_normal(E) * 0.1).astype(np.float32) if c[4] else None
    t = torch.from_numpy(l).to(F[dtype])
    return r, t, t.double().numpy(), bias


def _call(t, c, bias, scale=2.5, **more):
    n_group, topk_group, group_top = c[5]
    return m.moe_route_scored(t.to(DEV), c[2], score=KIND[c[3]], bias=None if bias is None else up(bias), n_group=n_group,
                              topk_group=topk_group, group_top=group_top, renormalize=c[6], scale=scale, **more)


def _check(got, scores, want, k, E):
    ids, w, s, _ = want
    assert np.array_equal(got.topk_ids.cpu().numpy(), ids)
    gw = got.topk_w.cpu().numpy()
    # float64 until one rounding to float32 (and 2^-40 for the float64 steps)
    assert (np.abs(gw.astype(np.float64) - w) <= np.abs(w) * U * (1 + 2.0 ** -15) + TINY["f32"]).all()
    if scores is not None:
        assert (np.abs(scores.double().cpu().numpy() - s) <= s * U * (1 + 2.0 ** -15) + TINY["f32"]).all()
    counts, offsets, src, row_of, row_w = OM.permute(ids, gw, E)
    for a, b in ((got.counts, counts), (got.offsets, offsets), (got.perm_src_token, src), (got.perm_of_assignment, row_of)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(got.perm_weight.cpu().numpy().view(np.uint32), row_w.view(np.uint32))


def _want(l, c, bias, scale=2.5):
    n_group, topk_group, group_top = c[5]
    return R.route(l, c[2], c[3], bias, n_group, topk_group, group_top, c[6], scale)


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_route(c):
    print("route", c, flush=True)
    _, t, l, bias = _logits(c)
    want = _want(l, c, bias)
    got, scores = _call(t, c, bias, save_scores=True)
    _check(got, scores, want, c[2], c[1])
    _check(_call(t, c, bias), None, want, c[2], c[1])          # without scores: fewer exponentials


def _edge_rows(E, bf16):
    r = np.random.default_rng(E)
    l = r.standard_normal((24, E)).astype(np.float32)
    l[0] = -INF                                 # nothing open
    l[1] = NAN
    l[2] = 0.25                                 # all equal
    l[3, : E - 1] = -INF                        # one open
    l[4, ::2] = NAN
    l[5, 1], l[5, 3] = INF, INF
    l[6] = -800.0 - r.random(E).astype(np.float32)      # a sigmoid that underflows in float64
    l[7] = -100.0 - r.random(E).astype(np.float32)      # ... in float32
    l[8] = 50.0 + r.random(E).astype(np.float32)        # ... that saturates
    l[9] = np.finfo(np.float32).min
    l[10] = np.where(np.arange(E) % 3 == 0, 1.0, -INF)
    l[11] = np.round(l[11])                     # many ties
    l[12, : E // 2] = -INF                      # whole groups closed
    if not bf16:
        # neighbours in float32, whose scores share a float32
        l[13] = (np.float32(3).view(np.uint32) + np.random.default_rng(1).permutation(E).astype(np.uint32)).view(np.float32)
        l[14] = (np.float32(-9).view(np.uint32) + np.random.default_rng(2).permutation(E).astype(np.uint32)).view(np.float32)
    l[15, 0] = 1e30
    return l


@pytest.mark.parametrize("repeat", [1, 100], ids=["few", "many"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 2), (4, 2, 1)], ids=str)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 72])
def test_edge_rows(E, kind, groups, bias, dtype, repeat):
    print("edges", E, kind, groups, bias, dtype, repeat, flush=True)
    t = torch.from_numpy(_edge_rows(E, dtype != "f32")).to(F[dtype])
    l = t.double().numpy()
    b = None
    if bias:
        b = (np.random.default_rng(3).standard_normal(E) * 0.01).astype(np.float32)
        b[3], b[5], b[9] = -INF, NAN, INF
    for renormalize in (True, False):
        c = (len(l), E, 6, kind, bias, groups, renormalize, dtype)
        ids, w, s, o = _want(l, c, b)
        big = np.tile(ids, (repeat, 1))
        got, scores = _call(t.repeat(repeat, 1), c, b, save_scores=True)
        _check(got, scores, (big, np.tile(w, (repeat, 1)), np.tile(s, (repeat, 1)), None), 6, E)
        r = np.random.default_rng(5)
        dw, ds = r.standard_normal(ids.shape).astype(np.float32), r.standard_normal((len(l), E)).astype(np.float32)
        d = m.moe_route_scored_backward(up(np.tile(dw, (repeat, 1))), t.repeat(repeat, 1).to(DEV), got.topk_ids,
                                        score=KIND[kind], bias=None if b is None else up(b), renormalize=renormalize,
                                        scale=2.5, d_scores=up(np.tile(ds, (repeat, 1))))
        want, tol = R.route_grad(dw, l, ids, o, kind, renormalize, 2.5, ds, dtype)
        err = np.abs(d.double().cpu().numpy() - np.tile(want, (repeat, 1)))
        assert (err <= np.tile(tol, (repeat, 1))).all(), np.argwhere(~(err <= np.tile(tol, (repeat, 1))))[:5]


@pytest.mark.parametrize("scores", ["none", "row", "full"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_gradient(c, scores):
    print("gradient", c, scores, flush=True)
    r, t, l, bias = _logits(c)
    ids, w, s, o = _want(l, c, bias)
    dw = r.standard_normal(ids.shape).astype(np.float32)
    ds = None if scores == "none" else r.standard_normal(c[1] if scores == "row" else (c[0], c[1])).astype(np.float32)
    got = m.moe_route_scored_backward(up(dw), t.to(DEV), up(ids), score=KIND[c[3]], renormalize=c[6], scale=2.5,
                                      d_scores=None if ds is None else up(ds))
    assert got.dtype == F[c[7]]
    want, tol = R.route_grad(dw, l, ids, o, c[3], c[6], 2.5, ds, c[7])
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_foreign_ids(kind, renormalize):
    """Ids outside the experts are left out; one that stands twice counts twice."""
    r = np.random.default_rng(8)
    T, E, k = 40, 20, 4
    l = r.standard_normal((T, E)).astype(np.float32)
    ids = r.integers(0, E, (T, k)).astype(np.int32)
    ids[::3, 1] = ids[::3, 0]
    ids[1, :2], ids[2], ids[4, 0] = (-1, E), (E, -7, 2 ** 31 - 1, -2 ** 31), E + 5
    dw = r.standard_normal((T, k)).astype(np.float32)
    got = m.moe_route_scored_backward(up(dw), up(l), up(ids), score=KIND[kind], renormalize=renormalize).double().cpu().numpy()
    want, tol = R.route_grad(dw, l, ids, np.ones((T, E), bool), kind, renormalize, 1.0)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("E", [24, 256])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_gradients_at_closed_experts_are_not_read(E, kind, renormalize, bad):
    """What the scores of closed logits and the weights of closed choices get is nothing, NaN and
    infinities too; the row's other gradients stay."""
    r = np.random.default_rng(E)
    T, k = 40, 6
    l = r.standard_normal((T, E)).astype(np.float32)
    l[:, 1::3] = -INF
    l[::2, 0] = NAN
    l[5, 4:] = -INF                             # fewer open ones than k: closed ones are chosen
    l[6] = -INF
    c = (T, E, k, kind, False, (1, 1, 1), renormalize, "f32")
    ids, w, s, o = _want(l.astype(np.float64), c, None)
    dw, ds = r.standard_normal((T, k)).astype(np.float32), r.standard_normal((T, E)).astype(np.float32)
    want, tol = R.route_grad(dw, l, ids, o, kind, renormalize, 2.5, ds)
    ds[~o] = bad
    dw[~o[np.arange(T)[:, None], ids]] = bad
    got = m.moe_route_scored_backward(up(dw), up(l), up(ids), score=KIND[kind], renormalize=renormalize, scale=2.5, d_scores=up(ds))
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all()


def test_default_is_the_plain_softmax_router():
    l = torch.randn((300, 96), device=DEV)
    a, b = m.moe_route_scored(l, 7), m.moe_route_permute(l, 7)
    for n in ("topk_ids", "counts", "offsets", "perm_src_token", "perm_of_assignment"):
        assert torch.equal(getattr(a, n), getattr(b, n))
    assert ((a.topk_w - b.topk_w).abs() <= 2.0 ** -23 * b.topk_w).all()


def test_unaligned_logits():
    """Rows of 256 values that start 4 (float32) or 2 bytes behind a 16-byte border."""
    for dtype in ("f32", "bf16", "f16"):
        c = (40, 256, 8, "sigmoid", True, (8, 4, 2), True, dtype)
        r, t, l, bias = _logits(c)
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1).to(DEV)
        x = flat[1:].view(t.shape)
        how = dict(score=KIND["sigmoid"], renormalize=True, scale=2.5)
        got, scores = m.moe_route_scored(x, 8, bias=up(bias), n_group=8, topk_group=4, group_top=2, save_scores=True, **how)
        ids, w, s, o = _want(l, c, bias)
        _check(got, scores, (ids, w, s, o), 8, 256)
        dw = r.standard_normal(ids.shape).astype(np.float32)
        d = flat.new_empty(t.numel() + 1)[1:].view(t.shape)
        m.moe_route_scored_backward(up(dw), x, got.topk_ids, dlogits=d, **how)
        want, tol = R.route_grad(dw, l, ids, o, "sigmoid", True, 2.5, None, dtype)
        assert (np.abs(d.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (3, 5, 72), (40, 8, 512), (33, 2, 520), (7, 33, 1032), (2049, 3, 1024), (2048, 9, 776),
                                   (5, 4, 6144), (1, 1024, 16)])
def test_combine_gradient(T, k, H, dt, yt):
    print("combine gradient", T, k, H, dt, yt, flush=True)
    r = np.random.default_rng([T, k, H])
    M = T * k
    dout = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(F[dt])
    y = torch.from_numpy(r.standard_normal((M, H)).astype(np.float32)).to(F[yt])
    rows, w = r.permutation(M).astype(np.int32).reshape(T, k), r.standard_normal((T, k)).astype(np.float32)
    args = (dout.to(DEV), y.to(DEV), up(rows.reshape(-1)), up(w))
    (dy, ty), (dw, tw) = R.combine_grad(dout.double().numpy(), y.double().numpy(), rows, w, yt)
    a, b = m.moe_unpermute_combine_backward(*args)
    assert a.dtype == F[yt] and (np.abs(a.double().cpu().numpy() - dy) <= ty).all()
    assert (np.abs(b.double().cpu().numpy() - dw) <= tw).all()
    assert torch.equal(m.moe_unpermute_combine_backward(*args, need_dw=False)[0], a)
    assert torch.equal(m.moe_unpermute_combine_backward(*args, need_dy=False)[1], b)
    # without a permutation: row t * k + j
    a2, b2 = m.moe_unpermute_combine_backward(args[0], args[1][args[2].long()].contiguous(), None, args[3])
    assert torch.equal(a2, a[args[2].long()]) and torch.equal(b2, b)


def test_combine_gradient_rows_apart():
    """Rows that no entry names: left in a given dy, zero in a new one; entries outside y are left out."""
    T, k, H, rows = 9, 2, 64, 40
    r = np.random.default_rng(2)
    perm = r.permutation(rows)[:T * k].astype(np.int32)
    perm[3], perm[7], perm[11] = -1, rows, 2 ** 31 - 1
    bad = np.isin(np.arange(T * k), (3, 7, 11)).reshape(T, k)
    dout, y, w = torch.randn((T, H), device=DEV), torch.randn((rows, H), device=DEV), torch.rand((T, k), device=DEV)
    dy = torch.full((rows, H), 7.0, device=DEV)
    _, dw = m.moe_unpermute_combine_backward(dout, y, up(perm), w, dy=dy)
    fresh, _ = m.moe_unpermute_combine_backward(dout, y, up(perm), w)
    named = torch.zeros(rows, dtype=torch.bool)
    named[torch.from_numpy(perm[~bad.reshape(-1)]).long()] = True
    assert (dy.cpu()[~named] == 7).all() and (fresh.cpu()[~named] == 0).all() and torch.equal(dy.cpu()[named], fresh.cpu()[named])
    assert (dw.cpu().numpy()[bad] == 0).all() and (dw.cpu().numpy()[~bad] != 0).all()


def test_combine_gradient_reads_no_other_rows():
    """Infinities and NaN in rows that none names, and y not read without its gradient."""
    T, k, H = 6, 2, 128
    y = torch.full((T * k + 3, H), float("nan"), device=DEV)
    perm = torch.arange(T * k, dtype=torch.int32, device=DEV).flip(0).contiguous()
    y[:T * k] = 1.0
    dout, w = torch.ones((T, H), device=DEV), torch.ones((T, k), device=DEV)
    _, dw = m.moe_unpermute_combine_backward(dout, y, perm, w)
    assert (dw == H).all()
    dy, _ = m.moe_unpermute_combine_backward(dout, torch.full_like(y, float("nan")), perm, w, need_dw=False)
    assert (dy[:T * k] == 1).all() and (dy[T * k:] == 0).all()
