"""Routing by scores (moe_route_scored and the layer calls that use it).

Ids and the permutation have to equal the plain 64-bit form's; the weights are
64-bit values rounded to fp32 once, so they are off by at most half a step
(2^-24 relative) plus the two 64-bit evaluations' own 1e-15 or so.
"""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_moe_router_amd as bq
import oracle
import scored_reference as ref
import synth
import workloads
from helpers import assert_parity

DEV = "cuda"
FAKE = 1 << 40  # a 256-aligned address that is never dereferenced: every call below fails first
SOFT, SIG = bq.MOE_SCORE_SOFTMAX, bq.MOE_SCORE_SIGMOID
W_RTOL = 2.0 ** -24 * 1.001


# --------------------------------------------------------------------- refusals (no GPU)
def _layer(E=16, k=2, **kw):
    p = dict(n_shared=0, router_w=FAKE, d=256, inter=128)
    p.update(kw)
    return bq.make_layer(p["d"], p["inter"], E, k, p["n_shared"], (2, 2, 2), FAKE, 30_720,
                         None, p["router_w"], None)


def _call(fn, L, S, T=2, flags=0, ws=FAKE, ws_bytes=None, R=None, x=FAKE, out=FAKE + (1 << 30)):
    lib = bq.load()
    if ws_bytes is None:
        ws_bytes = max(1, lib.moe_workspace_bytes(ctypes.byref(L.c), max(T, 0)))
    R = bq.moe_routing(*([FAKE] * 7)) if R is None else R
    args = [ctypes.byref(L.c) if L else None, ctypes.byref(S.c) if S else None, x, T, flags,
            ctypes.byref(R), ws, ws_bytes]
    if fn != "moe_route_scored":
        args.append(out)
    return getattr(lib, fn)(*args, None)


CALLS = ["moe_route_scored", "moe_forward_decode_scored", "moe_forward_prefill_scored"]


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("bad", [
    dict(score=0), dict(score=3), dict(n_groups=0), dict(n_groups=3), dict(n_groups=-4),
    dict(n_groups=4, topk_groups=0), dict(n_groups=4, topk_groups=5), dict(n_groups=4, group_top=0),
    dict(n_groups=4, topk_groups=2, group_top=3), dict(n_groups=16, topk_groups=8, group_top=2),
    dict(n_groups=16, topk_groups=1), dict(renorm=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(choice_bias=FAKE + 2)])
def test_scoring_outside_its_ranges_is_refused(fn, bad):
    p = dict(score=SOFT)
    p.update(bad)
    assert _call(fn, _layer(), bq.make_scoring(**p)) == bq.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", CALLS)
def test_argument_errors_are_those_of_the_other_router(fn):
    S = bq.make_scoring(SIG)
    assert _call(fn, _layer(), None) == bq.MOE_ERR_INVALID_ARG
    assert _call(fn, _layer(), S, T=-1) == bq.MOE_ERR_INVALID_ARG
    assert _call(fn, _layer(), S, flags=0x80) == bq.MOE_ERR_INVALID_ARG
    assert _call(fn, _layer(d=100), S) == bq.MOE_ERR_UNSUPPORTED
    assert _call(fn, _layer(E=2000), S) == bq.MOE_ERR_UNSUPPORTED
    assert _call(fn, _layer(router_w=None), S) == bq.MOE_ERR_INVALID_ARG
    assert _call(fn, _layer(), S, ws_bytes=10) == bq.MOE_ERR_WORKSPACE
    assert _call(fn, _layer(), S, ws=None) == bq.MOE_ERR_WORKSPACE
    assert _call(fn, _layer(), S, ws=FAKE + 8) == bq.MOE_ERR_INVALID_ARG
    R = bq.moe_routing(*([FAKE] * 7))
    R.inv_row = None
    assert _call(fn, _layer(), S, R=R) == bq.MOE_ERR_INVALID_ARG
    if fn != "moe_route_scored":
        assert _call(fn, _layer(), S, out=FAKE + 256) == bq.MOE_ERR_INVALID_ARG  # overlaps x
        assert _call(fn, _layer(), S, out=None) == bq.MOE_ERR_INVALID_ARG
    if fn == "moe_forward_decode_scored":
        assert _call(fn, _layer(), S, T=0) == bq.MOE_ERR_INVALID_ARG
        assert _call(fn, _layer(), S, T=9) == bq.MOE_ERR_INVALID_ARG
    else:
        assert _call(fn, _layer(), S, T=0) == bq.MOE_OK


def test_bias_tensor_must_be_contiguous_float32_on_the_gpu():
    for b in (torch.zeros(4, dtype=torch.float64), torch.zeros(8)[::2], torch.zeros(8)):
        with pytest.raises(bq.MoeError):
            bq.make_scoring(SIG, choice_bias=b)


def test_workspace_covers_both_routers():
    lib = bq.load()
    for E, k, T in ((1024, 1, 33), (1024, 32, 5000), (8, 2, 100_000)):
        L = _layer(E=E, k=k, d=128, router_w=FAKE)
        S = bq.make_scoring(SIG)
        need = lib.moe_workspace_bytes(ctypes.byref(L.c), T)
        assert _call("moe_route_scored", L, S, T=T, ws=FAKE + 8) == bq.MOE_ERR_INVALID_ARG
        assert need >= 4 * T * k


def test_reference_against_hand_worked_rows():
    # two groups of two; sigmoid(0) = 1/2; the bias steers the choice, not the weights
    l = np.float32([[0.0, 2.0, 1.0, 1.5]])
    ids, w, *_ = ref.route(l, 2, True, groups=2, topk_groups=1, group_top=1, renorm=True)
    assert ids.tolist() == [[1, 0]]
    assert np.allclose(w[0], np.array([0.8807970779778823, 0.5]) / 1.3807970779778823)
    b = np.float32([0, 0, 9, 0])
    ids, w, *_ = ref.route(l, 1, True, bias=b, renorm=False, scale=2.0)
    assert ids.tolist() == [[2]] and np.allclose(w, 2 * 0.7310585786300049)
    ids, w, *_ = ref.route(np.float32([[-np.inf] * 3]), 2, False)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


# ------------------------------------------------------------------------------- routing
def _inputs(T, E, kind, seed):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "ties":
        l = np.round(l)  # many equal logits in every row
    elif kind == "equal":
        l[:] = 0.25
    elif kind == "wide":
        l *= 300.0  # scores down to 0 and up to 1 in 64 bits
    elif kind == "near":
        # neighbours in fp32: scores that a 32-bit evaluation cannot tell apart
        l = (1.0 + rng.integers(0, 64, (T, E)) * 2.0 ** -23).astype(np.float32)
    elif kind == "tiny":
        # different logits with one 64-bit score, among the largest and in the middle of a row
        small = rng.integers(-3, 4, (T, E)).astype(np.float32) * np.float32(1e-20)
        l = np.where(rng.random((T, E)) < 0.5, small, l)
        l[::2] = np.minimum(l[::2], np.float32(3e-20))
    elif kind == "masked":
        l[rng.random((T, E)) < 0.6] = -np.inf
        l[0] = -np.inf
    elif kind == "odd":
        l[rng.random((T, E)) < 0.1] = np.nan
        l[rng.random((T, E)) < 0.05] = -np.inf
        if T > 1:
            l[1] = np.nan
            l[T - 1, 0] = np.inf
    return l


def _run(logits, k, bias, d=128, scratch=None, stream=None, **kw):
    T, E = logits.shape
    layer = bq.make_layer(d, 128, E, k, 0, (2, 2, 2), None, 0)
    lg = torch.from_numpy(logits).to(DEV)
    b = None if bias is None else torch.from_numpy(bias).to(DEV)
    S = bq.make_scoring(kw.pop("score"), choice_bias=b, **kw)
    R = bq.alloc_routing(T, E, k, DEV, logits=lg)
    for n in ("topk_ids", "topk_w", "counts", "offsets", "perm_tok", "inv_row"):
        getattr(R, n).fill_(-7)
    ws = bq.alloc_workspace(layer, T, DEV)
    ws.fill_(0xA5)
    bq.moe_route_scored(layer, S, None, T, bq.MOE_LOGITS_GIVEN, R, ws, stream)
    torch.cuda.synchronize()
    assert np.array_equal(lg.cpu().numpy().view(np.int32), logits.view(np.int32))
    return {n: getattr(R, n).cpu().numpy() for n in
            ("topk_ids", "topk_w", "counts", "offsets", "perm_tok", "inv_row")}


def _check(got, want):
    ids, w, counts, offsets, perm, inv = want
    assert np.array_equal(got["topk_ids"], ids)
    assert np.array_equal(got["counts"], counts)
    assert np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["perm_tok"], perm)
    assert np.array_equal(got["inv_row"], inv)
    assert np.allclose(got["topk_w"], w, rtol=W_RTOL, atol=2.0 ** -149, equal_nan=True)


SHAPES = [  # T, E, k, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (8, 256, 8, 1, 1, 1), (5, 8, 8, 2, 2, 1),
    (4, 64, 6, 64, 40, 1), (7, 40, 5, 8, 2, 2), (32, 256, 32, 4, 1, 2), (33, 256, 8, 8, 4, 2),
    (3, 160, 6, 8, 3, 1), (31, 1000, 12, 5, 2, 2), (32, 1024, 32, 16, 3, 2), (2, 512, 3, 32, 1, 2),
    (257, 130, 7, 13, 5, 2), (300, 64, 4, 1, 1, 1), (1237, 160, 6, 8, 3, 1), (2000, 1024, 5, 2, 1, 2),
    (24, 256, 32, 8, 2, 2), (25, 250, 31, 5, 2, 1), (8, 1024, 8, 32, 9, 2), (8, 600, 9, 6, 2, 1),
    (9, 513, 3, 27, 11, 2), (4, 256, 32, 8, 5, 1), (5, 200, 13, 4, 2, 2),
    (4099, 16, 2, 4, 2, 1), (4500, 256, 32, 1, 1, 1), (700, 384, 1, 3, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,tg,gt", SHAPES)
@pytest.mark.parametrize("sigmoid,bias,renorm", [(0, 0, 1), (1, 1, 1), (0, 1, 0), (1, 0, 0)])
def test_routing_matches_the_plain_form(T, E, k, G, tg, gt, sigmoid, bias, renorm):
    print(f"[route_scored] T={T} E={E} k={k} groups {G}/{tg}/{gt} sigmoid={sigmoid}", flush=True)
    l = _inputs(T, E, "normal", 1000 * T + E)
    b = np.random.default_rng(E).normal(0, 0.1, E).astype(np.float32) if bias else None
    kw = dict(topk_groups=tg, group_top=gt, renorm=bool(renorm), scale=2.5 if renorm else 16.0)
    got = _run(l, k, b, score=SIG if sigmoid else SOFT, n_groups=G, **kw)
    _check(got, ref.route(l, k, bool(sigmoid), groups=G, bias=b, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["ties", "equal", "wide", "near", "tiny", "masked", "odd"])
@pytest.mark.parametrize("T,E,k,G,tg,gt", [(6, 64, 8, 1, 1, 1), (30, 96, 8, 8, 3, 2),
                                           (130, 256, 8, 8, 4, 2), (70, 520, 9, 1, 1, 1)])
@pytest.mark.parametrize("sigmoid", [0, 1])
def test_ties_masks_and_specials(kind, T, E, k, G, tg, gt, sigmoid):
    print(f"[route_scored] {kind} T={T} E={E} groups {G} sigmoid={sigmoid}", flush=True)
    l = _inputs(T, E, kind, 7)
    for renorm in (True, False):
        got = _run(l, k, None, score=SIG if sigmoid else SOFT, n_groups=G, topk_groups=tg,
                   group_top=gt, renorm=renorm)
        _check(got, ref.route(l, k, bool(sigmoid), groups=G, topk_groups=tg, group_top=gt,
                              renorm=renorm))


@pytest.mark.gpu
def test_a_bias_of_minus_infinity_takes_an_expert_out_of_the_choice():
    l = _inputs(40, 32, "normal", 3)
    b = np.zeros(32, np.float32)
    b[::2] = -np.inf
    got = _run(l, 6, b, score=SIG)
    _check(got, ref.route(l, 6, True, bias=b))
    assert (got["topk_ids"] % 2 == 1).all()


@pytest.mark.gpu
def test_softmax_without_groups_is_the_layers_own_router():
    for T in (3, 500):
        l = _inputs(T, 256, "normal", T)
        got = _run(l, 8, None, score=SOFT)
        ids, w = oracle.topk_softmax(l, 8)
        assert np.array_equal(got["topk_ids"], ids)
        assert np.allclose(got["topk_w"], w, rtol=2e-6)


@pytest.mark.gpu
def test_bias_of_another_number_of_experts_is_refused():
    S = bq.make_scoring(SIG, choice_bias=torch.zeros(15, device=DEV))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    R = bq.alloc_routing(2, 16, 2)
    with pytest.raises(bq.MoeError):
        bq.moe_route_scored(_layer(), S, None, 2, bq.MOE_LOGITS_GIVEN, R, ws)
    for fn in (bq.moe_forward_decode_scored, bq.moe_forward_prefill_scored):
        with pytest.raises(bq.MoeError):
            fn(_layer(), S, None, 2, bq.MOE_LOGITS_GIVEN, R, ws, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(1, 96), (8, 96), (8, 1024), (77, 96), (900, 96), (40, 1024)])
def test_captured_into_a_graph_and_on_another_stream(T, E):
    k = 4
    layer = bq.make_layer(128, 128, E, k, 0, (2, 2, 2), None, 0)
    S = bq.make_scoring(SIG, n_groups=8, topk_groups=3, group_top=2)
    lg = torch.zeros((T, E), device=DEV)
    R = bq.alloc_routing(T, E, k, DEV, logits=lg)
    ws = bq.alloc_workspace(layer, T, DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        bq.moe_route_scored(layer, S, None, T, bq.MOE_LOGITS_GIVEN, R, ws)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            bq.moe_route_scored(layer, S, None, T, bq.MOE_LOGITS_GIVEN, R, ws)
    for seed in range(3):
        l = _inputs(T, E, "normal", seed)
        lg.copy_(torch.from_numpy(l))
        g.replay()
        torch.cuda.synchronize()
        want = ref.route(l, k, True, groups=8, topk_groups=3, group_top=2)
        got = {n: getattr(R, n).cpu().numpy() for n in
               ("topk_ids", "topk_w", "counts", "offsets", "perm_tok", "inv_row")}
        _check(got, want)
        eager = _run(l, k, None, score=SIG, n_groups=8, topk_groups=3, group_top=2)
        for n in got:
            assert np.array_equal(got[n], eager[n]), n  # also bit for bit the same


# --------------------------------------------------------------------- the layer's calls
CFG = synth.small_config(synth.CONFIGS["c0"], name="scored_small", n_shared=1, E=24, k=4)
CFG3 = synth.small_config(synth.CONFIGS["c0"], name="scored_int3", n_shared=1, E=24, k=4,
                          q_gate=3, q_up=3, q_down=2)


def _layer_reference(cfg, x, ids, w, residual):
    T = x.shape[0]
    y = np.zeros((T * cfg.k, cfg.d), np.uint16)
    inv = np.arange(T * cfg.k, dtype=np.int32).reshape(T, cfg.k)
    for e in np.unique(ids):
        mats = [synth.gen_matrix(cfg, 0, int(e), m) for m in range(3)]
        t, j = np.nonzero(ids == e)
        y[inv[t, j]] = oracle.expert_rows(cfg.qtypes, mats, x[t])[1]
    sh = None
    if cfg.n_shared:
        mats = [synth.gen_matrix(cfg, 0, cfg.E, m) for m in range(3)]
        sh = oracle.expert_rows(cfg.qtypes, mats, x)[1]
    return oracle.combine(w.astype(np.float32), inv, y, sh, x, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,T", [("decode", 1), ("decode", 2), ("decode", 8), ("prefill", 1),
                                    ("prefill", 8), ("prefill", 40), ("prefill", 301)])
@pytest.mark.parametrize("cfg", [CFG, CFG3], ids=["int2", "int3"])
@pytest.mark.parametrize("given", [True, False])
def test_layer_with_the_scored_router(mode, T, cfg, given):
    print(f"[scored layer] {mode} T={T} {cfg.name} logits given={given}", flush=True)
    dl = workloads.DeviceLayer(cfg, 0, DEV)
    x = synth.gen_x(cfg, seed=40 + T, T=T)
    xd = torch.from_numpy(x.view(np.int16)).to(DEV)
    b = np.random.default_rng(5).normal(0, 0.2, cfg.E).astype(np.float32)
    S = bq.make_scoring(SIG, n_groups=6, topk_groups=3, group_top=2, scale=1.5,
                        choice_bias=torch.from_numpy(b).to(DEV))
    R = bq.alloc_routing(T, cfg.E, cfg.k, DEV)
    if given:
        R.logits.copy_(torch.from_numpy(_inputs(T, cfg.E, "normal", T)))
    ws = bq.alloc_workspace(dl.handle, T, DEV)
    ws.fill_(0x5A)
    out = torch.full((T + 1, cfg.d), -3, dtype=torch.int16, device=DEV)
    fn = bq.moe_forward_decode_scored if mode == "decode" else bq.moe_forward_prefill_scored
    flags = bq.MOE_ADD_RESIDUAL | (bq.MOE_LOGITS_GIVEN if given else 0)
    fn(dl.handle, S, xd, T, flags, R, ws, out)
    torch.cuda.synchronize()
    logits = R.logits.cpu().numpy()
    want = ref.route(logits, cfg.k, True, groups=6, topk_groups=3, group_top=2, scale=1.5, bias=b)
    got = {n: getattr(R, n).cpu().numpy() for n in
           ("topk_ids", "topk_w", "counts", "offsets", "perm_tok", "inv_row")}
    _check(got, want)
    o = out.cpu().numpy().view(np.uint16)
    assert (o[T] == np.uint16(-3 & 0xFFFF)).all()  # nothing behind the last row
    assert_parity(o[:T], _layer_reference(cfg, x, want[0], want[1], True), f"scored {mode} T={T}")


@pytest.mark.gpu
def test_decode_with_a_second_expert_copy():
    cfg, T = CFG3, 3
    dl = workloads.DeviceLayer(cfg, 0, DEV)
    alt = workloads.DeviceLayer(cfg, 0, DEV)
    sel = torch.zeros(cfg.E, dtype=torch.uint8, device=DEV)
    sel[::2] = 1
    h = bq.make_layer(cfg.d, cfg.inter, cfg.E, cfg.k, cfg.n_shared, cfg.qtypes, dl.experts,
                      dl.stride, dl.shared, dl.router_w, dl.router_bias,
                      alt=(alt.experts, alt.stride, cfg.qtypes, sel))
    x = synth.gen_x(cfg, seed=9, T=T)
    xd = torch.from_numpy(x.view(np.int16)).to(DEV)
    S = bq.make_scoring(SOFT, n_groups=4, topk_groups=2)
    outs = []
    for handle in (dl.handle, h):
        R = bq.alloc_routing(T, cfg.E, cfg.k, DEV)
        ws = bq.alloc_workspace(handle, T, DEV)
        out = torch.empty((T, cfg.d), dtype=torch.int16, device=DEV)
        bq.moe_forward_decode_scored(handle, S, xd, T, 0, R, ws, out)
        torch.cuda.synchronize()
        outs.append(out.cpu().numpy())
    want = ref.route(R.logits.cpu().numpy(), cfg.k, False, groups=4, topk_groups=2)
    assert np.array_equal(R.topk_ids.cpu().numpy(), want[0])
    # a copy of the same experts in the same families: the same bytes, so the same layer
    a, b = (oracle.bf16_to_f64(o.view(np.uint16)) for o in outs)
    assert np.abs(a - b).max() <= 2e-2 * np.abs(a).max()
