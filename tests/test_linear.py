"""The dense product with packed weights and a fused epilogue (moe_linear_forward).

Two kinds of comparison.  On integers and powers of two every product and sum
is exact in fp32, so the result is the exact value rounded once and has to be
equal bit for bit.  On random values the bound is per value, from the roundings
that the call makes (see _bound), and the whole result's relative error is held
to a rounding's half step.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_quantized_moe_router_amd as bq
import oracle
import scored_reference
import synth
import workloads
from helpers import assert_parity

DEV = "cuda"
FAKE = 1 << 40  # a 256-aligned address that is never dereferenced: every call below fails first
OFFSET = {1: 1.0, 2: 1.5, 3: 3.5}
ACTS = {"none": bq.MOE_ACT_NONE, "silu": bq.MOE_ACT_SILU, "gelu": bq.MOE_ACT_GELU,
        "gelu_tanh": bq.MOE_ACT_GELU_TANH, "relu": bq.MOE_ACT_RELU, "relu2": bq.MOE_ACT_RELU2,
        "sigmoid": bq.MOE_ACT_SIGMOID}


# --------------------------------------------------------------------- refusals (no GPU)
def _call(P, T=2, x=FAKE, xs=None, mul=None, ms=None, res=None, rs=None, out=FAKE + (1 << 36),
          os_=None, ws=FAKE + (1 << 37), ws_bytes=None):
    lib = bq.load()
    K, N = P.K, P.N
    if ws_bytes is None:
        ws_bytes = max(256, lib.moe_linear_workspace_bytes(ctypes.byref(P), max(T, 0)))
    return lib.moe_linear_forward(ctypes.byref(P), x, K if xs is None else xs, T, mul,
                                  N if ms is None else ms, res, N if rs is None else rs, out,
                                  N if os_ is None else os_, ws, ws_bytes, None)


def _desc(K=256, N=48, q=2, act=0, w=FAKE + (1 << 35), bias=None):
    return bq.moe_linear(K, N, q, act, w, bias)


def test_a_null_or_senseless_description_is_refused():
    lib = bq.load()
    assert lib.moe_linear_workspace_bytes(None, 4) == 0
    assert lib.moe_linear_forward(None, FAKE, 256, 2, None, 0, None, 0, FAKE, 48, FAKE, 256,
                                  None) == bq.MOE_ERR_INVALID_ARG
    for bad in (dict(K=0), dict(N=-16), dict(act=-1), dict(act=7)):
        assert _call(_desc(**bad)) == bq.MOE_ERR_INVALID_ARG
        assert lib.moe_linear_workspace_bytes(ctypes.byref(_desc(**bad)), 4) == 0
    for bad in (dict(K=100), dict(N=40), dict(q=4), dict(q=0), dict(K=65536 + 128),
                dict(N=65536 + 16)):
        assert _call(_desc(**bad)) == bq.MOE_ERR_UNSUPPORTED
        assert lib.moe_linear_workspace_bytes(ctypes.byref(_desc(**bad)), 4) == 0


@pytest.mark.parametrize("T", [2, 100])
def test_operands_are_checked_before_any_launch(T):
    # (2048 x 48 at 100 rows: K is split, so the workspace is used)
    P, bad = _desc(K=256 if T == 2 else 2048), bq.MOE_ERR_INVALID_ARG
    other = FAKE + (1 << 34)
    for kw in (dict(T=-1), dict(x=None), dict(x=FAKE + 2), dict(xs=P.K - 8), dict(xs=P.K + 4),
               dict(out=None), dict(out=FAKE + 8), dict(os_=40), dict(os_=52),
               dict(mul=other + 2), dict(mul=other, ms=44), dict(res=other + 8),
               dict(res=other, rs=50),
               dict(out=FAKE), dict(out=FAKE + 256),              # over x
               dict(mul=FAKE + (1 << 36) + 16),                   # out shifted against mul
               dict(res=FAKE + (1 << 36), rs=56)):                # another stride
        kw = dict(T=T, **kw) if "T" not in kw else kw
        assert _call(P, **kw) == bad, kw
    assert _call(_desc(w=None), T=T) == bad
    assert _call(_desc(w=FAKE + 64), T=T) == bad
    assert _call(_desc(bias=FAKE + 2), T=T) == bad
    if T == 100:
        assert _call(P, T=T, ws=None) == bq.MOE_ERR_WORKSPACE
        assert _call(P, T=T, ws_bytes=8) == bq.MOE_ERR_WORKSPACE
        for ws in (FAKE + (1 << 37) + 8, FAKE, FAKE + (1 << 36)):  # unaligned, over x, over out
            assert _call(P, T=T, ws=ws) == bad
        assert _call(P, T=T, mul=other, ws=other) == bad
        assert _call(P, T=T, res=other, ws=other) == bad
    big = (1 << 23) + 8
    assert _call(P, T=T, xs=big) == bq.MOE_ERR_UNSUPPORTED
    assert _call(P, T=T, os_=big) == bq.MOE_ERR_UNSUPPORTED
    assert _call(P, T=T, res=other, rs=big) == bq.MOE_ERR_UNSUPPORTED
    assert _call(P, T=(1 << 24) + 1, ws_bytes=1 << 50) == bq.MOE_ERR_UNSUPPORTED
    assert _call(P, T=0, x=None, out=None, ws=None) == bq.MOE_OK


def test_binding_refuses_tensors_that_do_not_fit():
    P = _desc()
    lin = bq.Linear(P)
    ok = torch.zeros(4, 256, dtype=torch.bfloat16)
    o = torch.zeros(4, 48, dtype=torch.bfloat16)
    for args in ((ok, 4, o), (ok.float(), 4, o), (ok[:, :128], 4, o), (ok, 5, o)):
        with pytest.raises(bq.MoeError):  # host tensors, among others
            bq.moe_linear_forward(lin, *args, None)
    with pytest.raises(bq.MoeError):
        bq.make_linear(256, 48, 2, FAKE, bias=torch.zeros(47))
    with pytest.raises(bq.MoeError):
        bq.make_linear(256, 48, 2, torch.zeros(100, dtype=torch.uint8))
    with pytest.raises(bq.MoeError):  # a host tensor
        bq.make_linear(256, 48, 2, torch.zeros(bq.moe_packed_bytes(2, 256, 48), dtype=torch.uint8))


def test_a_workspace_for_many_rows_does_for_fewer():
    lib = bq.load()
    for K, N in ((256, 48), (8192, 4096), (4096, 16), (65536, 65536)):
        P = _desc(K=K, N=N)
        s = [lib.moe_linear_workspace_bytes(ctypes.byref(P), T) for T in (0, 1, 17, 65, 1000, 9000)]
        assert all(0 < v <= 16 << 20 for v in s) and s == sorted(s)
        for T in list(range(17, 400, 7)) + [1000, 3000, 9000]:
            # a size that covers T: the call passes that check and fails at the next one
            ws = lib.moe_linear_workspace_bytes(ctypes.byref(P), T)
            assert _call(P, T=T, ws_bytes=ws, ws=FAKE + (1 << 50) + 8, out=FAKE) == \
                bq.MOE_ERR_INVALID_ARG


# ------------------------------------------------------------------------------ the GPU's
def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _act64(name, v):
    if name in ("silu", "sigmoid"):
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-v))
        return v * s if name == "silu" else s
    if name == "gelu":
        return 0.5 * v * (1.0 + np.vectorize(math.erf)(v / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if name in ("relu", "relu2"):
        r = np.where(v < 0, 0.0, v)
        return r * r if name == "relu2" else r
    return v


class Case:
    def __init__(self, T, K, N, q, act="none", bias=False, mul=False, res=False, pad=0, seed=0,
                 exact=False, scale=0.05):
        rng = np.random.default_rng([T, K, N, q, seed])
        self.T, self.K, self.N, self.q, self.act, self.pad = T, K, N, q, act, pad
        self.codes = rng.integers(0, synth.LEVELS[q], (N, K)).astype(np.uint8)
        if exact:
            sc = 2.0 ** rng.integers(-2, 2, (N, K // 32)) * rng.choice([-1, 1], (N, K // 32))
            num = lambda *s: rng.integers(-2, 3, s).astype(np.float64)
        else:
            sc = np.abs(rng.normal(0, scale, (N, K // 32)))
            num = lambda *s: rng.standard_normal(s)
        self.scales = sc.astype(np.float16)
        self.x = self._rows(num(T, K))
        self.bias = num(N).astype(np.float32) if bias else None
        self.mul = self._rows(num(T, N)) if mul else None
        self.res = self._rows(num(T, N)) if res else None

    def _rows(self, a):
        return _bf16(a)

    def weights(self):
        w = self.codes.astype(np.float64) - OFFSET[self.q]
        return w * np.repeat(self.scales.astype(np.float64), 32, axis=1)

    def pre(self):
        v = self.x.double().numpy() @ self.weights().T
        return v if self.bias is None else v + self.bias

    def reference(self):
        v = _act64(self.act, self.pre())
        if self.mul is not None:
            v = v * self.mul.double().numpy()
        if self.res is not None:
            v = v + self.res.double().numpy()
        return v

    def _dev(self, t):
        """On the GPU, rows `pad` values apart, with NaN between them."""
        if t is None:
            return None
        full = torch.full((t.shape[0], t.shape[1] + self.pad), float("nan"), dtype=t.dtype,
                          device=DEV)
        full[:, :t.shape[1]] = t.to(DEV)
        return full[:, :t.shape[1]]

    def linear(self):
        blob = bq.moe_pack_weights(self.q, self.codes, self.scales.view(np.uint16))
        b = None if self.bias is None else torch.from_numpy(self.bias).to(DEV)
        return bq.make_linear(self.K, self.N, self.q, torch.from_numpy(blob).to(DEV), bias=b,
                              act=ACTS[self.act])

    def run(self, in_place=False):
        lin = self.linear()
        ws = bq.alloc_linear_workspace(lin, self.T)
        ws.fill_(0x7E)
        full = torch.full((self.T + 2, self.N + self.pad), 7.0, dtype=torch.bfloat16, device=DEV)
        out = full[1:self.T + 1, :self.N]
        res = self._dev(self.res)
        if in_place:
            out.copy_(res)
            res = out
        print(f"[linear] T={self.T} K={self.K} N={self.N} q={self.q} {self.act} pad={self.pad}",
              flush=True)
        bq.moe_linear_forward(lin, self._dev(self.x), self.T, out, ws, mul=self._dev(self.mul),
                              residual=res)
        torch.cuda.synchronize()
        # nothing before, behind or between the rows is touched
        assert (full[0] == 7).all() and (full[-1] == 7).all() and (full[:, self.N:] == 7).all()
        return out.cpu()


def _bound(c):
    """How far a result may be from the 64-bit one, value by value.

    Before the activation, with A = sum |x| |s| and S = sum |x W| + |bias|:
    * up to 16 rows (and perhaps to 64), levels on a base: two 32-term sums of magnitude at most
      1.25 sum |x| each per group, every term rounded once in each of at most
      34 steps (2^-23, whatever the order and rounding mode), times 32 s:
      32 * 2.5 * 34 * 2^-23 A; then K/32 + 10 steps over the groups, 2^-23 S;
    * beyond, weights rounded to 11 bits (half a step, 2^-11 S: three times a
      scale just above 4/3 lies just above 4 and is rounded by up to 2^-9;
      none of ternary ones) and at most K steps of 2^-23 S.
    The activation's slope is at most 1.13 (2 |v| for relu2); its hardware
    exponential takes an argument rounded by 2^-23 |v|, so it is off by 2^-16
    relative for |v| <= 80, and by less than 2^-16 absolute beyond.  Then one
    product, one sum (2^-23 each) and the rounding to bf16, half a step: 2^-8.
    """
    x, w = np.abs(c.x.double().numpy()), np.abs(c.weights())
    S = x @ w.T + (0 if c.bias is None else np.abs(c.bias))
    A = x @ np.repeat(np.abs(c.scales.astype(np.float64)), 32, axis=1).T
    few = 32 * 2.5 * 34 * 2.0 ** -23 * A + (c.K / 32 + 10) * 2.0 ** -23 * S
    e = (0 if c.q == 1 else 2.0 ** -11) * S + c.K * 2.0 ** -23 * S
    e = few if c.T <= 16 else np.maximum(few, e) if c.T <= 64 else e
    v = c.pre()
    a = _act64(c.act, v)
    if c.act == "relu2":
        e = 2 * (np.abs(v) + e) * e
    elif c.act != "none":
        e = 1.13 * e
    e = e + 2.0 ** -16 * (np.abs(a) + (c.act not in ("none", "relu", "relu2")))
    if c.mul is not None:
        e, a = e * np.abs(c.mul.double().numpy()), a * c.mul.double().numpy()
    ref = c.reference()
    e = e + 2.0 ** -22 * (np.abs(a) + np.abs(ref))
    return 2.0 ** -8 * (np.abs(ref) + e) + e


def _check(c, got):
    ref, g = c.reference(), got.double().numpy()
    err = np.abs(g - ref)
    assert np.isfinite(g).all()
    assert (err <= _bound(c)).all(), (err / _bound(c)).max()
    rel = np.linalg.norm(g - ref) / max(np.linalg.norm(ref), 1e-300)
    # all values rounded by half a step at most, and 11-bit weights of random sign: with
    # sum (xW)^2 <= S^2, three deviations of 2^-12 sqrt(sum (xW)^2)
    x2, w2 = c.x.double().numpy() ** 2, c.weights() ** 2
    spread = np.linalg.norm(np.sqrt(x2 @ w2.T) * (1 if c.mul is None
                                                  else np.abs(c.mul.double().numpy())))
    slack = 3 * 2.0 ** -12 * spread / max(np.linalg.norm(ref), 1e-300)
    print(f"  relative error {rel:.3e}", flush=True)
    if c.act not in ("relu2",):
        assert rel <= 2.0 ** -8 + slack


# The kernels: exact for few rows; chunks of K, split or not; tiles of 32, 64 and 128 rows.  The
# shapes below reach every one of them, each with ragged rows and columns.
ROWS = [1, 2, 4, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 300]
MANY = (2111, 4080)  # rows and columns that take the last one (at 256 and 384 deep)


@pytest.mark.gpu
@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("q", [1, 2, 3])
@pytest.mark.parametrize("K,N", [(128, 16), (384, 80), (1152, 272)])
def test_exact_values(T, q, K, N):
    c = Case(T, K, N, q, act=("none", "relu")[T % 2], bias=T % 3 == 0, res=T % 2 == 0, exact=True,
             pad=8 * (T % 4 == 1))
    # |sum| <= 1152 * 2 * 3.5 * 2 = 16128 in steps of 2^-3: exact in fp32
    want = _bf16(c.reference().astype(np.float32))
    assert torch.equal(c.run(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("q", [1, 2, 3])
@pytest.mark.parametrize("T,K,N", [(1, 4096, 528), (7, 1280, 1024), (64, 2176, 1040),
                                   (23, 4096, 16), (700, 2048, 1552), (2100, 640, 4112),
                                   (8200, 256, 2064), (2945, 384, 4080), (3001, 128, 4112),
                                   (530, 512, 4112), (1030, 640, 4080), (45, 384, 4112),
                                   (200, 4096, 1040), (220, 8192, 208),
                                   (MANY[0], 256, MANY[1]), (MANY[0], 384, MANY[1]),
                                   (4099, 128, 1040), (1000, 256, 1040)])
def test_exact_values_at_larger_shapes(q, T, K, N):
    c = Case(T, K, N, q, act="none", bias=True, res=True, exact=True)
    assert torch.equal(c.run(), _bf16(c.reference().astype(np.float32)))


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,K,N", [(3, 512, 160), (40, 640, 160), (90, 2048, 160), (90, 256, 4112),
                                   (MANY[0], 256, MANY[1])])
def test_epilogues(act, T, K, N):
    for q, bias, mul, res in ((1, True, False, True), (2, False, True, False),
                              (3, True, True, True)):
        if T * N > 1e6 and q != 1 + list(ACTS).index(act) % 3:
            continue
        c = Case(T, K, N, q, act, bias, mul, res, pad=8 * (q == 3))
        _check(c, c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (1, 8192, 208), (6, 3968, 1008), (16, 2176, 512),
                                   (50, 1664, 336), (77, 4096, 272), (200, 1152, 1040),
                                   (515, 896, 2000)])
@pytest.mark.parametrize("q", [1, 2, 3])
def test_random_values(T, K, N, q):
    c = Case(T, K, N, q, act="silu" if T % 2 else "none", mul=T > 100, res=T < 100)
    _check(c, c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(4, 512, 96), (80, 512, 96), (20, 2048, 96), (70, 1152, 4096),
                                   (1000, 256, 1040), (3000, 256, 1040), (4099, 128, 1040),
                                   (MANY[0], 256, MANY[1])])
@pytest.mark.parametrize("q", [1, 2, 3])
def test_very_small_and_very_large_scales_and_rows(T, K, N, q):
    for scale in (2.0 ** -22, 2.0 ** -14, 9000.0):
        c = Case(T, K, N, q, scale=scale)
        c.scales = np.minimum(c.scales, np.float16(60000))
        x = c.x.double().numpy()
        x[0] *= 2.0 ** 60
        x[1] *= 2.0 ** -60
        x[2] = 0.0
        x[3, ::3] *= 2.0 ** -12
        c.x = _bf16(x)
        g, ref, e = c.run().double().numpy(), c.reference(), _bound(c)
        assert (np.abs(g - ref) <= e).all(), (np.abs(g - ref) / e).max()
        assert (g[2] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(5, 256, 64), (70, 256, 64), (70, 2048, 64),
                                   (MANY[0], 256, MANY[1])])
def test_infinities_and_nan_stay_in_their_rows(T, K, N):
    c = Case(T, K, N, 2)
    clean = c.run()
    x = c.x.clone()
    x[1, 7] = float("inf")
    x[3, 200] = float("nan")
    c.x = x
    got = c.run()
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[1]).any() and torch.isnan(got[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(8, 512, 256), (200, 512, 256), (200, 1152, 256),
                                   (MANY[0], 256, MANY[1])])
def test_in_place_on_the_residual_stream_and_deterministic(T, K, N):
    c = Case(T, K, N, 3, res=True)
    a, b = c.run(), c.run(in_place=True)
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 640, 144), (33, 640, 144), (150, 2048, 144),
                                   (MANY[0], 256, MANY[1])])
def test_captured_into_a_graph(T, K, N):
    c = Case(T, K, N, 2, act="gelu_tanh", bias=True)
    lin = c.linear()
    ws = bq.alloc_linear_workspace(lin, T)
    x = torch.zeros(T, c.K, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(T, c.N, dtype=torch.bfloat16, device=DEV)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        bq.moe_linear_forward(lin, x, T, out, ws)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            bq.moe_linear_forward(lin, x, T, out, ws)
    for seed in range(3):
        d = Case(T, K, N, 2, act="gelu_tanh", bias=True, seed=seed)
        x.copy_(d.x)
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(out)
        bq.moe_linear_forward(lin, x, T, eager, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        c.x = d.x
        _check(c, out.cpu())


# --------------------------------------------------------------------- together
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 90])
def test_a_block_of_a_model(T):
    """Output projection onto the residual stream, the expert layer with the scored router, a
    gated dense feed-forward layer: each step against its own reference on the GPU's inputs."""
    cfg = synth.small_config(synth.CONFIGS["c0"], name="block", n_shared=1, E=24, k=4)
    dl = workloads.DeviceLayer(cfg, 0, DEV)
    d = cfg.d

    def step(q, K, N, x, act="none", mul=None, res=None, seed=0):
        c = Case(T, K, N, q, act, seed=seed)
        c.x, c.mul, c.res = x, mul, res
        got = c.run()
        _check(c, got)
        return got

    attn = _bf16(np.random.default_rng(1).standard_normal((T, 512)))
    stream = _bf16(np.random.default_rng(2).standard_normal((T, d)))
    h = step(2, 512, d, attn, res=stream, seed=1)

    S = bq.make_scoring(bq.MOE_SCORE_SIGMOID, n_groups=6, topk_groups=3, group_top=2, scale=2.5)
    R = bq.alloc_routing(T, cfg.E, cfg.k, DEV)
    ws = bq.alloc_workspace(dl.handle, T, DEV)
    out = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    fwd = bq.moe_forward_decode_scored if T <= 8 else bq.moe_forward_prefill_scored
    fwd(dl.handle, S, h.to(DEV), T, bq.MOE_ADD_RESIDUAL, R, ws, out)
    torch.cuda.synchronize()
    ids, w, *_ = scored_reference.route(R.logits.cpu().numpy(), cfg.k, True, groups=6,
                                        topk_groups=3, group_top=2, scale=2.5)
    assert np.array_equal(R.topk_ids.cpu().numpy(), ids)
    bits = h.view(torch.int16).numpy().view(np.uint16)
    y, inv = np.zeros((T * cfg.k, d), np.uint16), np.arange(T * cfg.k, dtype=np.int32)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        mats = [synth.gen_matrix(cfg, 0, int(e), m) for m in range(3)]
        y[t * cfg.k + j] = oracle.expert_rows(cfg.qtypes, mats, bits[t])[1]
    sh = oracle.expert_rows(cfg.qtypes, [synth.gen_matrix(cfg, 0, cfg.E, m) for m in range(3)],
                            bits)[1]
    want = oracle.combine(w.astype(np.float32), inv.reshape(T, cfg.k), y, sh, bits, True)
    o = out.cpu()
    assert_parity(o.view(torch.int16).numpy().view(np.uint16), want, f"block T={T}")

    up = step(3, d, 384, o, seed=2)
    gated = step(3, d, 384, o, act="silu", mul=up, seed=3)
    step(2, 384, d, gated, res=o, seed=4)
