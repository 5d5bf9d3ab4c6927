"""The operators around the mixer against their fp64 references (oracle/serve.py, where the
error bounds are derived): block norms, 8-bit rows and projections, beam selection and
state reordering, each alone and together as a beam-search decode step."""
import math

import numpy as np
import pytest
import torch

import gdn_testlib as L
from hybrid_linear_attention_mixer_b200 import gdn
from oracle import serve as S

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def on(x, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(DT[dt])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def worst(err, bound):
    return float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0


# ---------------------------------------------------------------------------
# Block norms
# ---------------------------------------------------------------------------
def norm_case(T, D, gate, act, res, seed):
    rng = np.random.default_rng(seed)
    c = {"o": on(rng.normal(size=(T, D)), act), "x": on(2 * rng.normal(size=(T, D)), res), "gate": None,
         "w_post": on(1 + 0.1 * rng.normal(size=D)), "w_pre": on(1 + 0.1 * rng.normal(size=D))}
    g = np.clip(2 * rng.normal(size={"token": (T,), "channel": (D,)}.get(gate, (T, D))), -7.5, 7.5)
    if gate != "none":
        c["gate"] = on(g, "f32" if gate == "channel" else act)
    return c


def norm_ref(c, cfg):
    g = None if c["gate"] is None else f64(c["gate"])
    if cfg.gate == "token":
        g = g[:, None]
    opt = lambda n: None if c[n] is None else f64(c[n])
    return S.block_norm(opt("o"), f64(c["x"]), g, opt("w_post"), opt("w_pre"), np.float64(np.float32(cfg.res_scale)),
                        np.float64(np.float32(cfg.eps)), cfg.gate_act == "sigmoid")


def check_norm(c, cfg, r, y, act, res):
    rr, ry, p = norm_ref(c, cfg)
    er, ey = S.block_norm_bounds(rr, ry, p)
    if r is not None:
        assert worst(np.abs(f64(r) - rr), S.U[res] * np.abs(rr) + (1 + S.U[res]) * er) <= 1
    if y is not None:
        assert worst(np.abs(f64(y) - ry), S.U[act] * np.abs(ry) + (1 + S.U[act]) * ey) <= 1


NORM_SHAPES = [(1, 8), (1, 2560), (3, 1032), (5, 2568), (33, 1024), (300, 2560), (2, 4096), (3, 6152), (2, 16384)]


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("gate,sigmoid", [("none", False), ("token", True), ("channel", False), ("full", True)])
def test_block_norm_bf16(T, D, gate, sigmoid):
    cfg = gdn.NormConfig(dim=D, res_scale=0.7, gate=gate, gate_act="sigmoid" if sigmoid else "linear")
    c = norm_case(T, D, gate, "bf16", "bf16", T * 31 + D)
    r, y, s = gdn.block_norm(cfg, c["o"], c["x"], c["gate"], c["w_post"], c["w_pre"])
    assert s is None
    check_norm(c, cfg, r, y, "bf16", "bf16")


@pytest.mark.parametrize("act,res", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,D", [(1, 2560), (19, 1336), (4, 5128), (2, 9000)])
def test_block_norm_types(T, D, act, res):
    for gate, sigmoid in (("full", False), ("token", False), ("channel", True)):
        cfg = gdn.NormConfig(dim=D, eps=1e-5, res_scale=-1.25, gate=gate, gate_act="sigmoid" if sigmoid else "linear",
                             act_dtype=DT[act], res_dtype=DT[res])
        c = norm_case(T, D, gate, act, res, T + D)
        r, y, _ = gdn.block_norm(cfg, c["o"], c["x"], c["gate"], c["w_post"], c["w_pre"])
        check_norm(c, cfg, r, y, act, res)


def test_block_norm_parts():
    """Without a norm after the block, without one before the next, without a block."""
    T, D = 37, 2560
    cfg = gdn.NormConfig(dim=D, res_scale=0.5)
    c = norm_case(T, D, "none", "bf16", "bf16", 5)
    r, y, _ = gdn.block_norm(cfg, c["o"], c["x"], None, None, c["w_pre"])
    check_norm(dict(c, w_post=None), cfg, r, y, "bf16", "bf16")
    r, y, _ = gdn.block_norm(cfg, c["o"], c["x"], None, c["w_post"], None)
    assert y is None
    check_norm(dict(c, w_pre=None), cfg, r, None, "bf16", "bf16")
    r, y, _ = gdn.block_norm(cfg, None, c["x"], None, None, c["w_pre"])
    assert r is None
    check_norm(dict(c, o=None, w_post=None), cfg, None, y, "bf16", "bf16")


def test_block_norm_in_place_equals_out_of_place():
    T, D = 65, 2560
    cfg = gdn.NormConfig(dim=D, gate="full", gate_act="sigmoid")
    c = norm_case(T, D, "full", "bf16", "bf16", 6)
    r, y, _ = gdn.block_norm(cfg, c["o"], c["x"], c["gate"], c["w_post"], c["w_pre"])
    o2, x2 = c["o"].clone(), c["x"].clone()
    gdn.block_norm(cfg, o2, x2, c["gate"], c["w_post"], c["w_pre"], r=x2, y=o2)
    assert torch.equal(x2, r) and torch.equal(o2, y)


@pytest.mark.parametrize("T,D", [(1, 2560), (40, 1040), (3, 8208)])
def test_block_norm_to_i8(T, D):
    cfg = gdn.NormConfig(dim=D, gate="full", gate_act="sigmoid")
    c = norm_case(T, D, "full", "bf16", "bf16", 7 + D)
    r, q, scale = gdn.block_norm(cfg, c["o"], c["x"], c["gate"], c["w_post"], c["w_pre"], quantize=True)
    assert q.dtype == torch.int8
    check_norm(c, cfg, r, None, "bf16", "bf16")
    rr, ry, p = norm_ref(c, cfg)
    _, ey = S.block_norm_bounds(rr, ry, p)
    # the scale is of the largest |y|: off by its error, and 2 roundings
    sc = f64(scale)
    ref = np.abs(ry).max(-1) / 127
    assert worst(np.abs(sc - ref), ey.max(-1) / 127 + 2 * S.U32 * ref) <= 1
    # half a quantum, y's error, and the roundings of 127 y, the quotient and the scale
    lim = 0.5 * sc[:, None] + ey + 4 * S.U32 * np.abs(ry)
    assert worst(np.abs(f64(q) * sc[:, None] - ry), lim) <= 1
    assert np.abs(f64(q)).max(-1).min() == 127


# Both sides of every bound between the forms for many rows (more than two to an SM), by dim.
MANY_DIMS = [8, 64, 504, 512, 520, 1024, 1032, 1536, 1544, 2048, 2056, 2560, 4040, 4096, 4104, 8192, 8200]


@pytest.mark.parametrize("D", MANY_DIMS)
@pytest.mark.parametrize("act,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_block_norm_many_rows(D, act, res):
    """The forms for many rows against the reference, in every type, to 8 bits too."""
    T = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    gate = ("none", "token", "channel", "full")[(D // 8 + len(act + res)) % 4]
    cfg = gdn.NormConfig(dim=D, res_scale=0.75, gate=gate, gate_act="sigmoid", act_dtype=DT[act], res_dtype=DT[res])
    c = norm_case(T, D, gate, act, res, D)
    args = (cfg, c["o"], c["x"], c["gate"], c["w_post"], c["w_pre"])
    r, y, _ = gdn.block_norm(*args)
    check_norm(c, cfg, r, y, act, res)
    r8, q, scale = gdn.block_norm(*args, quantize=True)
    assert torch.equal(r8, r)
    rr, ry, p = norm_ref(c, cfg)
    _, ey = S.block_norm_bounds(rr, ry, p)
    sc, ref = f64(scale), np.abs(ry).max(-1) / 127           # the bounds of test_block_norm_to_i8
    assert worst(np.abs(sc - ref), ey.max(-1) / 127 + 2 * S.U32 * ref) <= 1
    assert worst(np.abs(f64(q) * sc[:, None] - ry), 0.5 * sc[:, None] + ey + 4 * S.U32 * np.abs(ry)) <= 1
    assert np.abs(f64(q)).max(-1).min() == 127
    # the commonest call: a residual sum and the norm before the next block, nothing else
    plain = gdn.NormConfig(dim=D, act_dtype=DT[act], res_dtype=DT[res])
    r, y, _ = gdn.block_norm(plain, c["o"], c["x"], None, None, c["w_pre"])
    check_norm(dict(c, gate=None, w_post=None), plain, r, y, act, res)


def test_block_norm_rows_not_finite_or_zero():
    """Infinities and NaN stay in their rows; a row of zeros has the norm zero."""
    T, D = 6, 2560
    cfg = gdn.NormConfig(dim=D)
    c = norm_case(T, D, "none", "bf16", "bf16", 8)
    c["x"][1, 7], c["o"][2, 9], c["x"][3] = float("inf"), float("nan"), 0
    c["o"][3] = 0
    for quantize in (False, True):
        r, y, s = gdn.block_norm(cfg, c["o"], c["x"], None, c["w_post"], c["w_pre"], quantize=quantize)
        good = [0, 4, 5]
        one = {n: (t[good].contiguous() if n in "ox" else t) for n, t in c.items()}
        r1, y1, s1 = gdn.block_norm(cfg, one["o"], one["x"], None, c["w_post"], c["w_pre"], quantize=quantize)
        assert torch.equal(r[good], r1) and torch.equal(y[good], y1)
        assert torch.equal(r[3], torch.zeros_like(r[3])) and not y[3].any()
        if quantize:
            assert torch.equal(s[good], s1) and s[3] == 0
            assert torch.isnan(s[1]) and torch.isnan(s[2]) and not y[1].any() and not y[2].any()
        else:
            assert torch.isnan(y[2]).all() and torch.isnan(y[1, 7])


@pytest.mark.parametrize("T", [8, 600])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_block_norm_sigmoid_of_large_gates(gate, T):
    """o = 1 and x = 0 make r the gate's factor itself: within the error that gdn.h states (from
    the stated errors of the exponential, 2 + 1.173 |g| ulp, the sum, 1/2, and the quotient, 2)."""
    D = 1024
    rng = np.random.default_rng(31)
    n = T if gate == "token" else D
    g = np.concatenate([[-80.0, -20.0, -87.0, 20.0, 80.0, 0.0, -1e-30, -0.0], rng.uniform(-87.2, 100, max(n - 8, 0))])
    g = g if gate != "full" else np.stack([rng.permutation(g) for _ in range(T)])
    cfg = gdn.NormConfig(dim=D, gate=gate, gate_act="sigmoid", act_dtype=torch.float32, res_dtype=torch.float32)
    run = lambda g: gdn.block_norm(cfg, torch.ones((T, D), device=DEV), torch.zeros((T, D), device=DEV), g)[0]
    g = on(g)
    ref = 1 / (1 + np.exp(-f64(g)))
    lim = (5 + 1.2 * np.abs(f64(g))) * 2 * S.U32 * ref
    wide = lambda a: a[:, None] + np.zeros((T, D)) if gate == "token" else a + np.zeros((T, D))
    assert worst(np.abs(f64(run(g)) - wide(ref)), wide(lim)) <= 1
    # beyond: 0 and 1
    for value, want in ((-88.0, 0.0), (-1e30, 0.0), (-math.inf, 0.0), (1e30, 1.0), (math.inf, 1.0)):
        assert torch.equal(run(torch.full_like(g, value)), torch.full((T, D), want, device=DEV))
    assert torch.isnan(run(torch.full_like(g, math.nan))).all()


@pytest.mark.parametrize("T,D,dt", [(6, 2560, "bf16"), (400, 1336, "f32"), (400, 2560, "bf16")])
def test_block_norm_of_infinities_and_overflow(T, D, dt):
    """What gdn.h says of rows that hold an infinity or a NaN, and of finite ones beyond fp32's
    squares, entry by entry."""
    cfg = gdn.NormConfig(dim=D, act_dtype=DT[dt], res_dtype=DT[dt])
    inf, nan = float("inf"), float("nan")
    only = lambda t, row, at, rest: torch.isnan(t[row, at]) and torch.equal(
        torch.cat([t[row, :at], t[row, at + 1:]]), torch.cat([rest[:at], rest[at + 1:]]))
    c = norm_case(T, D, "none", dt, dt, 12)
    x, o, zero = c["x"], c["o"], torch.zeros(D, dtype=DT[dt], device=DEV)
    x[0, 7], o[1, 9], o[2, 11], x[3, 1], x[4] = inf, -inf, nan, nan, 1e19 * torch.sign(x[4].float()).to(DT[dt])
    o[5, ::2] = 1e19
    r, y, _ = gdn.block_norm(cfg, o, x, None, c["w_post"], c["w_pre"])
    assert r[0, 7] == inf and torch.isfinite(r[0]).sum() == D - 1 and only(y, 0, 7, zero)
    assert only(r, 1, 9, x[1]) and torch.isnan(y[1]).all()
    assert torch.isnan(r[2]).all() and torch.isnan(y[2]).all()
    assert torch.isnan(r[3, 1]) and torch.isfinite(r[3]).sum() == D - 1 and torch.isnan(y[3]).all()
    assert not y[4].any() and torch.equal(r[5], x[5])          # finite, but their squares are not
    _, q, s = gdn.block_norm(cfg, o, x, None, c["w_post"], c["w_pre"], quantize=True)
    assert torch.isnan(s[:4]).all() and not q[:5].any() and s[4] == 0 and torch.isfinite(s[5])
    # no norm after the block
    r, y, _ = gdn.block_norm(cfg, o, x, None, None, c["w_pre"])
    assert r[1, 9] == -inf and torch.isfinite(r[1]).sum() == D - 1 and only(y, 1, 9, zero)
    assert torch.isnan(r[2, 11]) and torch.isfinite(r[2]).sum() == D - 1 and torch.isnan(y[2]).all()
    # no block
    _, y, _ = gdn.block_norm(cfg, None, x, None, None, c["w_pre"])
    assert only(y, 0, 7, zero) and torch.isnan(y[3]).all() and not y[4].any() and torch.isfinite(y[1]).all()
    _, q, s = gdn.block_norm(cfg, None, x, None, None, c["w_pre"], quantize=True)
    assert torch.isnan(s[[0, 3]]).all() and not q[[0, 3, 4]].any() and s[4] == 0


# ---------------------------------------------------------------------------
# 8-bit rows and projections
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 2560), (7, 1040), (130, 6144), (3, 16400), (2, 40000)])
def test_quantize_rows_bf16_is_exact(rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = on(rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 20), "bf16")
    x[0, :8] = torch.tensor([1, 2, 3, 4, 5, 6, 7, 8.0])
    q, s = gdn.quantize_rows(x)
    rq, rs = S.quantize_rows(f64(x))
    np.testing.assert_array_equal(f64(q), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), (f64(x.abs().amax(-1)).astype(np.float32) / np.float32(127)))


@pytest.mark.parametrize("cols", [16, 512, 1024, 1040, 2560, 2576, 6144, 6160, 8192, 8208])
def test_quantize_rows_many_rows(cols):
    """Both sides of every bound between the forms, by columns, for more rows than two to an SM:
    exact in bf16, and half a step (and two roundings) in fp32."""
    rows = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 7
    rng = np.random.default_rng(cols)
    x = on(rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 20), "bf16")
    q, s = gdn.quantize_rows(x)
    rq, _ = S.quantize_rows(f64(x))
    np.testing.assert_array_equal(f64(q), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), x.float().abs().amax(-1).cpu().numpy() / np.float32(127))
    x = on(rng.normal(size=(rows, cols)))
    q, s = gdn.quantize_rows(x)
    t = 127 * f64(x) / np.abs(f64(x)).max(-1, keepdims=True)
    assert np.abs(f64(q) - t).max() <= 0.5 + 127 * 2 * S.U32
    np.testing.assert_array_equal(s.cpu().numpy(), x.abs().amax(-1).cpu().numpy() / np.float32(127))


@pytest.mark.parametrize("M,N,K", [(400, 264, 2560), (330, 1000, 1040), (600, 136, 6144), (301, 2312, 512)])
@pytest.mark.parametrize("x_dt", ["bf16", "f32"])
def test_linear_i8_makes_many_rows(M, N, K, x_dt):
    x, _, w, ws = i8_case(M, N, K, M + N + K, x_dt)
    y = gdn.linear_i8(x, w, ws, out_dtype=torch.float32)[0]
    q, xs = gdn.quantize_rows(x)
    assert torch.equal(y, gdn.linear_i8(q, w, ws, x_scale=xs, out_dtype=torch.float32)[0])
    check_linear(y, x, None, w, ws, "f32")


def test_quantize_rows_bf16_ties_and_range():
    """Halves of the largest entry are ties (63.5 -> 64); rows at both ends of the range, of
    zeros, and not finite."""
    rng = np.random.default_rng(3)
    x = on(rng.normal(size=(12, 256)), "bf16")
    for i, top in enumerate([1.0, 1.0078125, 1.9921875, 1.984375, 3e38, 1e-38, 1e-40, 0.0]):
        x[i] = x[i].clamp(-1, 1) * top
        x[i, 0], x[i, 1], x[i, 2] = top, top / 2, -top / 2
    x[8, 3], x[9, 4], x[10, 5] = float("inf"), float("nan"), float("-inf")
    q, s = gdn.quantize_rows(x)
    keep = [0, 1, 2, 3, 4, 5, 6, 7, 11]
    rq, _ = S.quantize_rows(f64(x[keep]))
    np.testing.assert_array_equal(f64(q[keep]), rq)
    assert s[7] == 0 and torch.isnan(s[8:11]).all() and not q[8:11].any()
    np.testing.assert_array_equal(s[keep].cpu().numpy(),
                                  x[keep].float().abs().amax(-1).cpu().numpy() / np.float32(127))


def test_quantize_rows_f32():
    rng = np.random.default_rng(4)
    x = on(rng.normal(size=(9, 2560)))
    x[1] *= 1e30
    x[2] *= 1e-36
    q, s = gdn.quantize_rows(x)
    t = 127 * f64(x) / np.abs(f64(x)).max(-1, keepdims=True)
    # half a step, and the roundings of 127 x and of the quotient (|t| <= 127)
    assert np.abs(f64(q) - t).max() <= 0.5 + 127 * 2 * S.U32


@pytest.mark.parametrize("rows,cols", [(9, 2560), (400, 2560), (700, 1040), (2, 16400)])
def test_quantize_rows_f32_is_that_of_two_fp32_operations(rows, cols):
    """Bit for bit, at both ends of the range too, with many quotients at a half and next to one."""
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(size=(rows, cols)).astype(np.float32)
    x[:, 0] = rng.uniform(3.5, 7, rows)                      # the largest entry, and quotients k + 1/2 of it
    half = (rng.integers(-127, 127, (rows, cols // 2)) + 0.5) / 127 * x[:, :1].astype(np.float64)
    x[:, 1:1 + cols // 2] = half.astype(np.float32)
    with np.errstate(over="ignore"):
        x[1::3] *= np.float32(2.0 ** 120)
        x[2::3] *= np.float32(2.0 ** -100)
        big = np.abs(x.astype(np.float64)).max(-1, keepdims=True)
        # (in fp64, so that 127 x stays in range; rounded to 24 bits each time, by way of [1, 2))
        def fp32(v):
            m, e = np.frexp(v)
            return np.ldexp(m.astype(np.float32).astype(np.float64), e)
        want = np.rint(fp32(fp32(127.0 * x.astype(np.float64)) / big))
    q, s = gdn.quantize_rows(on(x))
    np.testing.assert_array_equal(f64(q), want)
    np.testing.assert_array_equal(s.cpu().numpy(), np.abs(x).max(-1) / np.float32(127))


def i8_case(M, N, K, seed, x_dt="i8"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand(N, generator=g, device=DEV) + 0.5
    if x_dt == "i8":
        x = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
        return x, torch.rand(M, generator=g, device=DEV) + 0.5, w, ws
    return torch.randn((M, K), generator=g, device=DEV).to(DT[x_dt]), None, w, ws


def check_linear(y, x, xs, w, ws, out, rows=None, cols=None):
    """y (concatenated) against the exact sums, on some rows and columns of a large product."""
    if xs is None:
        q, xs = gdn.quantize_rows(x)   # (tested by itself)
    else:
        q = x
    rows = slice(None) if rows is None else rows
    cols = slice(None) if cols is None else cols
    ref = S.linear_i8(q[rows].cpu().numpy(), f64(xs[rows]), w[cols].cpu().numpy(), f64(ws[cols]))
    err = np.abs(f64(y[rows][:, cols]) - ref)
    assert worst(err, (S.U[out] + (1 + S.U[out]) * S.I8_ERR) * np.abs(ref)) <= 1


I8_SHAPES = [(1, 8, 16), (1, 16480, 2560), (5, 200, 144), (16, 136, 6144), (17, 1000, 272), (33, 2560, 6144),
             (64, 5000, 400), (100, 264, 2576), (128, 384, 160), (129, 264, 144), (257, 2312, 2560), (1000, 520, 1040),
             (300, 4040, 128), (1000, 2888, 64), (700, 3464, 32),
             # every pair tile width (160, 192, 224, 256, 128 with 74 pairs), then blocks of 128 tokens with K split
             (1000, 2600, 272), (1000, 3000, 272), (1000, 3496, 272), (1000, 4040, 272), (2500, 896, 272),
             (252, 1728, 3616), (130, 160, 6144), (513, 400, 2064), (900, 136, 1040), (129, 8, 16)]


@pytest.mark.parametrize("M,N,K", I8_SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_i8(M, N, K, out):
    x, xs, w, ws = i8_case(M, N, K, M * 7 + N + K)
    widths = [8, 120, N - 144, 16] if N > 144 else [N]
    outs = [torch.full((M, wd), float("nan"), dtype=DT[out], device=DEV) for wd in widths]
    got = gdn.linear_i8(x, w, ws, x_scale=xs, outs=outs)
    gdn.check_device_error()
    assert got is outs
    check_linear(torch.cat(outs, 1), x, xs, w, ws, out)


@pytest.mark.parametrize("M,N,K", [(1, 16480, 2560), (3, 80, 48), (16, 520, 2560), (65, 264, 6144), (200, 520, 2576),
                                   (8, 2560, 6144), (5, 20000, 6144), (2, 72, 16), (7, 1000, 2576), (8, 40, 12304),
                                   (1, 30000, 7000 // 16 * 16), (4, 24, 131056), (9, 2560, 2560),
                                   (1, 2560, 6144), (2, 2560, 2560), (1, 264, 144), (2, 5000, 2000), (1, 30000, 5104)])
@pytest.mark.parametrize("x_dt", ["bf16", "f32"])
def test_linear_i8_makes_the_rows(M, N, K, x_dt):
    """From bf16 / fp32 rows: bit for bit what gdn_quantize_rows and the 8-bit call give."""
    x, _, w, ws = i8_case(M, N, K, M + N + K, x_dt)
    y = gdn.linear_i8(x, w, ws, out_dtype=torch.float32)[0]
    q, xs = gdn.quantize_rows(x)
    y8 = gdn.linear_i8(q, w, ws, x_scale=xs, out_dtype=torch.float32)[0]
    assert torch.equal(y, y8)
    check_linear(y, x, None, w, ws, "f32")


def test_linear_i8_few_rows_not_finite_or_zero():
    """What gdn_quantize_rows does with such rows, where the product makes them 8-bit itself."""
    M, N, K = 6, 264, 2560
    x, _, w, ws = i8_case(M, N, K, 5, "bf16")
    x[1], x[2, 7], x[3, 2559], x[4] = 0, float("inf"), float("nan"), x[4] * 1e38
    for step in (1, 2, M):
        y = torch.cat([gdn.linear_i8(x[i:i + step], w, ws, out_dtype=torch.float32)[0] for i in range(0, M, step)])
        q, xs = gdn.quantize_rows(x)
        y8 = gdn.linear_i8(q, w, ws, x_scale=xs, out_dtype=torch.float32)[0]
        assert torch.equal(torch.nan_to_num(y, 7.0), torch.nan_to_num(y8, 7.0)) and torch.equal(torch.isnan(y), torch.isnan(y8))
        assert torch.isnan(y[2:4]).all() and not y[1].any() and torch.isfinite(y[[0, 1, 5]]).all()


def test_linear_i8_weights_written_just_before():
    """The weights a call reads may come from the kernel right before it on the stream."""
    M, N, K = 4, 16480, 2560
    x, _, _, _ = i8_case(M, 8, K, 1, "bf16")
    g = torch.Generator(device=DEV).manual_seed(2)
    wf = [torch.randn((N, K), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    ref = []
    for f in wf:
        q, s = gdn.quantize_rows(f)
        torch.cuda.synchronize()
        ref.append(gdn.linear_i8(x, q, s)[0])
    w, ws = torch.empty((N, K), dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    for i in (0, 1, 0, 1):
        gdn.quantize_rows(wf[i], w, ws)
        y = gdn.linear_i8(x, w, ws)[0]
        assert torch.equal(y, ref[i])


def test_linear_i8_extremes():
    """The largest sums (all -128, the longest K), and scales of zero, infinity and NaN."""
    M, N, K = 3, 136, 131056
    x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    one = lambda n: torch.ones(n, device=DEV)
    y = gdn.linear_i8(x, w, one(N), x_scale=one(M), out_dtype=torch.float32)[0]
    assert torch.equal(y, torch.full_like(y, float(K * 16384)))
    xs, ws = one(M), one(N)
    xs[1], ws[5], ws[6] = float("nan"), float("inf"), 0.0
    y = gdn.linear_i8(x, w, ws, x_scale=xs, out_dtype=torch.float32)[0]
    assert torch.isnan(y[1]).all() and torch.isinf(y[0, 5]) and y[0, 6] == 0 and torch.isfinite(y[0, :5]).all()


def test_linear_i8_many_rows_offsets_past_32_bits():
    """M x N past 2^31: the last rows and columns."""
    M, N, K = 131328, 16480, 32
    x, xs, w, ws = i8_case(M, N, K, 9)
    y = gdn.linear_i8(x, w, ws, x_scale=xs)[0]
    check_linear(y, x, xs, w, ws, "bf16", rows=slice(M - 300, M))
    check_linear(y, x, xs, w, ws, "bf16", rows=slice(0, 40))


@pytest.mark.parametrize("M", [3, 40, 100, 200])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_i8_writes_its_rows_only(M, out):
    """What lies behind the last row stays as it was (tiles reach past it)."""
    N, K = 392, 272
    x, xs, w, ws = i8_case(M, N, K, M, "i8")
    widths = (136, 256)
    big = [torch.full((M + 130, wd), 7.0, dtype=DT[out], device=DEV) for wd in widths]
    gdn.linear_i8(x, w, ws, x_scale=xs, outs=[b[:M] for b in big])
    check_linear(torch.cat([b[:M] for b in big], 1), x, xs, w, ws, out)
    assert all((b[M:] == 7.0).all() for b in big)


def test_projections_i8():
    cfg = gdn.Config()
    for T in (1, 70, 150):
        x, _, w, ws = i8_case(T, 16480, 2560, T, "bf16")
        p = gdn.in_proj_i8(cfg, x, w, ws)
        y = torch.cat([p[n].reshape(T, -1) for n in "qkvzab"], 1)
        check_linear(y, x, None, w, ws, "bf16")
        q, xs = gdn.quantize_rows(x)
        p8 = gdn.in_proj_i8(cfg, q, w, ws, hidden_scale=xs)
        assert all(torch.equal(p[n], p8[n]) for n in "qkvzab")
        o, _, wo, wos = i8_case(T, 2560, 6144, T + 1, "bf16")
        check_linear(gdn.out_proj_i8(cfg, o, wo, wos), o, None, wo, wos, "bf16")


# ---------------------------------------------------------------------------
# Beam selection
# ---------------------------------------------------------------------------
def beam_case(G, W, V, dt, seed, sigma=2.5):
    rng = np.random.default_rng(seed)
    return on(sigma * rng.normal(size=(G, W, V)), dt), on(-8 * rng.random(size=(G, W)))


def check_beam(logits, scores, n, got, finished=None, pad=0):
    ref = S.beam_select(logits.detach().cpu().float().numpy(), scores.cpu().numpy(), n, finished, pad)
    # inputs with a near tie between beams would say nothing: their results may be either way round
    assert ref[3] > 2 * S.BEAM_ERR, "choose other inputs: beams %.1e apart" % ref[3]
    np.testing.assert_array_equal(got[0].cpu().numpy(), ref[0])
    np.testing.assert_array_equal(got[1].cpu().numpy(), ref[1])
    g = f64(got[2])
    fin = np.isfinite(ref[2])
    assert np.array_equal(np.isfinite(g), fin) and (g[~fin] == -np.inf).all()
    assert worst(np.abs(g[fin] - ref[2][fin]), S.BEAM_ERR + 2 * S.U32 * np.abs(ref[2][fin])) <= 1


BEAM_SHAPES = [(1, 1, 1, 1), (1, 1, 5, 9), (1, 4, 248320, 4), (3, 5, 32003, 10), (2, 32, 1000, 64), (4, 3, 16384, 6),
               (2, 2, 16385, 3), (1, 8, 50001, 16), (5, 1, 777, 64), (1, 2, 1 << 20, 2)]


@pytest.mark.parametrize("G,W,V,n", BEAM_SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_beam_select(G, W, V, n, dt):
    logits, scores = beam_case(G, W, V, dt, G + W + V + n)
    check_beam(logits, scores, n, gdn.beam_select(logits, scores, n_out=n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [0.3, 0.999])
def test_beam_select_masks_finished_and_unused_beams(dt, masked):
    """Token masks, one beam with nothing allowed, beams that have ended (one of them not in
    use), and a group at its first step."""
    G, W, V, n, pad = 5, 4, 20011, 8, 17
    logits, scores = beam_case(G, W, V, dt, 11)
    rng = np.random.default_rng(12)
    logits.masked_fill_(torch.from_numpy(rng.random((G, 1, V)) < masked).to(DEV), -math.inf)
    logits[2, 3] = -math.inf
    scores[0, 1:] = -math.inf
    finished = np.zeros((G, W), np.uint8)
    finished[1, 2] = finished[3, 0] = finished[3, 1] = finished[4] = 1
    finished[0, 3] = 1
    logits[3, 0] = float("nan")   # (not read)
    for f in (torch.from_numpy(finished), torch.from_numpy(finished).bool()):
        check_beam(logits, scores, n, gdn.beam_select(logits, scores, n_out=n, finished=f.to(DEV), pad_token=pad),
                   finished, pad)


def test_beam_select_nothing_left():
    G, W, V, n = 2, 3, 5000, 4
    logits, scores = beam_case(G, W, V, "f32", 13)
    logits[0] = -math.inf
    scores[1] = -math.inf
    p, t, s = gdn.beam_select(logits, scores, n_out=n)
    assert (p == -1).all() and (t == -1).all() and (s == -math.inf).all()
    # one allowed token in one beam
    logits[0, 1, 4999] = 3.0
    p, t, s = gdn.beam_select(logits, scores, n_out=n)
    assert p[0].tolist() == [1, -1, -1, -1] and t[0].tolist() == [4999, -1, -1, -1]
    assert s[0, 0] == scores[0, 1]


def test_beam_select_rows_not_finite():
    """A NaN or +inf takes its beam out of the selection, wherever it stands."""
    W, V, n = 6, 40000, 5
    logits, scores = beam_case(1, W, V, "bf16", 14)
    scores[:] = scores[0, 0]
    logits[0, 1, 39999], logits[0, 2, 3], logits[0, 3, 20000] = float("nan"), float("inf"), float("-inf")
    logits[0, 4] = -math.inf
    logits[0, 4, 7] = float("nan")
    scores[0, 5] = float("nan")
    p, t, s = gdn.beam_select(logits, scores, n_out=n)
    ok = [0, 3]
    p2, t2, s2 = gdn.beam_select(logits[:, ok].contiguous(), scores[:, ok].contiguous(), n_out=n)
    assert torch.equal(p, p2 * 3) and torch.equal(t, t2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_beam_select_masks_of_the_lowest_value(dt):
    """Masks by the type's lowest finite value: such tokens are candidates still, behind all
    others; a row of nothing else is an even distribution."""
    G, W, V, n = 3, 2, 17000, 12
    logits, scores = beam_case(G, W, V, dt, 19)
    low = torch.finfo(DT[dt]).min
    rng = np.random.default_rng(20)
    logits.masked_fill_(torch.from_numpy(rng.random((G, W, V)) < 0.5).to(DEV), low)
    logits[1, :, 5:] = low          # 5 tokens left in each beam, and one tie of many
    logits[2, 1] = low
    scores[2, 0] = scores[2, 1] - 9
    check_beam(logits, scores, n, gdn.beam_select(logits, scores, n_out=n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 50001])
def test_beam_select_scores_that_hide_the_logits(dt, V):
    """Beams put out of use by a large finite score (the type's lowest value among them): fp64 does
    not tell their tokens' scores apart, their logits do, equal ones by the lowest token."""
    W, n = 4, 24
    logits, _ = beam_case(6, W, V, dt, 23)
    rng = np.random.default_rng(24)
    keep = torch.from_numpy(rng.permutation(V)[:5]).to(DEV)
    first = torch.full((V,), -math.inf, dtype=DT[dt], device=DEV)
    first[keep] = torch.arange(5, device=DEV).to(DT[dt])
    logits[:, 0] = first                                    # five tokens left in the beam in use
    logits[5, 1] = torch.round(logits[5, 1].float()).to(DT[dt])
    scores = torch.zeros((6, W), device=DEV)
    for g, low in enumerate((-1e12, -1e17, -1e30, torch.finfo(torch.float32).min, -3e20, -1e30)):
        scores[g, 1:] = low
        scores[g, 2] = -math.inf
    scores[4, 3] = -2e20                                    # (before beam 1)
    p, t, s = gdn.beam_select(logits, scores, n_out=n)
    assert not p[:, :5].any() and torch.equal(t[:, :5].long(), keep.flip(0).expand(6, 5))
    for g in range(6):
        if g > 0:   # (beside 1e12, with steps of 1e-4, the beams still take turns)
            w = 3 if g == 4 else 1
            assert (p[g, 5:] == w).all() and (s[g, 5:] == scores[g, w]).all()
        for w in (1, 3):
            x = logits[g, w].cpu().float().numpy().astype(np.float64)
            mine = t[g, 5:][p[g, 5:] == w].tolist()
            assert mine == np.lexsort((np.arange(V), -x))[:len(mine)].tolist()
        assert ((p[g, 5:] == 1) | (p[g, 5:] == 3)).all()


def test_beam_select_large_logits():
    """Rows with a large common offset, and of either sign of a large value."""
    G, W, V, n = 4, 2, 9000, 6
    logits, scores = beam_case(G, W, V, "f32", 21)
    for g, off in enumerate((1e4, -3e5, 1e20, 3e38)):
        logits[g] += off
    check_beam(logits, scores, n, gdn.beam_select(logits, scores, n_out=n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 20000, 33001])
def test_beam_select_ties(dt, V):
    """Equal logits go to the lowest token, equal beams to the lowest beam, at any alignment:
    constant rows, rows of two values, +0 beside -0."""
    W, n = 3, 40
    logits = torch.zeros((4, W, V), device=DEV, dtype=DT[dt])
    scores = torch.zeros((4, W), device=DEV)
    logits[1, :, V // 2:] = 1.0
    logits[2, :, ::2] = -0.0
    logits[3] = torch.from_numpy(np.random.default_rng(15).integers(-2, 3, (1, V)).astype(np.float32)).to(DEV)
    p, t, _ = gdn.beam_select(logits, scores, n_out=n)
    for g in range(4):
        ref = S.beam_select(logits[g:g + 1].cpu().float().numpy(), np.zeros((1, W)), n)
        np.testing.assert_array_equal(p[g:g + 1].cpu().numpy(), ref[0])
        np.testing.assert_array_equal(t[g:g + 1].cpu().numpy(), ref[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 30])
def test_beam_select_many_ties_below_a_few(dt, n):
    """A few distinct logits above, then thousands of equal ones spread over the row; the
    equal ones everywhere but at its start; and equal ones that are fewer than n."""
    W, V = 2, 70000
    rng = np.random.default_rng(17)
    x = np.full((3, W, V), -3.0)
    x[0] = np.where(rng.random((W, V)) < 0.1, 4.0, rng.integers(-12, 4, (W, V)))
    x[1, :, 60000:] = 2.5
    x[1, :, :60000] = rng.integers(-9, 0, (W, 60000))
    for w in range(W):
        x[:, w, rng.permutation(V)[:12]] = 8 + np.arange(12) * 0.25
    x[2, :, rng.permutation(V)[:5]] = 6.0
    logits, scores = on(x, dt), torch.zeros((3, W), device=DEV)
    # Two beams with the same logits in another order have the same sum of exponentials but for
    # its rounding, within BEAM_ERR: which of their equal candidates comes first is not said.
    # Their scores are.
    _, _, s = gdn.beam_select(logits, scores, n_out=n)
    ref = S.beam_select(logits.cpu().float().numpy(), np.zeros((3, W)), n)[2]
    assert worst(np.abs(f64(s) - ref), S.BEAM_ERR + 2 * S.U32 * np.abs(ref)) <= 1
    # each beam by itself, where nothing but the logits decides
    for w in range(W):
        one = logits[:, w:w + 1].contiguous()
        p, t, _ = gdn.beam_select(one, scores[:, :1].contiguous(), n_out=n)
        ref = S.beam_select(one.cpu().float().numpy(), np.zeros((3, 1)), n)
        np.testing.assert_array_equal(p.cpu().numpy(), ref[0])
        np.testing.assert_array_equal(t.cpu().numpy(), ref[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_beam_select_row_starts(dt):
    """Rows at every offset within 16 bytes, and rows further apart than the vocabulary."""
    W, V, n = 4, 16411, 8
    base, scores = beam_case(1, W, V, dt, 16)
    ref = gdn.beam_select(base, scores, n_out=n)
    check_beam(base, scores, n, ref)
    size = 2 if dt == "bf16" else 4
    for off in range(16 // size):
        for ld in (V, V + 1, V + 6):
            flat = torch.full((off + W * ld + 16,), float("nan"), dtype=DT[dt], device=DEV)
            view = flat[off:off + W * ld].as_strided((1, W, V), (W * ld, ld, 1), off)
            view.copy_(base)
            got = gdn.beam_select(view, scores, n_out=n)
            assert all(torch.equal(a, b) for a, b in zip(got, ref)), (off, ld)


def test_beam_select_scores_in_place():
    logits, scores = beam_case(6, 4, 9000, "bf16", 18)
    p, t, s = gdn.beam_select(logits, scores)
    mine = scores.clone()
    p2, t2, s2 = gdn.beam_select(logits, mine, out_scores=mine)
    assert s2 is mine and torch.equal(p, p2) and torch.equal(t, t2) and torch.equal(s, mine)


def test_beam_select_offsets_past_32_bits():
    G, W, V, n = 65, 32, 1 << 20, 3
    logits = torch.zeros((G, W, V), dtype=torch.bfloat16, device=DEV)
    scores = torch.zeros((G, W), device=DEV)
    scores[:, 30:] = 1.0
    logits[G - 1, 31, V - 5:] = torch.tensor([1.0, 3.0, 2.0, 9.0, 9.0]).to(torch.bfloat16)
    p, t, _ = gdn.beam_select(logits, scores, n_out=n)
    assert p[G - 1].tolist() == [31, 31, 31] and t[G - 1].tolist() == [V - 2, V - 1, V - 4]
    assert (p[:G - 1] == 30).all() and (t[:G - 1] == torch.arange(n, device=DEV)).all()


# ---------------------------------------------------------------------------
# State reordering
# ---------------------------------------------------------------------------
def states_of(n, seed, shapes):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randint(-2 ** 31, 2 ** 31 - 1, (n,) + s, generator=g, device=DEV, dtype=torch.int32) for s in shapes]


@pytest.mark.parametrize("G,W", [(1, 1), (1, 2), (3, 3), (2, 4), (5, 7), (1, 8), (2, 13), (1, 16), (2, 17), (1, 32)])
def test_reorder_states(G, W):
    shapes = [(4,), (48, 16), (1025, 4), (3, 5, 4), (9000,)]
    states = states_of(G * W, G * 100 + W, shapes)
    rng = np.random.default_rng(G + W)
    plan = gdn.reorder_plan(states, G, W)
    cases = [rng.integers(-1, W, (G, W)), np.tile(np.arange(W)[::-1], (G, 1)), np.tile((np.arange(W) + 1) % W, (G, 1)),
             np.zeros((G, W), int), np.tile(np.arange(W), (G, 1)), np.full((G, W), -1), np.full((G, W), W - 1)]
    for k, par in enumerate(cases):
        ref = [S.reorder(t.cpu().numpy(), par) for t in states]
        gdn.reorder_states(torch.from_numpy(par.astype(np.int32)).to(DEV), plan if k % 2 else states)
        gdn.check_device_error()
        for t, r in zip(states, ref):
            np.testing.assert_array_equal(t.cpu().numpy(), r)


def test_reorder_states_layouts():
    """Layers interleaved within a sequence's memory, states with gaps between them, the
    library's own states of several layers."""
    G, W, Lr = 2, 3, 4
    big = states_of(G * W, 1, [(Lr, 40, 4)])[0]                 # [sequences][layers][...]
    gap = states_of(G * W, 2, [(3, 64)])[0]
    rec = torch.randn((Lr, G * W, 6, 32, 32), device=DEV)
    conv = torch.randn((Lr, G * W, 320, 3), device=DEV).to(torch.bfloat16)
    par = np.array([[2, 0, 1], [1, 1, -1]])
    before = [t.cpu().clone() for t in (big, gap, rec, conv)]
    states = [big[:, i] for i in range(Lr)] + [gap[:, 1]] + list(rec) + list(conv)
    gdn.reorder_states(torch.from_numpy(par.astype(np.int32)).to(DEV), states)
    np.testing.assert_array_equal(big.cpu().numpy(), S.reorder(before[0].numpy(), par))
    ref = before[1].numpy().copy()
    ref[:, 1] = S.reorder(ref[:, 1], par)
    np.testing.assert_array_equal(gap.cpu().numpy(), ref)       # the gaps are as they were
    for i in range(Lr):
        np.testing.assert_array_equal(rec[i].cpu().numpy(), S.reorder(before[2][i].numpy(), par))
        np.testing.assert_array_equal(conv[i].cpu().view(torch.int16).numpy(),
                                      S.reorder(before[3][i].view(torch.int16).numpy(), par))


def test_reorder_states_bad_parent_leaves_its_group():
    G, W = 3, 4
    states = states_of(G * W, 3, [(5000,), (64,)])
    par = np.array([[1, 0, 3, 2], [0, 4, 0, 0], [0, 0, 0, -2]])
    ref = [S.reorder(t.cpu().numpy(), np.where((par < -1).any(1, keepdims=True) | (par >= W).any(1, keepdims=True), -1, par))
           for t in states]
    gdn.reorder_states(torch.from_numpy(par.astype(np.int32)).to(DEV), states)
    with pytest.raises(gdn.GdnError) as e:
        gdn.check_device_error()
    assert e.value.status == 8
    gdn.check_device_error()   # (cleared)
    for t, r in zip(states, ref):
        np.testing.assert_array_equal(t.cpu().numpy(), r)


def test_reorder_states_offsets_past_32_bits():
    """One buffer of 12 GiB, states 3 GiB apart."""
    W, n = 4, 3 << 28   # int32 entries a state
    t = torch.zeros((W, n), dtype=torch.int32, device=DEV)
    t[:, -1] = torch.arange(1, W + 1, device=DEV, dtype=torch.int32)
    t[:, 5] = torch.arange(11, 11 + W, device=DEV, dtype=torch.int32)
    gdn.reorder_states(torch.tensor([[3, 0, 0, 2]], dtype=torch.int32, device=DEV), [t])
    assert t[:, -1].tolist() == [4, 1, 1, 3] and t[:, 5].tolist() == [14, 11, 11, 13]
    assert int(torch.count_nonzero(t)) == 2 * W


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
class Step:
    """One beam-search decode step of a layer with 8-bit projections and its logits."""

    def __init__(self, G, W, V, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s, dt=torch.bfloat16, k=1.0: (torch.randn(s, generator=g, device=DEV) * k).to(dt)
        w8 = lambda n, k: gdn.quantize_rows(rnd(n, k, k=k ** -0.5))
        B, D = G * W, 2560
        self.G, self.W, self.V = G, W, V
        self.cfg, self.ncfg = gdn.Config(), gdn.NormConfig(gate="full", gate_act="sigmoid", res_scale=0.5)
        self.first = gdn.NormConfig()
        self.w = {"conv_w": rnd(10240, 4, dt=torch.float32, k=0.5), "A_log": torch.rand(48, generator=g, device=DEV),
                  "dt_bias": rnd(48, dt=torch.float32, k=0.1), "norm_w": torch.ones(128, device=DEV)}
        self.n1, self.n2, self.n3 = (1 + rnd(D, dt=torch.float32, k=0.1) for _ in range(3))
        self.w_in, self.w_out, self.w_lm = w8(16480, D), w8(D, 6144), w8(V, D)
        self.x, self.gate = rnd(B, D), rnd(B, D)
        self.conv0, self.rec0 = rnd(B, 10240, 3), rnd(B, 48, 128, 128, dt=torch.float32, k=0.02)
        self.scores0 = -torch.rand((G, W), generator=g, device=DEV)
        self.conv, self.rec, self.scores = self.conv0.clone(), self.rec0.clone(), self.scores0.clone()
        self.x_run = self.x.clone()
        self.ws = {n: torch.empty(s, dtype=torch.uint8, device=DEV) for n, s in
                   (("out", gdn.linear_i8_workspace_size(B, 6144)), ("lm", gdn.linear_i8_workspace_size(B, D)),
                    ("beam", gdn.beam_workspace_size(G, W, V, W, torch.float32)))}
        self.got = {}

    def reset(self):
        for a, b in ((self.conv, self.conv0), (self.rec, self.rec0), (self.scores, self.scores0), (self.x_run, self.x)):
            a.copy_(b)

    def run(self):
        x, c = self.x_run, self.cfg
        _, h, hs = gdn.block_norm(self.first, None, x, w_pre=self.n1, quantize=True)
        p = gdn.in_proj_i8(c, h, *self.w_in, hidden_scale=hs)
        o = gdn.decode(c, self.w, p["q"], p["k"], p["v"], p["a"], p["b"], p["z"], self.conv, self.rec)
        y = gdn.out_proj_i8(c, o, *self.w_out, workspace=self.ws["out"])
        _, f, _ = gdn.block_norm(self.ncfg, y, x, self.gate, self.n2, self.n3, r=x)
        lg = gdn.linear_i8(f, *self.w_lm, out_dtype=torch.float32, workspace=self.ws["lm"])[0]
        par, tok, sc = gdn.beam_select(lg.view(self.G, self.W, self.V), self.scores, out_scores=self.scores,
                                       workspace=self.ws["beam"])
        gdn.reorder_states(par, [self.conv, self.rec, x])
        self.got.update(h=h, hs=hs, p=p, o=o, y=y, f=f, lg=lg, par=par, tok=tok, sc=sc)


def test_decode_step_of_a_beam_search():
    """Each operator of the step against its reference on what it was given, the states after
    the reordering against those of the same step without it."""
    s = Step(2, 3, 5003 // 8 * 8, 21)
    s.run()
    gdn.check_device_error()
    g = s.got
    # the norm before the block, in 8 bits
    r, ry, p = S.block_norm(None, f64(s.x), None, None, f64(s.n1), 1.0, 1e-6, False)
    _, ey = S.block_norm_bounds(r, ry, p)
    sc = f64(g["hs"])[:, None]
    assert worst(np.abs(f64(g["h"]) * sc - ry), 0.5 * sc + ey + 4 * S.U32 * np.abs(ry)) <= 1
    check_linear(torch.cat([g["p"][n] for n in "qkvzab"], 1), g["h"], g["hs"], *s.w_in, "bf16")
    # the mixer: the library's decode on these inputs (its own parity tests cover it)
    conv, rec = s.conv0.clone(), s.rec0.clone()
    o = gdn.decode(s.cfg, s.w, *[g["p"][n] for n in "qkvabz"], conv, rec)
    assert torch.equal(o, g["o"])
    check_linear(g["y"], g["o"], None, *s.w_out, "bf16")
    c = {"o": g["y"], "x": s.x, "gate": s.gate, "w_post": s.n2, "w_pre": s.n3}
    rr, _, _ = gdn.block_norm(s.ncfg, g["y"], s.x, s.gate, s.n2, s.n3)
    check_norm(c, s.ncfg, rr, g["f"], "bf16", "bf16")
    check_linear(g["lg"], g["f"], None, *s.w_lm, "f32")
    check_beam(g["lg"].view(2, 3, -1), s.scores0, 3, (g["par"], g["tok"], g["sc"]))
    par = g["par"].cpu().numpy()
    for now, before in ((s.conv, conv), (s.rec, rec), (s.x_run, rr)):
        np.testing.assert_array_equal(f64(now), S.reorder(f64(before), par))


def test_decode_step_replays_from_a_graph():
    s = Step(2, 2, 4096, 22)
    s.run()
    torch.cuda.synchronize()
    ref = {n: s.got[n].clone() for n in ("o", "y", "f", "lg", "par", "tok", "sc")}
    ref.update(conv=s.conv.clone(), rec=s.rec.clone(), x=s.x_run.clone())
    s.reset()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            s.run()
    for _ in range(2):
        s.reset()
        graph.replay()
        torch.cuda.synchronize()
        gdn.check_device_error()
        assert all(torch.equal(s.got[n], ref[n]) for n in ("o", "y", "f", "lg", "par", "tok", "sc"))
        assert torch.equal(s.conv, ref["conv"]) and torch.equal(s.rec, ref["rec"]) and torch.equal(s.x_run, ref["x"])
    del graph


def test_graphs_that_share_a_workspace():
    """Two captured steps of different sizes over one set of workspaces, replayed in turn."""
    steps = [Step(2, 2, 4096, 25), Step(1, 3, 8192, 26)]
    size = {n: max(s.ws[n].numel() for s in steps) for n in steps[0].ws}
    shared = {n: torch.empty(v, dtype=torch.uint8, device=DEV) for n, v in size.items()}
    ref, graphs = [], []
    for s in steps:
        s.ws = shared
        s.run()
        torch.cuda.synchronize()
        ref.append((s.scores.clone(), s.rec.clone(), s.x_run.clone()))
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
            s.run()
        graphs.append(g)
    for _ in range(3):
        for s in steps:
            s.reset()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        gdn.check_device_error()
        for s, r in zip(steps, ref):
            assert torch.equal(s.scores, r[0]) and torch.equal(s.rec, r[1]) and torch.equal(s.x_run, r[2])
    del graphs


def test_prefill_between_8_bit_projections():
    """hidden -> norm to 8 bits -> in_proj -> prefill, whose work forks onto side streams ->
    out_proj -> norm with the residual, queued at once and from a graph: what the same calls
    give with a synchronisation after each."""
    T, cfg = 4200, gdn.Config(prefill_segments=3)
    g = torch.Generator(device=DEV).manual_seed(29)
    rnd = lambda *s, dt=torch.bfloat16, k=1.0: (torch.randn(s, generator=g, device=DEV) * k).to(dt)
    w = {"conv_w": rnd(10240, 4, dt=torch.float32, k=0.5), "A_log": torch.rand(48, generator=g, device=DEV),
         "dt_bias": rnd(48, dt=torch.float32, k=0.1), "norm_w": torch.ones(128, device=DEV)}
    n1, n2, n3 = (1 + rnd(2560, dt=torch.float32, k=0.1) for _ in range(3))
    w_in, w_out = (gdn.quantize_rows(rnd(n, k, k=k ** -0.5)) for n, k in ((16480, 2560), (2560, 6144)))
    x, gate = rnd(T, 2560), rnd(T, 2560)
    cu = torch.tensor([0, 1500, T], dtype=torch.int32, device=DEV)
    conv, rec = torch.zeros((2, 10240, 3), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 48, 128, 128), device=DEV)
    ws = torch.empty(gdn.workspace_size(cfg, T, 2), dtype=torch.uint8, device=DEV)
    ws8 = torch.empty(gdn.linear_i8_workspace_size(T, 6144), dtype=torch.uint8, device=DEV)
    ncfg = gdn.NormConfig(gate="full", gate_act="sigmoid", res_scale=0.5)

    def run(between=lambda: None):
        conv.zero_()
        rec.zero_()
        out = []
        _, h, hs = gdn.block_norm(gdn.NormConfig(), None, x, w_pre=n1, quantize=True)
        between()
        p = gdn.in_proj_i8(cfg, h, *w_in, hidden_scale=hs)
        between()
        o = gdn.prefill(cfg, w, p["q"], p["k"], p["v"], p["a"], p["b"], p["z"], conv, rec, cu, workspace=ws)
        between()
        y = gdn.out_proj_i8(cfg, o, *w_out, workspace=ws8)
        between()
        r, f, _ = gdn.block_norm(ncfg, y, x, gate, n2, n3)
        between()
        return [o, y, r, f]

    ref = [t.clone() for t in run(torch.cuda.synchronize)] + [conv.clone(), rec.clone()]
    gdn.check_device_error()
    for _ in range(3):
        got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + [conv, rec], ref))
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        got = run()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        gdn.check_device_error()
        assert all(torch.equal(a, b) for a, b in zip(got + [conv, rec], ref))
    del graph


FIRST_CALL = """
import sys
sys.path[:0] = [%r, %r]
import torch
import test_gpu_serve_ops as T
s = T.Step(1, 2, 4096, 27)   # (its weights' 8-bit rows are the library's first call)
torch.cuda.synchronize()
g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
st.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
    s.run()
g.replay()
torch.cuda.synchronize()
T.gdn.check_device_error()
got = (s.scores.clone(), s.rec.clone(), s.x_run.clone())
s.reset()
s.run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (s.scores, s.rec, s.x_run)))
print("captured first")
"""


def test_first_calls_may_be_captured():
    """A process that captures the products, the selection and the reordering before it has
    ever made such a call directly."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % (os.path.dirname(here), here)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def test_reorder_after_selection_of_a_whole_model():
    """The states of 36 layers in one call (72 buffers)."""
    G, W, Lr = 1, 4, 36
    rec = torch.randn((Lr, G * W, 6, 32, 32), device=DEV)
    conv = torch.randn((Lr, G * W, 320, 3), device=DEV).to(torch.bfloat16)
    before = rec.clone(), conv.clone()
    logits, scores = beam_case(G, W, 20000, "bf16", 28)
    par, _, _ = gdn.beam_select(logits, scores)
    gdn.reorder_states(par, gdn.reorder_plan(list(rec) + list(conv), G, W))
    gdn.check_device_error()
    at = par[0].long()
    assert torch.equal(rec, before[0][:, at]) and torch.equal(conv, before[1][:, at])


def test_two_streams_at_once():
    """Steps on two streams, with their own buffers, give what they give alone."""
    steps = [Step(2, 2, 4096, 23), Step(1, 3, 8192, 24)]
    ref = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        ref.append((s.scores.clone(), s.rec.clone(), s.x_run.clone()))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s in steps:
            s.reset()
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        gdn.check_device_error()
        for s, r in zip(steps, ref):
            assert torch.equal(s.scores, r[0]) and torch.equal(s.rec, r[1]) and torch.equal(s.x_run, r[2])


def test_stream_argument():
    """Calls with a stream of their own: their buffers come from that stream's pool."""
    st = torch.cuda.Stream()
    x, _, w, ws = i8_case(40, 264, 2560, 30, "bf16")
    logits, scores = beam_case(2, 3, 5000, "f32", 31)
    ref = gdn.linear_i8(x, w, ws)[0], gdn.quantize_rows(x), gdn.beam_select(logits, scores)
    torch.cuda.synchronize()
    got = gdn.linear_i8(x, w, ws, stream=st)[0], gdn.quantize_rows(x, stream=st), gdn.beam_select(logits, scores, stream=st)
    st.synchronize()
    assert torch.equal(got[0], ref[0])
    assert all(torch.equal(a, b) for i in (1, 2) for a, b in zip(got[i], ref[i]))


def test_binding_refuses():
    """Wrong types, shapes, layouts and devices reach no kernel."""
    T, D = 4, 2560
    cfg = gdn.NormConfig()
    c = norm_case(T, D, "none", "bf16", "bf16", 1)
    o, x, wq, wp = c["o"], c["x"], c["w_post"], c["w_pre"]
    for bad, err in ((lambda: gdn.block_norm(cfg, o.float(), x, None, wq, wp), TypeError),
                     (lambda: gdn.block_norm(cfg, o, x[:3], None, wq, wp), ValueError),
                     (lambda: gdn.block_norm(cfg, o, x.cpu(), None, wq, wp), ValueError),
                     (lambda: gdn.block_norm(cfg, o, x, None, wq, wp[:8]), ValueError),
                     (lambda: gdn.block_norm(cfg, o, x, None, wq, None, y=o), ValueError),
                     (lambda: gdn.block_norm(cfg, None, x, None, None, wp, r=x), ValueError),
                     (lambda: gdn.block_norm(cfg, o, x, o, wq, wp), gdn.GdnError),          # a gate that cfg has not
                     (lambda: gdn.block_norm(cfg, o, x, None, wq, wp, r=o), gdn.GdnError),   # r over o
                     (lambda: gdn.block_norm(cfg, o, o, None, wq, wp, r=torch.empty_like(o), y=o), gdn.GdnError)):
        with pytest.raises(err):
            bad()
    q, xs, w, ws = i8_case(4, 24, 64, 1)
    xb = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    for bad, err in ((lambda: gdn.linear_i8(q, w, ws), ValueError),                         # int8 without scales
                     (lambda: gdn.linear_i8(xb, w, ws, x_scale=xs), ValueError),
                     (lambda: gdn.linear_i8(xb, w.float(), ws), TypeError),
                     (lambda: gdn.linear_i8(xb, w, ws.double()), TypeError),
                     (lambda: gdn.linear_i8(xb, w[:, :32], ws), ValueError),
                     (lambda: gdn.linear_i8(xb, w, ws, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), gdn.GdnError),
                     (lambda: gdn.linear_i8(xb[:, :40].contiguous(), w[:, :40].contiguous(), ws), gdn.GdnError),
                     (lambda: gdn.quantize_rows(xb.t()), ValueError),
                     (lambda: gdn.quantize_rows(xb.half()), TypeError)):
        with pytest.raises(err):
            bad()
    lg, sc = beam_case(2, 3, 100, "f32", 1)
    for bad, err in ((lambda: gdn.beam_select(lg[0], sc), ValueError),
                     (lambda: gdn.beam_select(lg.half(), sc), TypeError),
                     (lambda: gdn.beam_select(lg.transpose(1, 2), sc), ValueError),
                     (lambda: gdn.beam_select(lg, sc[:1]), ValueError),
                     (lambda: gdn.beam_select(lg, sc, n_out=65), gdn.GdnError),
                     (lambda: gdn.beam_select(lg, sc, pad_token=100), gdn.GdnError),
                     (lambda: gdn.beam_select(lg, sc, n_out=2, out_scores=sc), ValueError)):
        with pytest.raises(err):
            bad()
    st = states_of(6, 1, [(64,), (64,)])
    par = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    for bad, err in ((lambda: gdn.reorder_states(par, [st[0], st[0]]), gdn.GdnError),       # the same buffer twice
                     (lambda: gdn.reorder_states(par, [st[0][:, :62]]), gdn.GdnError),      # not whole 16 bytes
                     (lambda: gdn.reorder_states(par, [st[0][:5]]), ValueError),
                     (lambda: gdn.reorder_states(par.long(), st), TypeError),
                     (lambda: gdn.reorder_states(par[0], st), ValueError),
                     (lambda: gdn.reorder_states(par, [st[0].t().contiguous().t()]), ValueError),
                     (lambda: gdn.reorder_states(par, [st[0][:1].expand(6, 64)]), gdn.GdnError)):
        with pytest.raises(err):
            bad()
    gdn.check_device_error()


def test_empty_calls():
    x = torch.empty((0, 2560), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(2560, device=DEV)
    r, y, _ = gdn.block_norm(gdn.NormConfig(), x, x, None, w, w)
    assert r.shape == y.shape == (0, 2560)
    _, _, w8, ws = i8_case(1, 24, 2560, 1)
    assert gdn.linear_i8(x, w8, ws)[0].shape == (0, 24)
    assert gdn.quantize_rows(x)[0].shape == (0, 2560)
    p, _, _ = gdn.beam_select(torch.empty((0, 3, 50), device=DEV), torch.empty((0, 3), device=DEV))
    assert p.shape == (0, 3)
    gdn.check_device_error()
