"""The operators around the mixer: their host-side argument checks, which answer without a
GPU, and the references they are tested against (CPU only)."""
import copy
import ctypes
import dataclasses
import pickle

import numpy as np
import pytest
import torch

from hybrid_linear_attention_mixer_b200 import build, gdn
from oracle import serve as S

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(6)
BF16, F32, I8 = 0, 1, 2
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.lib()


def test_norm_config_default(lib):
    c = gdn._CNormConfig()
    lib.gdn_norm_config_default(ctypes.byref(c))
    d = gdn.NormConfig().c()
    assert all(getattr(c, n) == getattr(d, n) for n, _ in c._fields_)
    assert (c.dim, c.gate, c.act_dtype, c.res_dtype) == (2560, 0, BF16, BF16) and c.res_scale == 1.0


MB = 1 << 20
ADDR = {"o": 16 * MB, "x": 32 * MB, "gate": 48 * MB, "w_post": 64 * MB, "w_pre": 65 * MB, "r": 80 * MB, "y": 96 * MB,
        "y_scale": 0}


def _norm(lib, T=4, cfg=None, **at):
    a = dict(ADDR, **at)
    if cfg is None:
        cfg = gdn.NormConfig(gate="full" if a["gate"] else "none")
    c = cfg if isinstance(cfg, gdn._CNormConfig) else cfg.c()
    return lib.gdn_block_norm(ctypes.byref(c), P(a["o"]), P(a["x"]), P(a["gate"]), P(a["w_post"]), P(a["w_pre"]), T,
                              P(a["r"]), P(a["y"]), P(a["y_scale"]), None)


def test_block_norm_argument_errors(lib):
    assert _norm(lib, T=0) == OK                                     # nothing to do
    assert lib.gdn_block_norm(None, *[P(16)] * 5, 4, *[P(16)] * 3, None) == INVALID
    assert _norm(lib, T=-1) == INVALID
    assert _norm(lib, T=1 << 31) == UNSUPPORTED
    for dim, want in ((0, INVALID), (-8, INVALID), (12, UNSUPPORTED), (16392, UNSUPPORTED)):
        assert _norm(lib, cfg=gdn.NormConfig(dim=dim, gate="full")) == want
    assert _norm(lib, cfg=gdn.NormConfig(eps=-1.0, gate="full")) == INVALID
    assert _norm(lib, cfg=gdn.NormConfig(eps=float("nan"), gate="full")) == INVALID
    assert _norm(lib, cfg=gdn.NormConfig(res_scale=float("inf"), gate="full")) == INVALID
    for field, value in (("gate", 4), ("gate", -1), ("act_dtype", I8), ("res_dtype", 7)):
        c = gdn.NormConfig(gate="full").c()
        setattr(c, field, value)
        assert _norm(lib, cfg=c) == INVALID
    # what goes with what
    assert _norm(lib, cfg=gdn.NormConfig()) == INVALID               # a gate without its kind
    assert _norm(lib, gate=0, cfg=gdn.NormConfig(gate="full")) == INVALID
    for missing in ("x", "r", "w_pre"):
        assert _norm(lib, **{missing: 0}) == INVALID
    assert _norm(lib, y=0) == INVALID                                # w_pre without y
    assert _norm(lib, y=0, w_pre=0, y_scale=112 * MB) == INVALID
    for extra in ({}, {"gate": 0}, {"gate": 0, "w_post": 0}):
        assert _norm(lib, o=0, **extra) == INVALID                   # no block: no gate, w_post or r
    assert _norm(lib, o=0, gate=0, w_post=0, r=0, y=0, w_pre=0) == INVALID   # nothing to compute
    # alignment
    for name in ("o", "x", "gate", "w_post", "w_pre", "r", "y"):
        assert _norm(lib, **{name: ADDR[name] + 8}) == INVALID
    assert _norm(lib, gate=ADDR["gate"] + 1, cfg=gdn.NormConfig(gate="token")) == INVALID
    assert _norm(lib, y_scale=112 * MB + 2) == INVALID
    # overlaps: only r on x and y (not int8) on o are open, and only exactly
    row = 2560 * 2
    assert _norm(lib, r=ADDR["o"]) == INVALID
    assert _norm(lib, r=ADDR["x"] + row) == INVALID
    assert _norm(lib, y=ADDR["o"] - row) == INVALID
    assert _norm(lib, y=ADDR["x"]) == INVALID
    assert _norm(lib, r=ADDR["y"]) == INVALID
    assert _norm(lib, y=ADDR["gate"]) == INVALID
    assert _norm(lib, y=ADDR["o"], y_scale=112 * MB) == INVALID
    assert _norm(lib, y_scale=ADDR["x"]) == INVALID
    assert _norm(lib, y_scale=ADDR["w_pre"] + 64) == INVALID


def test_quantize_argument_errors(lib):
    call = lambda dt=BF16, rows=4, cols=64, x=MB, q=2 * MB, s=3 * MB: lib.gdn_quantize_rows(P(x), dt, rows, cols, P(q), P(s), None)
    assert call(rows=0) == OK
    assert call(dt=I8) == INVALID and call(rows=-1) == INVALID and call(cols=0) == INVALID
    assert call(cols=72) == UNSUPPORTED and call(rows=1 << 31) == UNSUPPORTED
    assert call(x=0) == INVALID and call(q=0) == INVALID and call(s=0) == INVALID
    assert call(x=MB + 8) == INVALID and call(q=2 * MB + 8) == INVALID and call(s=3 * MB + 2) == INVALID
    assert call(q=MB) == INVALID and call(s=2 * MB + 16) == INVALID and call(s=MB + 32) == INVALID


def _segs(*widths, ptr=64 * MB):
    return (gdn._CSegment * len(widths))(*[gdn._CSegment(ptr, w) for w in widths])


def test_linear_i8_argument_errors(lib):
    def call(M=4, N=64, K=64, sg=None, n=None, x=MB, dt=I8, xs=2 * MB, w=3 * MB, ws=4 * MB, out=BF16, wk=0, wkb=0):
        sg = _segs(N) if sg is None else sg
        return lib.gdn_linear_i8(P(x), dt, P(xs), P(w), P(ws), M, N, K, out, sg, len(sg) if n is None else n, P(wk), wkb, None)
    assert call(M=0) == OK
    assert call(M=-1) == INVALID and call(N=0, sg=_segs(8)) == INVALID and call(K=0) == INVALID
    assert call(dt=3) == INVALID and call(out=I8) == INVALID
    assert call(K=72) == UNSUPPORTED and call(N=12) == UNSUPPORTED and call(K=131072) == UNSUPPORTED
    assert call(M=1 << 31) == UNSUPPORTED
    assert call(N=72, sg=_segs(*[8] * 9)) == UNSUPPORTED
    assert call(sg=_segs(32, 16)) == INVALID and call(sg=_segs(60, 4)) == INVALID and call(sg=_segs(64, 8)) == INVALID
    assert call(sg=_segs(2 ** 31 - 8, 72)) == INVALID
    assert call(sg=_segs(64, ptr=8)) == INVALID and call(sg=_segs(64, ptr=0)) == INVALID
    for bad in ({"x": 0}, {"w": 0}, {"ws": 0}, {"xs": 0}, {"x": MB + 8}, {"w": 3 * MB + 8}, {"ws": 4 * MB + 4}, {"xs": 2 * MB + 2}):
        assert call(**bad) == INVALID
    # rows that the call makes 8-bit itself: no scales, a workspace
    size = lib.gdn_linear_i8_workspace_size(4, 64)
    assert size == 512 and lib.gdn_linear_i8_workspace_size(-1, 64) == 0 and lib.gdn_linear_i8_workspace_size(1, 0) == 0
    assert gdn.linear_i8_workspace_size(4096, 2560) == 4096 * 2560 + 4096 * 4
    assert call(dt=BF16, wk=MB, wkb=size) == INVALID                          # scales given
    assert call(dt=BF16, xs=0, wk=0, wkb=size) == INVALID
    assert call(dt=BF16, xs=0, wk=8 * MB + 16, wkb=size) == INVALID
    assert call(dt=F32, xs=0, wk=8 * MB, wkb=size - 1) == WORKSPACE
    # nothing written may overlap anything else
    for ptr in (MB, MB + 128, 2 * MB, 3 * MB + 64 * 64 - 16, 4 * MB):
        assert call(sg=_segs(64, ptr=ptr)) == INVALID
    assert call(N=128, sg=_segs(64, 64)) == INVALID                            # one destination twice
    for wk in (MB, 3 * MB, 4 * MB, 64 * MB):
        assert call(dt=BF16, xs=0, wk=wk, wkb=size) == INVALID


def test_linear_i8_most_outputs(lib):
    """Output numbers, and a tile past the last of them, are 32 bits (x is null: the sizes
    are answered first)."""
    def call(N, M=4):
        return lib.gdn_linear_i8(None, I8, P(MB), P(MB), P(MB), M, N, 16, BF16, _segs(N), 1, None, 0, None)
    for M in (0, 1, 4, 4096):
        assert call(2 ** 31 - 8, M) == UNSUPPORTED and call(2 ** 31 - 256, M) == UNSUPPORTED
    assert call(2 ** 31 - 264) == INVALID and call(2 ** 31 - 264, 0) == OK


def test_projections_i8_argument_errors(lib):
    c = gdn.Config().c()
    inp = lambda cfg, T, D: lib.gdn_in_proj_i8(ctypes.byref(cfg), P(MB), I8, P(MB), P(MB), P(MB), T, D, *[P(MB)] * 6, None, 0, None)
    assert inp(gdn.Config(n_k_heads=2, n_v_heads=6, d_k=32, d_v=32).c(), 4, 64) == UNSUPPORTED
    assert inp(gdn.Config(d_k=48).c(), 4, 64) == UNSUPPORTED
    assert inp(c, 0, 2560) == OK and inp(c, -1, 2560) == INVALID and inp(c, 4, 2568) == UNSUPPORTED
    out = lambda T, D: lib.gdn_out_proj_i8(ctypes.byref(c), P(MB), I8, P(MB), P(MB), P(MB), T, D, P(MB), None, 0, None)
    assert out(0, 2560) == OK and out(-1, 2560) == INVALID and out(4, 2564) == UNSUPPORTED and out(4, 0) == INVALID
    assert lib.gdn_out_proj_i8(None, P(MB), I8, P(MB), P(MB), P(MB), 4, 2560, P(MB), None, 0, None) == INVALID


def test_beam_argument_errors(lib):
    size = lib.gdn_beam_workspace_size(2, 3, 1000, 4, BF16)
    assert size > 0 and gdn.beam_workspace_size(0, 3, 1000, 4) > 0
    base = dict(logits=16 * MB, dt=BF16, ld=1000, scores=32 * MB, fin=0, G=2, W=3, V=1000, n=4, pad=0, par=33 * MB,
                tok=34 * MB, out=35 * MB, ws=48 * MB, wsb=size)

    def call(**kw):
        a = dict(base, **kw)
        return lib.gdn_beam_select(P(a["logits"]), a["dt"], a["ld"], P(a["scores"]), P(a["fin"]), a["G"], a["W"], a["V"],
                                   a["n"], a["pad"], P(a["par"]), P(a["tok"]), P(a["out"]), P(a["ws"]), a["wsb"], None)
    assert call(G=0) == OK
    for bad in ({"G": -1}, {"W": 0}, {"V": 0}, {"n": 0}, {"dt": I8}, {"ld": 999}, {"pad": -1}, {"pad": 1000},
                {"ld": 1 << 62}):
        assert call(**bad) == INVALID
    for bad in ({"W": 33}, {"n": 65}, {"V": (1 << 20) + 1, "ld": 1 << 21}, {"G": 1 << 30}):
        assert call(**bad) == UNSUPPORTED
        a = dict(base, **bad)
        assert lib.gdn_beam_workspace_size(a["G"], a["W"], a["V"], a["n"], BF16) == 0
    for name in ("logits", "scores", "par", "tok", "out", "ws"):
        assert call(**{name: 0}) == INVALID
        assert call(**{name: base[name] + 1}) == INVALID
    assert call(ws=48 * MB + 128) == INVALID and call(wsb=size - 1) == WORKSPACE
    # overlaps
    assert call(par=34 * MB) == INVALID and call(out=33 * MB + 8) == INVALID
    assert call(out=32 * MB) == INVALID                        # n_out is not the number of beams
    assert call(n=3, out=32 * MB + 4) == INVALID
    assert call(par=32 * MB) == INVALID and call(tok=16 * MB + 100) == INVALID
    assert call(ws=16 * MB) == INVALID and call(fin=33 * MB) == INVALID


@pytest.mark.parametrize("dt,size", [(torch.bfloat16, 2), (torch.float32, 4)])
def test_beam_workspace_of_a_call_serves_smaller_ones(lib, dt, size):
    """No size that a request loses may make its step need more: batches that shrink, beams
    that are dropped, fewer results, a shorter vocabulary."""
    need = lambda G, W, V, n: gdn.beam_workspace_size(G, W, V, n, dt)
    for W, V, n in ((4, 128256, 4), (5, 32003, 10), (1, 1000, 1), (8, 248320, 16), (32, 1 << 20, 64), (3, 50001, 33), (16, 9000, 20)):
        sizes = [need(G, W, V, n) for G in range(0, 1400)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (W, V, n)
    for G, V, n in ((1, 248320, 4), (19, 128256, 64), (300, 1 << 20, 7)):
        sizes = [need(G, W, V, n) for W in range(1, 33)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (G, V, n)
    for G, W, V in ((1, 4, 248320), (64, 8, 32003), (1000, 3, 700)):
        sizes = [need(G, W, V, n) for n in range(1, 65)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (G, W, V)
    for G, W, n in ((1, 1, 1), (3, 5, 9), (70, 4, 64)):
        sizes = [need(G, W, V, n) for V in range(1, 1 << 20, 997)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (G, W, n)
    # every candidate list of any layout that the call can take fits (16 bytes of sums and n keys each)
    for G, W, V, n in ((18, 4, 128256, 4), (30, 5, 32003, 10), (1, 32, 1 << 20, 64), (2, 1, 30, 64), (500, 9, 70000, 2)):
        tiles, rows = -(-V * size // 2048), G * W
        each = min(max(rows * tiles // (148 * 32) + 1, 2, (n + 15) // 16), 32)
        slices = min(max(tiles // each, 1, -(-tiles // 32)), 4096 // W)
        assert need(G, W, V, n) >= rows * slices * (16 + 8 * n)


def test_reorder_argument_errors(lib):
    def call(bufs, G=2, W=3, par=MB, n=None):
        arr = (gdn._CStateBuffer * max(1, len(bufs)))(*[gdn._CStateBuffer(*b) for b in bufs])
        return lib.gdn_reorder_states(P(par), G, W, arr, len(bufs) if n is None else n, None)
    good = (16 * MB, 64, 64)
    assert call([good], G=0) == OK and call([]) == OK
    assert call([good], G=-1) == INVALID and call([good], W=0) == INVALID and call([good], n=-1) == INVALID
    assert call([good], W=33) == UNSUPPORTED
    assert call([(16 * MB + i * 4096, 16, 16) for i in range(129)]) == UNSUPPORTED
    assert call([good], par=0) == INVALID and call([good], par=MB + 2) == INVALID
    for bad in ((0, 64, 64), (16 * MB + 8, 64, 64), (16 * MB, 0, 64), (16 * MB, -64, 64), (16 * MB, 60, 64),
                (16 * MB, 64, 72), (16 * MB, 64, 48), (16 * MB, 64, 1 << 62)):
        assert call([bad]) == INVALID
    assert call([(16 * MB, (16 << 30) + 16, (16 << 30) + 16)]) == UNSUPPORTED
    # states that share memory, the parents among them
    assert call([good, good]) == INVALID
    assert call([good, (16 * MB + 64 * 5, 64, 64)]) == INVALID
    assert call([(16 * MB, 64, 128), (16 * MB + 48, 64, 128)]) == INVALID
    assert call([(16 * MB + 48, 64, 128), (16 * MB, 64, 128)]) == INVALID
    assert call([(16 * MB, 64, 128), (16 * MB + 64, 16, 256)]) == INVALID    # different strides, same span
    assert call([good], par=16 * MB + 64) == INVALID


@pytest.mark.parametrize("make", [gdn.Config, gdn.NormConfig])
def test_used_configs_copy_pickle_and_follow_their_fields(make):
    """A configuration that calls have been made with is copied, pickled and taken apart like
    a new one, and its next call has the values that its fields have then."""
    cfg, field = make(), "d_v" if make is gdn.Config else "dim"
    struct = gdn._CConfig if make is gdn.Config else gdn._CNormConfig
    seen = lambda c: getattr(ctypes.cast(c.ref(), ctypes.POINTER(struct)).contents, field)
    first = seen(cfg)
    setattr(cfg, field, 64)
    assert first != 64 and seen(cfg) == 64
    for twin in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), make(**vars(cfg)),
                 dataclasses.replace(cfg)):
        assert twin == cfg and vars(twin) == vars(cfg) and seen(twin) == 64
        setattr(twin, field, 32)
        assert seen(twin) == 32 and seen(cfg) == 64
    vars(cfg).update({field: 128})
    assert seen(cfg) == 128


def test_reorder_plan_keeps_its_memory(monkeypatch):
    """A plan's addresses stay those of memory that it keeps, whatever its tensors are
    pointed at afterwards."""
    monkeypatch.setattr(gdn, "_index_of", lambda t, name: t.get_device())
    states = [torch.zeros(4, 8), torch.zeros(4, 16, requires_grad=True)]
    plan = gdn.reorder_plan(states, 2, 2)
    old = [t.data_ptr() for t in states]
    states[0].data = torch.ones(4, 8)
    with torch.no_grad():
        states[1].set_(torch.ones(4, 16))
    assert [b.base for b in plan.buffers] == old
    assert [t.data_ptr() for t in plan.states] == old
    assert all(int(torch.count_nonzero(t)) == 0 for t in plan.states)


def test_binding_refuses_sizes_that_the_library_cannot_take(monkeypatch):
    """Sizes that are 32 bits in the C interface are not cut off to other sizes (shapes alone
    here: tensors without memory, and no call may get as far as the library)."""
    monkeypatch.setattr(gdn, "_index_of", lambda t, name: t.get_device())
    reached = lambda *a: pytest.fail("reached the library")
    monkeypatch.setattr(gdn, "_call", reached)
    over = 2 ** 32
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")
    f, i8 = (lambda *s: e(*s, dt=torch.float32)), (lambda *s: e(*s, dt=torch.int8))
    lg, sc = f(2, 3, 1000), f(2, 3)
    layer = gdn.Config()
    for bad in (lambda: gdn.block_norm(gdn.NormConfig(dim=over + 64), None, e(1, over + 64), w_pre=f(over + 64)),
                lambda: gdn.quantize_rows(e(1, over + 64)),
                lambda: gdn.linear_i8(i8(1, over + 64), i8(8, over + 64), f(8), x_scale=f(1)),
                lambda: gdn.linear_i8(i8(1, 64), i8(over + 8, 64), f(over + 8), x_scale=f(1)),
                lambda: gdn.in_proj_i8(layer, i8(1, over + 64), i8(16480, over + 64), f(16480), hidden_scale=f(1)),
                lambda: gdn.out_proj_i8(layer, i8(1, 6144), i8(over + 64, 6144), f(over + 64), o_scale=f(1)),
                lambda: gdn.beam_select(lg, sc, pad_token=over),
                lambda: gdn.beam_select(lg, sc, pad_token=-over),
                lambda: gdn.beam_select(lg, sc, n_out=over + 3),
                lambda: gdn.beam_select(lg, sc, n_out=-1),
                lambda: gdn.beam_select(f(over, 1, 1), f(over, 1)),
                lambda: gdn.reorder_states(e(over, 1, dt=torch.int32), [f(over, 4)]),
                lambda: gdn.linear_i8_workspace_size(4, over + 64),
                lambda: gdn.beam_workspace_size(2, 3, 1000, over + 4),
                lambda: gdn.beam_workspace_size(2, over + 3, 1000, 4)):
        with pytest.raises(ValueError):
            bad()


def test_status_string_of_the_index_check():
    assert gdn.status_string(8) not in {gdn.status_string(s) for s in range(8)} | {"unknown status"}


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 2560, dtype=torch.bfloat16), torch.ones(2560)
    with pytest.raises(ValueError):
        gdn.block_norm(gdn.NormConfig(), x, x, None, w, w)
    with pytest.raises(ValueError):
        gdn.quantize_rows(x)
    with pytest.raises(ValueError):
        gdn.linear_i8(x, torch.zeros(8, 2560, dtype=torch.int8), torch.ones(8))
    with pytest.raises(ValueError):
        gdn.beam_select(torch.zeros(1, 2, 10), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        gdn.reorder_states(torch.zeros(1, 2, dtype=torch.int32), [torch.zeros(2, 8)])


# ---------------------------------------------------------------------------
# The references themselves
# ---------------------------------------------------------------------------
def test_reference_norm_closed_forms():
    x = np.full((2, 8), 3.0)
    r, y, p = S.block_norm(np.full((2, 8), -5.0), x, np.zeros((2, 8)), np.ones(8), 2 * np.ones(8), 4.0, 0.0, True)
    np.testing.assert_allclose(p, -2.0)          # 4 * sigmoid(0) * (-5 / 5)
    np.testing.assert_allclose(r, 1.0)
    np.testing.assert_allclose(y, 2.0)
    _, y, _ = S.block_norm(None, x, None, None, np.ones(8), 1.0, 7.0, False)
    np.testing.assert_allclose(y, 0.75)          # 3 / sqrt(9 + 7)


def test_reference_rows_and_product():
    q, s = S.quantize_rows(np.array([[2.0, 1.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0]]))
    np.testing.assert_array_equal(q, [[127, 64, -64, 0], [0, 0, 0, 0]])      # 63.5 to even
    np.testing.assert_array_equal(s, [2 / 127, 0])
    y = S.linear_i8([[1, -2]], [0.5], [[3, 4], [5, -6]], [2.0, 4.0])
    np.testing.assert_array_equal(y, [[-5.0, 34.0]])


def test_reference_beam_and_reorder():
    lg = np.log(np.array([[[1.0, 2.0, 1.0], [2.0, 1.0, 1.0]]]))
    p, t, s, gap = S.beam_select(lg, np.zeros((1, 2)), 4)
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[1, 0, 0, 2]]      # ties: lowest w * V + v
    np.testing.assert_allclose(s, np.log([[0.5, 0.5, 0.25, 0.25]]))
    p, t, s, _ = S.beam_select(lg, np.zeros((1, 2)), 7, np.array([[0, 1]]), 2)
    assert p.tolist() == [[1, 0, 0, 0, -1, -1, -1]] and t[0, 0] == 2 and s[0, 0] == 0
    st = np.arange(4)
    np.testing.assert_array_equal(S.reorder(st, np.array([[1, 1], [-1, 0]])), [1, 1, 2, 2])
