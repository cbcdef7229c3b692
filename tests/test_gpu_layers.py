"""The layer operators (include/ma_layers.h) on the GPU against float64
references: norm, rotary positions and token log probabilities, forward and backward, at the sizes, types,
strides and values where each can go wrong."""

import numpy as np
import pytest

from tests import _grads_ref as G
from tests import _layers_ref as R
from tests.test_gpu_grads import DT, _close, _dev, _f64, _strided

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.load_library()
    yield
    torch.cuda.synchronize()


def _stream(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp(0.7 * rng.standard_normal(cols))
    if rows > 2:
        x[1] = 0.0
    return x


# --------------------------------------------------------------------- norm --

NORM_SHAPES = [(1, 1, 0), (1, 7, 0), (5, 32, 0), (70, 64, 0), (33, 100, 3), (16, 128, 8), (17, 129, 0), (9, 256, 0),
               (3, 257, 1), (50, 1000, 0), (50, 1024, 0), (6, 1025, 0), (5, 2048, 8), (4, 2049, 0), (3, 4096, 0),
               (3, 4104, 0), (2, 8192, 0), (3, 8191, 0), (1, 8001, 1)]


@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", NORM_SHAPES)
def test_norm_forward(kind, wkind, rows, cols, pad):
    rng = np.random.default_rng(rows * 131 + cols)
    x, _ = _strided(_stream(rng, rows, cols), pad, kind)
    res, _ = _strided(_stream(rng, rows, cols), 2 * pad, kind)
    w = _dev(1 + 0.3 * rng.standard_normal(cols), wkind)
    for off, r in ((0.0, None), (0.0, res), (1.0, res)):
        y, s, inv, c = M.ma_rms_norm_forward(x, w, r, eps=1e-5, weight_offset=off, y_ckpt=True)
        yy, ss, ii, dy, ds, di = R.rms_norm(_f64(x), _f64(w), None if r is None else _f64(r), 1e-5, off)
        _close(y, yy, R.rounded(yy, dy, kind), "y")
        assert (s is x) if r is None else True
        _close(s, ss, R.rounded(ss, ds, kind), "s")
        _close(inv, ii, di, "inv")
        # what is held is y as it is stored, byte for byte
        p = M.ma_act_pack(y)
        assert torch.equal(p.codes, c.codes)
        groups = c.codes.shape[1] // 32
        assert torch.equal(p.exps[:, :groups], c.exps[:, :groups])
        again = M.ma_rms_norm_forward(x, w, r, eps=1e-5, weight_offset=off)
        assert again[3] is None and torch.equal(again[0], y) and torch.equal(again[2], inv)
        none, _, _, only = M.ma_rms_norm_forward(x, w, r, eps=1e-5, weight_offset=off, out=False, y_ckpt=True)
        assert none is None and torch.equal(only.codes, c.codes)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_norm_forward_into_strided_outputs(kind):
    rng = np.random.default_rng(4)
    x, r = _dev(_stream(rng, 37, 200), kind), _dev(_stream(rng, 37, 200), kind)
    w = _dev(rng.standard_normal(200))
    y, s, _, c = M.ma_rms_norm_forward(x, w, r, y_ckpt=True)
    y2, yw = _strided(np.zeros((37, 200)), 5, kind)
    s2, sw = _strided(np.zeros((37, 200)), 8, kind)
    held = M.ActCheckpoint.empty((37, 200), "cuda")
    got = M.ma_rms_norm_forward(x, w, r, out=y2, sum_out=s2, y_ckpt=held)
    assert got[0] is y2 and got[1] is s2 and got[3] is held
    assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(held.codes, c.codes)
    assert torch.all(yw[:, 200:] == 7.0) and torch.all(sw[:, 200:] == 7.0)
    # a row alone, and a row repeated
    one = M.ma_rms_norm_forward(x[3], w, r[3])
    assert torch.equal(one[0], y[3]) and one[2].shape == ()
    rep = M.ma_rms_norm_forward(x[3].expand(5, 200), w, r[3].expand(5, 200))
    assert torch.equal(rep[0], y[3].expand(5, 200))
    none = M.ma_rms_norm_forward(x[:0], w, r[:0], y_ckpt=True)
    assert none[0].shape == (0, 200) and none[3].rows == 0


@pytest.mark.parametrize("cols", [96, 1000, 5000])
def test_norm_extremes(cols):
    """Rows of zeros, tiny values, values whose squares leave float32, an infinity, a NaN."""
    x = np.ones((8, cols), np.float32)
    x[0] = 0
    x[1] = 1e-30
    x[2] = 1e30
    x[3] = -3e38
    x[4, ::2], x[4, 1::2] = 2e25, 3e19
    x[5, 3] = np.inf
    x[6, 5] = np.nan
    w = _dev(np.ones(cols))
    y, _, inv, c = M.ma_rms_norm_forward(torch.from_numpy(x).cuda(), w, eps=1e-6, y_ckpt=True)
    yy, _, ii, dy, _, di = R.rms_norm(x[:5].astype(np.float64), np.ones(cols), None, 1e-6, 0.0)
    # (an inverse below 2^-126 keeps fewer bits: 2^-149 apart)
    _close(inv[:5], ii, di + 2.0 ** -149)
    _close(y[:5], yy, dy + np.abs(x[:5]) * 2.0 ** -149 + G.TINY)
    assert inv[5] == 0 and torch.isnan(y[5, 3]) and torch.all(y[5, 4:] == 0)
    assert torch.isnan(y[6]).all() and torch.isnan(inv[6])
    assert torch.all(c.exps[6, :(cols + 31) // 32] == 255)
    assert torch.equal(M.ma_act_pack(y).codes, c.codes)
    # the gradient at such rows is finite and near the formula's
    d = np.ones((5, cols), np.float32)
    d[:, ::3] = -1
    ds, dw = M.ma_rms_norm_backward(torch.from_numpy(d).cuda(), torch.from_numpy(x[:5]).cuda(), inv[:5].contiguous(), w)
    want, dwant, tol, wtol = R.rms_norm_backward(d.astype(np.float64), x[:5].astype(np.float64), _f64(inv[:5]),
                                                 np.ones(cols))
    _close(ds, want, tol + 2.0 ** -140)
    _close(dw, dwant, wtol + G.TINY)


@pytest.mark.parametrize("kind,wkind,gkind", [("fp32", "fp32", "fp32"), ("bf16", "fp32", "fp32"),
                                              ("bf16", "bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", NORM_SHAPES + [(3000, 72, 0), (4000, 256, 0), (900, 2048, 0), (1601, 301, 0)])
def test_norm_backward(kind, wkind, gkind, rows, cols, pad):
    rng = np.random.default_rng(rows * 17 + cols)
    s, _ = _strided(_stream(rng, rows, cols), pad, kind)
    dy, _ = _strided(rng.standard_normal((rows, cols)), pad, kind)
    dsum, _ = _strided(rng.standard_normal((rows, cols)), 0, kind)
    w = _dev(rng.standard_normal(cols), wkind)
    inv = M.ma_rms_norm_forward(s, w, eps=1e-5)[2]
    for off, add in ((0.0, None), (1.0, dsum)):
        ds, dw = M.ma_rms_norm_backward(dy, s, inv, w, add, weight_offset=off, grad_dtype=DT[gkind])
        want, dwant, tol, wtol = R.rms_norm_backward(_f64(dy), _f64(s), _f64(inv), _f64(w), off,
                                                     None if add is None else _f64(add))
        _close(ds, want, R.rounded(want, tol, kind), "ds")
        _close(dw, dwant, R.rounded(dwant, wtol, gkind), "dw")
        # reruns are bitwise equal, whatever the workspace held; without a weight gradient too
        ws = torch.full((M.ma_rms_norm_backward_workspace_size(rows, cols),), 255, dtype=torch.uint8, device="cuda")
        ds2, dw2 = M.ma_rms_norm_backward(dy, s, inv, w, add, weight_offset=off, workspace=ws, grad_dtype=DT[gkind])
        assert torch.equal(ds, ds2) and torch.equal(dw, dw2)
        ds3, none = M.ma_rms_norm_backward(dy, s, inv, w, add, weight_offset=off, dweight=False)
        assert none is None and torch.equal(ds, ds3)
        old = _dev(rng.standard_normal(cols), gkind)
        acc = old.clone()
        M.ma_rms_norm_backward(dy, s, inv, w, add, weight_offset=off, dweight=acc, accumulate=True)
        _, dwant, _, wtol = R.rms_norm_backward(_f64(dy), _f64(s), _f64(inv), _f64(w), off, None, _f64(old))
        _close(acc, dwant, R.rounded(dwant, wtol, gkind), "dw added to")


def test_norm_backward_of_no_rows():
    w = torch.ones(40, device="cuda")
    e = torch.zeros((0, 40), device="cuda")
    i = torch.zeros(0, device="cuda")
    ds, dw = M.ma_rms_norm_backward(e, e, i, w)
    assert ds.shape == (0, 40) and torch.all(dw == 0)
    acc = torch.full((40,), 3.0, device="cuda")
    M.ma_rms_norm_backward(e, e, i, w, dweight=acc, accumulate=True)
    assert torch.all(acc == 3)


def test_norm_gradient_against_differences():
    """f(x, w) = sum(c y): its slope along a random direction, by central differences of the
    reference in 64 bits."""
    rng = np.random.default_rng(11)
    x, w, c = rng.standard_normal((7, 90)), rng.standard_normal(90), rng.standard_normal((7, 90))
    y, s, inv, _ = M.ma_rms_norm_forward(_dev(x), _dev(w), eps=1e-5)
    ds, dw = M.ma_rms_norm_backward(_dev(c), s, inv, _dev(w))
    f = lambda a, b: np.sum(c * R.rms_norm(a, b, None, 1e-5)[0])
    for seed in range(4):
        u, v = np.random.default_rng(seed).standard_normal((7, 90)), np.random.default_rng(seed + 9).standard_normal(90)
        h = 1e-5
        slope = (f(x + h * u, w + h * v) - f(x - h * u, w - h * v)) / (2 * h)
        got = np.sum(_f64(ds) * u) + np.sum(_f64(dw) * v)
        # float32 inputs and gradients: 630 terms of magnitude about 1, each off by some 2^-22
        assert abs(got - slope) < 1e-3 * max(1, abs(slope))


# ------------------------------------------------------------------- rotary --

PLANS = [((64,), "half", "blocks", False), ((16, 24, 24), "half", "blocks", False), ((16, 24, 24), "pairs", "cycled", False),
         ((18, 18), "half", "blocks", True), ((18, 18), "pairs", "blocks", True), ((5, 0, 3), "half", "cycled", True),
         ((1,), "half", "blocks", False), ((128,), "half", "blocks", False), ((3, 5, 2, 1), "pairs", "cycled", False)]


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("sections,layout,order,restart", PLANS)
@pytest.mark.parametrize("tokens,heads,rest", [(1, 1, 0), (37, 5, 0), (130, 3, 8), (700, 2, 7)])
def test_rotary(kind, sections, layout, order, restart, tokens, heads, rest):
    rng = np.random.default_rng(tokens + sum(sections))
    dim, axes = 2 * sum(sections) + rest, len(sections)
    plan = M.Rotary(sections, theta=10000.0, layout=layout, order=order, restart=restart)
    table = R.rotary_table(sections, 10000.0, order, restart)
    assert plan.pair_axis == tuple(a for a, _ in table)
    assert np.allclose(plan.frequencies, [f for _, f in table], rtol=1e-14, atol=0)
    x = _dev(rng.standard_normal((tokens, heads, dim)), kind)
    pos = rng.integers(-50, 1 << 20, (axes, tokens))
    for ptype in (torch.int64, torch.int32):
        p = torch.from_numpy(pos).to("cuda", ptype)
        for inverse in (False, True):
            got = M.ma_rotary(x, p if axes > 1 else p[0], plan, inverse=inverse)
            want, tol = R.rotary(_f64(x), pos, table, layout, inverse)
            _close(got, want, R.rounded(want, tol, kind))
            assert torch.equal(got[..., 2 * plan.pairs:], x[..., 2 * plan.pairs:])
    # in place, and in a part of a wider array whose other heads stay
    wide = torch.full((tokens, heads + 2, dim + 3), 7.0, dtype=DT[kind], device="cuda")
    part = wide[:, 1:1 + heads, :dim]
    part.copy_(x)
    assert M.ma_rotary(part, p, plan, inverse=True, out=part) is part
    assert torch.equal(part, got)
    assert torch.all(wide[:, 0] == 7) and torch.all(wide[:, -1] == 7) and torch.all(wide[:, :, dim:] == 7)
    # heads outside, tokens inside
    turned = torch.empty((heads, tokens, dim), dtype=DT[kind], device="cuda").transpose(0, 1)
    M.ma_rotary(x, p, plan, inverse=True, out=turned)
    assert torch.equal(turned, got)


def test_rotary_far_positions_and_back():
    plan = M.Rotary((16, 24, 24))
    x = torch.randn(500, 4, 128, device="cuda")
    pos = torch.randint(0, 1 << 31, (3, 500), device="cuda")
    got = M.ma_rotary(x, pos, plan)
    want, tol = R.rotary(_f64(x), pos.cpu().numpy(), R.rotary_table((16, 24, 24), 10000.0, "blocks", False), "half")
    _close(got, want, R.rounded(want, tol, "fp32"))
    back = M.ma_rotary(got, pos, plan, inverse=True)
    # two turns, each off by its bound on values of at most |u| + |v|
    assert (back - x).abs().max() < 1e-5
    # a turn keeps the product of a pair of vectors: <R g, R x> = <g, x>, so the inverse is the gradient
    g = torch.randn_like(x)
    a = (g.double() * got.double()).sum()
    b = (M.ma_rotary(g, pos, plan, inverse=True).double() * x.double()).sum()
    assert abs(a - b) < 1e-3 * x.numel() ** 0.5


def test_rotary_shapes_and_empty():
    plan = M.Rotary(8)
    x = torch.randn(2, 9, 3, 16, device="cuda")
    pos = torch.arange(18, device="cuda").view(2, 9)
    flat = M.ma_rotary(x.view(18, 3, 16), pos.view(18), plan)
    assert torch.equal(M.ma_rotary(x, pos, plan).view(18, 3, 16), flat)
    assert torch.equal(M.ma_rotary(x, pos[None], plan).view(18, 3, 16), flat)
    assert M.ma_rotary(x[:0], pos[:0], plan).shape == (0, 9, 3, 16)
    one = M.ma_rotary(x[0, 4], pos[0, 4], plan)
    assert torch.equal(one, flat[4])
    assert torch.equal(M.ma_rotary(x, torch.zeros_like(pos), plan), x)


# -------------------------------------------------- log probabilities of tokens --

def _check_logprob(z, ids, scale, top, tok=torch.int64):
    got = M.ma_token_logprob_forward(z, torch.from_numpy(ids).to("cuda", tok), scale=scale, top=top)
    want, tol = R.logprob(_f64(z), ids, float(np.float32(scale)), top)
    for name, k in (("logprob", 0), ("entropy", 1), ("lse", 2)):
        _close(got[k], want[k], tol[k], name)
    if top:
        assert got[3].dtype == tok and np.array_equal(got[3].cpu().numpy(), want[3])
        _close(got[4], want[4], tol[4], "top")
    else:
        assert got[3] is None and got[4] is None
    return got


def _logits(rng, rows, vocab, spread=3.0):
    return rng.standard_normal((rows, vocab)) * spread


LOGIT_SHAPES = [(1, 1, 0), (3, 2, 0), (5, 7, 1), (2, 9, 0), (37, 64, 0), (3, 100, 4), (4, 519, 3), (130, 1000, 0),
                (3, 1001, 0), (2, 4096, 0), (3, 4097, 0), (2, 8200, 0), (3, 16385, 1), (1, 32003, 0), (700, 4133, 0),
                (600, 17001, 0), (1, 151000, 0), (2, 151003, 5)]


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", LOGIT_SHAPES)
def test_logprob(kind, rows, vocab, pad):
    rng = np.random.default_rng(rows + vocab)
    z, _ = _strided(_logits(rng, rows, vocab), pad, kind)
    ids = rng.integers(0, vocab, rows)
    ids[rows // 2] = vocab if rows > 2 else ids[rows // 2]
    for top, scale in ((0, 1.0), (1, 0.5), (min(vocab, 20), 1.3), (min(vocab, 64), 1.0)):
        got = _check_logprob(z, ids, scale, top, torch.int32 if top == 1 else torch.int64)
    need = M.ma_token_logprob_workspace_size(rows, vocab, min(vocab, 64))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    again = M.ma_token_logprob_forward(z, torch.from_numpy(ids).cuda(), scale=1.0, top=min(vocab, 64), workspace=ws)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [300, 1000, 5001, 20011, 151000])
def test_logprob_orders(kind, vocab):
    """Rows in rising and falling order, of one value, of few values, with the highest side by side, at the
    stride of a workgroup's rounds, at both ends; masked but for a few; with zeros of both signs."""
    rng = np.random.default_rng(vocab)
    z = np.zeros((12, vocab))
    z[0] = np.linspace(-5, 5, vocab)
    z[1] = z[0][::-1]
    z[2] = 0.25
    z[3] = rng.integers(0, 3, vocab)
    z[4] = rng.standard_normal(vocab)
    z[4, vocab // 3:vocab // 3 + 70] = 9 + rng.random(70)
    z[5] = rng.standard_normal(vocab)
    z[5, ::512 * 8 if vocab > 16384 else 64 * 8] = 7.0
    z[6, :5], z[6, -5:] = 3.0, 3.0
    z[7] = -np.inf
    z[7, rng.integers(0, vocab, 5)] = rng.random(5)
    z[8] = -3.3e38
    z[9] = -3.3e38
    z[9, -1] = 1.0
    z[10] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)
    z[11] = -np.inf
    t = _dev(z, kind)
    ids = rng.integers(0, vocab, 12)
    for top in (1, 5, 20, 64):
        _check_logprob(t, ids, 1.0, top)
    # from an odd address on, so that a row's first elements are no whole unit
    for off in (1, 3):
        w = torch.zeros(12 * vocab + 8, dtype=DT[kind], device="cuda")
        o = w[off:off + 12 * vocab].view(12, vocab)
        o.copy_(t)
        _check_logprob(o, ids, 1.0, 20)


def test_logprob_more_keys_than_the_list():
    """Thousands of values above the bound that the threads' largest give: the 64 highest threads hold
    only such values."""
    z = torch.randn(2, 151000, device="cuda")
    unit = (torch.arange(151000, device="cuda") // 8) % 512
    hot = unit < 64
    z[:, hot] = 20 + torch.rand(2, int(hot.sum()), device="cuda")
    # (one row, and the same among enough rows for a workgroup each)
    ids = np.array([5, 77])
    _check_logprob(z, ids, 1.0, 64)
    many = z.repeat(300, 1)
    got = M.ma_token_logprob_forward(many, torch.zeros(600, dtype=torch.int64, device="cuda"), top=64)
    want = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :64]
    assert torch.equal(got[3], want.repeat(300, 1))


def test_logprob_nonfinite():
    z = torch.randn(6, 5000, device="cuda")
    z[0, 17] = float("nan")
    z[1, 4000] = float("inf")
    z[3] = float("nan")
    ids = torch.tensor([1, 2, 3, 4, 5, 6], device="cuda")
    lp, ent, lse, top, tl = M.ma_token_logprob_forward(z, ids, top=10)
    for r in (0, 1, 3):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(lse[r]) and torch.isnan(tl[r]).any()
        assert len(set(top[r].tolist())) == 10 and 0 <= int(top[r].min()) and int(top[r].max()) < 5000
    clean = M.ma_token_logprob_forward(z[[2, 4, 5]].contiguous(), ids[[2, 4, 5]], top=10)
    for a, b in zip((lp, ent, lse, top, tl), clean):
        assert torch.equal(a[[2, 4, 5]], b)
    d = M.ma_token_logprob_backward(z, ids, lse, torch.ones(6, device="cuda"))
    assert torch.isnan(d[0]).all() and torch.isfinite(d[2]).all()


@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,vocab,pad", LOGIT_SHAPES)
def test_logprob_backward(kind, gkind, rows, vocab, pad):
    rng = np.random.default_rng(rows * 3 + vocab)
    z = _logits(rng, rows, vocab)
    if vocab > 50:
        z[:, 5:40:3] = -np.inf
    if rows > 4:
        z[3] = -np.inf
    z, _ = _strided(z, pad, kind)
    ids = rng.integers(0, vocab, rows)
    ids[0] = -1 if rows > 1 else 0
    tok = torch.from_numpy(ids).cuda()
    g, h = _dev(rng.standard_normal(rows)), _dev(rng.standard_normal(rows))
    scale = 1.25
    _, ent, lse, _, _ = M.ma_token_logprob_forward(z, tok, scale=scale)
    out, wide = _strided(np.zeros((rows, vocab)), pad + 1, gkind)
    for e, k in ((None, None), (ent, h)):
        M.ma_token_logprob_backward(z, tok, lse, g, entropy=e, dentropy=k, scale=scale, out=out)
        want, tol = R.logprob_backward(_f64(z), ids, scale, _f64(lse), _f64(g), None if e is None else _f64(e),
                                       None if k is None else _f64(k))
        _close(out, want, R.rounded(want, tol, gkind))
        assert torch.all(wide[:, vocab:] == 7.0)
        assert torch.equal(M.ma_token_logprob_backward(z, tok.to(torch.int32), lse, g, entropy=e, dentropy=k,
                                                       scale=scale, grad_dtype=DT[gkind]), out)
    if kind == gkind:                                        # over the logits themselves
        into = z.clone()
        M.ma_token_logprob_backward(into, tok, lse, g, entropy=ent, dentropy=h, scale=scale, out=into)
        assert torch.equal(into, out)


def test_logprob_gradient_against_differences():
    rng = np.random.default_rng(8)
    z, ids = rng.standard_normal((5, 300)) * 2, rng.integers(0, 300, 5)
    g, h = rng.standard_normal(5), rng.standard_normal(5)
    _, ent, lse, _, _ = M.ma_token_logprob_forward(_dev(z), torch.from_numpy(ids).cuda(), scale=0.7)
    d = _f64(M.ma_token_logprob_backward(_dev(z), torch.from_numpy(ids).cuda(), lse, _dev(g), entropy=ent,
                                         dentropy=_dev(h), scale=0.7))

    def f(a):
        (lp, e, _, _, _), _ = R.logprob(a, ids, 0.7)
        return np.sum(g * lp + h * e)

    for seed in range(4):
        u = np.random.default_rng(seed).standard_normal(z.shape)
        slope = (f(z + 1e-5 * u) - f(z - 1e-5 * u)) / 2e-5
        # gradients sum to a few units, in float32: 2^-20 or so of their magnitudes
        assert abs(np.sum(d * u) - slope) < 1e-4 * max(1.0, abs(slope))


def test_logprob_shapes_and_empty():
    z = torch.randn(2, 3, 50, device="cuda")
    ids = torch.randint(0, 50, (2, 3), device="cuda")
    lp, ent, lse, top, tl = M.ma_token_logprob_forward(z, ids, top=4)
    flat = M.ma_token_logprob_forward(z.view(6, 50), ids.view(6), top=4)
    assert lp.shape == (2, 3) and top.shape == (2, 3, 4)
    assert torch.equal(top.view(6, 4), flat[3]) and torch.equal(lp.view(6), flat[0])
    d = M.ma_token_logprob_backward(z, ids, lse, torch.ones_like(lp))
    assert d.shape == z.shape and d.sum(-1).abs().max() < 1e-5
    e = M.ma_token_logprob_forward(z[:0], ids[:0], top=4)
    assert e[0].shape == (0, 3) and e[3].shape == (0, 3, 4)
    assert M.ma_token_logprob_backward(z[:0], ids[:0], lse[:0], lp[:0]).shape == (0, 3, 50)


# ---------------------------------------------------------------- attention --

def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def _cu(off):
    return torch.from_numpy(off.astype(np.int32)).cuda()


def _heads_first(x):
    """The same values with heads outside and tokens inside."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def _inputs(rng, nq, nk, heads, kv, dim, kind):
    return [_dev(rng.standard_normal(s), kind) for s in ((nq, heads, dim), (nk, kv, dim), (nk, kv, dim), (nq, heads, dim))]


def _check_attention(q, k, v, do, cq, ck, causal, scale, kind):
    nq = int(cq[-1])
    cu = (_cu(cq), _cu(ck))
    o, lse = torch.full_like(q, 7.0), None
    o, lse = M.ma_attention_forward(q, k, v, *cu, causal=causal, scale=scale, out=o)
    s = q.shape[2] ** -0.5 if scale is None else float(np.float32(scale))
    want, wl, ot, lt = R.attention(_f64(q), _f64(k), _f64(v), cq, ck, causal, s, kind)
    _close(o[:nq], want[:nq], R.rounded(want, ot, kind)[:nq], "o")
    _close(lse[:, :nq], wl[:, :nq], lt[:, :nq], "lse")
    assert torch.all(o[nq:] == 7.0)
    g = [torch.full_like(x, 7.0) for x in (q, k, v)]
    M.ma_attention_backward(do, q, k, v, o, lse, *cu, causal=causal, scale=scale, dq=g[0], dk=g[1], dv=g[2])
    want, tol = R.attention_backward(_f64(do), _f64(q), _f64(k), _f64(v), _f64(o), _f64(lse), cq, ck, causal, s, kind)
    for x, w, t, n, name in zip(g, want, tol, (nq, int(ck[-1]), int(ck[-1])), ("dq", "dk", "dv")):
        _close(x[:n], w[:n], R.rounded(w, t, kind)[:n], name)
        assert torch.all(x[n:] == 7.0), name
    return o, lse, g


ATTN = [  # lengths of queries, of keys (None: the same), heads, key heads, dim, causal
    ([1], None, 1, 1, 64, True), ([1], [1], 2, 1, 128, False), ([33], None, 2, 2, 64, True), ([7, 1, 0, 70], None, 4, 2, 128, True),
    ([128], None, 1, 1, 128, True), ([129], [257], 2, 1, 64, True), ([50, 50], [261, 130], 4, 1, 256, False),
    ([200, 3, 140], None, 4, 4, 80, True), ([64, 65], [64, 1], 2, 1, 72, False), ([90, 5], [30, 200], 2, 2, 128, True),
    ([5, 0, 9], [0, 7, 300], 3, 1, 40, False), ([300], None, 6, 2, 24, True), ([31], [500], 1, 1, 200, True),
    ([260], [129], 2, 1, 33, True), ([100, 28], None, 2, 1, 7, True), ([513], None, 2, 1, 256, True), ([1] * 40, None, 2, 1, 64, True),
    ([3], [2000], 2, 2, 128, False), ([700], None, 2, 1, 128, True)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,heads,kv,dim,causal", ATTN)
def test_attention(kind, lq, lk, heads, kv, dim, causal):
    rng = np.random.default_rng(sum(lq) + dim)
    cq, ck = _offsets(lq), _offsets(lk or lq)
    # (rows behind the last sequence)
    q, k, v, do = _inputs(rng, int(cq[-1]) + 3, int(ck[-1]) + 5, heads, kv, dim, kind)
    for x in (q, do):
        x[int(cq[-1]):] = float("nan")
    for x in (k, v):
        x[int(ck[-1]):] = float("nan")
    o, lse, g = _check_attention(q, k, v, do, cq, ck, causal, None, kind)
    # bitwise the same for other layouts: heads outside, a part of wider rows, odd addresses
    cu = (_cu(cq), _cu(ck))
    nq, nk = int(cq[-1]), int(ck[-1])
    q2, k2, v2, do2 = (_heads_first(x) for x in (q, k, v, do))
    o2, lse2 = M.ma_attention_forward(q2, k2, v2, *cu, causal=causal, out=_heads_first(torch.zeros_like(q)))
    assert torch.equal(o2[:nq], o[:nq]) and torch.equal(lse2[:, :nq], lse[:, :nq])
    wide = [torch.zeros((x.shape[0], x.shape[1], dim + 3), dtype=x.dtype, device="cuda")[:, :, 1:1 + dim] for x in (q, k, v, do)]
    for a, b in zip(wide, (q, k, v, do)):
        a.copy_(b)
    o3, _ = M.ma_attention_forward(*wide[:3], *cu, causal=causal)
    assert torch.equal(o3[:nq], o[:nq])
    g2 = M.ma_attention_backward(do2, q2, k2, v2, o2, lse2, *cu, causal=causal)
    g3 = M.ma_attention_backward(wide[3], *wide[:3], o3, lse, *cu, causal=causal)
    for a, b, c, n in zip(g, g2, g3, (nq, nk, nk)):
        assert torch.equal(a[:n], b[:n]) and torch.equal(a[:n], c[:n])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,heads,kv,dim", [([1500, 900], None, 4, 1, 64), ([40, 1200, 7], [900, 1300, 64], 2, 2, 128),
                                                ([1111], None, 8, 1, 136)])
def test_attention_causal_walks_in_pieces(kind, lq, lk, heads, kv, dim):
    rng = np.random.default_rng(sum(lq) * 3 + dim)
    cq, ck = _offsets(lq), _offsets(lk or lq)
    _check_attention(*_inputs(rng, int(cq[-1]), int(ck[-1]), heads, kv, dim, kind), cq, ck, True, None, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_attention_one_sequence_without_offsets(kind):
    rng = np.random.default_rng(2)
    q, k, v, do = _inputs(rng, 150, 190, 4, 2, 64, kind)
    cu = (_cu(_offsets([150])), _cu(_offsets([190])))
    for causal in (True, False):
        o, lse = M.ma_attention_forward(q, k, v, causal=causal, scale=0.3)
        o2, lse2 = M.ma_attention_forward(q, k, v, *cu, causal=causal, scale=0.3)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(M.ma_attention_backward(do, q, k, v, o, lse, causal=causal, scale=0.3),
                        M.ma_attention_backward(do, q, k, v, o, lse, *cu, causal=causal, scale=0.3)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_attention_sharp_rows(kind):
    """Scores far apart, rising and falling along the keys (the softmax's reference moves at every tile, or
    never), and one key that takes everything."""
    rng = np.random.default_rng(5)
    n, d = 400, 64
    q, k, v, do = _inputs(rng, n, n, 3, 3, d, kind)
    ramp = torch.linspace(-30, 30, n, device="cuda")
    q[:, :, 0] = 8.0
    k[:, 0, 0], k[:, 1, 0], k[:, 2, 0] = ramp, -ramp, 0.0
    k[17, 2, 0] = 60.0
    _check_attention(q, k, v, do, _offsets([n]), _offsets([n]), False, 0.25, kind)
    _check_attention(q, k, v, do, _offsets([150, 250]), _offsets([150, 250]), True, 0.25, kind)


def test_attention_nan_stays_in_its_sequence():
    rng = np.random.default_rng(6)
    lens = [40, 100, 60]
    cq = _offsets(lens)
    q, k, v, do = _inputs(rng, 200, 200, 2, 1, 64, "bf16")
    o, lse = M.ma_attention_forward(q, k, v, _cu(cq), _cu(cq))
    g = M.ma_attention_backward(do, q, k, v, o, lse, _cu(cq), _cu(cq))
    for bad in (float("nan"), float("inf")):
        q2, k2, v2, do2 = (x.clone() for x in (q, k, v, do))
        for x in (q2, k2, v2, do2):
            x[60:130] = bad
        o2, lse2 = M.ma_attention_forward(q2, k2, v2, _cu(cq), _cu(cq))
        g2 = M.ma_attention_backward(do2, q2, k2, v2, o2, lse2, _cu(cq), _cu(cq))
        for s in (slice(0, 40), slice(140, 200)):
            assert torch.equal(o2[s], o[s]) and torch.equal(lse2[:, s], lse[:, s])
            for a, b in zip(g2, g):
                assert torch.equal(a[s], b[s])
        assert torch.isnan(o2[70:140]).all()


def test_attention_bad_offsets_stay_inside():
    """Offsets that fall, are negative or too large: what is computed is not defined, but nothing outside the
    arrays is touched."""
    rng = np.random.default_rng(7)
    for cu in ([0, 500, 100], [-7, 30, 100], [50, 20, 90], [0, 2 ** 31 - 1, 5], [90, 100, 300]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        q, k, v, do = _inputs(rng, 100, 100, 2, 1, 64, "bf16")
        guard = torch.full((300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        o, lse = M.ma_attention_forward(q, k, v, c, c, out=guard[100:200])
        M.ma_attention_backward(do, q, k, v, o, lse.nan_to_num(), c, c)
        assert torch.all(guard[:100] == 7.0) and torch.all(guard[200:] == 7.0)


def test_attention_gradient_against_differences():
    rng = np.random.default_rng(9)
    n, heads, kv, d = 20, 2, 1, 8
    x = [rng.standard_normal(s) for s in ((n, heads, d), (n, kv, d), (n, kv, d))]
    c = rng.standard_normal((n, heads, d))
    cq = _offsets([12, 8])
    t = [_dev(a) for a in x]
    o, lse = M.ma_attention_forward(*t, _cu(cq), _cu(cq))
    g = [_f64(a) for a in M.ma_attention_backward(_dev(c), *t, o, lse, _cu(cq), _cu(cq))]

    def f(y):
        return np.sum(c * R.attention(*y, cq, cq, True, d ** -0.5, "fp32")[0])

    for seed in range(4):
        r = np.random.default_rng(seed)
        u = [r.standard_normal(a.shape) for a in x]
        slope = (f([a + 1e-5 * b for a, b in zip(x, u)]) - f([a - 1e-5 * b for a, b in zip(x, u)])) / 2e-5
        got = sum(np.sum(a * b) for a, b in zip(g, u))
        # some 640 terms of about 1, each off by a few 2^-24 of its parts
        assert abs(got - slope) < 1e-3 * max(1.0, abs(slope))


def test_attention_empty():
    e = torch.zeros((0, 2, 64), device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = M.ma_attention_forward(e, e, e)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert M.ma_attention_backward(e, e, e, e, o, lse)[0].shape == (0, 2, 64)
    x = torch.randn(5, 2, 64, device="cuda")
    o, lse = M.ma_attention_forward(x, x, x, z, z, out=torch.full_like(x, 7.0))        # no sequence
    assert torch.all(o == 7.0)
    o, lse = M.ma_attention_forward(x, e, e, causal=False)                              # no keys
    assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    dq, dk, dv = M.ma_attention_backward(x, x, e, e, o, lse, causal=False)
    assert torch.all(dq == 0) and dk.shape == (0, 2, 64)
    dq, dk, dv = M.ma_attention_backward(e, e, x, x, e, lse[:, :0].contiguous(), causal=False)   # no queries
    assert torch.all(dk == 0) and torch.all(dv == 0)


def test_attention_refuses_heads_without_features():
    x = torch.zeros((4, 2, 8), device="cuda")
    many = torch.zeros((1, 1, 8), device="cuda").expand(1, 2 ** 31, 8)
    none = x[:, :, :0]
    for q, k in ((none, none), (many, many), (x, many)):
        with pytest.raises(ValueError, match="heads"):
            M.ma_attention_forward(q, k, k)
        with pytest.raises(ValueError, match="heads"):
            M.ma_attention_backward(q, q, k, k, q, torch.zeros((2, 4), device="cuda"))


def test_attention_of_the_most_rows():
    """2^28 queries of one feature and one key: launches longer than 2^32 threads, done in rounds."""
    n = 2 ** 28
    q = torch.empty((n, 1, 1), dtype=torch.bfloat16, device="cuda")
    q.view(-1)[:] = (torch.arange(n, device="cuda", dtype=torch.int32) % 5).to(torch.bfloat16)
    k = torch.ones((1, 1, 1), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 1.5)
    o, lse = M.ma_attention_forward(q, k, v, causal=False, scale=1.0)
    # a probability of 1 (off by less than 2^-20, and bfloat16's half step is 2^-8)
    assert torch.all(o == 1.5)
    assert (lse.view(-1) - q.view(-1).float()).abs().max() <= 2.0 ** -20
    # dv sums 2^28 ones: 2^23 a piece and 2^28 in all, exact in float32
    dq, dk, dv = M.ma_attention_backward(torch.ones_like(q), q, k, v, o, lse, causal=False, scale=1.0)
    assert torch.all(dq == 0) and dk.item() == 0 and dv.item() == 2.0 ** 28


# ------------------------------------------------------------ used together --

LENS = [13, 1, 50, 32]
HEADS, KV, DIM, VOCAB, HIDDEN = 4, 2, 16, 300, 64
SECTIONS = (2, 3, 3)
WEIGHTS = ("table", "w1", "wqkv", "wo", "w2", "head")
LAYER_NAMES = ["action_expert.embed_tokens.weight", "action_expert.layers.0.input_layernorm.weight",
               "action_expert.layers.0.self_attn.qkv_proj.weight", "action_expert.layers.0.self_attn.o_proj.weight",
               "action_expert.norm.weight", "action_expert.lm_head.weight"]


def _block_inputs(seed, kind="fp32"):
    rng = np.random.default_rng(seed)
    n = sum(LENS)
    p = dict(ids=torch.from_numpy(rng.integers(0, VOCAB, n)).cuda(), answer=torch.from_numpy(rng.integers(0, VOCAB, n)).cuda(),
             pos=torch.from_numpy(rng.integers(0, 1000, (3, n))).cuda(),
             g=_dev(rng.standard_normal(n) / n), h=_dev(np.full(n, 0.1 / n)))
    for name, shape, std in (("table", (VOCAB, HIDDEN), 0.1), ("wqkv", ((HEADS + 2 * KV) * DIM, HIDDEN), 0.125),
                             ("wo", (HIDDEN, HEADS * DIM), 0.125), ("head", (VOCAB, HIDDEN), 0.125)):
        p[name] = _dev(std * rng.standard_normal(shape), kind)
    for name in ("w1", "w2"):
        p[name] = _dev(1 + 0.2 * rng.standard_normal(HIDDEN), kind)
    return p


def _block(p, cu, plan):
    """A transformer block with its loss: embedding, norm, turned queries and keys, attention, residual, norm,
    answers' log probabilities with a bonus on entropy; forward and backward with the operators, plain matrix
    products for the layers themselves.  (loss parts, gradients or their sources in the order of WEIGHTS)"""
    n = p["ids"].numel()
    x = M.ma_embedding_lookup(p["table"], p["ids"], scale=8.0)
    y1, s1, inv1, c1 = M.ma_rms_norm_forward(x, p["w1"], y_ckpt=True)
    qkv = (y1 @ p["wqkv"].t()).view(n, HEADS + 2 * KV, DIM)
    qk = qkv[:, :HEADS + KV]
    M.ma_rotary(qk, p["pos"], plan, out=qk)
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    o, lse = M.ma_attention_forward(q, k, v, cu, cu)
    a = o.view(n, -1)
    y2, s2, inv2, c2 = M.ma_rms_norm_forward(a @ p["wo"].t(), p["w2"], x, y_ckpt=True)
    z = y2 @ p["head"].t()
    lp, ent, zl, _, _ = M.ma_token_logprob_forward(z, p["answer"])
    # backward
    dz = M.ma_token_logprob_backward(z, p["answer"], zl, p["g"], entropy=ent, dentropy=p["h"], out=z)
    ds2, dw2 = M.ma_rms_norm_backward(dz @ p["head"], s2, inv2, p["w2"])
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv[:, :HEADS], dqkv[:, HEADS:HEADS + KV], dqkv[:, HEADS + KV:]
    M.ma_attention_backward((ds2 @ p["wo"]).view_as(o), q, k, v, o, lse, cu, cu, dq=dq, dk=dk, dv=dv)
    dqk = dqkv[:, :HEADS + KV]
    M.ma_rotary(dqk, p["pos"], plan, inverse=True, out=dqk)
    dqkv = dqkv.view(n, -1)
    dx, dw1 = M.ma_rms_norm_backward(dqkv @ p["wqkv"], s1, inv1, p["w1"], ds2)
    return (lp, ent), [M.EmbeddingGrad(dx, p["ids"], 8.0), dw1, M.LinearGrad(dqkv, c1), M.LinearGrad(ds2, M.ma_act_pack(a)),
                       dw2, M.LinearGrad(dz, c2)]


def _formed(src):
    return [M.ma_embedding_grad(s.dout, s.tokens, VOCAB, scale=s.scale) if isinstance(s, M.EmbeddingGrad) else
            M.ma_linear_grad(s.dy, s.x) if isinstance(s, M.LinearGrad) else s for s in src]


def _plain_block(p):
    """The same in torch autograd, float64 on the CPU."""
    q = {k: t.double().cpu() if t.is_floating_point() else t.cpu() for k, t in p.items()}
    for k in WEIGHTS:
        q[k].requires_grad_()
    n = q["ids"].numel()

    def norm(x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    x = q["table"][q["ids"]] * 8.0
    qkv = (norm(x, q["w1"]) @ q["wqkv"].t()).view(n, -1, DIM)
    ang = torch.stack([q["pos"][a].double() * f for a, f in R.rotary_table(SECTIONS, 10000.0, "blocks", False)], 1)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = qkv[:, :HEADS + KV, :DIM // 2], qkv[:, :HEADS + KV, DIM // 2:]
    qk = torch.cat([a * c - b * s, a * s + b * c], -1)
    o, at = [], 0
    for m in LENS:
        r = slice(at, at + m)
        at += m
        z = torch.einsum("qhd,khd->hqk", qk[r, :HEADS], qk[r, HEADS:].repeat_interleave(2, 1)) / DIM ** 0.5
        z = z.masked_fill(torch.ones(m, m, dtype=torch.bool).triu(1), -np.inf)
        o.append(torch.einsum("hqk,khd->qhd", torch.softmax(z, -1), qkv[r, HEADS + KV:].repeat_interleave(2, 1)))
    s2 = torch.cat(o).reshape(n, -1) @ q["wo"].t() + x
    lp = torch.log_softmax(norm(s2, q["w2"]) @ q["head"].t(), -1)
    ent = -(lp.exp() * lp).sum(-1)
    got = lp[torch.arange(n), q["answer"]]
    ((got * q["g"]).sum() + (ent * q["h"]).sum()).backward()
    return got.detach().numpy(), ent.detach().numpy(), [q[k].grad.numpy() for k in WEIGHTS]


def test_block_gradients():
    """float32 throughout.  Sums of at most 300 terms in a chain of some eight operators, each result off by
    at most its terms' 2^-24 and twice as much again where one is divided by a norm: 8 x 2 x 300 x 2^-24 = 2.9e-4
    of a result's norm even if all errors were aligned.  The linear layers' weights see inputs held in 8 bits,
    off by at most half a step: 1.8 % of a group of 32 normal values."""
    p = _block_inputs(1)
    cu, plan = _cu(_offsets(LENS)), M.Rotary(SECTIONS)
    (lp, ent), src = _block(p, cu, plan)
    wl, we, want = _plain_block(p)
    assert np.abs(_f64(lp) - wl).max() < 3e-4 * np.abs(wl).max() and np.abs(_f64(ent) - we).max() < 3e-4 * np.abs(we).max()
    for g, w, s, name in zip(_formed(src), want, src, WEIGHTS):
        rel = np.linalg.norm(_f64(g) - w) / np.linalg.norm(w)
        assert rel < (0.019 if isinstance(s, M.LinearGrad) else 3e-4), (name, rel)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_block_feeds_the_optimizer(kind):
    """The step with gradients and their sources is the step with the formed gradients."""
    p = _block_inputs(2, kind)
    cu, plan = _cu(_offsets(LENS)), M.Rotary(SECTIONS)
    outs = []
    for form in (False, True):
        params = [p[k].clone() for k in WEIGHTS]
        opt = M.MuonAdamW(list(zip(LAYER_NAMES, params, [True] * 6)), lr=1e-3)
        for _ in range(2):
            src = [s.to(DT[kind]) if isinstance(s, torch.Tensor) else s for s in _block(p, cu, plan)[1]]
            if form:
                src = [g.to(DT[kind]) if isinstance(s, torch.Tensor) else
                       M.ma_embedding_grad(s.dout, s.tokens, VOCAB, scale=s.scale, grad_dtype=DT[kind])
                       if isinstance(s, M.EmbeddingGrad) else M.ma_linear_grad(s.dy, s.x, grad_dtype=DT[kind])
                       for s, g in zip(src, src)]
            opt.step(src)
        outs.append(params)
    for a, b, k in zip(*outs, WEIGHTS):
        assert torch.equal(a, b), k
        # (an AdamW step moves a weight by about lr = 1e-3: in bfloat16 less than half the 2^-7 or 2^-8
        # between values near 1, so the norms' weights stay)
        assert not torch.equal(a, p[k]) or (kind == "bf16" and k in ("w1", "w2")), k


def _everything(p, cu, plan, big):
    """The block, and calls whose work is cut into pieces and joined."""
    (lp, ent), src = _block(p, cu, plan)
    q, k, z, ids = big
    o, lse = M.ma_attention_forward(q, k, k, causal=False)
    got = M.ma_attention_backward(o, q, k, k, o, lse, causal=False)
    return [lp, ent, *_formed(src), o, lse, *got, *M.ma_token_logprob_forward(z, ids, top=7)]


def _big(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    return [r(40, 2, 128), r(3000, 1, 128), r(3, 90000), torch.tensor([5, 80000, 17], device="cuda")]


def test_block_captured_and_replayed():
    """Captured once and replayed on changed inputs, with eager work in between, equals the eager
    results each time."""
    p, big = _block_inputs(20), _big(20)
    cu, plan = _cu(_offsets(LENS)), M.Rotary(SECTIONS)
    _everything(p, cu, plan, big)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _everything(p, cu, plan, big)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _everything(p, cu, plan, big)
    del plan                                     # (the graph holds its own frequencies)
    plan = M.Rotary(SECTIONS)
    for seed in (21, 22, 23, 24):
        for k, v in _block_inputs(seed).items():
            p[k].copy_(v)
        for a, b in zip(big, _big(seed)):
            a.copy_(b)
        for o in outs:
            o.fill_(float("nan") if o.is_floating_point() else -1)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for i, (a, b) in enumerate(zip(got, _everything(p, cu, plan, big))):
            assert torch.equal(a, b), (seed, i)
        torch.cuda.synchronize()


def test_two_graphs_and_two_streams():
    """Two graphs of the same operators on different data replayed in turn, then at once, and two eager
    streams at once."""
    ps, bigs = [_block_inputs(50 + k) for k in range(2)], [_big(50 + k) for k in range(2)]
    cu, plan = _cu(_offsets(LENS)), M.Rotary(SECTIONS)
    want = [_everything(p, cu, plan, b) for p, b in zip(ps, bigs)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p, b in zip(ps, bigs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_everything(p, cu, plan, b))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    for r in range(4):
        for o in outs:
            for t in o:
                t.fill_(float("nan") if t.is_floating_point() else -1)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
            if r < 2:
                st.synchronize()
        for st in streams:
            st.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w)), r
    for _ in range(3):
        got = []
        for p, b, st in zip(ps, bigs, streams):
            with torch.cuda.stream(st):
                got.append(_everything(p, cu, plan, b))
        for st in streams:
            st.synchronize()
        for o, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_streams_are_taken_as_arguments():
    """Each call on another stream than the current one, as an object and as a raw handle."""
    rng = np.random.default_rng(3)
    x, w, r = _dev(_stream(rng, 30, 96)), _dev(np.ones(96)), _dev(_stream(rng, 30, 96))
    q, k, v, do = _inputs(rng, 60, 500, 2, 1, 64, "bf16")
    ids, plan, pos = torch.arange(30, device="cuda"), M.Rotary(32), torch.arange(60, device="cuda")
    z = _dev(_logits(rng, 30, 20000))

    def all_calls(**kw):
        y, s, inv, c = M.ma_rms_norm_forward(x, w, r, y_ckpt=True, **kw)
        ds, dw = M.ma_rms_norm_backward(y, s, inv, w, r, **kw)
        lp, ent, lse, top, best = M.ma_token_logprob_forward(z, ids, top=3, **kw)
        dz = M.ma_token_logprob_backward(z, ids, lse, lp, entropy=ent, dentropy=ent, **kw)
        t = M.ma_rotary(q, pos, plan, **kw)
        o, l = M.ma_attention_forward(t, k, v, causal=False, **kw)
        return [y, s, inv, c.codes, ds, dw, lp, ent, lse, top, best, dz, t, o, l,
                *M.ma_attention_backward(do, t, k, v, o, l, causal=False, **kw)]

    want = all_calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        got = all_calls(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Every operator at random sizes, types and strides (each a view of a wider array filled with NaN)."""
    rng = np.random.default_rng(2000 + seed)

    def size(most):
        return int(np.exp(rng.random() * np.log(most)))

    def kind():
        return ("fp32", "bf16")[rng.integers(2)]

    def view(x, k):
        v, wide = _strided(x, int(rng.integers(0, 20)), k)
        wide[:, x.shape[1]:] = float("nan")
        return v

    rows, cols, t, wk = size(3000), size(3000), kind(), kind()
    x, r, w = view(_stream(rng, rows, cols), t), view(_stream(rng, rows, cols), t), _dev(rng.standard_normal(cols), wk)
    y, s, inv, c = M.ma_rms_norm_forward(x, w, r, eps=1e-5, weight_offset=0.5, y_ckpt=True)
    yy, ss, ii, dy, ds, di = R.rms_norm(_f64(x), _f64(w), _f64(r), 1e-5, 0.5)
    _close(y, yy, R.rounded(yy, dy, t), "y")
    _close(inv, ii, di, "inv")
    assert torch.equal(M.ma_act_pack(y).codes, c.codes)
    g = view(rng.standard_normal((rows, cols)), t)
    a, b = M.ma_rms_norm_backward(g, s, inv, w, r, weight_offset=0.5, grad_dtype=DT[wk])
    want, dwant, tol, wtol = R.rms_norm_backward(_f64(g), _f64(s), _f64(inv), _f64(w), 0.5, _f64(r))
    _close(a, want, R.rounded(want, tol, t), "ds")
    _close(b, dwant, R.rounded(dwant, wtol, wk), "dw")

    rows, vocab, t = size(300), size(40000), kind()
    z = view(_logits(rng, rows, vocab), t)
    ids = rng.integers(0, vocab, rows)
    _check_logprob(z, ids, 0.8, min(vocab, int(rng.integers(0, 30))))
    lse = M.ma_token_logprob_forward(z, torch.from_numpy(ids).cuda(), scale=0.8)[2]
    g = _dev(rng.standard_normal(rows))
    want, tol = R.logprob_backward(_f64(z), ids, float(np.float32(0.8)), _f64(lse), _f64(g))
    _close(M.ma_token_logprob_backward(z, torch.from_numpy(ids).cuda(), lse, g, scale=0.8), want, R.rounded(want, tol, t))

    tokens, heads, dim, t = size(2000), int(rng.integers(1, 9)), int(rng.integers(2, 257)), kind()
    axes = int(rng.integers(1, 5))
    cut = np.sort(rng.integers(0, dim // 2, axes - 1)) if axes > 1 else np.zeros(0, int)
    sections = [int(n) for n in np.diff(np.concatenate([[0], cut, [max(1, int(rng.integers(1, dim // 2 + 1)))]]))]
    if min(sections) >= 0 and sum(sections) > 0:
        how = (("half", "pairs")[rng.integers(2)], ("blocks", "cycled")[rng.integers(2)], bool(rng.integers(2)))
        x = view(rng.standard_normal((tokens, heads * dim)), t).unflatten(1, (heads, dim))
        pos = rng.integers(0, 5000, (axes, tokens))
        got = M.ma_rotary(x, torch.from_numpy(pos).cuda(), M.Rotary(sections, layout=how[0], order=how[1], restart=how[2]))
        want, tol = R.rotary(_f64(x), pos, R.rotary_table(sections, 10000.0, how[1], how[2]), how[0])
        _close(got, want, R.rounded(want, tol, t))

    kv, t = int(rng.integers(1, 4)), kind()
    heads, dim, n = kv * int(rng.integers(1, 4)), int(rng.integers(1, 257)), int(rng.integers(1, 6))
    cq, ck = _offsets(rng.integers(0, size(400) + 1, n)), _offsets(rng.integers(0, size(400) + 1, n))
    arr = [view(rng.standard_normal((max(1, int(m)), h * dim)), t).unflatten(1, (h, dim))
           for m, h in ((cq[-1], heads), (ck[-1], kv), (ck[-1], kv), (cq[-1], heads))]
    _check_attention(*arr, cq, ck, bool(rng.integers(2)), None, t)


# ----------------------------------------------------- offsets past 32 bits --

def test_long_offsets():
    """Arrays of more than 2^31 elements (4.4 GB): their far ends."""
    rows, cols = 540_000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    w = torch.full((cols,), 3.0, device="cuda")
    y, _, inv, c = M.ma_rms_norm_forward(x, w, eps=1e-6, y_ckpt=True)
    assert torch.all(y[-1] == 3.0) and float(y[:-1].abs().max()) == 0.0 and abs(float(inv[-1]) - 0.5) < 1e-6
    assert torch.all(M.ma_act_unpack(M.ActCheckpoint(c.codes[-1:], c.exps[-1:], cols)) == 3.0)
    del y, c
    ds, dw = M.ma_rms_norm_backward(x, x, inv, w)
    assert float(ds[-1].abs().max()) < 1e-2 and torch.all((dw - 2.0).abs() < 1e-5)
    del ds
    t = M.ma_rotary(x.view(rows, 32, 128), torch.arange(rows, device="cuda"), M.Rotary(64))
    want = M.ma_rotary(x[-1:].view(1, 32, 128), torch.tensor([rows - 1], device="cuda"), M.Rotary(64))
    assert torch.equal(t[-1:], want) and float(t[:-1].abs().max()) == 0.0
    del t
    ids = torch.full((rows,), 7, device="cuda")
    lp, _, lse, top, _ = M.ma_token_logprob_forward(x, ids, top=2)
    assert torch.all((lp + np.log(cols)).abs() < 1e-5) and top[-1].tolist() == [0, 1]
    x[-1, 9] = 12.0
    lp2 = M.ma_token_logprob_forward(x, torch.full((rows,), 9, device="cuda"))[0]
    assert float(lp2[-1]) > -1 and torch.equal(lp2[:-1], lp[:-1])
    d = M.ma_token_logprob_backward(x, ids, lse, torch.ones(rows, device="cuda"), out=x)
    assert abs(float(d[-1, 7]) - (1 - 1 / cols)) < 1e-2 and abs(float(d[0, 7]) - (1 - 1 / cols)) < 1e-2
    del x, d
    torch.cuda.empty_cache()
    # attention over rows that lie far apart in a cache of 2^32 elements
    n = 1 << 13
    cache = torch.empty((n, 1 << 19), dtype=torch.bfloat16, device="cuda")
    k, v = cache[:, :128].unflatten(1, (1, 128)), cache[:, -128:].unflatten(1, (1, 128))
    k.normal_(), v.normal_()
    q = torch.randn(70, 2, 128, device="cuda").to(torch.bfloat16)
    o, lse = M.ma_attention_forward(q, k, v)
    o2, lse2 = M.ma_attention_forward(q, k.contiguous(), v.contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = M.ma_attention_backward(o, q, k, v, o, lse, dk=torch.empty_like(k, memory_format=torch.contiguous_format))
    for a, b in zip(g, M.ma_attention_backward(o, q, k.contiguous(), v.contiguous(), o, lse)):
        assert torch.equal(a, b)
    del cache, k, v
    torch.cuda.empty_cache()
