"""The gradient operators (include/ma_grads.h) on the GPU against float64
references: embedding lookup and gradient, activations held in 8 bits, the
linear layer's weight gradient from them and the gated activation, at the sizes,
types, strides and values where each can go wrong; their use together up to an
optimizer step; graph capture, streams and reruns."""

import numpy as np
import pytest

from tests import _grads_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.load_library()
    yield
    torch.cuda.synchronize()


def _dev(x, kind="fp32"):
    """x on the GPU in the given type."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda").to(DT[kind])


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, want, tol, what=""):
    got = _f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    bad_nan = np.isnan(got) != np.isnan(want)
    assert not bad_nan.any(), "%s: NaN in %d other places" % (what, bad_nan.sum())
    m = ~np.isnan(want)
    inf = m & np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    m &= ~inf
    off = np.abs(got[m] - want[m]) - (tol[m] if isinstance(tol, np.ndarray) else tol)
    assert off.size == 0 or off.max() <= 0, "%s: %g over the bound" % (what, off.max())


def _activation(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))
    x[:, rng.random(cols) < 0.02] *= 50
    if rows > 2:
        x[1] = 0.0
    return x


def _strided(x, pad, kind):
    """x as a view of a wider array (rows pad elements apart more)."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, device="cuda", dtype=DT[kind])
    v = wide[:, :x.shape[1]]
    v.copy_(_dev(x, kind))
    return v, wide


# ------------------------------------------------------------ 8-bit form --

@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 31, 0), (2, 32, 0), (5, 33, 0),
                                           (4, 64, 8), (7, 100, 0), (3, 128, 3), (2, 1000, 0),
                                           (50, 256, 0), (1, 4097, 1)])
def test_pack_is_the_definition(kind, rows, cols, pad):
    rng = np.random.default_rng(rows * 10007 + cols)
    x, _ = _strided(_activation(rng, rows, cols), pad, kind)
    c = M.ma_act_pack(x)
    codes, exps = R.pack(_f64(x))
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.exps.cpu().numpy()[:, :codes.shape[1] // 32], exps[:, :codes.shape[1] // 32])
    want = R.unpack(codes, exps, cols)
    for out in ("fp32", "bf16"):        # every held value is exact in bf16
        assert np.array_equal(_f64(M.ma_act_unpack(c, DT[out])), want)
    into, wide = _strided(np.zeros((rows, cols)), 5, "fp32")
    M.ma_act_unpack(c, out=into)
    assert np.array_equal(_f64(into), want)
    assert torch.all(wide[:, cols:] == 7.0)


def test_pack_borders():
    """Around each power of two, the quotients 127, 127.5 and 128; the smallest
    and largest floats; signed zeros; ties."""
    f = np.float32
    tops = []
    for k in (-149, -140, -130, -127, -126, -121, -120, -119, -20, -1, 0, 1, 60, 126, 127):
        for m in (1.0, 1.5, 127 / 64, 127.5 / 64, np.nextafter(f(127.5 / 64), f(0)),
                  np.nextafter(f(2.0), f(0))):
            with np.errstate(over="ignore"):
                v = f(np.ldexp(float(m), k))
            if np.isfinite(v):
                tops.append(v)
    x = np.zeros((len(tops), 40), np.float32)
    rng = np.random.default_rng(0)
    for r, t in enumerate(tops):
        x[r, 0] = t if r % 2 else -t
        x[r, 1:32] = (t * rng.integers(-255, 256, 31) / 256).astype(f)     # ties among them
        x[r, 32:] = -0.0
    d = torch.from_numpy(x).cuda()
    c = M.ma_act_pack(d)
    codes, exps = R.pack(x.astype(np.float64))
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.exps.cpu().numpy()[:, :2], exps[:, :2])
    got = _f64(M.ma_act_unpack(c))
    assert np.isfinite(got).all()
    assert np.array_equal(got, R.unpack(codes, exps, 40))


def test_pack_nonfinite_group_stands_for_nan():
    x = np.ones((4, 96), np.float32)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 95] = -np.inf
    for kind in ("fp32", "bf16"):
        c = M.ma_act_pack(_dev(x, kind))
        got = _f64(M.ma_act_unpack(c))
        want = np.ones((4, 96))
        want[0, :32] = want[1, 32:64] = want[2, 64:] = np.nan
        assert np.array_equal(got, want, equal_nan=True)


def test_pack_token_alone():
    """A token's form depends on that token only: any batch gives the same bytes."""
    rng = np.random.default_rng(3)
    x = _dev(_activation(rng, 37, 200), "bf16")
    whole = M.ma_act_pack(x)
    for r in (0, 1, 17, 36):
        one = M.ma_act_pack(x[r])
        assert torch.equal(one.codes[0], whole.codes[r]) and torch.equal(one.exps[0], whole.exps[r])
        assert tuple(M.ma_act_unpack(one).shape) == (200,)


def test_pack_empty_and_leading_dimensions():
    c = M.ma_act_pack(torch.zeros((0, 70), device="cuda"))
    assert tuple(M.ma_act_unpack(c).shape) == (0, 70)
    x = torch.randn(2, 3, 5, 70, device="cuda")
    c = M.ma_act_pack(x)
    assert c.shape == (2, 3, 5, 70) and c.rows == 30
    assert torch.equal(M.ma_act_unpack(c).view(30, 70), M.ma_act_unpack(M.ma_act_pack(x.view(30, 70))))
    # a repeated row (stride 0)
    r = torch.randn(70, device="cuda").expand(4, 70)
    assert torch.equal(M.ma_act_pack(r).codes, M.ma_act_pack(r.contiguous()).codes)


# -------------------------------------------------------------- embedding --

@pytest.mark.parametrize("ti,to", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16"),
                                   ("bf16", "fp32")])
@pytest.mark.parametrize("n,v,h,pad", [(1, 1, 1, 0), (1, 50, 256, 0), (37, 1000, 256, 0),
                                       (130, 33, 100, 4), (65, 7, 1001, 0), (9, 40, 2048, 8)])
def test_lookup(ti, to, n, v, h, pad):
    rng = np.random.default_rng(n + v + h)
    table, _ = _strided(rng.standard_normal((v, h)), pad, ti)
    ids = rng.integers(0, v, n)
    for tok in (torch.int64, torch.int32):
        got = M.ma_embedding_lookup(table, torch.from_numpy(ids).to("cuda", tok), scale=h ** 0.5,
                                    out_dtype=DT[to])
        assert got.dtype == DT[to] and tuple(got.shape) == (n, h)
        want = _f64(table)[ids] * h ** 0.5
        _close(got, want, R.rounded(want, 2 * R.F32 * np.abs(want), to))


def test_lookup_tokens_outside_and_shapes():
    table = torch.randn(10, 24, device="cuda")
    table[3] = float("nan")
    ids = torch.tensor([[0, -1, 9], [10, 5, -2 ** 40], [2 ** 32 + 1, 2 ** 62, 1]], device="cuda")
    out = torch.full((3, 3, 32), 5.0, device="cuda")
    M.ma_embedding_lookup(table, ids, scale=2.0, out=out[:, :, :24])
    want = torch.zeros(3, 3, 24, device="cuda")
    for r, c, t in ((0, 0, 0), (0, 2, 9), (1, 1, 5), (2, 2, 1)):
        want[r, c] = 2.0 * table[t]
    assert torch.equal(out[:, :, :24], want)
    assert torch.all(out[:, :, 24:] == 5.0)
    assert tuple(M.ma_embedding_lookup(table, ids[:0].reshape(0, 3)).shape) == (0, 3, 24)
    got = M.ma_embedding_lookup(table, torch.tensor(3, device="cuda"))
    assert got.shape == (24,) and torch.isnan(got).all()


def _tokens(rng, how, n, v):
    if how == "uniform":
        return rng.integers(0, v, n)
    if how == "one":
        return np.full(n, v // 2)
    if how == "last":
        return np.full(n, v - 1)
    if how == "zipf":
        return np.minimum(np.exp(rng.random(n) * np.log(v + 1)).astype(np.int64) - 1, v - 1)
    if how == "mixed":         # runs of one row, ids outside, padding
        t = rng.integers(-2, v + 2, n)
        t[n // 3:n // 2] = v // 3
        return t
    return np.full(n, -1)      # "none"


def test_lookup_of_more_rows_than_one_grid_axis():
    n, v, h = 4 * 65536 + 5, 301, 1032          # 4 rows a workgroup
    table = torch.randn(v, h, device="cuda").to(torch.bfloat16)
    tok = torch.randint(-1, v, (n,), device="cuda")
    out = torch.full((n + 1, h), 7.0, dtype=torch.bfloat16, device="cuda")
    M.ma_embedding_lookup(table, tok, out=out[:n])
    want = torch.cat([table, torch.zeros_like(table[:1])])[tok]
    assert torch.equal(out[:n], want)
    assert torch.all(out[n] == 7.0)


@pytest.mark.parametrize("td,tg", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"),
                                   ("fp32", "bf16")])
@pytest.mark.parametrize("n,v,h,how", [
    (1, 1, 1, "uniform"), (1, 1000, 256, "last"), (2, 3, 8, "one"), (31, 7, 33, "uniform"),
    (32, 40, 16, "zipf"), (33, 40, 16, "one"), (64, 5, 24, "mixed"), (512, 1000, 256, "zipf"),
    (1000, 1023, 40, "mixed"), (1025, 1024, 8, "uniform"), (3000, 70000, 24, "zipf"),
    (5000, 300, 17, "mixed"), (4097, 2, 8, "uniform"), (2500, 1100000, 8, "mixed"),
    (700, 50, 2048, "one"), (257, 9, 12, "none"), (1024, 40, 520, "one"), (1024, 9000, 16, "zipf"),
    (2048, 3, 40, "mixed"), (2049, 40, 264, "one"), (4096, 600, 16, "zipf"), (4096, 9, 8, "none"),
    (9000, 5000, 300, "zipf"), (20000, 3, 24, "one"), (140000, 700, 8, "mixed")])
def test_embedding_grad(td, tg, n, v, h, how):
    rng = np.random.default_rng(n * 31 + v + h)
    ids = _tokens(rng, how, n, v)
    pad = v - 1 if how == "mixed" else -1
    d = _dev(rng.standard_normal((n, h)), td)
    scale = h ** 0.5
    tok = torch.from_numpy(ids).cuda()
    got = M.ma_embedding_grad(d, tok, v, scale=scale, padding_token=pad, grad_dtype=DT[tg])
    want, tol = R.embedding_grad(_f64(d), ids, v, scale, pad)
    _close(got, want, R.rounded(want, tol, tg), "grad")
    # reruns are bitwise equal, whatever the workspace held
    need = M.ma_embedding_grad_workspace_size(n, v, h)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    again = M.ma_embedding_grad(d, tok.to(torch.int32), v, scale=scale, padding_token=pad,
                                out=torch.full_like(got, float("nan")), workspace=ws)
    assert torch.equal(got, again)


@pytest.mark.parametrize("td,tg", [("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("n,v,h,how", [
    # chunks of 20, 18, 35 and 69 sorted entries, one to four workgroups per CU
    (5003, 400, 2040, "mixed"), (5003, 2, 2040, "one"), (9001, 5000, 1001, "zipf"),
    (70001, 900, 300, "mixed"), (140001, 30, 520, "mixed")])
def test_embedding_grad_of_long_chunks(td, tg, n, v, h, how):
    test_embedding_grad(td, tg, n, v, h, how)


@pytest.mark.parametrize("tg", ["fp32", "bf16"])
@pytest.mark.parametrize("n,v,h,off", [
    # many more rows than tokens: few tokens, and tables whose zeroing is told the rows of tokens,
    # at any address; rows of more than 32 KB; three passes of the sort; one row
    (0, 4001, 33, 1), (3000, 30011, 264, 0), (3000, 30011, 263, 3), (4097, 40009, 264, 0),
    (4097, 40009, 264, 8), (4100, 40009, 264, 9), (5000, 50021, 251, 5), (4500, 900, 16392, 16),
    (5000, 1100003, 16, 24), (200000, 1100003, 8, 64), (200000, 2200003, 4, 0), (5000, 1, 16, 8),
    (4097, 3, 1, 1)])
def test_embedding_grad_zeroes_the_other_rows(tg, n, v, h, off):
    """Rows without a token are zero, whatever they held, and what lies before and
    behind the gradient is left alone."""
    rng = np.random.default_rng(n + v + h)
    ids = torch.from_numpy(rng.integers(-1, v, n)).cuda()
    d = torch.randn(n, h, device="cuda").to(torch.bfloat16)
    buf = torch.full((off + v * h + 300,), 7.0, dtype=DT[tg], device="cuda")
    out = buf[off:off + v * h].view(v, h)
    M.ma_embedding_grad(d, ids, v, out=out)
    assert torch.all(buf[:off] == 7.0) and torch.all(buf[off + v * h:] == 7.0)
    hit = torch.zeros(v, dtype=torch.bool, device="cuda")
    real = ids >= 0
    hit[ids[real]] = True
    assert torch.all(out[~hit] == 0)
    rows = torch.nonzero(hit)[:, 0]
    want = torch.zeros(len(rows), h, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    at = torch.searchsorted(rows, ids[real])
    want.index_add_(0, at, d[real].double())
    mag.index_add_(0, at, d[real].double().abs())
    count = torch.bincount(at, minlength=len(rows))[:, None].double()
    want, tol = want.cpu().numpy(), ((count + 4) * R.F32 * mag).cpu().numpy()
    _close(out[rows], want, R.rounded(want, tol, tg))


@pytest.mark.parametrize("tg", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1100, 5000])
@pytest.mark.parametrize("v,h,off", [(3, 1, 0), (1, 3, 0), (2, 1, 5), (7, 4, 4), (30, 1, 1), (5, 3, 33)])
def test_embedding_grad_of_few_bytes(tg, n, v, h, off):
    """A gradient inside one 128-byte line, mostly without a whole 16-byte piece, whose rows have
    one to three tokens in a batch of padding: each row is written by the launch of the sums
    itself, beside which nothing may zero it."""
    rng = np.random.default_rng(n + 7 * v + h + off)
    ids = np.full(n, -1)
    places = rng.permutation(n)
    for r in range(v):
        for k in range(1 + r % 3):
            ids[places[3 * r + k]] = r
    d = _dev(rng.standard_normal((n, h)), "fp32")
    buf = torch.full((off + v * h + 64,), 7.0, dtype=DT[tg], device="cuda")
    out = buf[off:off + v * h].view(v, h)
    want, tol = R.embedding_grad(_f64(d), ids, v, 1.5, -1)
    for tok in (torch.from_numpy(ids).cuda(), torch.from_numpy(ids).cuda().to(torch.int32)):
        out.fill_(7.0)
        M.ma_embedding_grad(d, tok, v, scale=1.5, out=out)
        _close(out, want, R.rounded(want, tol, tg))
        assert torch.all(buf[:off] == 7.0) and torch.all(buf[off + v * h:] == 7.0)


@pytest.mark.parametrize("tg", ["fp32", "bf16"])
@pytest.mark.parametrize("n,v,h,how", [(1, 4, 8, "uniform"), (300, 20, 40, "mixed"),
                                       (3000, 900, 33, "zipf"), (0, 6, 8, "none")])
def test_embedding_grad_accumulates(tg, n, v, h, how):
    rng = np.random.default_rng(n + v)
    ids = _tokens(rng, how, n, v)
    d = _dev(rng.standard_normal((n, h)), "bf16")
    old = _dev(rng.standard_normal((v, h)), tg)
    old[v // 2] = float("nan") if n == 0 else old[v // 2]
    out = old.clone()
    M.ma_embedding_grad(d, torch.from_numpy(ids).cuda(), v, scale=0.5, out=out, accumulate=True)
    want, tol = R.embedding_grad(_f64(d), ids, v, 0.5, -1, _f64(old))
    hit = np.isin(np.arange(v), ids)
    assert torch.equal(out[~torch.from_numpy(hit).cuda()].nan_to_num(3.0),
                       old[~torch.from_numpy(hit).cuda()].nan_to_num(3.0))
    _close(out[torch.from_numpy(hit).cuda()], want[hit], R.rounded(want, tol, tg)[hit])


def test_embedding_grad_strides_and_nan():
    rng = np.random.default_rng(5)
    d, wide = _strided(rng.standard_normal((90, 40)), 8, "bf16")
    wide[:, 40:] = float("nan")
    ids = torch.from_numpy(rng.integers(0, 9, 90)).cuda()
    ids[7] = -1
    d[7] = float("nan")               # a masked position's gradient is never read in
    got = M.ma_embedding_grad(d, ids, 9)
    assert torch.isfinite(got).all()
    assert torch.equal(got, M.ma_embedding_grad(d.contiguous(), ids, 9))
    # one gradient row for every token (stride 0), two leading dimensions
    one = torch.randn(40, device="cuda").expand(6, 15, 40)
    got = M.ma_embedding_grad(one, ids.view(6, 15), 9)
    assert torch.equal(got, M.ma_embedding_grad(one.contiguous(), ids.view(6, 15), 9))
    # NaN and infinity reach their row and no other
    d2 = torch.ones(4, 8, device="cuda")
    d2[2, 3] = float("inf")
    d2[3, 5] = float("nan")
    g = M.ma_embedding_grad(d2, torch.tensor([0, 1, 1, 2], device="cuda"), 4)
    assert torch.isinf(g[1, 3]) and torch.isnan(g[2, 5])
    assert torch.isfinite(g[0]).all() and torch.isfinite(g[3]).all()
    assert torch.isfinite(g).sum() == 30
    # no tokens at all: a gradient of zeros
    g = M.ma_embedding_grad(torch.zeros(0, 8, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"),
                            5, out=torch.full((5, 8), 3.0, device="cuda"))
    assert torch.all(g == 0)


# ------------------------------------------------------------ linear grad --

def _ckpt(x):
    """x held in 8 bits, and the values that stands for."""
    c = M.ma_act_pack(_dev(x, "bf16"))
    return c, R.unpack(c.codes.cpu().numpy(), c.exps.cpu().numpy(), x.shape[1])


@pytest.mark.parametrize("td,tg", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32"),
                                   ("fp32", "bf16")])
@pytest.mark.parametrize("m,n,k,pad", [
    (1, 1, 1, 0), (1, 256, 256, 0), (0, 40, 33, 0), (31, 16, 32, 0), (32, 128, 128, 8),
    (33, 130, 70, 1), (77, 256, 256, 0), (64, 257, 129, 0), (300, 24, 1000, 0),
    (5000, 24, 40, 0), (2049, 264, 136, 8), (1000, 520, 300, 4), (700, 7, 8, 0),
    (1024, 1024, 256, 0), (1025, 1032, 300, 8), (2100, 1288, 513, 0), (1500, 1030, 256, 3),
    (8191, 1024, 257, 16)])
def test_linear_grad(td, tg, m, n, k, pad):
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    dy, wide = _strided(rng.standard_normal((m, n)), pad, td)
    if pad:
        wide[:, n:] = float("nan")
    c, x = _ckpt(_activation(rng, m, k))
    got = M.ma_linear_grad(dy, c, grad_dtype=DT[tg])
    want, tol = R.linear_grad(_f64(dy), x)
    _close(got, want, R.rounded(want, tol, tg), "grad")
    old = _dev(rng.standard_normal((n, k)), tg)
    need = M.ma_linear_grad_workspace_size(m, n, k, DT[td])
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    out = old.clone()
    M.ma_linear_grad(dy, c, out=out, accumulate=True, workspace=ws)
    want, tol = R.linear_grad(_f64(dy), x, _f64(old))
    _close(out, want, R.rounded(want, tol, tg), "accumulated")
    assert torch.equal(got, M.ma_linear_grad(dy, c, out=torch.full_like(got, float("nan"))))


@pytest.mark.parametrize("td", ["bf16", "fp32"])
def test_linear_grad_units(td):
    """One product per output: dy and x are rows of an identity, so every output
    is one value of the other, exactly."""
    m, n, k = 200, 200, 136
    rng = np.random.default_rng(1)
    c, x = _ckpt(_activation(rng, m, k))
    eye = torch.eye(m, n, device="cuda", dtype=DT[td])
    assert np.array_equal(_f64(M.ma_linear_grad(eye, c)), x)
    dy = _dev(rng.standard_normal((m, n)), td)
    ident = M.ma_act_pack(torch.eye(m, k, device="cuda"))
    # (float32 dy: the three parts add up to it)
    assert np.array_equal(_f64(M.ma_linear_grad(dy, ident)), _f64(dy)[:k].T)


@pytest.mark.parametrize("tg", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k,pad", [(3000, 3001, 2048, 0), (4100, 3004, 2047, 1),
                                       (3000, 3000, 2048, 7), (8192, 1024, 4096, 0)])
def test_linear_grad_large_odd(tg, m, n, k, pad):
    """Large products whose dY rows are not 16-byte aligned (they are copied into
    ones that are), and one that is cut into slices, against float64 on the GPU."""
    rng = np.random.default_rng(m + n)
    dy, wide = _strided(rng.standard_normal((m, n)), pad, "bf16")
    if pad:
        wide[:, n:] = float("nan")
    c = M.ma_act_pack(_dev(_activation(rng, m, k), "bf16"))
    x = M.ma_act_unpack(c).double()
    d = dy.double()
    want = (d.t().contiguous() @ x).cpu().numpy()
    mag = (d.abs().t().contiguous() @ x.abs()).cpu().numpy()
    tol = (4 * m + 4) * 2 * R.F32 * mag          # as in the reference module
    got = M.ma_linear_grad(dy, c, grad_dtype=DT[tg])
    _close(got, want, R.rounded(want, tol, tg))
    out = got.clone()
    M.ma_linear_grad(dy, c, out=out, accumulate=True)
    twice = want + _f64(got)
    _close(out, twice, R.rounded(twice, tol + 4 * R.F32 * np.abs(twice), tg))
    # a sharper look than the bound for any signs: the M / 16 additions of a sum of
    # random products err by at most a step, 2^-23, of a partial sum that is no larger in
    # root mean square than the result, and independently, so by less than 2^-23
    # sqrt(M / 16) = 2.7e-6 of it for M = 8192; rounding to bf16 by at most 2^-8
    rel = np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)
    assert rel < (2.7e-6 if tg == "fp32" else 2 ** -8 + 2.7e-6), rel


def _taken_in_parts(m, n, k):
    """Whether a float32 dY is cut into its three parts before the product: the
    workspace then holds them."""
    return M.ma_linear_grad_workspace_size(m, n, k, torch.float32) >= 6 * m * n


@pytest.mark.parametrize("tg", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k,pad", [
    # one slice, two, three (each a part), four, and six of three parts; odd rows and columns
    (2050, 700, 300, 0), (2050, 512, 520, 4), (700, 2001, 2051, 0), (1025, 700, 4100, 3),
    (2050, 2001, 1030, 7), (4096, 1024, 2048, 8)])
def test_linear_grad_large_float32(tg, m, n, k, pad):
    """Large products of a float32 dY, against float64 on the GPU."""
    assert _taken_in_parts(m, n, k)
    rng = np.random.default_rng(m + n)
    dy, wide = _strided(rng.standard_normal((m, n)), pad, "fp32")
    if pad:
        wide[:, n:] = float("nan")
    c = M.ma_act_pack(_dev(_activation(rng, m, k), "bf16"))
    x = M.ma_act_unpack(c).double()
    d = dy.double()
    want = (d.t().contiguous() @ x).cpu().numpy()
    mag = (d.abs().t().contiguous() @ x.abs()).cpu().numpy()
    tol = (4 * m + 4) * 2 * R.F32 * mag          # as in the reference module
    need = M.ma_linear_grad_workspace_size(m, n, k, torch.float32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = M.ma_linear_grad(dy, c, grad_dtype=DT[tg], workspace=ws)
    _close(got, want, R.rounded(want, tol, tg))
    # the 3 M / 16 additions of a sum of random products err by at most a step, 2^-23, of
    # a partial sum, independently: by less than 2^-23 sqrt(3 M / 16) = 3.4e-6 for M = 4096
    # in root mean square; rounding to bf16 by at most 2^-8
    rel = np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)
    assert rel < (3.4e-6 if tg == "fp32" else 2 ** -8 + 3.4e-6), rel
    out = got.clone()
    M.ma_linear_grad(dy, c, out=out, accumulate=True, workspace=ws)
    twice = want + _f64(got)
    _close(out, twice, R.rounded(twice, tol + 4 * R.F32 * np.abs(twice), tg))
    assert torch.equal(got, M.ma_linear_grad(dy, c, out=torch.full_like(got, float("nan"))))


@pytest.mark.parametrize("m,n,k", [(2050, 700, 300), (700, 2001, 2051)])
def test_linear_grad_large_float32_values(m, n, k):
    """Value by value: x is all ones and one token of each output's dy is not zero, so
    the output's row is that float32 value, whole: the parts add up to it."""
    assert _taken_in_parts(m, n, k)
    rng = np.random.default_rng(8)
    c = M.ma_act_pack(torch.ones(m, k, device="cuda"))
    v = (torch.randn(n, device="cuda") * torch.exp2(torch.randint(-40, 40, (n,), device="cuda").float()))
    v[3] = torch.finfo(torch.float32).max
    v[4] = -torch.finfo(torch.float32).max
    at = torch.from_numpy(rng.integers(0, m, n)).cuda()
    at[:6] = m - 1
    dy = torch.zeros((m, n), device="cuda")
    dy[at, torch.arange(n, device="cuda")] = v
    assert torch.equal(M.ma_linear_grad(dy, c), v[:, None].expand(n, k))
    dy.view(torch.int32)[m - 1, 5] = 0x7f800001
    dy[m // 2, 333] = float("inf")
    xs = torch.ones(m, k, device="cuda")
    xs[m - 1, 40] = float("nan")
    got = M.ma_linear_grad(dy, c)
    assert torch.isnan(got[5]).all() and torch.isinf(got[333]).all()
    got = M.ma_linear_grad(dy, M.ma_act_pack(xs))
    assert torch.isnan(got[:, 32:64]).all()
    rest = torch.ones(n, k, dtype=torch.bool, device="cuda")
    rest[5] = rest[333] = False
    rest[:, 32:64] = False
    assert torch.isfinite(got[rest]).all()


@pytest.mark.parametrize("pad,copies", [(0, False), (1, True)])
def test_linear_grad_allocates_what_its_dy_needs(pad, copies):
    """Without a workspace of the caller's, a call allocates the gradient, x as bf16 and partial
    sums, and a copy of dy only where its rows are not aligned."""
    m, n, k = 16384, 4096, 1024
    dy, _ = _strided(np.zeros((m, n)), pad, "bf16")
    c = M.ma_act_pack(torch.ones((m, k), dtype=torch.bfloat16, device="cuda"))
    M.ma_linear_grad(dy, c)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    base = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    M.ma_linear_grad(dy, c)
    used = torch.cuda.max_memory_allocated() - base
    # (the few slices' partial sums, of the gradient's size each, are less than a copy of dy)
    assert (used >= 2 * m * k + 4 * n * k + 2 * m * n) == copies, used


@pytest.mark.parametrize("m,n,k", [(64, 96, 64), (2050, 700, 300)])
def test_linear_grad_float32_small_values(m, n, k):
    """Float32 values down to the smallest denormal, on the small tiles and in parts: x is all
    ones and one token of each output's dy is not zero.  A value of at least 2^-110 has no bit
    under 2^-133, the smallest bf16, and comes out whole; a smaller one has those bits
    cut off, so it is off by less than 2^-133."""
    assert _taken_in_parts(m, n, k) == (m > 64)
    rng = np.random.default_rng(9)
    v = np.ldexp(1.0 + rng.random(n), rng.integers(-140, -100, n)) * rng.choice([-1.0, 1.0], n)
    v[:8] = np.ldexp([1.0, 2 - 2.0 ** -23, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -23, 1.0, 1.0, 1.0],
                     [-110, -110, -110, -111, -126, -126, -133, -149])
    v = v.astype(np.float32)
    dy = np.zeros((m, n), np.float32)
    dy[rng.integers(0, m, n), np.arange(n)] = v
    got = _f64(M.ma_linear_grad(torch.from_numpy(dy).cuda(), M.ma_act_pack(torch.ones(m, k, device="cuda"))))
    want = np.repeat(v.astype(np.float64)[:, None], k, 1)
    whole = np.abs(v) >= 2.0 ** -110
    assert np.array_equal(got[whole], want[whole])
    assert np.all(np.abs(got - want) < 2.0 ** -133)
    assert whole.sum() > 10 and (~whole).sum() > 10


@pytest.mark.parametrize("m", [1024, 1055])
def test_linear_grad_large_product_values(m):
    """The large-product kernel, value by value: one token of dy is one, so the
    gradient's rows are that token's x; and NaN stays in its row or columns, although
    the last stage of tokens is partly empty."""
    n, k = 1024, 320
    rng = np.random.default_rng(6)
    xs = _activation(rng, m, k)
    c, x = _ckpt(xs)
    dy = torch.zeros((m, n), device="cuda", dtype=torch.bfloat16)
    at = torch.from_numpy(rng.integers(0, m, n)).cuda()
    at[-1] = m - 1
    dy[at, torch.arange(n, device="cuda")] = 1.0
    assert np.array_equal(_f64(M.ma_linear_grad(dy, c)), x[at.cpu().numpy()])
    dy[m - 1, 5] = float("nan")
    dy[m // 2, 700] = float("inf")
    xs[m - 1, 40] = np.nan
    c2, _ = _ckpt(xs)
    got = _f64(M.ma_linear_grad(dy, c))
    assert np.isnan(got[5]).all() and not np.isfinite(got[700]).any()
    assert np.isfinite(np.delete(got, [5, 700], axis=0)).all()
    got = _f64(M.ma_linear_grad(dy, c2))
    assert np.isnan(got[:, 32:64]).all()
    assert np.isfinite(np.delete(np.delete(got, [5, 700], axis=0), np.s_[32:64], axis=1)).all()


@pytest.mark.parametrize("td", ["bf16", "fp32"])
def test_linear_grad_nonfinite(td):
    """NaN and infinity in dy reach their output row, a NaN group of x its 32
    columns, and nothing else; extreme finite values stay finite."""
    m, n, k = 70, 48, 96
    rng = np.random.default_rng(2)
    xs = np.abs(rng.standard_normal((m, k))) + 0.5
    xs[:, 5] = 0.0                                       # infinity times zero
    c, x = _ckpt(xs)
    dy = rng.standard_normal((m, n))
    dy[69, 3] = np.nan
    dy[10, 20] = np.inf
    got = _f64(M.ma_linear_grad(_dev(dy, td), c))
    assert np.isnan(got[3]).all()
    assert np.isinf(np.delete(got[20], 5)).all() and np.isnan(got[20, 5])
    rest = np.delete(got, [3, 20], axis=0)
    assert np.isfinite(rest).all()
    bad = xs.copy()
    bad[33, 40] = np.nan
    c2, _ = _ckpt(bad)
    got = _f64(M.ma_linear_grad(_dev(np.abs(rng.standard_normal((m, n))) + 1, td), c2))
    assert np.isnan(got[:, 32:64]).all()
    assert np.isfinite(np.delete(got, np.s_[32:64], axis=1)).all()
    # the largest float and NaN patterns whose payload is in the low bits only
    big = torch.zeros(32, 8, device="cuda")
    big[0, 0] = torch.finfo(torch.float32).max
    big[1, 1] = -torch.finfo(torch.float32).max
    big.view(torch.int32)[2, 2] = 0x7f800001
    one = M.ma_act_pack(torch.ones(32, 32, device="cuda"))
    if td == "fp32":
        g = M.ma_linear_grad(big, one)
        assert torch.all(g[0] == torch.finfo(torch.float32).max)
        assert torch.all(g[1] == -torch.finfo(torch.float32).max)
        assert torch.isnan(g[2]).all() and torch.all(g[3:] == 0)


@pytest.mark.parametrize("td", ["bf16", "fp32"])
def test_linear_grad_broadcast_and_batch(td):
    """dy of one repeated row (stride 0), leading dimensions, and a padded
    batch: zero rows of dy change nothing."""
    rng = np.random.default_rng(4)
    c, x = _ckpt(_activation(rng, 150, 64))
    row = _dev(rng.standard_normal((1, 72)), td)
    a = M.ma_linear_grad(row.expand(150, 72), c)
    assert torch.equal(a, M.ma_linear_grad(row.expand(150, 72).contiguous(), c))
    dy = _dev(rng.standard_normal((5, 30, 72)), td)
    c3 = M.ActCheckpoint(c.codes, c.exps, 64, (5, 30, 64))
    assert torch.equal(M.ma_linear_grad(dy, c3), M.ma_linear_grad(dy.view(150, 72), c))


def test_linear_grad_order_of_a_dy_elsewhere():
    """A dy whose rows are not 16-byte aligned may be cut into other slices: its gradient is as
    near to the exact one, not bitwise that of the same values in aligned rows; each is bitwise
    equal on every run."""
    import ctypes as C
    from muon_newton_schulz_02_amd import _abi
    m, n, k = 16001, 256, 1024
    rng = np.random.default_rng(10)
    c = M.ma_act_pack(_dev(_activation(rng, m, k), "bf16"))
    x = M.ma_act_unpack(c).double()
    flat = torch.empty(m * n + 8, dtype=torch.bfloat16, device="cuda")
    values = _dev(rng.standard_normal((m, n)), "bf16")
    sizes = set()
    for off, pad in ((0, 0), (1, 0), (0, 3)):
        dy = flat[off:off + m * n].view(m, n) if not pad else _strided(np.zeros((m, n)), pad, "bf16")[0]
        dy.copy_(values)
        size = C.c_size_t()
        assert _abi.load().ma_linear_grad_workspace_size_at(dy.data_ptr(), 1, m, n, n + pad, k,
                                                            C.byref(size)) == 0
        sizes.add(size.value)
        got = M.ma_linear_grad(dy, c)
        want = (values.double().t().contiguous() @ x).cpu().numpy()
        mag = (values.double().abs().t().contiguous() @ x.abs()).cpu().numpy()
        tol = (4 * m + 4) * 2 * R.F32 * mag          # as in the reference module
        _close(got, want, R.rounded(want, tol, "fp32"))
        for _ in range(2):
            assert torch.equal(got, M.ma_linear_grad(dy, c))
    assert len(sizes) == 2          # (two plans)


# ---------------------------------------------------------- gated activation --

@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 256, 0), (3, 33, 0), (50, 100, 4),
                                           (9, 128, 8), (2, 1001, 0)])
def test_glu(kind, act, rows, cols, pad):
    rng = np.random.default_rng(rows + cols)
    g, _ = _strided(_activation(rng, rows, cols), pad, kind)
    u, _ = _strided(_activation(rng, rows, cols), pad, kind)
    dh, _ = _strided(rng.standard_normal((rows, cols)), pad, kind)
    h, cg, cu = M.ma_glu_forward(g, u, act)
    g64, u64, d64 = _f64(g), _f64(u), _f64(dh)
    a, _, a_tol, _ = R.act(act, g64)
    want = a * u64
    _close(h, want, R.rounded(want, a_tol * np.abs(u64) + 2 * R.F32 * np.abs(want), kind), "h")
    for c, x in ((cg, g64), (cu, u64)):
        codes, exps = R.pack(x)
        assert np.array_equal(c.codes.cpu().numpy(), codes)
        ng = codes.shape[1] // 32
        assert np.array_equal(c.exps.cpu().numpy()[:, :ng], exps[:, :ng])
    into, wide = _strided(np.zeros((rows, cols)), 3, kind)
    dg, du, ch = M.ma_glu_backward(dh, cg, cu, act, dup=into, h_ckpt=True)
    assert torch.all(wide[:, cols:] == 7.0)
    gh, uh = R.held(g64), R.held(u64)
    a, s, a_tol, s_tol = R.act(act, gh)
    want = d64 * a
    _close(du, want, R.rounded(want, a_tol * np.abs(d64) + 2 * R.F32 * np.abs(want), kind), "dup")
    want = d64 * uh * s
    _close(dg, want, R.rounded(want, np.abs(d64 * uh) * s_tol + 4 * R.F32 * np.abs(want), kind),
           "dgate")
    # h as held: within half a step of h at the held values
    hv = a * uh
    e = ch.exps.cpu().numpy()[:, :ch.codes.shape[1] // 32].astype(np.float64)
    step = np.repeat(2.0 ** (e - 127), 32, axis=1)[:, :cols]
    _close(M.ma_act_unpack(ch), hv, 0.5 * step + a_tol * np.abs(uh) + 2 * R.F32 * np.abs(hv) + R.TINY,
           "held h")
    two = M.ma_glu_backward(dh, cg, cu, act)
    assert len(two) == 2 and torch.equal(two[0], dg) and torch.equal(two[1], du)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_glu_extremes(act):
    """Saturated, zero, huge and non-finite gates: slopes 0 and 1 at the far
    ends, NaN groups to NaN gradients, and no NaN elsewhere."""
    v = np.array([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 90.0, -90.0, 1e4, -1e4, 1e19, -1e19, 1e38,
                  -1e38])
    g = np.zeros((len(v), 64))
    g[:, :32] = v[:, None]
    g[:, 32:] = 1.0
    g[3, 40] = np.nan
    h, cg, cu = M.ma_glu_forward(_dev(g), torch.ones(len(v), 64, device="cuda"), act)
    dg, du = M.ma_glu_backward(torch.ones(len(v), 64, device="cuda"), cg, cu, act)
    h, dg, du = _f64(h), _f64(dg), _f64(du)
    assert np.isnan(h[3, 40]) and np.isfinite(np.delete(h.ravel(), 3 * 64 + 40)).all()
    assert np.isnan(dg[3, 32:]).all() and np.isnan(du[3, 32:]).all()
    dg[3, 32:] = du[3, 32:] = 0
    assert np.isfinite(dg).all() and np.isfinite(du).all()
    for r in (8, 10, 12):
        assert np.all(dg[r, :32] == 1.0) and np.all(dg[r + 1, :32] == 0.0)
        assert np.all(h[r, :32] == np.float32(v[r])) and np.all(h[r + 1, :32] == 0.0)


def test_glu_halves_of_one_array():
    """gate and up, and their gradients, as the two halves of one fused array."""
    x = torch.randn(40, 2 * 96, device="cuda").to(torch.bfloat16)
    dh = torch.randn(40, 96, device="cuda").to(torch.bfloat16)
    h, cg, cu = M.ma_glu_forward(x[:, :96], x[:, 96:])
    h2, cg2, cu2 = M.ma_glu_forward(x[:, :96].contiguous(), x[:, 96:].contiguous())
    assert torch.equal(h, h2) and torch.equal(cg.codes, cg2.codes) and torch.equal(cu.codes, cu2.codes)
    d = torch.empty_like(x)
    M.ma_glu_backward(dh, cg, cu, dgate=d[:, :96], dup=d[:, 96:])
    dg, du = M.ma_glu_backward(dh, cg, cu)
    assert torch.equal(d, torch.cat([dg, du], 1))
    for bad in (dict(dgate=d[:, :96], dup=d[:, 95:191]), dict(dgate=d[:, :96], dup=d[:, :96]),
                dict(dgate=dh)):
        with pytest.raises(M.MuonAdamWError) as e:
            M.ma_glu_backward(dh, cg, cu, **bad)
        assert e.value.code == M.MA_ERR_INVALID_ARG


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_glu_gradient_against_differences(act):
    """dgate and dup against central differences of h at the held values.  The
    float64 difference over step e errs by e^2/6 |act'''| |u dh| < e^2 |u dh| (all third
    derivatives of both acts stay below 2) plus its own rounding."""
    rng = np.random.default_rng(8)
    g, u, dh = (rng.standard_normal((6, 64)) for _ in range(3))
    _, cg, cu = M.ma_glu_forward(_dev(g), _dev(u), act)
    dg, du = M.ma_glu_backward(_dev(dh), cg, cu, act)
    gh, uh, d = R.held(_dev(g).cpu().numpy().astype(np.float64)), \
        R.held(_dev(u).cpu().numpy().astype(np.float64)), _dev(dh).cpu().numpy().astype(np.float64)
    e = 1e-4
    num = (R.act(act, gh + e)[0] - R.act(act, gh - e)[0]) / (2 * e) * uh * d
    _close(dg, num, e * e * np.abs(uh * d) + 1e-11 + 2 ** -18 * np.abs(uh * d))
    num = (R.act(act, gh)[0] * (uh + e) - R.act(act, gh)[0] * (uh - e)) / (2 * e) * d
    _close(du, num, 1e-11 + 2 ** -18 * np.abs(d * gh))


# ----------------------------------------------------------- used together --

def _layer_inputs(seed, tokens=96, hidden=64, mlp=128, vocab=300, kind="fp32"):
    rng = np.random.default_rng(seed)
    return dict(
        ids=torch.from_numpy(rng.integers(0, vocab, tokens)).cuda(),
        table=_dev(0.1 * rng.standard_normal((vocab, hidden)), kind),
        wg=_dev(rng.standard_normal((mlp, hidden)) / 8, kind),
        wu=_dev(rng.standard_normal((mlp, hidden)) / 8, kind),
        wd=_dev(rng.standard_normal((hidden, mlp)) / 11, kind),
        dout=_dev(rng.standard_normal((tokens, hidden)), kind))


def _layer(p):
    """Embedding, then a gated MLP: forward and backward with the operators;
    plain matrix products for the layers themselves.  Gradient sources."""
    x = M.ma_embedding_lookup(p["table"], p["ids"], scale=8.0)
    cx = M.ma_act_pack(x)
    _, cg, cu = M.ma_glu_forward(x @ p["wg"].t(), x @ p["wu"].t())
    dh = p["dout"] @ p["wd"]
    dg, du, ch = M.ma_glu_backward(dh, cg, cu, h_ckpt=True)
    dx = dg @ p["wg"] + du @ p["wu"]
    return [M.EmbeddingGrad(dx, p["ids"], 8.0), M.LinearGrad(dg, cx), M.LinearGrad(du, cx),
            M.LinearGrad(p["dout"], ch)]


NAMES = ["action_expert.embed_tokens.weight", "action_expert.layers.0.mlp.gate_proj.weight",
         "action_expert.layers.0.mlp.up_proj.weight", "action_expert.layers.0.mlp.down_proj.weight"]


def _optimizer(p):
    params = [p[k].clone() for k in ("table", "wg", "wu", "wd")]
    return M.MuonAdamW(list(zip(NAMES, params, [True] * 4)), lr=1e-3), params


def _plain_gradients(p):
    """The same layer in torch autograd, float64 on the CPU."""
    q = {k: v.double().cpu() for k, v in p.items() if k != "ids"}
    for k in ("table", "wg", "wu", "wd"):
        q[k].requires_grad_()
    x = q["table"][p["ids"].cpu()] * 8.0
    h = torch.nn.functional.silu(x @ q["wg"].t()) * (x @ q["wu"].t())
    (h @ q["wd"].t()).backward(q["dout"])
    return [q[k].grad.numpy() for k in ("table", "wg", "wu", "wd")]


def test_layer_gradients_near_plain_ones():
    """Gradients through 8-bit activations against exact ones.  Every use of a
    held value errs by at most half a step, 1/128 of its group's largest value; with
    groups of 32 normal values that is under 1.2 % of their root mean square each
    (uniform over half a step of at most amax/64, amax < 4 sigma: 4/128/sqrt(3) =
    1.8 %).  Held x enters the linear gradients once, held gate and up and the held h
    each once more, so relative errors of the whole gradients stay below 4 x 1.8 %
    in norm even if all were aligned."""
    p = _layer_inputs(11)
    src = _layer(p)
    got = [M.ma_embedding_grad(src[0].dout, src[0].tokens, 300, scale=8.0)] + \
        [M.ma_linear_grad(s.dy, s.x) for s in src[1:]]
    for g, w, name in zip(got, _plain_gradients(p), NAMES):
        rel = np.linalg.norm(_f64(g) - w) / np.linalg.norm(w)
        assert rel < 0.072, (name, rel)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_optimizer_step_takes_gradient_sources(kind):
    """A step given gradient sources equals, bit for bit, a step given the
    gradients that the operators form from them."""
    p = _layer_inputs(12, kind=kind)
    src = _layer(p)
    opt, params = _optimizer(p)
    opt.step(src)
    ref, want = _optimizer(p)
    grads = [M.ma_embedding_grad(src[0].dout, src[0].tokens, 300, scale=8.0, grad_dtype=DT[kind])] + \
        [M.ma_linear_grad(s.dy, s.x, grad_dtype=DT[kind]) for s in src[1:]]
    ref.step(grads)
    for a, b in zip(params, want):
        assert torch.equal(a, b)
    for a, b in zip(opt.grad_buffers, grads):
        assert torch.equal(a, b)
    # a tensor beside sources
    opt.step([grads[0]] + src[1:])
    ref.step(grads)
    for a, b in zip(params, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_optimizer_step_adds_micro_batches(kind):
    """A list of sources is the sum over micro-batches, rounded once."""
    p, q = _layer_inputs(13, kind=kind), _layer_inputs(14, tokens=51, kind=kind)
    for k in ("table", "wg", "wu", "wd"):
        q[k] = p[k]
    a, b = _layer(p), _layer(q)
    opt, _ = _optimizer(p)
    opt.step([[x, y] for x, y in zip(a, b)])
    for i in range(4):
        def form(s, out=None):
            if i == 0:
                return M.ma_embedding_grad(s.dout, s.tokens, 300, scale=8.0, out=out,
                                           accumulate=out is not None)
            return M.ma_linear_grad(s.dy, s.x, out=out, accumulate=out is not None)
        want = form(b[i], form(a[i])).to(DT[kind])
        assert torch.equal(opt.grad_buffers[i], want), NAMES[i]


def test_step_sources_on_another_stream():
    p = _layer_inputs(15)
    src = _layer(p)
    opt, params = _optimizer(p)
    ref, want = _optimizer(p)
    ref.step(src)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    opt.step(src, stream=side)
    del src
    side.synchronize()
    for a, b in zip(params, want):
        assert torch.equal(a, b)


def test_step_buffers_belong_to_the_step_stream():
    """A step on another stream, right after work of the current stream whose memory has been
    given back: the gradient buffers are not that memory.  Then a step on the current stream."""
    p = _layer_inputs(16)
    ref, want = _optimizer(p)
    src = _layer(p)
    for _ in range(2):
        ref.step(src)
    opt, params = _optimizer(p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # freed blocks of the buffers' sizes in the current stream's pool
    freed = [torch.empty_like(q) for q in params for _ in range(4)]
    held = {t.data_ptr() for t in freed}
    del freed
    opt.step(src, stream=side)
    assert not held & {t.data_ptr() for t in opt.grad_buffers}
    side.synchronize()
    opt.step(src)
    torch.cuda.synchronize()
    for a, b in zip(params, want):
        assert torch.equal(a, b)
    # a third stream, current and given; and a buffer of the caller's
    third = torch.cuda.Stream()
    opt.grad_buffers[1] = torch.empty_like(params[1])
    with torch.cuda.stream(third):
        opt.step(src, stream=third)
    third.synchronize()
    ref.step(src)
    torch.cuda.synchronize()
    for a, b in zip(params, want):
        assert torch.equal(a, b)


# --------------------------------------------------------- graphs, streams --

def test_capture_and_replay():
    """The layer's backward pass captured once and replayed on changed inputs,
    with eager work in between, equals the eager results each time."""
    p = _layer_inputs(20, tokens=1500, vocab=3000)

    def work():
        src = _layer(p)
        return [M.ma_embedding_grad(src[0].dout, src[0].tokens, 3000, scale=8.0)] + \
            [M.ma_linear_grad(s.dy, s.x) for s in src[1:]]

    work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = work()
    for seed in (21, 22, 23, 24):
        for k, v in _layer_inputs(seed, tokens=1500, vocab=3000).items():
            p[k].copy_(v)
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, work()):
            assert torch.equal(a, b), seed
        torch.cuda.synchronize()


def test_capture_step_with_sources():
    """The whole training step captured: gradients formed from sources, then the
    optimizer step with its counter on the device.  Replays equal eager steps."""
    outs = []
    for captured in (False, True):
        p = _layer_inputs(40)
        opt, params = _optimizer(p)
        opt.state.device_step = torch.zeros(1, dtype=torch.int64, device="cuda")
        opt.step(_layer(p))                       # (allocates the gradient buffers)
        torch.cuda.synchronize()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                opt.step(_layer(p))
        for seed in (41, 42, 43):
            q = _layer_inputs(seed)
            for k in ("ids", "dout"):
                p[k].copy_(q[k])
            if captured:
                g.replay()
            else:
                opt.step(_layer(p))
            torch.cuda.synchronize()
            M.ma_act_pack(p["dout"])              # eager work in between
        assert int(opt.state.device_step.item()) == 4
        outs.append(params)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_two_captured_graphs():
    """Two graphs of the same operators on different data, replayed in turn and
    then at once on two streams."""
    ps = [_layer_inputs(50 + k, tokens=3000, vocab=2000) for k in range(2)]

    def work(p):
        s = _layer(p)
        return [M.ma_embedding_grad(s[0].dout, s[0].tokens, 2000, scale=8.0)] + \
            [M.ma_linear_grad(x.dy, x.x) for x in s[1:]]

    want = [work(p) for p in ps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(p))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    for r in range(4):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
            if r < 2:
                st.synchronize()
        for st in streams:
            st.synchronize()
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a, b), r


def test_stream_zero_is_the_default_stream():
    """A raw handle of 0 names the default stream, whatever stream is current."""
    from muon_newton_schulz_02_amd import grads as G
    dev = torch.device("cuda", torch.cuda.current_device())
    x = torch.randn(50, 96, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with G._At(dev, 0, (x,)):
            assert torch.cuda.current_stream().cuda_stream == 0
        c = M.ma_act_pack(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(c.codes, M.ma_act_pack(x).codes)


def test_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    other = SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1), cuda_stream=0)
    x = torch.randn(5, 96, device="cuda")
    with pytest.raises(ValueError, match="stream is on"):
        M.ma_act_pack(x, stream=other)


def test_workspace_is_checked_before_the_stream_is_taken():
    dy = torch.randn(40, 24, device="cuda")
    c = M.ma_act_pack(torch.randn(40, 32, device="cuda"))
    ids = torch.zeros(40, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    for ws, error in ((torch.empty(1 << 20, dtype=torch.uint8), ValueError), ([0], TypeError),
                      (torch.empty(4, 4, device="cuda").t(), ValueError)):
        for stream in (None, side):
            with pytest.raises(error, match="workspace"):
                M.ma_linear_grad(dy, c, workspace=ws, stream=stream)
            with pytest.raises(error, match="workspace"):
                M.ma_embedding_grad(dy, ids, 9, workspace=ws, stream=stream)


def test_copies_of_a_checkpoint_hold_arrays_of_their_own():
    import copy
    import io
    x = torch.randn(6, 7, 100, device="cuda", dtype=torch.bfloat16)
    c = M.ma_act_pack(x)
    want = M.ma_act_unpack(c)
    f = io.BytesIO()
    torch.save((c.codes.clone(), c.exps.clone(), c.cols, c.shape), f)
    f.seek(0)
    loaded = M.ActCheckpoint(*torch.load(f, weights_only=True))
    g = io.BytesIO()
    torch.save(c, g)
    g.seek(0)
    whole = torch.load(g, weights_only=False)
    deep = copy.deepcopy(c)
    copies = (deep, loaded, whole, copy.copy(c))
    for d in copies:
        assert d._pc == d.codes.data_ptr() != c._pc and d._pe == d.exps.data_ptr() != c._pe
        assert d.shape == c.shape and d.cols == c.cols and d.rows == c.rows
    c.codes.zero_()
    del c
    for d in copies:
        assert torch.equal(M.ma_act_unpack(d), want)


def test_checkpoint_whose_arrays_move():
    """Arrays given other memory since are read there; on the CPU, or freed, they are refused."""
    x = torch.randn(6, 100, device="cuda")
    c = M.ma_act_pack(x)
    own = M.ActCheckpoint(c.codes.clone(), c.exps.clone(), 100)
    twice = (2 * M.ma_act_unpack(c)).clone()
    for d in (c, own):
        d.exps.data = d.exps + (d.exps > 0).to(torch.uint8)      # (groups of the padding are 0)
        d.codes.data = d.codes.clone()
        assert torch.equal(M.ma_act_unpack(d), twice)
        g = M.ma_linear_grad(torch.eye(6, device="cuda"), d)
        assert torch.equal(g, twice)
        d.codes.data = d.codes.cpu()
        with pytest.raises(ValueError, match="codes are on cpu"):
            M.ma_act_unpack(d)
        d.exps.data = d.exps.cpu()
        with pytest.raises(ValueError, match="GPU"):
            M.ma_linear_grad(torch.eye(6, device="cuda"), d)
    one = M.ma_act_pack(x)
    for freed in (one, M.ActCheckpoint(torch.zeros_like(one.codes), torch.zeros(9, 4, dtype=torch.uint8,
                                                                                device="cuda")[3:], 100)):
        freed.exps.untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="freed"):
            M.ma_act_unpack(freed)


def test_two_streams_at_once():
    """Two calls of each operator in flight at once, on two streams."""
    ps = [_layer_inputs(30 + k, tokens=4000, vocab=2000) for k in range(2)]
    want = []
    for p in ps:
        s = _layer(p)
        want.append([M.ma_embedding_grad(s[0].dout, s[0].tokens, 2000, scale=8.0)] +
                    [M.ma_linear_grad(x.dy, x.x) for x in s[1:]])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [None, None]
    for _ in range(3):
        for k, (p, st) in enumerate(zip(ps, streams)):
            with torch.cuda.stream(st):
                s = _layer(p)
                got[k] = [M.ma_embedding_grad(s[0].dout, s[0].tokens, 2000, scale=8.0)] + \
                    [M.ma_linear_grad(x.dy, x.x) for x in s[1:]]
        for st in streams:
            st.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


# ---------------------------------------------------------- random calls --

@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Every operator at random sizes, types and strides (each a view of a wider
    array filled with NaN)."""
    rng = np.random.default_rng(1000 + seed)

    def size(most):
        return int(np.exp(rng.random() * np.log(most)))

    def kind():
        return ("fp32", "bf16")[rng.integers(2)]

    def view(x, k):
        pad = int(rng.integers(0, 20))
        v, wide = _strided(x, pad, k)
        wide[:, x.shape[1]:] = float("nan")
        return v

    n, v, h = size(3000), size(5000), size(700)
    ids, td, tg = _tokens(rng, ("uniform", "zipf", "mixed", "one")[rng.integers(4)], n, v), kind(), kind()
    tok = torch.from_numpy(ids).cuda()
    table = view(rng.standard_normal((v, h)), td)
    got = M.ma_embedding_lookup(table, tok, scale=-1.5, out_dtype=DT[tg])
    ok = (ids >= 0) & (ids < v)
    want = np.where(ok[:, None], -1.5 * _f64(table)[np.where(ok, ids, 0)], 0.0)
    _close(got, want, R.rounded(want, 2 * R.F32 * np.abs(want), tg), "lookup")
    d = view(rng.standard_normal((n, h)), td)
    pad = int(rng.integers(-1, v))
    got = M.ma_embedding_grad(d, tok, v, scale=-1.5, padding_token=pad, grad_dtype=DT[tg])
    want, tol = R.embedding_grad(_f64(d), ids, v, -1.5, pad)
    _close(got, want, R.rounded(want, tol, tg), "embedding grad")

    rows, cols, act = size(400), size(900), ("silu", "gelu_tanh")[rng.integers(2)]
    g, u = view(_activation(rng, rows, cols), td), view(_activation(rng, rows, cols), td)
    out, cg, cu = M.ma_glu_forward(g, u, act)
    a, _, a_tol, _ = R.act(act, _f64(g))
    want = a * _f64(u)
    _close(out, want, R.rounded(want, a_tol * np.abs(_f64(u)) + 2 * R.F32 * np.abs(want), td), "h")
    assert torch.equal(cg.codes, M.ma_act_pack(g).codes)
    dh = view(rng.standard_normal((rows, cols)), td)
    dg, du = M.ma_glu_backward(dh, cg, cu, act)
    gh, uh, dd = R.held(_f64(g)), R.held(_f64(u)), _f64(dh)
    a, s, a_tol, s_tol = R.act(act, gh)
    want = dd * a
    _close(du, want, R.rounded(want, a_tol * np.abs(dd) + 2 * R.F32 * np.abs(want), td), "dup")
    want = dd * uh * s
    _close(dg, want, R.rounded(want, np.abs(dd * uh) * s_tol + 4 * R.F32 * np.abs(want), td), "dgate")

    m, n, k = size(3000), size(1500), size(600)
    dy = view(rng.standard_normal((m, n)), td)
    c, x = _ckpt(_activation(rng, m, k))
    want, tol = R.linear_grad(_f64(dy), x)
    _close(M.ma_linear_grad(dy, c, grad_dtype=DT[tg]), want, R.rounded(want, tol, tg), "linear grad")


# ----------------------------------------------------- offsets past 32 bits --

def test_long_offsets_embedding():
    """A table and a gradient of more than 2^31 elements (4.6 GB and 9.2 GB)."""
    v, h = 1_130_000, 2048
    table = torch.zeros((v, h), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([v - 1, 0, v - 2, v - 1], device="cuda")
    table[v - 1], table[v - 2] = 3.0, 2.0
    out = M.ma_embedding_lookup(table, ids)
    assert out[:, 0].tolist() == [3.0, 0.0, 2.0, 3.0] and out[0].eq(3.0).all()
    del table
    d = torch.ones((4, h), dtype=torch.bfloat16, device="cuda")
    g = M.ma_embedding_grad(d, ids, v)
    assert g[v - 1].eq(2.0).all() and g[v - 2].eq(1.0).all() and g[0].eq(1.0).all()
    assert float(g.sum(dtype=torch.float64)) == 4.0 * h
    del g
    torch.cuda.empty_cache()


def test_long_offsets_rows():
    """Activations of more than 2^32 elements: pack, unpack, the gated
    activation's rows and the linear gradient's token axis at their far ends."""
    rows, cols = 530_000, 8192
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = 5.0
    x[-2, ::32] = 1.0
    c = M.ma_act_pack(x)
    assert torch.equal(M.ma_act_unpack(M.ActCheckpoint(c.codes[-2:], c.exps[-2:], cols), torch.bfloat16), x[-2:])
    small = M.ma_act_pack(torch.ones((rows, 32), dtype=torch.bfloat16, device="cuda"))
    g = M.ma_linear_grad(x, small)
    want = torch.full((cols,), 5.0, device="cuda")
    want[::32] += 1.0
    assert torch.equal(g, want[:, None].expand(cols, 32))
    wide = M.ma_act_pack(torch.ones((rows, 256), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(M.ma_linear_grad(x, wide), want[:, None].expand(cols, 256))
    del wide
    dy = torch.zeros((rows, 8), dtype=torch.bfloat16, device="cuda")
    dy[-1] = 1.0
    assert torch.equal(M.ma_linear_grad(dy, c), torch.full((8, cols), 5.0, device="cuda"))
    y = M.ma_act_unpack(c, torch.bfloat16)
    assert torch.equal(y[-2:], x[-2:]) and float(y[:-2].abs().max()) == 0.0
    del x, y, c
    torch.cuda.empty_cache()
