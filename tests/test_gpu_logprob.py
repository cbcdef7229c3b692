"""Log probabilities of tokens on the GPU in each of the kernels a call may take: rows far from zero, every
order of a row's values, and more high values than are listed at once."""

import numpy as np
import pytest

from tests import _layers_ref as R
from tests.test_gpu_grads import DT, _close, _dev, _f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")

# (times the 12 rows of a test, vocabulary): one workgroup of 256 threads a row where there are few; of 64,
# 128 and 256 where there are many; rows cut into pieces that are joined, of 256 threads and of 64
PLANS = [(1, 64), (1, 1000), (22, 64), (22, 519), (22, 1000), (43, 17003), (43, 33001), (1, 16400), (22, 20000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.load_library()
    yield
    torch.cuda.synchronize()


def _check(z, times, ids, scale, top, off=0):
    """z (rows, vocab) repeated `times` times, from element `off` of an allocation on, against the reference."""
    rows, vocab = z.shape
    flat = torch.zeros(times * rows * vocab + off, dtype=z.dtype, device="cuda")
    t = flat[off:].view(times * rows, vocab)
    t.view(times, rows, vocab).copy_(z)
    got = M.ma_token_logprob_forward(t, torch.from_numpy(np.tile(ids, times)).cuda(), scale=scale, top=top)
    want, tol = R.logprob(_f64(z), ids, float(np.float32(scale)), top)
    each = lambda x: np.tile(x, (times,) + (1,) * (x.ndim - 1))
    for name, k in (("logprob", 0), ("entropy", 1), ("lse", 2)):
        _close(got[k], each(want[k]), each(tol[k]), name)
    if top:
        assert np.array_equal(got[3].cpu().numpy(), each(want[3]))
        _close(got[4], each(want[4]), each(tol[4]), "top")
    return t, got


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("times,vocab", PLANS)
def test_rows_far_from_zero(kind, times, vocab):
    """A constant added to a row's logits changes neither its log probabilities nor its entropy: with logits of
    float32 and bfloat16 as they are, the bounds of rows around zero hold.  (lse has the constant's own
    rounding.)"""
    rng = np.random.default_rng(vocab + times)
    add = np.array([100, -100, 1000, -1000, 1e4, -1e4, 3.3, -25, 65504, -65504, 1e6, -1e6])
    z = _dev(rng.standard_normal((12, vocab)) * 3 + add[:, None], kind)
    ids = rng.integers(0, vocab, 12)
    for scale, top in ((1.0, 5), (0.7, 0)):
        _check(z, times, ids, scale, top)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("times,vocab", PLANS)
def test_rows_of_large_values(kind, times, vocab):
    """Rows of nothing but a finite mask value, such a mask beside a few entries, and logits of up to float32's
    largest, some of which differ by a few steps of float32 only."""
    rng = np.random.default_rng(vocab * 3 + times)
    few = lambda: rng.integers(0, 9, vocab)
    z = np.zeros((12, vocab))
    for r, mask in enumerate((-1e9, -1e10, -1e20, -1e30, -3.3e38, 1e10, 3e38)):
        z[r] = mask
    z[7] = -1e10
    z[7, rng.integers(0, vocab, 5)] = rng.standard_normal(5)
    z[8] = 1e10 + 1024.0 * few()             # (float32 is 1024 apart there)
    z[9] = -1e10 - 1024.0 * few()
    z[10] = 2.0 ** 24 * np.log(2) - 4 + few()    # (their exponents of 2 lie around 2^24)
    z[11] = -2.0 ** 24 * np.log(2) - 4 + few()
    t = _dev(z, kind)
    ids = rng.integers(0, vocab, 12)
    for scale, top in ((1.0, 5), (2.0 ** -10, 20), (0.7, 0)):
        _check(t, times, ids, scale, top)


# threads of the workgroups that rows of a vocabulary get, 264 of them or (for 128 threads) 516
ORDERS = [(64, 22, 300), (64, 22, 1000), (64, 22, 5001), (64, 22, 20011), (128, 43, 17001), (128, 43, 20011), (256, 1, 5001)]


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("threads,times,vocab", ORDERS)
def test_orders_in_each_kernel(kind, threads, times, vocab):
    """Rows in rising and falling order, of one value, of few values, with the highest side by side, in one thread's
    rounds, at both ends; masked but for a few; with zeros of both signs; from odd addresses on too."""
    rng = np.random.default_rng(vocab)
    z = np.zeros((12, vocab))
    z[0] = np.linspace(-5, 5, vocab)
    z[1] = z[0][::-1]
    z[2] = 0.25
    z[3] = rng.integers(0, 3, vocab)
    z[4] = rng.standard_normal(vocab)
    z[4, vocab // 3:vocab // 3 + 70] = 9 + rng.random(70)
    z[5] = rng.standard_normal(vocab)
    z[5, ::threads * 8] = 7.0
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
    for top in (1, 20, 64):
        _check(t, times, ids, 1.0, top)
    for off in (1, 3):
        _check(t, times, ids, 1.0, 20, off)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("threads,rows,vocab,pieces", [(64, 300, 4096, 1), (128, 600, 20000, 1), (256, 3, 8184, 1),
                                                       (256, 530, 40000, 1), (256, 2, 16384, 2), (64, 300, 20000, 2)])
def test_more_high_values_than_are_listed(kind, threads, rows, vocab, pieces):
    """63 threads of a workgroup hold nothing but high values, a 64th a single value below them: that one is the
    bound of the top 64, and more keys reach it than a workgroup lists (576) at once."""
    rng = np.random.default_rng(threads + vocab)
    piece = -(-vocab // pieces)
    assert piece % 8 == 0
    at = np.arange(vocab) % piece
    thread = at // 8 % threads
    base = rng.standard_normal((4, vocab)).clip(-4, 4)
    base = np.where(thread < 63, 20 + rng.random((4, vocab)), base)
    base[:, (thread == 63) & (at % 8 == 5) & (at < 8 * threads)] = 10.0
    for p in range(pieces):
        assert all((base[:, p * piece:(p + 1) * piece] >= 10.0).sum(1) > 576)
    z = _dev(base, kind).repeat(-(-rows // 4), 1)[:rows].contiguous()
    ids = torch.zeros(rows, dtype=torch.int64, device="cuda")
    got = M.ma_token_logprob_forward(z, ids, top=64)
    want = torch.sort(z[:4].float(), dim=1, descending=True, stable=True)[1][:, :64]
    assert torch.equal(got[3], want.repeat(-(-rows // 4), 1)[:rows])
    lse = torch.logsumexp(z[:4].double(), 1)
    lp = torch.gather(z[:4].double(), 1, want) - lse[:, None]
    # (values of at most 21 and lse of at most 32 in float32: a few of their half steps, and the sum's own)
    tol = (vocab / 8 + 40) * 2.0 ** -24 + 8 * 32 * 2.0 ** -24
    assert (got[4].double() - lp.repeat(-(-rows // 4), 1)[:rows]).abs().max() <= tol
