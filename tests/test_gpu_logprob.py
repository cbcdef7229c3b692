"""Log probabilities of tokens on the GPU in each of the kernels a call may take: rows far from zero."""

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
