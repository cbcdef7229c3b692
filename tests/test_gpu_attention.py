"""Attention on the GPU at scores far beyond those of a trained model."""

import numpy as np
import pytest

from tests._grads_ref import F32, U
from tests.test_gpu_grads import DT, _f64

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


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [8, 128, 256])
@pytest.mark.parametrize("n,m,causal", [(1, 70, False), (40, 3000, False), (300, 300, True), (2500, 100, False)])
@pytest.mark.parametrize("sign", [1, -1])
def test_forward_of_large_scores(kind, dim, n, m, causal, sign):
    """Scores of +-2^40 + 2^17 j, j < 4, exact in float32 and in either type's products, so that softmax sees their
    differences alone: of 2^17 j and, with scale 2^-14, of 8 j."""
    rng = np.random.default_rng(n + m + dim)
    q, k = torch.zeros((n, 2, dim), device="cuda"), torch.zeros((m, 1, dim), device="cuda")
    j = rng.integers(0, 4, m)
    q[:, :, 0], q[:, :, dim // 2] = 2.0 ** 20, 2.0 ** 17
    k[:, 0, 0], k[:, 0, dim // 2] = sign * 2.0 ** 20, torch.from_numpy(j).cuda().float()
    v = torch.from_numpy(rng.standard_normal((m, 1, dim))).cuda()
    q, k, v = (x.to(DT[kind]) for x in (q, k, v))
    for scale in (1.0, 2.0 ** -14):
        o, lse = M.ma_attention_forward(q, k, v, causal=causal, scale=scale)
        z = scale * (sign * 2.0 ** 40 + 2.0 ** 17 * j)[None] + np.zeros((n, 1))
        if causal:
            z = np.where(np.arange(m)[None] <= np.arange(n)[:, None] + m - n, z, -np.inf)
        top = z.max(1, keepdims=True)
        e = np.exp(z - top)
        p = e / e.sum(1, keepdims=True)
        want = p @ _f64(v)[:, 0]
        # an argument of at most 24 ln units errs by 4 u of itself, a sum of m terms by m u and the product
        # with v by 2 m u; probabilities and results of a bfloat16 call are rounded once each
        tol = (p @ np.abs(_f64(v)[:, 0])) * ((4 * 24 + 3 * m + 16) * F32 + (2.1 * U[kind] if kind == "bf16" else F32))
        for h in range(2):
            assert (np.abs(_f64(o)[:, h] - want) <= tol + 1e-30).all()
            assert (np.abs(_f64(lse)[h] - top[:, 0] - np.log(e.sum(1))) <= 2 * F32 * np.abs(top[:, 0]) + 1).all()
