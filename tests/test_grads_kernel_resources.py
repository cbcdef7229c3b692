"""Resource budgets of the gradient operators' kernels, read from the gfx950
assembly the compiler writes (no GPU needed): nothing spills, and each kernel
leaves room for the workgroups per compute unit that its launch counts on (a
SIMD holds 512 registers per lane, a compute unit 160 KB of LDS)."""

import pytest

from tests.test_kernel_resources import _kernels

KB = 1024


def _fits(ks, part, per_cu, waves, least=1):
    """Every kernel named so runs per_cu workgroups of `waves` waves on a compute unit."""
    found = {n: r for n, r in ks.items() if part in n}
    assert len(found) >= least, sorted(ks)
    for name, r in found.items():
        regs = -(-(r["vgpr"] + r["agpr"]) // 8) * 8
        assert regs * (per_cu * waves // 4) <= 512, (name, r)
        assert r["lds"] * per_cu <= 160 * KB, (name, r)


@pytest.mark.parametrize("src", ["act8.hip", "embedding.hip", "linear_grad.hip"])
def test_gradient_kernels_do_not_spill(src, tmp_path):
    for name, r in _kernels(src, tmp_path).items():
        assert r["spill"] == 0, (name, r)


def test_linear_grad_budgets(tmp_path):
    ks = _kernels("linear_grad.hip", tmp_path)
    _fits(ks, "k_linear_grad_big", 1, 8, 2)
    _fits(ks, "k_linear_gradIDF16b", 3, 4, 4)         # bf16 dY: up to three share a CU
    _fits(ks, "k_linear_gradIf", 2, 4, 4)             # float32 dY: two


def test_embedding_grad_budgets(tmp_path):
    ks = _kernels("embedding.hip", tmp_path)
    _fits(ks, "k_sort_count", 2, 16)                  # the zeroing beside the sort
    _fits(ks, "k_sort_scatter", 2, 16)
    _fits(ks, "k_sort_lds", 1, 16, 3)
    _fits(ks, "k_emb_sum", 4, 4, 12)
