"""Resource budgets of the layer operators, read from the gfx950 assembly the compiler writes (no
GPU needed).

The norm, the rotary positions and the token log probabilities are bound by memory and live on
waves in flight: four on a SIMD need at most 128 of its 512 registers each. The attention kernels
hold their tiles in registers, one or two waves on a SIMD, and their workgroups' LDS is what
decides how many of them a compute unit runs."""

import re

import pytest

from tests.test_kernel_resources import _kernels


def _one(ks, *parts):
    return {n: r for n, r in ks.items() if all(p in n for p in parts)}


@pytest.mark.parametrize("src, kernels", [("norm.hip", 3), ("rotary.hip", 1), ("logprob.hip", 3)])
def test_streaming_kernels_fit_four_waves_a_simd(tmp_path, src, kernels):
    ks = _kernels(src, tmp_path)
    names = {re.search(r"k_[a-z0-9_]+?(?=I)", n).group(0) for n in ks if re.search(r"k_[a-z0-9_]+?(?=I)", n)}
    assert len(names) >= kernels, names
    for name, r in ks.items():
        assert r["vgpr"] + r["agpr"] <= 128, (name, r)
        assert r["spill"] == 0, (name, r)
        assert r["lds"] <= 160 * 1024 // 16, (name, r)


@pytest.mark.parametrize("src, kernel", [
    ("attention.hip", "k_attention_forward"),
    ("attention_dq.hip", "k_attention_dq"),
    ("attention_dkv.hip", "k_attention_dkv"),
])
def test_attention_tiles_stay_in_registers(tmp_path, src, kernel):
    ks = _kernels(src, tmp_path)
    tiles = _one(ks, kernel)
    assert len(tiles) == (9 if kernel == "k_attention_forward" else 12), sorted(ks)
    for name, r in ks.items():
        if name not in tiles:
            assert r["vgpr"] <= 80 and r["spill"] == 0, (name, r)      # (six waves a SIMD)
    for name, r in tiles.items():
        assert r["vgpr"] <= 512 and r["lds"] <= 160 * 1024, (name, r)
        # (key gradients of 256 features share a head with two waves: a few values outside the
        # products spill rather than halve the waves)
        wide = kernel == "k_attention_dkv" and "IDF16bLi256ELi4E" in name
        assert r["spill"] <= (16 if wide else 0), (name, r)
        # bfloat16 of at most 128 features: two workgroups of four waves on a compute unit
        if "IDF16bLi64E" in name or re.search(r"IDF16bLi128E(Li64E)?Li4E", name):
            assert r["vgpr"] <= 512 // 2, (name, r)
            assert r["lds"] <= 160 * 1024 // 2, (name, r)
