"""Python integers that do not fit the C type they go into, and types without kernels, are refused by the
binding: ctypes would take the lowest bits of one, and a bare dictionary names neither argument nor type."""

import resource

import pytest

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")
from muon_newton_schulz_02_amd import layers  # noqa: E402

BIG32 = [2 ** 32 + 5, 2 ** 31, -2 ** 31 - 1, -2 ** 32 + 5]
BIG64 = [2 ** 64 + 5, 2 ** 63, -2 ** 63 - 1]


@pytest.mark.parametrize("n", BIG32)
def test_top(n):
    with pytest.raises(ValueError, match="top"):
        M.ma_token_logprob_workspace_size(3, 40000, n)


def test_top_of_a_call_is_checked_before_it_sizes_anything(monkeypatch):
    """The call itself, up to the first thing that needs a GPU."""
    z, ids = torch.zeros(3, 40000), torch.zeros(3, dtype=torch.int64)
    monkeypatch.setattr(layers, "_check_cuda", lambda x, what: None)
    monkeypatch.setattr(layers, "_elsewhere", lambda dev, stream: False)
    with pytest.raises(ValueError, match="top"):
        M.ma_token_logprob_forward(z, ids, top=2 ** 32 + 5)


@pytest.mark.parametrize("n", BIG64)
def test_sizes(n):
    for call, name in ((lambda: M.ma_token_logprob_workspace_size(n, 40000, 5), "n_tokens"),
                       (lambda: M.ma_token_logprob_workspace_size(3, n, 5), "vocab"),
                       (lambda: M.ma_rms_norm_backward_workspace_size(n, 40), "rows"),
                       (lambda: M.ma_rms_norm_backward_workspace_size(6, n), "cols"),
                       (lambda: M.ma_embedding_grad_workspace_size(n, 10, 10), "n_tokens"),
                       (lambda: M.ma_embedding_grad_workspace_size(10, n, 10), "vocab"),
                       (lambda: M.ma_embedding_grad_workspace_size(10, 10, n), "hidden"),
                       (lambda: M.ma_linear_grad_workspace_size(n, 10, 10), "n_tokens"),
                       (lambda: M.ma_linear_grad_workspace_size(10, n, 10), "n_out"),
                       (lambda: M.ma_linear_grad_workspace_size(10, 10, n), "n_in")):
        with pytest.raises(ValueError, match=name):
            call()


ATTN = dict(n_queries=100, n_keys=100, heads=4, kv_heads=2, head_dim=64, n_seqs=3)


@pytest.mark.parametrize("size", [M.ma_attention_forward_workspace_size, M.ma_attention_backward_workspace_size])
def test_attention_sizes(size):
    size(**ATTN)
    for name in ATTN:
        for n in BIG64 + (BIG32 if not name.startswith("n_q") and not name.startswith("n_k") else []):
            with pytest.raises(ValueError, match=name):
                size(**dict(ATTN, **{name: n}))
    with pytest.raises(TypeError, match="float16"):
        size(**ATTN, dtype=torch.float16)


def test_linear_grad_size_names_the_type():
    with pytest.raises(TypeError, match="float16"):
        M.ma_linear_grad_workspace_size(10, 10, 10, dy_dtype=torch.float16)


@pytest.mark.parametrize("sections", [(2 ** 32 + 4,), (4, 2 ** 32 + 4), (-2 ** 32 + 4,)])
def test_rotary_sections(sections):
    with pytest.raises(ValueError, match="section"):
        M.Rotary(sections)


def test_rotary_sections_are_counted_before_they_are_allocated():
    """Two sections of 2^30 pairs: refused without the 16 GB that their frequencies would take."""
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    with pytest.raises(M.MuonAdamWError):
        M.Rotary((2 ** 30, 2 ** 30))
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 1 << 20      # KB
