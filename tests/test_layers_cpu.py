"""Host-side tests of the layer operators' C ABI (include/ma_layers.h) and binding:
declared and exported names, sizes, and every refusal.  No GPU is needed: a
refused call launches nothing, so the addresses are never used."""

import ctypes as C
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")
from muon_newton_schulz_02_amd import _abi  # noqa: E402
from tests import _layers_ref as R  # noqa: E402
from tests.test_grads_cpu import _err, _refused, at  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I, S, W, OK = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE, M.MA_ERR_WORKSPACE, M.MA_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return M.load_library()


def test_declared_names_and_constants(lib):
    text = open(os.path.join(ROOT, "include", "ma_layers.h")).read()
    bare = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"^int (ma_\w+)\s*\(", bare, flags=re.M)))
    assert names == sorted(s[0] for s in _abi.LAYER_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    for k, v in re.findall(r"#define\s+(MA_\w+)\s+(\d+)", text):
        assert getattr(_abi, k) == int(v) == getattr(M, k)
    for n in M._LAYERS:
        assert getattr(M, n) is not None and n in M.__all__


def test_header_compiles_as_c_and_structs_match(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ma_layers.h"\nint main(void) { printf("%zu %zu", '
                   'sizeof(ma_attention), sizeof(ma_heads));\n' +
                   "".join('printf(" %%zu", offsetof(ma_attention, %s));\n' % f for f, _ in _abi.ma_attention._fields_) +
                   "return 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(_abi.ma_attention), C.sizeof(_abi.ma_heads)] + \
        [getattr(_abi.ma_attention, f).offset for f, _ in _abi.ma_attention._fields_]


def test_norm_forward_refusals(lib):
    base = dict(x=at(0), xs=40, res=at(1), rs=40, dtype=1, rows=6, cols=40, w=at(2), wdt=0, off=0.0, eps=1e-6, sum=at(3),
                ss=40, y=at(4), ys=40, codes=at(5), exps=at(6), inv=at(7), stream=None)
    for code, change in [
            (I, dict(dtype=2)), (I, dict(wdt=-1)), (S, dict(rows=-1)), (S, dict(cols=0)), (S, dict(cols=8193)),
            (S, dict(rows=2 ** 30 + 1)), (I, dict(xs=-1)), (I, dict(rs=-1)), (I, dict(ss=39)), (I, dict(ys=39)),
            (I, dict(eps=0.0)), (I, dict(eps=-1.0)), (I, dict(eps=NAN)), (I, dict(eps=1e39)), (I, dict(off=INF)),
            (I, dict(x=None)), (I, dict(w=None)), (I, dict(inv=None)), (I, dict(res=None)), (I, dict(sum=None)),
            (I, dict(codes=None)), (I, dict(exps=None)), (I, dict(y=None, codes=None, exps=None)), (I, dict(x=at(0) + 1)),
            (I, dict(codes=at(5) + 8)), (I, dict(exps=at(6) + 2)), (I, dict(inv=at(7) + 2)), (I, dict(w=at(2) + 2)),
            (I, dict(y=at(0))), (I, dict(sum=at(1))), (I, dict(sum=at(4))), (I, dict(inv=at(2))), (I, dict(codes=at(0))),
            (I, dict(y=at(3) + 40))]:
        _refused(lib.ma_rms_norm_forward, base, code, **change)


def test_norm_backward_refusals(lib):
    need = M.ma_rms_norm_backward_workspace_size(6, 40)
    assert need > 0 and need % 256 == 0
    base = dict(dy=at(0), dys=40, s=at(1), ss=40, dsum=at(2), dss=40, dtype=1, rows=6, cols=40, inv=at(3), w=at(4), wdt=1,
                off=1.0, ds=at(5), dss2=40, dw=at(6), gdt=0, acc=0, ws=at(7), wsb=need, stream=None)
    for code, change in [
            (I, dict(dtype=5)), (I, dict(wdt=2)), (I, dict(gdt=2)), (I, dict(acc=2)), (S, dict(rows=-1)), (S, dict(cols=0)),
            (S, dict(cols=8193)), (I, dict(dys=-1)), (I, dict(ss=-1)), (I, dict(dss=-2)), (I, dict(dss2=39)),
            (I, dict(off=NAN)), (W, dict(ws=None)), (W, dict(wsb=need - 1)), (W, dict(ws=at(7) + 64)), (I, dict(dy=None)),
            (I, dict(s=None)), (I, dict(inv=None)), (I, dict(w=None)), (I, dict(ds=None)), (I, dict(ds=at(0))),
            (I, dict(ds=at(2))), (I, dict(dw=at(4))), (I, dict(dw=at(5))), (I, dict(ws=at(1) - 256 + 256)),
            (I, dict(dw=at(6) + 2)), (I, dict(inv=at(3) + 1))]:
        _refused(lib.ma_rms_norm_backward, base, code, **change)
    n = C.c_size_t()
    assert lib.ma_rms_norm_backward_workspace_size(4, 4, None) == I
    assert lib.ma_rms_norm_backward_workspace_size(-1, 4, C.byref(n)) == S
    assert lib.ma_rms_norm_backward_workspace_size(4, 8193, C.byref(n)) == S
    assert M.ma_rms_norm_backward_workspace_size(0, 40) == 0


@pytest.mark.parametrize("sections,order,restart", [((64,), 0, 0), ((16, 24, 24), 0, 0), ((16, 24, 24), 1, 0),
                                                    ((5, 0, 3), 1, 1), ((1, 2, 3, 4), 1, 1), ((0, 7), 0, 1)])
def test_rotary_frequencies(lib, sections, order, restart):
    n = sum(sections)
    f, a = (C.c_double * n)(), (C.c_uint8 * n)()
    assert lib.ma_rotary_frequencies((C.c_int32 * len(sections))(*sections), len(sections), 500.0, order, restart, f,
                                     a) == OK
    want = R.rotary_table(sections, 500.0, ("blocks", "cycled")[order], bool(restart))
    assert list(a) == [x for x, _ in want]
    assert np.allclose(list(f), [x for _, x in want], rtol=1e-14, atol=0)


def test_rotary_frequency_refusals(lib):
    f, a, s = (C.c_double * 256)(), (C.c_uint8 * 256)(), (C.c_int32 * 5)(4, 4, 4, 4, 4)
    base = dict(s=s, axes=2, theta=1e4, order=0, restart=0, f=f, a=a)
    for code, change in [(I, dict(s=None)), (I, dict(f=None)), (I, dict(a=None)), (S, dict(axes=0)), (S, dict(axes=5)),
                         (I, dict(theta=0.0)), (I, dict(theta=NAN)), (I, dict(theta=INF)), (I, dict(order=2)),
                         (I, dict(restart=2)), (S, dict(s=(C.c_int32 * 2)(-1, 4))), (S, dict(s=(C.c_int32 * 2)(0, 0))),
                         (S, dict(s=(C.c_int32 * 2)(200, 57))), (S, dict(s=(C.c_int32 * 2)(257, 0)))]:
        _refused(lib.ma_rotary_frequencies, base, code, **change)
    with pytest.raises(M.MuonAdamWError):
        M.Rotary((300,))
    with pytest.raises(M.MuonAdamWError):
        M.Rotary(())
    with pytest.raises(ValueError, match="layout"):
        M.Rotary(4, layout="quarter")
    with pytest.raises(ValueError, match="order"):
        M.Rotary(4, order="none")


def test_rotary_refusals(lib):
    f, a = (C.c_double * 8)(*[0.5] * 8), (C.c_uint8 * 8)(*[0, 1] * 4)
    base = dict(x=at(0), dtype=0, n=5, heads=3, dim=20, ts=60, hs=20, pos=at(1), pb=8, axes=2, axs=5, f=f, a=a, pairs=8,
                layout=0, inverse=0, out=at(2), ots=60, ohs=20, stream=None)
    for code, change in [
            (I, dict(dtype=2)), (S, dict(n=-1)), (S, dict(heads=0)), (S, dict(dim=0)), (S, dict(dim=513)),
            (S, dict(pairs=0)), (S, dict(pairs=11)), (S, dict(axes=0)), (S, dict(axes=5)), (I, dict(pb=2)),
            (I, dict(layout=2)), (I, dict(inverse=2)), (I, dict(ts=-1)), (I, dict(hs=-1)), (I, dict(ts=2 ** 31)),
            (I, dict(ohs=19)), (I, dict(ots=59)), (I, dict(axs=-1)), (I, dict(f=None)), (I, dict(a=None)),
            (I, dict(axes=1)), (I, dict(f=(C.c_double * 8)(*[NAN] * 8))), (I, dict(x=None)), (I, dict(pos=None)),
            (I, dict(out=None)), (I, dict(out=at(0) + 4)), (I, dict(out=at(0), ots=80)), (I, dict(out=at(1))),
            (I, dict(pos=at(1) + 4)), (I, dict(x=at(0) + 2)), (I, dict(ots=10, ohs=10))]:
        _refused(lib.ma_rotary, base, code, **change)


def test_logprob_refusals(lib):
    need = M.ma_token_logprob_workspace_size(3, 40000, 5)
    assert need > 0 and need % 256 == 0 and M.ma_token_logprob_workspace_size(3000, 40000, 5) == 0
    base = dict(z=at(0), dtype=1, n=3, v=40000, stride=40000, tok=at(1), tb=8, scale=1.0, lp=at(2), ent=at(3), lse=at(4),
                top=5, ids=at(5), best=at(6), ws=at(7), wsb=need, stream=None)
    for code, change in [
            (I, dict(dtype=2)), (S, dict(n=-1)), (S, dict(v=0)), (S, dict(v=2 ** 31)), (I, dict(stride=-1)), (I, dict(tb=3)),
            (I, dict(scale=0.0)), (I, dict(scale=-1.0)), (I, dict(scale=NAN)), (I, dict(scale=1e39)), (S, dict(top=-1)),
            (S, dict(top=65)), (S, dict(v=4, top=5)), (I, dict(z=None)), (I, dict(tok=None)), (I, dict(lp=None)),
            (I, dict(lse=None)), (I, dict(ids=None)), (I, dict(best=None)), (W, dict(ws=None)), (W, dict(wsb=need - 1)),
            (W, dict(ws=at(7) + 8)), (I, dict(lp=at(3))), (I, dict(lse=at(0))), (I, dict(ids=at(6))), (I, dict(best=at(1))),
            (I, dict(ids=at(5) + 4)), (I, dict(tok=at(1) + 4)), (I, dict(z=at(0) + 1)), (I, dict(ent=at(7)))]:
        _refused(lib.ma_token_logprob_forward, base, code, **change)
    base = dict(z=at(0), dtype=1, n=3, v=400, stride=400, tok=at(1), tb=4, scale=1.0, lse=at(2), ent=at(3), g=at(4),
                h=at(5), d=at(6), ddt=0, ds=400, stream=None)
    for code, change in [
            (I, dict(dtype=2)), (I, dict(ddt=3)), (S, dict(n=-1)), (S, dict(v=0)), (I, dict(ds=399)), (I, dict(scale=0.0)),
            (I, dict(z=None)), (I, dict(tok=None)), (I, dict(lse=None)), (I, dict(g=None)), (I, dict(ent=None)),
            (I, dict(h=None)), (I, dict(d=None)), (I, dict(d=at(0))), (I, dict(d=at(0), ddt=1, ds=401)),
            (I, dict(d=at(0) + 2, ddt=1)), (I, dict(d=at(4))), (I, dict(d=at(6) + 2)), (I, dict(tb=0))]:
        _refused(lib.ma_token_logprob_backward, base, code, **change)
    n = C.c_size_t()
    assert lib.ma_token_logprob_workspace_size(4, 4, 0, None) == I
    assert lib.ma_token_logprob_workspace_size(4, 4, 5, C.byref(n)) == S
    assert lib.ma_token_logprob_workspace_size(-4, 4, 0, C.byref(n)) == S


def _attention(back=True, **change):
    a = _abi.ma_attention()
    a.dtype, a.heads, a.kv_heads, a.head_dim, a.causal, a.n_seqs = 1, 4, 2, 64, 1, 3
    a.n_queries, a.n_keys, a.scale, a.cu_q, a.cu_k, a.lse = 100, 3000, 0.125, at(0), at(1), at(2)
    for k, (name, n) in enumerate((("q", 4), ("k", 2), ("v", 2), ("o", 4), ("dout", 4), ("dq", 4), ("dk", 2), ("dv", 2))):
        x = getattr(a, name)
        x.p, x.token_stride, x.head_stride = at(3 + k), n * 64, 64
    for k, v in change.items():
        if "." in k:
            x, f = k.split(".")
            setattr(getattr(a, x), f, v)
        else:
            setattr(a, k, v)
    return a


SHARED = [
    (I, {"dtype": 2}), (S, {"heads": 0}), (S, {"kv_heads": 0}), (S, {"heads": 3}), (S, {"head_dim": 0}),
    (S, {"head_dim": 257}), (I, {"causal": 2}), (S, {"n_seqs": -1}), (S, {"n_seqs": 2 ** 21}), (S, {"n_queries": -1}),
    (S, {"n_keys": -1}), (S, {"n_queries": 2 ** 28}), (S, {"n_keys": 2 ** 28}), (I, {"scale": 0.0}), (I, {"scale": -1.0}),
    (I, {"scale": NAN}), (I, {"scale": INF}), (I, {"cu_q": None}), (I, {"cu_k": None}),
    (I, {"cu_q": None, "cu_k": None}), (I, {"cu_q": at(0) + 2}), (I, {"lse": None}), (I, {"lse": at(2) + 2}),
    (I, {"q.p": None}), (I, {"k.p": None}), (I, {"v.p": None}), (I, {"o.p": None}), (I, {"q.p": at(3) + 1}),
    (I, {"q.token_stride": -1}), (I, {"k.head_stride": -1}), (I, {"v.token_stride": 2 ** 31})]


def test_attention_refusals(lib):
    n = C.c_size_t()
    a = _attention()
    assert lib.ma_attention_forward_workspace_size(C.byref(a), C.byref(n)) == OK
    need = n.value
    assert need > 0 and need % 256 == 0
    assert lib.ma_attention_forward(None, at(20), need, None) == I
    assert lib.ma_attention_forward_workspace_size(C.byref(a), None) == I
    assert lib.ma_attention_forward_workspace_size(None, C.byref(n)) == I
    for code, change in SHARED + [
            (I, {"o.p": at(3)}), (I, {"o.p": at(2)}), (I, {"lse": at(0)}), (I, {"o.head_stride": 63}),
            (I, {"o.token_stride": 255}), (I, {"o.token_stride": 0})]:
        a = _attention(**change)
        rc = lib.ma_attention_forward(C.byref(a), at(20), 1 << 40, None)
        assert rc == code, (change, rc, _err())
    a = _attention()
    for ws, size in ((None, need), (at(20), need - 1), (at(20) + 64, need)):
        assert lib.ma_attention_forward(C.byref(a), ws, size, None) == W
    assert lib.ma_attention_forward(C.byref(a), at(4), need, None) == I          # over k

    assert lib.ma_attention_backward_workspace_size(C.byref(a), C.byref(n)) == OK
    need = n.value
    for code, change in SHARED + [
            (I, {"dout.p": None}), (I, {"dq.p": None}), (I, {"dk.p": None}), (I, {"dv.p": None}), (I, {"dq.p": at(3)}),
            (I, {"dk.p": at(4)}), (I, {"dk.p": at(10)}), (I, {"dv.p": at(6)}), (I, {"dq.p": at(7)}),
            (I, {"dk.head_stride": 63}), (I, {"dv.token_stride": 127}), (I, {"dq.token_stride": 255}),
            (I, {"dout.token_stride": -4})]:
        a = _attention(**change)
        rc = lib.ma_attention_backward(C.byref(a), at(20), 1 << 40, None)
        assert rc == code, (change, rc, _err())
    a = _attention()
    for ws, size in ((None, need), (at(20), need - 1), (at(20) + 128, need)):
        assert lib.ma_attention_backward(C.byref(a), ws, size, None) == W
    assert lib.ma_attention_backward(C.byref(a), at(8), need, None) == I         # over dq


def test_attention_workspace_follows_the_arrays(lib):
    """Rows that are not whole 16-byte chunks at 16-byte addresses are copied; few rows take pieces."""
    def need(back, **change):
        n = C.c_size_t()
        a = _attention(**change)
        fn = lib.ma_attention_backward_workspace_size if back else lib.ma_attention_forward_workspace_size
        assert fn(C.byref(a), C.byref(n)) == OK
        return n.value

    long = dict(n_queries=60000, n_keys=60000)
    assert need(False, **long) == 0
    plain = need(True, **long)
    assert plain >= 60000 * 4 * 8
    for name, n in (("q", 4), ("k", 2), ("v", 2), ("dout", 4)):
        size = 60000 * n * 64 * 2
        for change in ({name + ".p": at(30) + 2}, {name + ".token_stride": n * 64 + 1}, {name + ".token_stride": 1 << 23}):
            assert need(True, **long, **change) == plain + size, change
            assert need(False, **long, **change) == (0 if name == "dout" else size), change
    assert M.ma_attention_forward_workspace_size(60000, 60000, 4, 2, 64, 3) == 0
    assert M.ma_attention_backward_workspace_size(60000, 60000, 4, 2, 64, 3) == plain
    assert M.ma_attention_forward_workspace_size(100, 60000, 4, 2, 64, 3) > 0


def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros(4, 40), torch.ones(40)
    ids = torch.zeros(4, dtype=torch.int64)
    q = torch.zeros(4, 2, 64)
    for call in (lambda: M.ma_rms_norm_forward(x, w), lambda: M.ma_rms_norm_backward(x, x, ids, w),
                 lambda: M.ma_rotary(q, ids, M.Rotary(32)), lambda: M.ma_token_logprob_forward(x, ids),
                 lambda: M.ma_token_logprob_backward(x, ids, w, w), lambda: M.ma_attention_forward(q, q, q),
                 lambda: M.ma_attention_backward(q, q, q, q, q, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        M.ma_rms_norm_forward([0.0], w)


def test_rotary_plans_are_copied():
    import copy
    import pickle
    p = M.Rotary((3, 5), theta=77.0, layout="pairs", order="cycled", restart=True)
    for q in (copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert (q.sections, q.theta, q.layout, q.order, q.restart) == (p.sections, 77.0, "pairs", "cycled", True)
        assert q.frequencies == p.frequencies and q.pair_axis == p.pair_axis
