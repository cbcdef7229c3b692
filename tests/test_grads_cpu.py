"""Host-side tests of the gradient operators' C ABI (include/ma_grads.h) and
binding: declared and exported names, sizes, and every refusal.  No GPU is
needed: a refused call launches nothing, so the addresses are never used."""

import ctypes as C
import os
import re

import pytest

torch = pytest.importorskip("torch")
M = pytest.importorskip("muon_newton_schulz_02_amd")
from muon_newton_schulz_02_amd import _abi  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40            # fake addresses, far apart
GAP = 1 << 32


def at(k):
    return A + k * GAP


@pytest.fixture(scope="module")
def lib():
    return M.load_library()


def _err():
    return M.muon_adamw_last_error()


def test_declared_names_and_constants(lib):
    text = open(os.path.join(ROOT, "include", "ma_grads.h")).read()
    bare = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ma_\w+)\s*\(", bare)))
    assert names == sorted(s[0] for s in _abi.GRAD_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    for k, v in re.findall(r"#define\s+(MA_ACT\w+)\s+(\d+)", text):
        assert getattr(_abi, k) == int(v) == getattr(M, k)


def test_header_compiles_as_c(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "ma_grads.h"\nint main(void) { return MA_ACT_GROUP - 32; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-c", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "t.o")], check=True)


@pytest.mark.parametrize("cols,cp,ep", [(1, 32, 4), (32, 32, 4), (33, 64, 4), (128, 128, 4),
                                        (129, 160, 8), (1000, 1024, 32), (8192, 8192, 256)])
def test_pitch(lib, cols, cp, ep):
    a, b = C.c_int64(), C.c_int64()
    assert lib.ma_act_pitch(cols, C.byref(a), C.byref(b)) == M.MA_OK
    assert (a.value, b.value) == (cp, ep)
    c = M.ActCheckpoint.empty((3, cols), "cpu")
    assert tuple(c.codes.shape) == (3, cp) and tuple(c.exps.shape) == (3, ep)


def test_pitch_refusals(lib):
    a, b = C.c_int64(), C.c_int64()
    assert lib.ma_act_pitch(0, C.byref(a), C.byref(b)) == M.MA_ERR_SHAPE
    assert lib.ma_act_pitch(2 ** 30 + 1, C.byref(a), C.byref(b)) == M.MA_ERR_SHAPE
    assert lib.ma_act_pitch(4, None, C.byref(b)) == M.MA_ERR_INVALID_ARG


def _refused(fn, base, code, **change):
    args = dict(base)
    for k in change:
        assert k in args, k
    args.update(change)
    rc = fn(*args.values())
    assert rc == code, (change, rc, _err())
    assert fn.__name__ in _err() or "ma_" in _err()


def test_pack_refusals(lib):
    base = dict(x=at(0), dtype=0, rows=4, cols=40, stride=40, codes=at(1), exps=at(2), stream=None)
    I, S = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE
    for code, change in [(I, dict(dtype=2)), (I, dict(x=None)), (I, dict(codes=None)),
                         (I, dict(exps=None)), (S, dict(rows=-1)), (S, dict(cols=0)),
                         (S, dict(rows=2 ** 30, cols=2 ** 30)), (I, dict(stride=-1)),
                         (I, dict(stride=2 ** 39)), (I, dict(x=at(0) + 2)),
                         (I, dict(codes=at(1) + 8)), (I, dict(exps=at(2) + 2)),
                         (I, dict(codes=at(0))), (I, dict(exps=at(1) + 64)),
                         (I, dict(exps=at(0) + 4 * 40 * 4 - 4))]:
        _refused(lib.ma_act_pack, base, code, **change)


def test_unpack_refusals(lib):
    base = dict(codes=at(1), exps=at(2), rows=4, cols=40, out=at(0), dtype=1, stride=40, stream=None)
    I, S = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE
    for code, change in [(I, dict(dtype=-1)), (I, dict(out=None)), (I, dict(codes=None)),
                         (I, dict(exps=None)), (S, dict(rows=2 ** 31)), (S, dict(cols=-3)),
                         (I, dict(stride=39)), (I, dict(out=at(0) + 1)), (I, dict(out=at(1)))]:
        _refused(lib.ma_act_unpack, base, code, **change)


def test_lookup_refusals(lib):
    base = dict(table=at(0), tdt=0, vocab=10, hidden=8, tstride=8, tokens=at(1), tb=8, n=5,
                scale=1.0, out=at(2), odt=1, ostride=8, stream=None)
    I, S = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE
    for code, change in [(I, dict(tdt=3)), (I, dict(odt=-1)), (I, dict(tb=2)), (S, dict(n=-1)),
                         (S, dict(vocab=0)), (S, dict(hidden=0)), (S, dict(hidden=2 ** 20 + 1)),
                         (S, dict(vocab=2 ** 31)), (S, dict(vocab=2 ** 30, hidden=2 ** 20)),
                         (I, dict(tstride=-1)), (I, dict(ostride=7)),
                         (I, dict(scale=float("nan"))), (I, dict(scale=1e39)),
                         (I, dict(table=None)), (I, dict(tokens=None)), (I, dict(out=None)),
                         (I, dict(tokens=at(1) + 4)), (I, dict(out=at(0) + 16)),
                         (I, dict(out=at(1) + 8)), (I, dict(table=at(0) + 2))]:
        _refused(lib.ma_embedding_lookup, base, code, **change)


def test_embedding_grad_refusals(lib):
    need = M.ma_embedding_grad_workspace_size(5000, 50, 16)
    assert need % 256 == 0 and need > 0
    base = dict(dout=at(0), ddt=1, dstride=16, tokens=at(1), tb=4, n=5000, vocab=50, hidden=16,
                scale=2.0, pad=-1, grad=at(2), gdt=0, acc=0, ws=at(3), wsb=need, stream=None)
    I, S, W = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE, M.MA_ERR_WORKSPACE
    for code, change in [(I, dict(ddt=2)), (I, dict(gdt=2)), (I, dict(tb=1)), (I, dict(acc=2)),
                         (S, dict(n=-1)), (S, dict(vocab=0)), (S, dict(hidden=0)),
                         (I, dict(dstride=-16)), (I, dict(scale=float("inf"))),
                         (W, dict(ws=None)), (W, dict(wsb=need - 1)), (W, dict(ws=at(3) + 64)),
                         (I, dict(dout=None)), (I, dict(tokens=None)), (I, dict(grad=None)),
                         (I, dict(dout=at(0) + 1)), (I, dict(grad=at(2) + 2)),
                         (I, dict(grad=at(0))), (I, dict(grad=at(3) + 256)),
                         (I, dict(tokens=at(2) + 50 * 16 * 4 - 4)), (I, dict(ws=at(1) - 256))]:
        _refused(lib.ma_embedding_grad, base, code, **change)
    n = C.c_size_t()
    assert lib.ma_embedding_grad_workspace_size(4, 4, 4, None) == I
    assert lib.ma_embedding_grad_workspace_size(-1, 4, 4, C.byref(n)) == S
    assert lib.ma_embedding_grad_workspace_size(4, 0, 4, C.byref(n)) == S
    assert M.ma_embedding_grad_workspace_size(0, 4, 4) == 0


def test_linear_grad_refusals(lib):
    need = M.ma_linear_grad_workspace_size(5000, 24, 40)
    assert need > 0
    base = dict(dy=at(0), ddt=1, m=5000, n=24, stride=24, codes=at(1), exps=at(2), k=40, grad=at(3),
                gdt=0, acc=0, ws=at(4), wsb=need, stream=None)
    I, S, W = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE, M.MA_ERR_WORKSPACE
    for code, change in [(I, dict(ddt=5)), (I, dict(gdt=-1)), (I, dict(acc=-1)), (S, dict(m=-1)),
                         (S, dict(n=0)), (S, dict(k=0)), (S, dict(n=2 ** 20 + 1)),
                         (S, dict(m=2 ** 30, n=2 ** 20)), (S, dict(n=2 ** 20, k=2 ** 20)),
                         (I, dict(stride=-1)), (W, dict(ws=None)), (W, dict(wsb=need - 1)),
                         (W, dict(ws=at(4) + 128)), (I, dict(dy=None)), (I, dict(codes=None)),
                         (I, dict(exps=None)), (I, dict(grad=None)), (I, dict(codes=at(1) + 4)),
                         (I, dict(exps=at(2) + 1)), (I, dict(dy=at(0) + 1)), (I, dict(grad=at(0))),
                         (I, dict(grad=at(1) + 64)), (I, dict(ws=at(3))), (I, dict(grad=at(2)))]:
        _refused(lib.ma_linear_grad, base, code, **change)
    n = C.c_size_t()
    assert lib.ma_linear_grad_workspace_size(4, 4, 4, 0, None) == I
    assert lib.ma_linear_grad_workspace_size(4, 4, 4, 7, C.byref(n)) == I
    assert lib.ma_linear_grad_workspace_size(4, -4, 4, 0, C.byref(n)) == S


def test_glu_refusals(lib):
    base = dict(gate=at(0), up=at(1), dtype=1, rows=6, cols=40, gs=40, us=40, act=0, h=at(2), hs=40,
                gc=at(3), ge=at(4), uc=at(5), ue=at(6), stream=None)
    I, S, U = M.MA_ERR_INVALID_ARG, M.MA_ERR_SHAPE, M.MA_ERR_UNSUPPORTED
    for code, change in [(I, dict(dtype=2)), (U, dict(act=2)), (U, dict(act=-1)), (S, dict(rows=-1)),
                         (S, dict(cols=0)), (I, dict(gs=-1)), (I, dict(us=-1)), (I, dict(hs=39)),
                         (I, dict(gate=None)), (I, dict(up=None)), (I, dict(h=None)),
                         (I, dict(gc=None)), (I, dict(ge=None)), (I, dict(uc=None)),
                         (I, dict(ue=None)), (I, dict(h=at(0))), (I, dict(gc=at(5))),
                         (I, dict(ue=at(4))), (I, dict(gc=at(1))), (I, dict(uc=at(5) + 1))]:
        _refused(lib.ma_glu_forward, base, code, **change)
    base = dict(dh=at(0), dtype=0, rows=6, cols=40, ds=40, gc=at(1), ge=at(2), uc=at(3), ue=at(4),
                act=1, dg=at(5), dgs=40, du=at(6), dus=40, hc=at(7), he=at(8), stream=None)
    for code, change in [(I, dict(dtype=2)), (U, dict(act=5)), (S, dict(rows=-1)), (S, dict(cols=0)),
                         (I, dict(ds=-1)), (I, dict(dgs=39)), (I, dict(dus=0)), (I, dict(dh=None)),
                         (I, dict(gc=None)), (I, dict(ge=None)), (I, dict(uc=None)),
                         (I, dict(ue=None)), (I, dict(dg=None)), (I, dict(du=None)),
                         (I, dict(hc=None)), (I, dict(he=None)), (I, dict(dg=at(6))),
                         (I, dict(du=at(0))), (I, dict(hc=at(1))), (I, dict(he=at(4))),
                         (I, dict(du=at(5) + 160))]:
        _refused(lib.ma_glu_backward, base, code, **change)


def test_interleaved_rows_are_told_apart(lib):
    """dgate and dup may be columns of one array only where their columns do not
    meet (the accepted case runs on a GPU: here each is refused for another
    reason, an unknown act, or for the overlap itself)."""
    base = dict(dh=at(0), dtype=0, rows=6, cols=40, ds=40, gc=at(1), ge=at(2), uc=at(3), ue=at(4),
                act=0, dg=at(5), dgs=80, du=at(5) + 160, dus=80, hc=None, he=at(8), stream=None)
    rc = lib.ma_glu_backward(*base.values())
    assert rc == M.MA_ERR_INVALID_ARG and "go together" in _err()
    for off, dus in ((156, 80), (164, 80), (0, 80), (160, 81), (80 * 4 * 5 + 40, 80)):
        args = dict(base, he=None, du=at(5) + off, dus=dus)
        rc = lib.ma_glu_backward(*args.values())
        assert rc == M.MA_ERR_INVALID_ARG and "overlaps" in _err(), (off, dus, _err())


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 40)
    with pytest.raises(ValueError, match="GPU"):
        M.ma_act_pack(x)
    with pytest.raises(TypeError):
        M.ma_act_pack([1.0])
    with pytest.raises(ValueError, match="GPU"):
        M.ma_embedding_lookup(x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        M.ma_embedding_grad(x, torch.zeros(4, dtype=torch.int64), 7)
    c = M.ActCheckpoint.empty((4, 40), "cpu")
    with pytest.raises(ValueError, match="GPU"):
        M.ma_act_unpack(c)
    with pytest.raises(ValueError, match="GPU"):
        M.ma_linear_grad(x, c)
    with pytest.raises(ValueError, match="GPU"):
        M.ma_glu_forward(x, x)
    with pytest.raises(ValueError, match="GPU"):
        M.ma_glu_backward(x, c, c)


def test_checkpoint_layout_is_checked():
    codes, exps = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8)
    c = M.ActCheckpoint(codes, exps, 40)
    assert c.shape == (4, 40) and c.rows == 4
    assert M.ActCheckpoint(codes, exps, 40, (2, 2, 40)).shape == (2, 2, 40)
    for bad in [(codes.int(), exps, 40), (codes, exps.int(), 40), (codes, exps, 0)]:
        with pytest.raises(TypeError):
            M.ActCheckpoint(*bad)
    for bad in [(codes, exps, 65), (codes, exps, 32), (codes[:3], exps, 40),
                (codes, exps[:, :3], 40), (codes.t().contiguous().t(), exps, 40),
                (codes, exps, 40, (3, 40)), (codes, exps, 40, (4, 41))]:
        with pytest.raises(ValueError):
            M.ActCheckpoint(*bad)


def test_rows_of_a_tensor():
    from muon_newton_schulz_02_amd.grads import _rows
    x = torch.zeros(2, 3, 5, 8)
    assert _rows(x, "x") == (30, 8, 8)
    assert _rows(x[0, 0, 0], "x") == (1, 8, 8)
    assert _rows(x[..., :6], "x") == (30, 6, 8)
    assert _rows(x[:, :, 0], "x") == (6, 8, 40)
    assert _rows(torch.zeros(8).expand(5, 8), "x") == (5, 8, 0)
    assert _rows(torch.zeros(8).expand(5, 3, 8), "x") == (15, 8, 0)
    assert _rows(torch.zeros(1, 8).t(), "x") == (8, 1, 1)
    assert _rows(torch.zeros(0, 8), "x")[:2] == (0, 8)
    for bad in (x[:, :2], x.transpose(1, 2), x.transpose(2, 3), torch.zeros(4, 8)[:, ::2],
                torch.zeros(())):
        with pytest.raises(ValueError):
            _rows(bad, "x")


def _holder(**kw):
    """A MuonAdamW without a GPU: only what _formed looks at."""
    o = object.__new__(M.MuonAdamW)
    o.names, o.params, o.groups = ["a"], [torch.zeros(4, 4)], [M.MA_GROUP_MUON]
    o.grad_buffers, o.sum_buffers = [None], [None]
    o.__dict__.update(kw)
    return o


def test_step_refuses_wrong_sources():
    for bad in ([torch.zeros(4, 4)], [], (1, 2), [M.LinearGrad(None, None), None]):
        with pytest.raises(TypeError, match="LinearGrad"):
            _holder()._formed(0, bad, None)
        with pytest.raises(TypeError, match="LinearGrad"):
            _holder().step([bad])
    with pytest.raises(ValueError, match="matrix"):
        _holder(params=[torch.zeros(4)])._formed(0, M.LinearGrad(None, None), None)
    with pytest.raises(ValueError, match="entries"):
        _holder().step([M.LinearGrad(None, None), None])
    frozen = _holder(groups=[M.MA_GROUP_NONE])
    assert frozen._formed(0, M.LinearGrad(None, None), None) is None


@pytest.mark.parametrize("dtype,buffers", [(torch.float32, 1), (torch.bfloat16, 2)])
def test_step_allocates_on_the_stream_that_writes(dtype, buffers, monkeypatch):
    """The buffers that gradients are formed into come from the pool of the step's stream: each
    allocation is made while that stream is current.  A later step on another stream, given or
    current, is made known to the allocator."""
    from types import SimpleNamespace
    from muon_newton_schulz_02_amd import grads as G
    side, other = SimpleNamespace(cuda_stream=7), SimpleNamespace(cuda_stream=9)
    now, made, recorded = [other], [], []

    class At:
        def __init__(self, dev, stream, tensors):
            self.stream = stream or now[-1]

        def __enter__(self):
            now.append(self.stream)

        def __exit__(self, *exc):
            now.pop()

    def noted(make):
        def f(*a, **k):
            made.append(now[-1])
            return make(*a, **k)
        return f

    monkeypatch.setattr(G, "_At", At)
    monkeypatch.setattr(G, "_raw_stream", lambda index: now[-1].cuda_stream)
    monkeypatch.setattr(G, "form_gradient", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append(s))
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    opt = _holder(params=[torch.zeros(4, 4, dtype=dtype)])
    src = M.LinearGrad(None, None)
    out = opt._formed(0, [src, src], side)
    assert out is opt.grad_buffers[0] and out.shape == (4, 4) and out.dtype == dtype
    assert made == [side] * buffers and recorded == []
    for stream, want in ((side, []), (7, []), (None, [other]), (other, [other])):
        del recorded[:]
        assert opt._formed(0, [src, src], stream) is out and len(made) == buffers     # kept
        assert recorded == want * buffers, stream


@pytest.mark.parametrize("torch_there", [False, True])
def test_star_import_with_and_without_torch(torch_there):
    """The optimizer step's names need no torch to be imported; the gradient operators' join
    them where torch is installed."""
    import subprocess
    import sys
    code = ("import sys\n"
            + ("" if torch_there else "sys.modules['torch'] = None\n") +
            "sys.path.insert(0, %r)\n"
            "from muon_newton_schulz_02_amd import *\n"
            "print(muon_adamw_version(), MuonAdamW.__name__, 'ma_act_pack' in globals())\n" % ROOT)
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.split()[-2:] == ["MuonAdamW", str(torch_there)]


@pytest.mark.parametrize("m,n,k", [(0, 8, 8), (5, 24, 40), (16001, 256, 1024), (32768, 8192, 2048),
                                   (3000, 3001, 2048), (8192, 1024, 4096), (4096, 1024, 1024)])
@pytest.mark.parametrize("dt", [0, 1])
def test_linear_grad_workspace_of_one_dy(lib, m, n, k, dt):
    """What a call needs for its own dy: its size is taken and one byte less is refused; never
    more than the size for any dy, and no copy of a bf16 dy with aligned rows."""
    worst, size = C.c_size_t(), C.c_size_t()
    assert lib.ma_linear_grad_workspace_size(m, n, k, dt, C.byref(worst)) == M.MA_OK
    es = 2 if dt else 4
    for addr in (at(0), at(0) + es, at(0) + 16):
        for stride in (n, n + 1, n + 8, 0):
            assert lib.ma_linear_grad_workspace_size_at(addr, dt, m, n, stride, k,
                                                        C.byref(size)) == M.MA_OK
            assert size.value <= worst.value

            def call(bytes_):       # (no gradient: refused after the workspace is looked at)
                return lib.ma_linear_grad(addr, dt, m, n, stride, at(1), at(2), k, None, 0, 0, at(3),
                                          bytes_, None)
            assert call(size.value) == M.MA_ERR_INVALID_ARG and "grad is NULL" in _err()
            if size.value:
                assert call(size.value - 1) == M.MA_ERR_WORKSPACE
            if dt and n % 8 == 0 and m >= 512 and addr % 16 == 0 and stride >= n and stride % 8 == 0:
                # x as bf16 in whole tiles, and at most 64 slices of partial sums that together
                # fill 8 workgroups of 128 x 128 outputs per CU
                x = -(-m // 32) * 32 * (-(-k // 256) * 256) * 2
                assert size.value <= x + (2 * 8 * 256 * 128 * 128 + 256) * 4
    assert lib.ma_linear_grad_workspace_size_at(None, dt, m, n, n, k, None) == M.MA_ERR_INVALID_ARG
    assert lib.ma_linear_grad_workspace_size_at(None, 7, m, n, n, k, C.byref(size)) == M.MA_ERR_INVALID_ARG
    assert lib.ma_linear_grad_workspace_size_at(None, dt, m, n, -1, k, C.byref(size)) == M.MA_ERR_INVALID_ARG
    assert lib.ma_linear_grad_workspace_size_at(None, dt, -1, n, n, k, C.byref(size)) == M.MA_ERR_SHAPE


@pytest.mark.parametrize("where", ["record", "stream"])
def test_a_failed_switch_of_device_and_stream_is_undone(where, monkeypatch):
    """A call for another device that fails while it takes the device and the stream leaves the
    current ones as they were."""
    from types import SimpleNamespace
    from muon_newton_schulz_02_amd import grads as G
    current = ["first"]

    class device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.was

    def fails(*a):
        raise RuntimeError("no")

    dev = SimpleNamespace(index=1)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", fails)
    monkeypatch.setattr(G, "_raw_stream", lambda index: 0)
    t = SimpleNamespace(record_stream=fails if where == "record" else lambda s: None)
    with pytest.raises(RuntimeError, match="no"):
        G._At(dev, SimpleNamespace(device=dev, cuda_stream=5), (t, None))
    assert current == ["first"]


def test_checkpoint_follows_its_arrays():
    """Arrays that their owner has given other memory since are looked at again by the next
    call: nothing reads where they once were."""
    def used(c):
        with pytest.raises(ValueError, match="GPU"):      # (the layout has been looked at)
            M.ma_act_unpack(c)
        assert (c._pc, c._pe) == (c.codes.data_ptr(), c.exps.data_ptr())

    codes, exps = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8)
    c = M.ActCheckpoint(codes, exps, 40, (2, 2, 40))
    used(c)
    kept = codes.data, exps.data
    codes.data = codes.clone()
    used(c)
    exps.data = exps.clone()
    used(c)
    assert c._pc != kept[0].data_ptr() and c._pe != kept[1].data_ptr()
    for bad in (torch.zeros(4, 32), torch.zeros(3, 64), torch.zeros(64, 4).t()):
        codes.data = bad.to(torch.int8)
        with pytest.raises(ValueError):
            M.ma_act_unpack(c)
    # arrays that lie in one allocation
    c = M.ActCheckpoint.empty((4, 40), "cpu")
    used(c)
    c.codes.data = c.codes.clone()
    used(c)
    c = M.ActCheckpoint.empty((4, 40), "cpu")
    c.exps.data = torch.zeros(4, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="do not hold"):
        M.ma_act_unpack(c)
    for c in (M.ActCheckpoint.empty((4, 40), "cpu"),
              M.ActCheckpoint(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(7, 4, dtype=torch.uint8)[3:], 40)):
        c.exps.untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="freed"):
            M.ma_act_unpack(c)
