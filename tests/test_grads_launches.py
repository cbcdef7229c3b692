"""The launches that ma_embedding_grad makes, looked at without a GPU: a
preloaded library reports them instead of making them (tests/c/launch_trace.c).

Zeroing rides along in the launches of the sort and of the sums.  Its shares
have to cover the gradient exactly once, and those beside the sums, which write
rows at the same time, may only take rows that a flag tells to be empty."""

import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

DRIVER = """
import ctypes as C, json, sys
sys.path.insert(0, %(root)r)
trace = C.CDLL(None)
import muon_newton_schulz_02_amd._abi as A
lib = A.load()

class Fill(C.Structure):
    _fields_ = [("p", C.c_uint64), ("pieces", C.c_int64), ("groups", C.c_int64),
                ("flags", C.c_uint64), ("first", C.c_int64), ("row", C.c_uint32),
                ("magic", C.c_uint32), ("edge", C.c_uint64 * 2), ("edge_n", C.c_int32 * 2)]

AT = {"k_sort_count": 2, "k_sort_scatter": 4, "k_sort_lds": 4, "k_emb_sum": 1}
seen = []

@C.CFUNCTYPE(None, C.c_char_p, C.c_uint, C.c_uint, C.c_uint, C.POINTER(C.c_void_p))
def report(name, gx, gy, threads, args):
    name = name.decode()
    for k, i in AT.items():
        if k in name:
            f = Fill.from_address(args[i])
            seen.append(dict(kernel=k, grid=gx, groups=f.groups, p=f.p, pieces=f.pieces,
                             flags=f.flags, edge=list(f.edge), edge_n=list(f.edge_n)))
            return
    seen.append(dict(kernel=name, grid=gx))

trace.launch_trace_report(report)
out = []
for n, v, h, dtype, addr, acc in json.loads(sys.argv[1]):
    need = C.c_size_t()
    assert lib.ma_embedding_grad_workspace_size(n, v, h, C.byref(need)) == 0
    del seen[:]
    rc = lib.ma_embedding_grad(1 << 40, 0, h, 1 << 41, 8, n, v, h, 1.0, -1, addr, dtype, acc,
                               (1 << 42) if need.value else None, need.value, None)
    assert rc == 0, lib.muon_adamw_last_error()
    out.append(list(seen))
print(json.dumps(out))
"""

G = 1 << 43         # the gradient's address: nothing is read or written there


def _cases():
    """(tokens, vocab, hidden, dtype, address, accumulate): every size of sort, from gradients of
    a few bytes that lie inside one 128-byte line to ones of many shares, at each kind of
    address."""
    cases = []
    for n in (1100, 3000, 5000, 140000):
        for v, h in ((1, 1), (2, 1), (3, 1), (30, 1), (7, 4), (1, 3), (1, 16), (5, 8), (3, 33), (40, 24),
                     (40009, 264), (30011, 263)):
            for dtype, size in ((0, 4), (1, 2)):
                for off in (0, 1, 4, 8, 31, 63):
                    cases.append((n, v, h, dtype, G + off * size, 0))
    cases += [(0, 7, 3, 0, G + 4, 0), (0, 1, 1, 1, G + 2, 0), (200000, 1100003, 8, 1, G + 128, 0),
              (16384, 151000, 2048, 1, G, 0), (5000, 3, 1, 0, G, 1), (3000, 40, 24, 1, G + 2, 1)]
    return cases


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lib = str(tmp_path_factory.mktemp("trace") / "liblaunch_trace.so")
    subprocess.run([cc, "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-o", lib,
                    os.path.join(HERE, "c", "launch_trace.c"), "-ldl"], check=True)
    cases = _cases()
    preload = ":".join([lib] + [x for x in [os.environ.get("LD_PRELOAD")] if x])
    res = subprocess.run([sys.executable, "-c", DRIVER % {"root": ROOT}, json.dumps(cases)],
                         cwd=ROOT, env=dict(os.environ, LD_PRELOAD=preload), capture_output=True, text=True,
                         timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    return list(zip(cases, json.loads(res.stdout.splitlines()[-1])))


def test_every_byte_is_zeroed_once(launches):
    for case, seen in launches:
        n, v, h, dtype, addr, acc = case
        spans = []
        for s in seen:
            if "groups" not in s:
                continue
            if s["groups"] == 0:
                assert s["pieces"] == 0 and s["edge_n"] == [0, 0], (case, s)
                continue
            assert s["grid"] >= s["groups"], (case, s)
            spans.append((s["p"], 16 * s["pieces"]))
            spans += [(e, 2 * k) for e, k in zip(s["edge"], s["edge_n"])]
        spans = sorted(x for x in spans if x[1])
        if acc:
            assert not spans, case
            continue
        at = addr
        for p, size in spans:
            assert p == at, (case, spans[:6])
            at += size
        assert at == addr + v * h * (2 if dtype else 4), (case, spans[-3:])


def test_sums_ride_with_flagged_zeroing_only(launches):
    met = 0
    for case, seen in launches:
        sums = [s for s in seen if s["kernel"] == "k_emb_sum"]
        assert len(sums) == (1 if case[0] > 1024 else 0), case
        for s in sums:
            assert s["groups"] == 0 or s["flags"] != 0, (case, s)
            met += s["groups"] > 0
    assert met > 0
