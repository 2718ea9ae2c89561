"""Dense attention whose waits give up.  A build of its own lets them: every
wait that does not pass at once, or one in eight of those (then the rest give
up after some 16 ms).  The call has to end, say so in the error word and leave
nothing behind that reaches the calls after it: no copy, commit or MMA still
under way in the shared memory and TMEM of a CTA that has left."""
import ctypes as C
import os
import subprocess
import time

import pytest
import torch

from test_gpu_dense_pa import Case

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    from block_sparse_paged_score_gb300 import bsp, build
    bsp.lib()
    where = tmp_path_factory.mktemp("impatient")
    objs = [os.path.join(build.BUILD_DIR, f.replace(".cu", ".o")) for f in build.SOURCES if f != "dense_pa.cu"]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True)
    cmds, libs = [], []
    for name, rounds in (("at_once", "0u"), ("now_and_then", "((clock() & 7) ? 1u << 14 : 0u)")):
        obj, so = str(where / f"{name}.o"), str(where / f"lib{name}.so")
        cmds.append([build.nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.INCLUDE,
                    "--expt-relaxed-constexpr", f"-DBSP_DENSE_PA_WAIT_ROUNDS={rounds}", "-c",
                    os.path.join(build.CSRC, "dense_pa.cu"), "-o", obj])
        libs.append((so, obj))
    running = [subprocess.Popen(c) for c in cmds]
    assert [p.wait() for p in running] == [0, 0]
    out = []
    for so, obj in libs:
        subprocess.check_call([build.nvcc()] + build.ARCH + ["-shared", "-o", so] + objs + [obj, "-cudart", "static"])
        L = C.CDLL(so)
        for f, args in bsp.SYMBOLS.items():
            getattr(L, f).argtypes, getattr(L, f).restype = args, bsp.RESTYPES.get(f, C.c_int32)
        out.append(L)
    return out


CASES = [dict(lens=[700, 31], q_len=1), dict(lens=[700, 31], q_len=1, q8=False), dict(lens=[2500, 128, 900], q_len=2),
         dict(lens=[1500, 4000], q_len=4), dict(lens=[1500, 4000], q_len=4, q8=False),
         dict(lens=[300, 5, 900, 77], q_len=8), dict(lens=[40] * 1500, q_len=1)]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_waits_that_give_up_end_the_call_and_reach_no_other(monkeypatch, impatient, which, case):
    from block_sparse_paged_score_gb300 import bsp
    c = Case(seed=3, **case).device()
    want = c.call().clone()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    own = bsp.lib()
    for i in range(3):
        c.err.zero_()
        monkeypatch.setattr(bsp, "_lib", impatient[which])
        t = time.perf_counter()
        c.call()
        monkeypatch.setattr(bsp, "_lib", own)
        # the very next kernel takes over the shared memory and TMEM
        got = c.call()
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        # the drain has a limit of about a second for each barrier: it did not need one
        assert t < 0.9, t
        assert torch.equal(got, want), i
        assert c.err.item() in ((TIMEOUT,) if which == 0 else (0, TIMEOUT))
