"""Prompt attention and dense attention over fp8 whose waits give up.  A build of
its own lets them: every wait, those that do not pass within about a microsecond, or
some of them (then the rest give up after some 16 ms).  In the prompt kernel a warp
votes in each round, so that all of its lanes must count the same rounds: which give
up goes by the warp and the CTA, not by the clock.  The call has to end, say so in the error word and leave nothing behind
that reaches the calls after it."""
import ctypes as C
import os
import subprocess
import time

import numpy as np
import pytest
import torch

import test_gpu_dense_pa_fp8 as D
import test_gpu_prompt as A

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    from block_sparse_paged_score_gb300 import bsp, build
    bsp.lib()
    where = tmp_path_factory.mktemp("impatient")
    own = ("prompt.cu", "dense_pa_fp8.cu")
    objs = [os.path.join(build.BUILD_DIR, f.replace(".cu", ".o")) for f in build.SOURCES if f not in own]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True)
    running, out = [], []
    some = {"prompt.cu": "(((threadIdx.x >> 5) + 3 * blockIdx.x) % 29 ? 1u << 14 : 0u)",
            "dense_pa_fp8.cu": "((clock() & 7) ? 1u << 14 : 0u)"}
    kinds = (("at_once", dict.fromkeys(own, "0u")), ("soon", dict.fromkeys(own, "1u")), ("some", some))
    for name, macro in kinds:
        for f in own:
            running.append(subprocess.Popen(
                [build.nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.INCLUDE,
                 "--expt-relaxed-constexpr", f"-DBSP_WAIT_ROUNDS={macro[f]}", "-c", os.path.join(build.CSRC, f), "-o",
                 str(where / f"{name}_{f}.o")]))
    assert not any([p.wait() for p in running])
    for name, _ in kinds:
        so = str(where / f"lib{name}.so")
        subprocess.check_call([build.nvcc()] + build.ARCH + ["-shared", "-o", so] + objs +
                              [str(where / f"{name}_{f}.o") for f in own] + ["-cudart", "static"])
        L = C.CDLL(so)
        for f, args in bsp.SYMBOLS.items():
            getattr(L, f).argtypes, getattr(L, f).restype = args, bsp.RESTYPES.get(f, C.c_int32)
        out.append(L)
    return out


def prompt(nq, nk, hkv, group):
    from block_sparse_paged_score_gb300 import bsp
    p = A.problem(31, nq, nk, hkv, group)
    cu = [torch.from_numpy(np.asarray(p[x], np.int32)).cuda() for x in ("cu_q", "cu_k")]
    ws = bsp.prompt_attention_workspace(len(p["q"]), len(nq), hkv, group)
    out = torch.zeros_like(p["q"])
    return lambda err: bsp.prompt_attention(p["q"], p["k"], p["v"], *cu, out=out, ws=ws, dev_err=err)


def decode(lens, q_len, q8, group=16):
    from block_sparse_paged_score_gb300 import bsp
    d = D.problem(32, len(lens), q_len, 1, group, lens, q8)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    c = bsp.BlockScaledKvCache(1, d["blocks"], buffer=t(d["cache"]), k_scales=t(d["scales"][0]), v_scales=t(d["scales"][1]))
    q, table, seq, rl = d["q"].cuda(), t(d["table"]), t(d["row_seq"]), t(d["row_len"])
    ws, out = bsp.dense_pa_fp8_workspace(len(rl), 1, group, q_len), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    return lambda err: bsp.dense_pa_decode_fp8(c, q, bsp.FP8_E4M3 if q8 else bsp.BF16, group, table, seq, rl, q_len,
                                               out=out, ws=ws, dev_err=err)


CASES = [(prompt, ((100,), (100,), 1, 4)), (prompt, ((700, 31, 300), (700, 31, 2000), 2, 8)),
         (prompt, ((5, 2000), (9000, 3000), 1, 16)), (prompt, ([3] * 600, [3] * 600, 2, 1)),
         (decode, ([700, 31], 1, True)), (decode, ([2500, 128, 900], 2, False)), (decode, ([1500, 4000], 4, True)),
         (decode, ([300, 5, 900, 77], 8, False)), (decode, ([40] * 700, 1, False))]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("make,args", CASES, ids=range(len(CASES)))
def test_waits_that_give_up_end_the_call_and_reach_no_other(monkeypatch, impatient, which, make, args):
    from block_sparse_paged_score_gb300 import bsp
    call, err = make(*args), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(err).clone()
    torch.cuda.synchronize()
    assert err.item() == 0
    own = bsp.lib()
    for i in range(3):
        err.zero_()
        monkeypatch.setattr(bsp, "_lib", impatient[which])
        t = time.perf_counter()
        call(err)
        monkeypatch.setattr(bsp, "_lib", own)
        # the very next kernel takes over the shared memory and TMEM
        got = call(err)
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        # the drain has a limit of about a second for each barrier: it did not need one
        assert t < 0.9, t
        assert torch.equal(got, want), i
        assert err.item() in ((TIMEOUT,) if which == 0 else (0, TIMEOUT))
