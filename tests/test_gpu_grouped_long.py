"""The block-scaled product over routed experts' rows at the batches that a
grid of its tiles holds: the choice on the host (CPU), and batches of more
16-row blocks x 16 columns than the few-row kernel's grid holds, which the
tiles take, against the formula in 64 bits (tolerances as in
test_gpu_fp8_block)."""
import ctypes
import math
import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_fp8_block import _rand, block_rows, block_weights
from tests.test_gpu_linear import reference


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    """The host's count of a grouped call's threads, compiled alone."""
    d = tmp_path_factory.mktemp("plan")
    src = d / "plan.cpp"
    src.write_text('#include "%s"\n' % os.path.join(ROOT, "fp4_expert_ffn_amd", "csrc", "linear_block_plan.h") + """
extern "C" long long threads(int T, int E, int N, int gated, int K, int exact, int fits) {
  return moe::grouped_threads(T, E, N, gated != 0, K, exact != 0, fits != 0);
}
""")
    out = str(d / "plan.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(out).threads
    f.restype = ctypes.c_longlong
    return f


# rows, experts, columns, gated: 32768 and 65535 tokens by 8 of 256, the largest route of 1024 experts, one expert
@pytest.mark.parametrize("T,E,N,gated", [(262144, 256, 7168, 0), (524280, 256, 4096, 0), (524280, 256, 8192, 1),
                                         (131072, 1024, 16384, 1), (1 << 20, 1, 16384, 0), (150000, 8, 7200, 1)])
def test_long_batches_fit_a_grid(threads, T, E, N, gated):
    for K in (128, 256, 2048):
        for exact in (0, 1):
            assert 0 < threads(T, E, N, gated, K, exact, 1) < 2 ** 32, (K, exact)


def test_what_no_grid_holds(threads):
    for fits in (0, 1):
        assert threads(1 << 23, 4, 100000, 0, 128, 0, fits) >= 2 ** 32
    # 16 x 16 outputs for 256 and, from K = 4096 on, 512 threads
    assert threads(1 << 16, 1, 65536 - 16, 0, 2048, 0, 0) < 2 ** 32 <= threads(1 << 16, 1, 65536 - 16, 0, 4096, 0, 0)
    assert threads(1, 1, 16, 0, 128, 0, 1) == 256 and threads(0, 4, 16, 0, 128, 0, 1) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("gated,K", [(False, 256), (True, 384)])
def test_more_rows_than_a_grid_of_small_tiles(gated, K):
    """150000 rows of 8 experts, 7200 columns: 4.2 million blocks of 16 x 16; every 97th row and both ends of every
    expert's, all columns."""
    need_gpu()
    import fp4_expert_ffn_amd as m
    T, E, N, k = 150000, 8, 7200, 8
    R = 2 * N if gated else N
    w = [block_weights(_rand(e + 1, R, K) / math.sqrt(K), 2 if gated else 1) for e in range(2)]  # two slots for all
    wq = torch.stack([q.view(torch.uint8) for q, _, _ in w]).view(torch.float8_e4m3fn).to(DEV)
    ws = torch.stack([s for _, s, _ in w]).to(DEV)
    wv = [v.to(DEV) for _, _, v in w]
    xq, xs, xv = (t.to(DEV) for t in block_rows(_rand(5, T // k, K)))
    at = torch.tensor([0, 31000, 31001, 31001, 77777, 120000, 120127, 149900, T - 3])  # three rows behind the last
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(7)).int().to(DEV)
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    slot = torch.tensor([e % 2 for e in range(E)], dtype=torch.int32, device=DEV)
    say("grouped, long batch", gated, K)
    m.moe_linear_grouped(m.grouped_args(x=xq, x_scale=xs, w=wq, w_scale=ws, offsets=at.int().to(DEV), rows=perm,
                                        rows_div=k, slot_of_expert=slot, act="silu" if gated else "none", gated=gated, out=out))
    torch.cuda.synchronize()
    for e in range(E):
        lo, hi = int(at[e]), int(at[e + 1])
        rows = torch.tensor(sorted(set(range(lo, hi, 97)) | set(range(lo, min(lo + 2, hi))) | set(range(max(hi - 2, lo), hi))),
                            dtype=torch.long, device=DEV)
        if len(rows):
            want, tol = reference(xv[perm[rows].long() // k], wv[e % 2], None, "silu" if gated else "none", gated, None, N, K, True)
            bad = ~((out[rows].double() - want).abs() <= tol + want.abs() * 2.0 ** -8 + 1e-30)
            assert not bad.any(), (e, int(bad.sum()), torch.nonzero(bad)[:4])
    assert torch.all(out[T - 3:] == 7.0)
