"""Tiles of prompt_attention over so many rows that they take longer than the limit of an ordinary wait (2 s: 200 million
rows).  The warps that write results wait for a whole tile, with a limit of their own.  Here the kernels are
built with waits of a million clocks (0.5 ms), a hundred times what any step takes, and a tile takes several
times that."""
import importlib
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from test_gpu_attention_timeout import library

pytestmark = pytest.mark.gpu
DEV = "cuda"
CLOCKS = 1000000


@pytest.fixture(scope="module")
def short(gkr, tmp_path_factory):
    b = importlib.import_module("gather_kv_rope_gb300.build")
    tmp = tmp_path_factory.mktemp("short_waits")

    def run(*args):
        subprocess.run([b.nvcc(), *b.ARCH, *map(str, args)], check=True, capture_output=True)

    def compile_one(src):
        run(*b.NVCC_FLAGS, f"-DGKR_WAIT_CLOCKS={CLOCKS}", "-c", src, "-o", tmp / f"{src.stem}.o")
        return tmp / f"{src.stem}.o"

    with ThreadPoolExecutor(8) as ex:
        objs = list(ex.map(compile_one, b.sources()))
    run("-shared", "-cudart", "static", "-o", tmp / "libgkr.so", *objs)
    return tmp / "libgkr.so"


@pytest.mark.parametrize("queries", [1, 80])
def test_long_tiles(gkr, short, queries):
    """One request; 80 queries of 128 heads are a tile or more for each pair, a query is cut over all pairs."""
    rows = 400000 if queries > 1 else 8000000          # 3125 (822) chunks of about 2200 clocks a pair
    g = torch.Generator(device=DEV).manual_seed(queries)
    q = (2 * torch.randn(queries, 128, 512, generator=g, device=DEV)).to(torch.bfloat16)
    kv = torch.randn(1000, 512, generator=g, device=DEV).to(torch.bfloat16).repeat(rows // 1000, 1)
    starts, kv_starts = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (queries, rows))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = gkr.prompt_attention(q, kv, starts, 512 ** -0.5, kv_starts=kv_starts, causal=False, err_flag=err)
    with library(short):
        got = gkr.prompt_attention(q, kv, starts, 512 ** -0.5, kv_starts=kv_starts, causal=False, err_flag=err)
        torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # rows / 1000 times the same rows: their attention, and the log of how often
    once = gkr.prompt_attention(q, kv[:1000], starts, 512 ** -0.5, kv_starts=kv_starts.clamp(max=1000), causal=False)
    # the same terms in sums of up to a chunk's count more fp32 additions (and those of a row's threads and pieces), and
    # the roundings of lse values below 32
    off = (rows / 128 + 200) * 2.0 ** -24 + 4 * 32 * 2.0 ** -24
    assert (want[1] - once[1] - np.log(rows / 1000)).abs().max() < off
