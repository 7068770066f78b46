"""What prefix_attention leaves behind when a bounded wait gives up (GKR_ERR_TIMEOUT) where the prefix is read once
for all queries and joined with lists of their own: a row whose prefix part, own part or any piece of them was left
out is not written, and its lse is a NaN of its own; any other row is right.  As in test_gpu_prompt_timeout the
kernels are built with waits that run out after few clocks, while those for what is under way when a CTA leaves keep
their full limit; here those of the own lists, those of the prefix, and both."""
import importlib
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import test_gpu_prefix
from test_gpu_attention_timeout import library
from test_gpu_prompt_timeout import ALL_RUN_OUT, DEV, check

pytestmark = pytest.mark.gpu
# clocks of the own lists' waits and of the prefix's (None: the full limit); those between are about what the first
# rows take to come, so that some rows are missing and some are not
LIMITS = [(ALL_RUN_OUT, None), (5000, None), (9000, None), (None, ALL_RUN_OUT), (None, 8000), (None, 10000),
          (None, 16000), (9000, 16000)]
# tiles whole and cut, own lists whole and cut; the first and a middle query have no records of their own
SIZES = [(230, 16, 3000, 40), (100, 16, 2000, 1000), (400, 64, 900, 70), (1000, 2, 130, 100)]


@pytest.fixture(scope="module")
def libraries(gkr, tmp_path_factory):
    """{limits: library}."""
    b = importlib.import_module("gather_kv_rope_gb300.build")
    tmp = tmp_path_factory.mktemp("short_waits")

    def run(*args):
        subprocess.run([b.nvcc(), *b.ARCH, *map(str, args)], check=True, capture_output=True)

    def compile_one(job):
        src, limit = job
        obj = tmp / f"{src.stem}{limit}.o"
        defines = [] if limit is None else [f"-DGKR_WAIT_CLOCKS={limit}"]
        run(*b.NVCC_FLAGS, *defines, "-c", src, "-o", obj)
        return obj

    def limit_of(src, limits):
        return {"attention": limits[0], "prompt": limits[1]}.get(src.stem)

    jobs = sorted({(s, limit_of(s, x)) for s in b.sources() for x in (*LIMITS, (None, None))}, key=str)
    with ThreadPoolExecutor(8) as ex:
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
    out = {}
    for x in LIMITS:
        out[x] = tmp / f"libgkr{x[0]}_{x[1]}.so"
        run("-shared", "-cudart", "static", "-o", out[x], *(objs[(s, limit_of(s, x))] for s in b.sources()))
    return out


@pytest.mark.parametrize("Q,H,L,K", SIZES)
@pytest.mark.parametrize("limits", LIMITS)
def test_joined_rows_are_right_or_not_written(gkr, libraries, Q, H, L, K, limits):
    size = gkr.prefix_attention_workspace(H, Q, L, K)
    assert size != gkr.sparse_attention_workspace(H, Q, L + K)    # every list with the prefix in front
    c = test_gpu_prefix.Case(gkr, Q, H, L, K, seed=Q + K, empty=(0, Q // 2))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    q, cache, prefix, indices, sm = c.args
    other = q.flip(0).flip(1).neg()

    def call(out, lse, err):
        gkr.prefix_attention(q, cache, prefix, indices, sm, out=out, lse=lse, workspace=ws, err_flag=err)

    def spoil():
        gkr.prefix_attention(other, cache, prefix, indices, -sm, workspace=ws)

    check(gkr, libraries, limits, 2 if ALL_RUN_OUT in limits else 8, call, spoil, (Q, H))
    if ALL_RUN_OUT in limits:        # one part of every row is missing
        out, lse, err = torch.full_like(q, 7.0), torch.zeros(Q, H, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        with library(libraries[limits]):
            call(out, lse, err)
            torch.cuda.synchronize()
        assert torch.isnan(lse).all() and (out == 7.0).all() and int(err.item()) == gkr.ERR_TIMEOUT
