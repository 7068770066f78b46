"""What prompt_attention and prefix_attention leave behind when a bounded wait gives up (GKR_ERR_TIMEOUT):
every row is either right or not written, with a NaN of its own as lse.  The kernels are built once more
with waits that run out after few clocks (GKR_WAIT_CLOCKS); the waits for what is under way when a CTA
leaves keep their full limit, so that such a call ends by itself and leaves the device as any other does."""
import importlib
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import test_gpu_prefix
import test_gpu_prompt
from test_gpu_attention_timeout import library

pytestmark = pytest.mark.gpu
DEV = "cuda"
ALL_RUN_OUT = -1                       # clocks: only what is complete at once counts
SOME_RUN_OUT = (2500, 4000, 6000)      # about what the first rows take to come


@pytest.fixture(scope="module")
def libraries(gkr, tmp_path_factory):
    """{limit: library}: the sources with waits of that many clocks at most."""
    b = importlib.import_module("gather_kv_rope_gb300.build")
    tmp = tmp_path_factory.mktemp("short_waits")
    limits = (ALL_RUN_OUT, *SOME_RUN_OUT)

    def compile_one(job):
        src, limit = job
        obj = tmp / f"{src.stem}{limit}.o"
        defines = [] if limit is None else [f"-DGKR_WAIT_CLOCKS={limit}"]
        subprocess.run([b.nvcc(), *b.ARCH, *b.NVCC_FLAGS, *defines, "-c", str(src), "-o", str(obj)],
                       check=True, capture_output=True)
        return obj

    jobs = [(s, limit) for s in b.sources()
            for limit in (limits if s.stem in ("attention", "prompt") else (None,))]
    with ThreadPoolExecutor(8) as ex:
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
    out = {}
    for limit in limits:
        out[limit] = tmp / f"libgkr{limit}.so"
        used = [str(o) for (_, x), o in objs.items() if x in (None, limit)]
        subprocess.run([b.nvcc(), *b.ARCH, "-shared", "-cudart", "static", "-o", str(out[limit]), *used],
                       check=True, capture_output=True)
    return out


def check(gkr, libraries, limit, times, call, spoil, shape):
    """call(out, lse, err) under the limit against the same without one; spoil() fills the workspace with
    another call's results."""
    want, want_lse = torch.empty(*shape, 512, dtype=torch.bfloat16, device=DEV), torch.empty(*shape, device=DEV)
    call(want, want_lse, None)
    for _ in range(times):
        spoil()
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        with library(libraries[limit]):
            call(out, lse, err)
            torch.cuda.synchronize()
        missing = torch.isnan(lse)
        assert int(err.item()) in (0, gkr.ERR_TIMEOUT)
        assert torch.equal(lse[~missing], want_lse[~missing])
        assert torch.equal(out[~missing], want[~missing])
        assert (out[missing] == 7.0).all()
        if missing.any():
            assert int(err.item()) == gkr.ERR_TIMEOUT
        if limit == ALL_RUN_OUT:
            assert missing[torch.isfinite(want_lse)].all()
    again, again_lse = torch.empty_like(want), torch.empty_like(want_lse)
    call(again, again_lse, None)
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse)


LIMITS = [(ALL_RUN_OUT, 2)] + [(x, 10) for x in SOME_RUN_OUT]


# whole tiles, cut ones of few and of many pieces, tiles without rows, a single query
@pytest.mark.parametrize("added,past,H", [
    ([1], 0, 1), ([60], 0, 16), ([1], 5000, 128), ([700], 0, 64), ([300, 5, 200], [0, 900, -250], 32),
    ([1] * 100, 300, 128)])
@pytest.mark.parametrize("limit,times", LIMITS)
def test_prompt_rows_are_right_or_not_written(gkr, libraries, added, past, H, limit, times):
    c = test_gpu_prompt.Case(added, past, H, seed=sum(added))
    ws = torch.zeros(gkr.prompt_attention_workspace(H, c.T), dtype=torch.uint8, device=DEV)
    q, kv, starts, sm, kv_starts, causal = c.args()
    other = q.flip(0).flip(1).neg()

    def call(out, lse, err):
        gkr.prompt_attention(q, kv, starts, sm, kv_starts, causal, out=out, lse=lse, workspace=ws, err_flag=err)

    def spoil():
        gkr.prompt_attention(other, kv, starts, -sm, kv_starts, causal, workspace=ws)

    check(gkr, libraries, limit, times, call, spoil, (c.T, H))


@pytest.mark.parametrize("Q,H,L,K", [(40, 128, 2000, 90), (100, 16, 3000, 0), (3, 16, 700, 50)])
@pytest.mark.parametrize("limit,times", LIMITS)
def test_prefix_rows_are_right_or_not_written(gkr, libraries, Q, H, L, K, limit, times):
    c = test_gpu_prefix.Case(gkr, Q, H, L, K, seed=Q + K)
    ws = torch.zeros(max(16, gkr.prefix_attention_workspace(H, Q, L, K)), dtype=torch.uint8, device=DEV)
    q, cache, prefix, indices, sm = c.args
    other = q.flip(0).flip(1).neg()

    def call(out, lse, err):
        gkr.prefix_attention(q, cache, prefix, indices, sm, out=out, lse=lse, workspace=ws, err_flag=err)

    def spoil():
        gkr.prefix_attention(other, cache, prefix, indices, -sm, workspace=ws)

    check(gkr, libraries, limit, times, call, spoil, (Q, H))
