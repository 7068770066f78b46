"""What sparse_attention leaves behind when a bounded wait gives up (GKR_ERR_TIMEOUT): every result is
either the right one or not written, and nothing is added to the running weights from results that were
not.  The kernels are built once more with waits that run out after few clocks (GKR_WAIT_CLOCKS); the waits
for what is under way when a CTA leaves keep their full limit, so that such a call ends by itself and
leaves the device as any other does."""
import contextlib
import importlib
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from test_gpu_mxfp4 import DEV, Case

pytestmark = pytest.mark.gpu
ALL_RUN_OUT = -1        # clocks: only what is complete at once counts
SOME_RUN_OUT = (4000, 5000)   # about what the first records take to come


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

    jobs = [(s, limit) for s in b.sources() for limit in (limits if s.stem == "attention" else (None,))]
    with ThreadPoolExecutor(8) as ex:
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
    out = {}
    for limit in limits:
        out[limit] = tmp / f"libgkr{limit}.so"
        used = [str(o) for (_, x), o in objs.items() if x in (None, limit)]
        subprocess.run([b.nvcc(), *b.ARCH, "-shared", "-cudart", "static", "-o", str(out[limit]), *used],
                       check=True, capture_output=True)
    return out


@contextlib.contextmanager
def library(path):
    from gather_kv_rope_gb300 import _binding as b
    kept = b._lib, b.LIB
    b._lib, b.LIB = None, path
    try:
        yield
    finally:
        b._lib, b.LIB = kept


# many whole queries, cut ones of few and of many pieces, both widths of the weights' kernel
@pytest.mark.parametrize("Q,H,K", [(64, 128, 130), (5, 128, 1000), (3, 16, 700), (1, 64, 9000), (200, 8, 70)])
@pytest.mark.parametrize("limit,times", [(ALL_RUN_OUT, 2)] + [(x, 12) for x in SOME_RUN_OUT])
def test_results_are_right_or_not_written(gkr, libraries, Q, H, K, limit, times):
    c = Case(gkr, Q, H, K, seed=Q + K)
    size = max(gkr.sparse_attention_workspace(H, Q, K), 16)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    want_w = c.weights.clone()
    want, want_lse = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=want_w, workspace=ws)
    other = c.q.flip(0).flip(1).neg()
    for _ in range(times):
        # the workspace holds another call's pieces: they look like results
        gkr.sparse_attention(other, c.cache, c.indices, -c.sm, workspace=ws)
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        w = c.weights.clone()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        with library(libraries[limit]):
            gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, out=out, lse=lse, weights=w, workspace=ws,
                                 err_flag=err)
            torch.cuda.synchronize()
        missing = torch.isnan(lse)
        assert int(err.item()) in (0, gkr.ERR_TIMEOUT)
        assert torch.equal(lse[~missing], want_lse[~missing])
        assert torch.equal(out[~missing], want[~missing])
        assert (out[missing] == 7.0).all()
        kept, added = w == c.weights, w == want_w
        assert (kept | added).all()
        assert kept[missing.any(1)].all()
        if missing.any() or not added.all():
            assert int(err.item()) == gkr.ERR_TIMEOUT
        if limit == ALL_RUN_OUT:
            assert missing.all() and kept.all()
    # and the device is as before
    again_w = c.weights.clone()
    again, again_lse = gkr.sparse_attention(c.q, c.cache, c.indices, c.sm, weights=again_w, workspace=ws)
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse) and torch.equal(again_w, want_w)
