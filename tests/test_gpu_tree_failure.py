"""The failure path of mla_decode_tree on the GPU, without a fault: MLA_FLAG_TEST_GIVE_UP lets a short wait run out
in every pair of SMs that has two steps or more.  The call returns, the error word says so, nothing outside the
outputs is written, whatever the workspace held, and the next call is exact."""
import time

import pytest
import torch

from tests.test_gpu_tree import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,n,heads", [([40000], [3], 16), ([6000, 3000, 10, 9000], [40, 17, 3, 64], 128), ([33000, 17001], [4, 3], 128),
                                         ([300] * 400, [1] * 400, 128)])
@pytest.mark.parametrize("fill", [0, 0x3F, 0xFF])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_exact(kv, ctx, n, heads, fill):
    from mla_latent_kv_mqa_b200 import layer as L, native as N
    b = Batch(ctx, n, heads=heads, kv=kv, seed=3)
    want, want_lse = b.decode()
    assert N.mla_get_last_device_error() == N.MLA_OK
    guard = 1 << 16
    rows = b.T * heads
    big_o = torch.full((rows * 512 + 2 * guard,), 5.0, device="cuda")
    big_l = torch.full((rows + 2 * guard,), 6.0, device="cuda")
    o = big_o[guard:guard + rows * 512].view(b.T, heads, 512)
    lse = big_l[guard:guard + rows].view(b.T, heads)
    need = N.mla_decode_tree_workspace_size(b.dims, b.B, b.T, b.max_len)
    ws = torch.full((need + 2 * guard,), fill, dtype=torch.uint8, device="cuda")
    at = guard + -(ws.data_ptr() + guard) % 256
    work = ws[at:at + need]
    bad = L.dims_for(heads, 128, 512, 64, kv=kv, flags=N.MLA_FLAG_TEST_GIVE_UP)
    c = b.cache

    def call(dims):
        N.mla_decode_tree(dims, b.B, b.trees.cu_nodes, b.T, b.most, b.q, c.kv_pool, c.kr_pool, c.kv_scale, b.table,
                          b.table.shape[1], c.num_blocks, b.lens, b.max_len, b.trees.mask, b.trees.mask_words, work, need, o,
                          N.MLA_DTYPE_F32, lse)
        torch.cuda.synchronize()

    t0 = time.perf_counter()
    call(bad)
    assert time.perf_counter() - t0 < 10.0
    assert N.mla_get_last_device_error() == N.MLA_ERR_DEVICE_TIMEOUT
    assert (big_o[:guard] == 5).all() and (big_o[-guard:] == 5).all()
    assert (big_l[:guard] == 6).all() and (big_l[-guard:] == 6).all()
    assert (ws[:at] == fill).all() and (ws[at + need:] == fill).all()
    call(b.dims)
    assert N.mla_get_last_device_error() == N.MLA_OK
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
