"""Drafted trees and pages at the edges of what the calls allow: values at the ends of their types, infinities, scales
far from one, streams, graphs and threads."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R
from tests.test_gpu_tree import Batch, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


# ---- lengths at the ends of their type ---------------------------------------------------------------

LOWEST = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 5, 2 ** 31 - 1]


@pytest.mark.parametrize("L", LOWEST)
@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1)])
def test_a_length_whose_difference_to_the_nodes_passes_the_type(kv, flags, L):
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([100, 300, 90], [6, 4, 3], kv=kv, flags=flags, heads=16)
    good, good_lse = b.decode()
    b.lens[1] = L
    o, lse = b.decode()
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    others = [0, 1, 2, 3, 4, 5, 10, 11, 12]
    assert torch.equal(o[others], good[others]) and torch.equal(lse[others], good_lse[others])
    assert (o[6:10] == 0).all() and (lse[6:10] == float("-inf")).all()


@pytest.mark.parametrize("L", LOWEST[:3])
def test_prepare_and_keep_refuse_such_a_length(L):
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([100, 300, 90], [6, 7, 3], heads=1)
    b.lens[1] = L
    b.trees.seq_idx.fill_(1)
    b.trees.prepare(b.lens)
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    assert b.trees.seq_idx.tolist() == [0] * 6 + [-1] * 7 + [2] * 3
    before = b.cache.kv_pool.clone()
    new = b.trees.keep([b.cache], b.table, b.lens, dev([[0, 1], [1, 3], [0, 1]]), dev([2, 2, 1]))
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    assert new.tolist() == [102, L, 91]
    assert torch.equal(b.cache.kv_pool.view(torch.int16), before.view(torch.int16))


# ---- refusals that need a device ---------------------------------------------------------------------

def test_host_tensors_among_device_ones_are_refused():
    from mla_latent_kv_mqa_b200 import layer as L, pages as P
    b = Batch([100, 30], [6, 4], heads=4)
    with pytest.raises(ValueError):
        b.decode(o_lat=torch.zeros(10, 4, 512))
    with pytest.raises(ValueError):
        b.decode(lse=torch.zeros(10, 4))
    for ws in (torch.zeros(1 << 26, dtype=torch.uint8), torch.zeros(1 << 24, device="cuda")):
        with pytest.raises(ValueError):
            b.decode(workspace=ws)
    keep, num = dev([[0], [0]]), dev([1, 1])
    other = L.PagedLatentCache(b.dims, b.cache.num_blocks, device="cpu")
    with pytest.raises(ValueError):
        b.trees.keep([b.cache, other], b.table, b.lens, keep, num)
    seqs = P.PagedSequences(64, 2, 4, b.cache.num_blocks)
    for moves in ((dev([0, 1]), dev([1])), (dev([[0, 1, 2]]), dev([1])), (dev([[0, 1]]), dev([])), (torch.zeros(1, 2, dtype=torch.int32), None)):
        with pytest.raises(ValueError):
            seqs.copy_pages([b.cache], moves)
    b.check(b.decode())
