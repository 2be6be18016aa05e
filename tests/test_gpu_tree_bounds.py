"""The drafted-tree attention against its formula in 64 bits, each kernel held to what it rounds (tests/tree_bounds.py):
few tokens, where a weight's rounding shows whole, and many."""
import numpy as np
import pytest
import torch

from tests import tree_bounds as T, tree_ref as R
from tests.test_gpu_tree import TOY, V3, Batch, no_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


def check(b, got, out="f32", sample=9):
    o, lse = got
    worst = 0.0
    for s in range(b.B):
        nodes = np.unique(np.linspace(0, b.n[s] - 1, min(sample, b.n[s])).astype(int))
        t, (ro, rl, size, reach) = b.reference(s, nodes)
        bound = T.o_bound(ro, size, reach, b.row, int(b.ctx[s] + b.n[s]), out == "bf16", T.kind_of(b))
        lb = R.lse_bound(rl, reach, b.row)
        if T.kind_of(b) == "fp8":
            bound = bound + 2 * size * b.extra[0][..., None] + b.extra[1]
            lb = lb + b.extra[0]
        worst = max(worst, float(((o[t].double() - ro).abs() / bound).max()))
        assert ((lse[t].double() - rl).abs() <= lb).all()
    assert worst <= 1, worst
    no_error()


@pytest.mark.parametrize("kv,act,shape,flags", [("bf16", "bf16", V3, 0), ("fp8", "bf16", V3, 0), ("bf16", "bf16", V3, 1), ("fp8", "bf16", V3, 1),
                                                ("f32", "f32", TOY, 0)])
@pytest.mark.parametrize("ctx,n,heads", [([1], [1], 128), ([2, 3, 0], [1, 3, 7], 128), ([5, 9], [2, 30], 20), ([250, 700], [3, 2], 64),
                                         ([4000], [3], 16), ([9000], [2], 64)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("spread", [1.0, 6.0])
def test_each_kernel_rounds_what_it_says(kv, act, shape, flags, ctx, n, heads, out, spread):
    b = Batch(ctx, n, heads=heads, kv=kv, act=act, shape=shape, flags=flags, seed=91, spread=spread)
    check(b, b.decode(out), out)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,n,heads", [([70000, 66001], [4, 3], 128), ([70000, 300, 33000], [4, 1, 9], 64), ([40000] * 3, [1, 1, 1], 128),
                                         ([66000, 5], [40, 2], 16)])
def test_long_sequences_with_tiles_that_share_them_and_without(kv, ctx, n, heads):
    b = Batch(ctx, n, heads=heads, kv=kv, seed=95)
    first = b.decode()
    check(b, first, sample=2)
    assert all(torch.equal(x, y) for x, y in zip(first, b.decode()))


@pytest.mark.parametrize("ctx", [3, 300, 5000])
@pytest.mark.parametrize("power", [-70, -90, -100, -140, 50, 100])
@pytest.mark.parametrize("flags", [0, 1])
def test_scales_far_from_one(ctx, power, flags):
    """All scales times a power of two, down to denormals.  fp16 keeps 2^-27 of the row's largest weight times scale,
    or of 2^-80 where that is larger.  A query's content is taken to 2^-17 of its row's largest, or of 2^-61 where
    that is larger: the row is multiplied by 2^68 at most, and behind its nearest e4m3 value the rest is off by half of
    e4m3's smallest step, 2^-10, so an element by 2^-78.  (power 100 passes that by far: weights are any then.)"""
    b = Batch([ctx], [4], heads=24, kv="fp8", flags=flags, seed=93)
    b.cache.kv_scale.mul_(2.0 ** power)
    if power > 0:
        b.q[:, :, :512] *= 2.0 ** -power
    o, lse = b.decode()
    t, (ro, rl, size, reach) = b.reference(0)
    bound = T.o_bound(ro, size, reach, b.row, ctx + 4, False, T.kind_of(b)) + 2.0 ** -149
    lb = R.lse_bound(rl, reach, b.row)
    if T.kind_of(b) == "fp8":
        ds, da = b.extra
        ds = ds * (2.0 ** -61 / b.q[t][..., :512].double().abs().amax(-1)).clamp(min=1)
        largest = float(b.cache.kv_scale[b.owned[0]].nan_to_num(0).max())
        bound = bound + 2 * size * ds[..., None] + da * max(1.0, 2.0 ** -80 / largest)
        lb = lb + ds
        if float(ds.max()) > 0.1:                                    # 2 ds is the first order of exp(2 ds) - 1
            bound = torch.full_like(bound, 2 * 448 * largest)
    assert torch.isfinite(o[t]).all()
    worst = float(((o[t].double() - ro).abs() / bound).max()), float(((lse[t].double() - rl).abs() / lb).max())
    assert max(worst) <= 1, worst
    if power > -110:
        assert (o[t] != 0).any()
    no_error()
