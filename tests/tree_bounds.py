"""Bounds of mla_decode_tree's errors by what each kernel rounds, once each:

  a score      row + 1 roundings in fp32 of terms whose sum of sizes is `reach`, twice that where the tensor core
               truncates; it moves every weight by as much, the sum of the weights again
  exp2         2^-21 each, weight and sum
  P            "bf16": 2^-8, over a bf16 cache on the tensor cores; "fp8": 2^-11, P times the scale as fp16 (what fp16 has
               no 11 bits for is tree_ref.fp8_terms'); "cores": fp32
  the sums     of L weights times values: a rounding a token on the CUDA cores; on the tensor cores one of 16 tokens at a
               time, each of 2 units in the last place at most, truncated: 4 half steps; a few more where runs are joined
  the output   once
"""
from tests import tree_ref as R

P_ROUNDING = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -11, "cores": 2.0 ** -24}


def o_bound(o, size, reach, row, L, out_bf16, kind):
    ds = (row + 1) * R.EPS_F32 * 2 * reach
    sums = (64 + (L if kind == "cores" else L / 4)) * R.EPS_F32
    rel = 2 * ds[..., None] + 2.0 ** -20 + sums + P_ROUNDING[kind]
    return size * rel + (R.EPS_BF16 if out_bf16 else R.EPS_F32) * o.abs() + 1e-30


def kind_of(batch):
    return "cores" if not batch.tensor_core() else "fp8" if batch.kv == "fp8" else "bf16"
