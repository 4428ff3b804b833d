"""Shared by the cache and attention tests: seeded ragged batches and the error
bounds of the attention results, derived from the roundings that occur."""
import numpy as np
import torch

from oracle import kv as okv

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def random_cache(r, blocks, H, block, D, spread=3):
    """Finite random codes of normal values, exponents within `spread` binades."""
    def codes(*shape):
        x = torch.from_numpy((r.standard_normal(shape) * 80).clip(-448, 448).astype(np.float32))
        return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()

    def exps():
        return r.integers(119, 119 + spread, (blocks, H)).astype(np.uint8)

    return okv.Cache(codes(blocks, H, block, D), codes(blocks, H, block // 16, D, 16), exps(), exps())


def batch(r, n, lens, block, blocks=None, extra=1):
    """(cu, lens, table, blocks) of a ragged batch; every sequence has its own
    shuffled blocks, `extra` more columns than the longest needs."""
    need = [-(-L // block) for L in lens]
    blocks = blocks or sum(need) + 2
    order = r.permutation(blocks)
    table = np.zeros((len(lens), max(max(need), 1) + extra), dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return cu, np.array(lens, dtype=np.int32), table, blocks


def to_dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def dev_cache(c):
    from column_scaled_gemm_amd import fp8sm
    return fp8sm.KVCache(*to_dev(c.codes[0], c.codes[1], c.exp[0], c.exp[1]))


def attention_bounds(ref, lse, spread, qk, scale, D, length, dtype):
    """Largest allowed |out - ref| and |lse - ref|.

    u = 2^-24.  A score is a sum of D products taken in fp32 in any order, each
    step rounded or truncated (2u), times scale * log2(e) (two roundings of up to
    u each, relative): ds = 2 (D + 2) u scale sum|q||k|.  The exponent's
    difference to the running maximum rounds again and the hardware 2^x is
    within 2 ulp; the factors that rescale a sum when the maximum moves add such
    an error a few times over: dp = 2 ds + 16 u (1 + range), with the range of
    the scores at most 2 scale sum|q||k|.  p is rounded to 16 bits for the
    product (2^-8 of it for bf16 calls, 2^-11 for fp16 ones) but not for the sum
    l; the sums over `length` tokens add 2u each.  The result is rounded to its
    type once: half a step, 2^-8 or 2^-11, and for fp16 at most 2^-25 absolute
    below its normal range.  A factor 1.01 covers the products of these.
    """
    u = 2.0 ** -24
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    ds = 2 * (D + 2) * u * scale * qk
    dp = 2 * ds + 16 * u * (1 + 2 * scale * qk)
    rel = dp + half + 4 * length * u
    out = 1.01 * (spread * rel[..., None] + np.abs(ref) * half) + 2.0 ** -24
    with np.errstate(invalid="ignore"):
        dl = ds + dp + 4 * length * u + 8 * u * np.abs(lse)
    return out, 1.01 * dl
