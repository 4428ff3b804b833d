"""Head norm + rotation and the E4M3 cache against the 64-bit oracle: codes and
exponents exactly, widened values exactly, the rotation within its roundings."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from kv_util import DT, batch, dev_cache, random_cache, rng, to_dev
from oracle import kv as okv

pytestmark = pytest.mark.gpu


def table_of(P, rot):
    ang = np.arange(P)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,norm,inter,dtype", [
    (1, 1, 0, 128, 128, True, False, "bf16"), (1, 0, 1, 64, 64, True, True, "fp16"),
    (5, 4, 1, 128, 64, True, False, "fp16"), (3, 7, 7, 64, 16, False, False, "bf16"),
    (33, 17, 3, 128, 128, True, True, "bf16"), (9, 40, 8, 64, 32, True, False, "bf16"),
    (4, 5, 5, 128, 16, False, True, "fp16"), (2, 3, 2, 128, 0, True, False, "bf16"),
    (257, 9, 1, 64, 48, True, False, "fp16"), (6, 65, 2, 128, 96, True, False, "bf16")])
def test_norm_rope(T, Hq, Hk, D, rot, norm, inter, dtype):
    print(f"[case] rope {T} {Hq} {Hk} {D} {rot} {norm} {inter} {dtype}", flush=True)
    r = rng(T * 1000 + Hq)
    dt, W = DT[dtype], (Hq + Hk) * D
    x = torch.from_numpy(r.standard_normal((T, W + 24)).astype(np.float32)).to(dt)
    x[T // 2, :D] *= 0     # an all-zero head
    wq, wk = (torch.from_numpy(r.standard_normal(D).astype(np.float32)).to(dt) for _ in range(2))
    P = 5000
    pos = r.integers(0, P, T).astype(np.int32)
    if T > 3:
        pos[1], pos[2] = -1, P      # padding
    cs = table_of(P, rot) if rot else None
    args = dict(q_weight=wq.cuda(), k_weight=wk.cuda()) if norm else {}
    out = torch.full((T, W + 8), 7.0, dtype=dt, device="cuda")
    got = fp8sm.qk_norm_rope(x.cuda(), Hq, Hk, D, to_dev(pos)[0], to_dev(cs)[0] if rot else None,
                             interleaved=inter, out=out, **args)
    ref, mag = okv.norm_rope(x.double().numpy(), Hq, Hk, D, pos, cs, wq.double().numpy() if norm else None,
                             wk.double().numpy() if norm else None, 1e-6, inter)
    assert got is out and torch.all(out[:, W:] == 7)
    g = got[:, :W].double().cpu().numpy().reshape(ref.shape)
    pad = np.isnan(ref).all((1, 2))
    assert np.all(g[pad] == 7)
    # one rounding to the type, half a step; in fp32 before it, relative to the
    # summands: the mean of D squares (D + 2 roundings, halved by the root), root
    # and reciprocal (4), the weight, product and sum (4): D / 2 + 10 roundings
    half = torch.finfo(dt).eps / 2
    tol = 1.01 * (np.abs(ref) * half + mag * (D / 2 + 10) * 2.0 ** -24) + 2.0 ** -25
    assert np.all(np.abs(g - ref)[~pad] <= tol[~pad]), np.nanmax(np.abs(g - ref) / tol)


def test_norm_rope_in_place_leaves_the_value_heads():
    r = rng(8)
    x = torch.from_numpy(r.standard_normal((70, 4 * 128 + 3 * 128 * 2)).astype(np.float32)).to(torch.bfloat16).cuda()
    pos, cs = to_dev(np.arange(70, dtype=np.int32), table_of(70, 128))
    want = fp8sm.qk_norm_rope(x, 4, 3, 128, pos, cs)
    y = x.clone()
    assert fp8sm.qk_norm_rope(y, 4, 3, 128, pos, cs, out=y) is y
    assert torch.equal(y[:, :7 * 128], want) and torch.equal(y[:, 7 * 128:], x[:, 7 * 128:])


def check_cache(dev, ref):
    for g, c in ((dev.k, ref.codes[0]), (dev.v, ref.codes[1]), (dev.k_exp, ref.exp[0]), (dev.v_exp, ref.exp[1])):
        assert np.array_equal(g.cpu().numpy(), c)


CASES = [  # n, lens, H, D, block, dtype
    ([1], [1], 1, 64, 16, "bf16"),
    ([1, 1, 1, 1], [1, 16, 17, 32], 2, 128, 16, "bf16"),
    ([5, 0, 16, 1], [37, 9, 16, 50], 3, 64, 16, "fp16"),
    ([33, 7, 64], [40, 7, 100], 2, 128, 32, "fp16"),
    ([130, 1, 3], [131, 64, 66], 1, 64, 64, "bf16"),
    ([200, 129, 2], [290, 129, 300], 5, 128, 128, "bf16"),
    ([100, 28], [300, 28], 1, 64, 128, "fp16"),
]


@pytest.mark.parametrize("n,lens,H,D,block,dtype", CASES)
def test_write_and_read(n, lens, H, D, block, dtype):
    print(f"[case] write {n} {lens} {H} {D} {block} {dtype}", flush=True)
    r = rng(sum(lens))
    cu, L, table, blocks = batch(r, n, lens, block)
    ref = random_cache(r, blocks, H, block, D, spread=8)
    T = sum(n)
    rows = torch.from_numpy((r.standard_normal((T, 3 * H * D)) * np.exp(r.uniform(-3, 3, (T, 1)))).astype(np.float32)).to(DT[dtype])
    k, v = rows[:, H * D:2 * H * D], rows[:, 2 * H * D:].unflatten(1, (H, D))
    rd = rows.cuda()
    kd, vd = rd[:, H * D:2 * H * D], rd[:, 2 * H * D:].unflatten(1, (H, D))
    dev = dev_cache(ref)
    d = to_dev(cu, L, table)
    fp8sm.kv_cache_write(kd, vd, dev, *d)
    okv.write(ref, k.double().numpy().reshape(T, H, D), v.double().numpy(), cu, L, table)
    check_cache(dev, ref)           # what is not the batch's is as it was, too
    fp8sm.kv_cache_write(kd, vd, dev, *d)   # the same tokens again change nothing
    check_cache(dev, ref)
    # every cached token of every sequence, into rows wider than the heads
    cu2 = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = sum(lens) + 2
    ko = torch.full((total, H * D + 8), 3.0, dtype=DT[dtype], device="cuda")
    vo = torch.full((total, H, D), 3.0, dtype=DT[dtype], device="cuda")
    fp8sm.kv_cache_read(dev, to_dev(cu2)[0], d[1], d[2], total, dtype=DT[dtype], k=ko[:, :H * D], v=vo)
    want = okv.read(ref, cu2, L, table, total)
    for got, w in ((ko[:, :H * D].reshape(total, H, D), want[0]), (vo, want[1])):
        w = torch.from_numpy(np.where(np.isnan(w), 3.0, w)).to(DT[dtype])
        assert torch.equal(got.cpu(), w)
    assert torch.all(ko[:, H * D:] == 3)


def test_many_sequences_and_padded_or_bad_batch_data():
    """More sequences than one probe round; rows of none; lengths below the new
    tokens; lengths beyond the table; blocks that do not exist."""
    r = rng(30)
    B, H, D, block = 150, 1, 64, 16
    n = r.integers(0, 4, B)
    lens = n + r.integers(0, 40, B)
    cu, L, table, blocks = batch(r, list(n), list(lens), block)
    L[3] = max(int(n[3]) - 2, 0)
    L[5], table[5] = 10 ** 6, np.resize(np.arange(blocks, blocks + 3), table.shape[1])
    table[7, 0], table[9, 0] = -1, blocks + 5
    cu = cu + 2                     # two rows before the first sequence
    T = int(cu[-1]) + 3
    ref = random_cache(r, blocks, H, block, D)
    x = torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).to(torch.bfloat16)
    dev = dev_cache(ref)
    d = to_dev(cu, L, table)
    fp8sm.kv_cache_write(x.cuda(), x.cuda(), dev, *d)
    okv.write(ref, x.double().numpy(), x.double().numpy(), cu, L, table)
    check_cache(dev, ref)
    got = fp8sm.kv_cache_read(dev, *d, T, k=torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda"),
                              v=torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda"))
    for g, w in zip(got, okv.read(ref, cu, L, table, T)):
        assert torch.equal(g.cpu(), torch.from_numpy(np.where(np.isnan(w), 3.0, w)).to(torch.bfloat16))


def test_non_finite_and_extreme_values():
    r = rng(31)
    H, D, block = 2, 64, 16
    ref = random_cache(r, 3, H, block, D)
    x = r.standard_normal((20, H, D)).astype(np.float32)
    x[0, 0, :3] = [np.inf, -np.inf, np.nan]
    x[4] *= 1e30
    x[5] *= 1e-30
    x[17:] = 0
    x = torch.from_numpy(x).to(torch.bfloat16)
    cu, L, table = np.int32([0, 20]), np.int32([20]), np.int32([[2, 0]])
    dev = dev_cache(ref)
    fp8sm.kv_cache_write(x.cuda(), x.cuda(), dev, *to_dev(cu, L, table))
    okv.write(ref, x.double().numpy(), x.double().numpy(), cu, L, table)
    for g, c in ((dev.k, ref.codes[0]), (dev.v, ref.codes[1])):
        g = g.cpu().numpy()
        nan = (c & 0x7F) == 0x7F
        assert np.array_equal(nan, (g & 0x7F) == 0x7F) and np.array_equal(g[~nan], c[~nan])
    assert np.array_equal(dev.k_exp.cpu().numpy(), ref.exp[0])
    # appending to it raises no exponent and keeps the NaN
    y = torch.full((1, H, D), 1e35, dtype=torch.bfloat16)
    cu, L = np.int32([0, 1]), np.int32([21])
    fp8sm.kv_cache_write(y.cuda(), y.cuda(), dev, *to_dev(cu, L, table))
    okv.write(ref, y.double().numpy(), y.double().numpy(), cu, L, table)
    assert np.array_equal(dev.v_exp.cpu().numpy(), ref.exp[1])
    assert np.array_equal(dev.v[0].cpu().numpy(), ref.codes[1][0])


@pytest.mark.parametrize("byte", [0, 1, 60, 127, 200, 247])
def test_read_of_any_exponent(byte):
    r = rng(32)
    ref = random_cache(r, 1, 1, 16, 64)
    for e in ref.exp:
        e[:] = byte
    d = to_dev(np.int32([0, 16]), np.int32([16]), np.zeros((1, 1), np.int32))
    want = okv.read(ref, [0, 16], [16], np.zeros((1, 1), np.int32), 16)
    for dtype in (torch.bfloat16, torch.float16):
        for g, w in zip(fp8sm.kv_cache_read(dev_cache(ref), *d, 16, dtype=dtype), want):
            w = torch.from_numpy(w).to(dtype)   # exact in fp64: one rounding, overflow to infinity
            assert torch.equal(g.cpu(), w)


@pytest.mark.parametrize("byte", [0, 246, 253, 254])
def test_append_to_a_block_of_any_exponent(byte):
    """A block that was written elsewhere may hold every exponent of the format."""
    r = rng(33)
    ref = random_cache(r, 1, 2, 16, 64)
    for e in ref.exp:
        e[:] = byte
    x = r.standard_normal((4, 2, 64)).astype(np.float32)
    x[0] = np.sign(x[0]) * np.float32(3e38)
    x[1] *= np.float32(3e37)
    x = torch.from_numpy(x).to(torch.bfloat16)
    cu, L, table = np.int32([0, 4]), np.int32([9]), np.int32([[0]])
    dev = dev_cache(ref)
    fp8sm.kv_cache_write(x.cuda(), x.cuda(), dev, *to_dev(cu, L, table))
    okv.write(ref, x.double().numpy(), x.double().numpy(), cu, L, table)
    for g, c in zip(dev, ref.codes + ref.exp):
        assert np.array_equal(g.cpu().numpy(), c)


def test_cache_offsets_beyond_32_bits():
    """A cache of 5 GiB a side: the blocks at its end."""
    H, D, block = 8, 128, 128
    blocks = (5 << 30) // (H * D * block)
    c = fp8sm.kv_cache_empty(blocks, H, D, block)
    r = rng(33)
    x = torch.from_numpy(r.standard_normal((150, H, D)).astype(np.float32)).to(torch.bfloat16)
    d = to_dev(np.int32([0, 150]), np.int32([150]), np.int32([[blocks - 1, blocks - 2]]))
    fp8sm.kv_cache_write(x.cuda(), x.cuda(), c, *d)
    k, v = fp8sm.kv_cache_read(c, *d, 150)
    small = random_cache(r, 2, H, block, D)
    t = np.int32([[1, 0]])
    okv.write(small, x.double().numpy(), x.double().numpy(), [0, 150], [150], t)
    for g, w in zip((k, v), okv.read(small, [0, 150], [150], t, 150)):
        assert np.array_equal(g.double().cpu().numpy(), w)
    q = x[-1:].cuda()
    d1 = to_dev(np.int32([0, 1])) + d[1:]
    out = fp8sm.attention_cache(q, c, *d1, 1)
    dev = dev_cache(small)
    assert torch.equal(out, fp8sm.attention_cache(q, dev, d1[0], d1[1], to_dev(t)[0], 1))
