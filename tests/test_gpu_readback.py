"""GPU parity of the caches read back as bf16 rows: FP4 entries (contiguous and paged, ranges and ids) and FP8 window
rows, bit-exact against the oracle's dequantisation rounded as the header states."""
import numpy as np
import pytest
import torch

from csa_workloads import gen, normal
from oracle import csa_oracle as O
from tests.cmp_utils import f64, np_u8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def fp4_rows(codes, scales, rope, d_n, g):
    """bf16(fp32(e2m1 * e4m3 * g)) of every entry, the RoPE slice as it is."""
    v = O.dequant_fp4(codes, scales, d_n, 1.0).astype(np.float32) * np.float32(g)
    return np.concatenate([O.bf16_round(v.astype(np.float64)), rope], -1)


def paged_table(B, width, seed):
    return torch.as_tensor(np.random.default_rng(seed).permutation(B * width + 2)[: B * width].reshape(B, width).astype(np.int32))


CASES = [  # B, n_max, d, d_r, g, page
    (1, 1, 512, 64, 1.0, 0), (3, 130, 512, 64, 2.0 ** -4, 0), (2, 77, 128, 32, 0.05, 0), (2, 40, 128, 0, 1.0, 0),
    (2, 300, 512, 64, 1.0, 128), (3, 700, 512, 64, 0.3, 256), (2, 9, 96, 0, 1.0, 0), (1, 5, 64, 64, 1.0, 0)]


@pytest.mark.parametrize("B,n_max,d,d_r,g,page", CASES)
def test_fp4_read_back(cuda_lib, B, n_max, d, d_r, g, page):
    csa = cuda_lib
    src = normal((B, n_max, d), 1.0, gen(n_max)).to(DEV)
    if page:
        width = -(-n_max // page)
        cache = csa.PagedCache(B, n_max, d, d_r, DEV, page, B * width + 2, paged_table(B, width, n_max), g)
    else:
        cache = csa.PackedCache(B, n_max, d, d_r, DEV, g)
    if d > d_r:
        csa.pack_fp4(src, cache)
    else:
        cache.rope.copy_(src)
    ref = []
    for b in range(B):
        if d > d_r:
            codes, scales, rope = O.pack_fp4(f64(src[b]), d_r, g)
            ref.append(fp4_rows(codes, scales, rope, d - d_r, g))
        else:
            ref.append(f64(src[b]))
    ref = np.stack(ref)
    assert np.array_equal(f64(csa.unpack_fp4(cache)), ref)
    # a range that starts inside, a range that leaves the cache on both sides, and ids in any order
    n = max(1, n_max // 2)
    row0 = torch.tensor([(7 * b + 1) % (n_max - n + 1) for b in range(B)], dtype=torch.int32)
    got = f64(csa.unpack_fp4(cache, n=n, row0=row0.to(DEV)))
    for b in range(B):
        assert np.array_equal(got[b], ref[b, int(row0[b]): int(row0[b]) + n])
    out = torch.full((B, n_max + 9, d), 3.0, dtype=torch.bfloat16, device=DEV)
    got = f64(csa.unpack_fp4(cache, n=n_max + 9, row0=torch.full((B,), -4, dtype=torch.int32, device=DEV), out=out))
    assert (got[:, :4] == 0).all() and (got[:, n_max + 4:] == 0).all() and np.array_equal(got[:, 4:n_max + 4], ref)
    rng = np.random.default_rng(1)
    ids = rng.integers(0, n_max, (B, 50)).astype(np.int32)
    ids[:, ::7] = [-1, n_max, 2 ** 31 - 1, -2 ** 31, n_max + 5, -7, -1, 0][: len(ids[0, ::7])]
    got = f64(csa.unpack_fp4(cache, idx=torch.as_tensor(ids, device=DEV)))
    for b in range(B):
        for j, i in enumerate(ids[b]):
            want = ref[b, i] if 0 <= i < n_max else np.zeros(d)
            assert np.array_equal(got[b, j], want), (b, j, i)
    csa.device_status()


def test_pages_outside_the_pool_read_as_zero(cuda_lib):
    csa = cuda_lib
    cache = csa.PagedCache(1, 384, 512, 64, DEV, 128, 3, torch.tensor([[2, 3, -1]], dtype=torch.int32))
    src = normal((1, 128, 512), 1.0, gen(0)).to(DEV)
    csa.pack_fp4(src, cache)                                # rows 0..127: page 2
    got = csa.unpack_fp4(cache)
    codes, scales, rope = O.pack_fp4(f64(src[0]), 64, 1.0)
    assert np.array_equal(f64(got[0, :128]), fp4_rows(codes, scales, rope, 448, 1.0))
    assert (got[0, 128:] == 0).all()


@pytest.mark.parametrize("B,Wn,d,d_r", [(1, 1, 512, 64), (3, 132, 512, 64), (2, 50, 128, 64), (2, 33, 64, 0)])
def test_fp8_window_read_back(cuda_lib, B, Wn, d, d_r):
    csa = cuda_lib
    src = normal((B, Wn, d), 2.0, gen(Wn)).to(DEV)
    src[0, 0, :64] = 0.0
    win = csa.Fp8Window(B, Wn, d, d_r, DEV)
    csa.pack_fp8_window(src, win)
    codes, scales = np_u8(win.codes), f64(win.scales)
    v = O.e4m3_decode(codes).astype(np.float32) * np.repeat(scales[..., : (d - d_r) // 64], 64, -1).astype(np.float32)
    ref = np.concatenate([O.bf16_round(v.astype(np.float64)), f64(src[..., d - d_r:])], -1)
    assert np.array_equal(f64(csa.unpack_fp8_window(win)), ref)
    ids = torch.tensor([[Wn - 1, -1, 0, Wn, 0]] * B, dtype=torch.int32, device=DEV)
    got = f64(csa.unpack_fp8_window(win, idx=ids))
    assert np.array_equal(got[:, 0], ref[:, -1]) and (got[:, 1] == 0).all() and (got[:, 3] == 0).all()
    assert np.array_equal(got[:, 2], ref[:, 0]) and np.array_equal(got[:, 4], ref[:, 0])
    row0 = torch.full((B,), Wn - 1, dtype=torch.int32, device=DEV)
    got = f64(csa.unpack_fp8_window(win, n=2, row0=row0))
    assert np.array_equal(got[:, 0], ref[:, -1]) and (got[:, 1] == 0).all()


def test_read_back_is_what_the_attention_reads(cuda_lib):
    """Entries read back and packed again (unit scales on the grid) give the same bytes, and attention over one selected
    entry returns that entry's row."""
    csa = cuda_lib
    B, n, d, H = 2, 64, 512, 8
    cache = csa.PackedCache(B, n, d, 64, DEV)
    csa.pack_fp4(normal((B, n, d), 1.0, gen(7)).to(DEV), cache)
    rows = csa.unpack_fp4(cache)
    q = normal((B, 1, H, d), 1.0, gen(8)).to(DEV)
    n_c = torch.full((B,), n, dtype=torch.int32, device=DEV)
    q_pos = torch.full((B, 1), 4 * n, dtype=torch.int64, device=DEV)
    for i in (0, 31, 63):
        idx = torch.full((B, 1, 1), i, dtype=torch.int32, device=DEV)
        out, _ = csa.sparse_attn(q, q_pos, cache, n_c, idx)
        assert torch.equal(out, rows[:, i][:, None, None].expand_as(out))


def test_empty_reads(cuda_lib):
    csa = cuda_lib
    cache = csa.PackedCache(2, 4, 512, 64, DEV)
    assert csa.unpack_fp4(cache, n=0).shape == (2, 0, 512)
    assert csa.unpack_fp4(cache, idx=torch.empty((2, 0), dtype=torch.int32, device=DEV)).shape == (2, 0, 512)
    none = csa.PackedCache(2, 0, 512, 64, DEV)
    assert (csa.unpack_fp4(none, n=3) == 0).all()
