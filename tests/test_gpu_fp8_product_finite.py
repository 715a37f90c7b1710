"""The FP8 product with NaN, infinite and zero blocks over each of its tile arrangements: outputs that should be NaN are,
and all others are finite and within the product's bound (a comparison of errors alone lets a NaN pass)."""
import numpy as np
import pytest
import torch

from csa_workloads import gen, normal
from oracle import csa_oracle as O
from tests.cmp_utils import f64
from tests.test_gpu_fp8_projection import product_bound, quantised

DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def check_finite_product(got, ref, mag, K, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: {np.isnan(got).sum()} NaN, expected {np.isnan(ref).sum()}"
    keep = ~np.isnan(ref)
    with np.errstate(invalid="ignore"):
        bad = keep & ~(np.abs(got - ref) <= product_bound(ref, mag, K))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}"


def test_the_check_sees_nan_and_infinity():
    ref, mag = np.ones((3, 4)), np.ones((3, 4))
    check_finite_product(ref, ref, mag, 128)
    for bad in (NAN, INF, -INF, 1.1):
        got = ref.copy()
        got[1, 2] = bad
        with pytest.raises(AssertionError):
            check_finite_product(got, ref, mag, 128)
    ref[0, 0] = NAN
    with pytest.raises(AssertionError):
        check_finite_product(np.ones((3, 4)), ref, mag, 128)


# channels as the MMA's rows with 16, 32 and 64 tokens, tiles of 128 x 128 in one and several parts of K, pairs of CTAs
SIZES = [(5, 256, 640), (20, 136, 1040), (50, 384, 2048), (300, 256, 640), (140, 1032, 4096), (2500, 1288, 400)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_nan_and_infinity_stay_in_their_row_and_column(cuda_lib, M, N, K):
    """A NaN or infinity in a token makes that token's outputs NaN, one in a weight the outputs of its channel (NaN) or of its
    block of 128 channels (an infinity makes the block's scale infinite), and no others."""
    csa = cuda_lib
    G = gen(M + N)
    xb, wb = normal((M, K), 1.0, G), normal((N, K), K ** -0.5, G)
    xb[3, 200] = NAN
    xb[1, K - 1] = INF
    wb[7, 130] = NAN
    wb[N - 1, 5] = -INF
    x, xc, xs = quantised(csa, xb, 1)
    w, wc, ws = quantised(csa, wb, 128)
    w2, w2c, w2s = quantised(csa, normal((N, K), K ** -0.5, G), 128)
    outs = csa.gemm_fp8(x, w, w2)
    csa.device_status()
    rows, cols = np.zeros(M, bool), np.zeros(N, bool)
    rows[[1, 3]] = True
    cols[7] = True
    cols[(N - 1) // 128 * 128:] = True
    for o, codes, scales, c in ((outs[0], wc, ws, cols), (outs[1], w2c, w2s, np.zeros(N, bool))):
        with np.errstate(invalid="ignore"):
            ref, mag = O.gemm_fp8(xc, xs, codes, scales)
        nan = rows[:, None] | c[None, :]
        assert np.isnan(ref[nan]).all() and np.isfinite(ref[~nan]).all()
        check_finite_product(f64(o), ref, mag, K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_zero_blocks_add_nothing(cuda_lib, M, N, K):
    csa = cuda_lib
    G = gen(M + K)
    xb, wb = normal((M, K), 1.0, G), normal((N, K), K ** -0.5, G)
    xb[0] = 0.0
    xb[1, 128:256] = 0.0
    wb[:128, 256:384] = 0.0
    wb[128:] = 0.0
    x, xc, xs = quantised(csa, xb, 1)
    w, wc, ws = quantised(csa, wb, 128)
    out, = csa.gemm_fp8(x, w)
    csa.device_status()
    check_finite_product(f64(out), *O.gemm_fp8(xc, xs, wc, ws), K)
    assert (out[0] == 0).all() and (out[:, 128:] == 0).all()


@pytest.mark.gpu
def test_every_output_of_a_prefill_chunk_is_finite(cuda_lib):
    csa = cuda_lib
    M, N, K = 4096, 512, 4096
    G = gen(9)
    x, _, _ = quantised(csa, normal((M, K), 1.0, G), 1)
    ws = [quantised(csa, normal((N, K), K ** -0.5, G), 128)[0] for _ in range(2)]
    outs = csa.gemm_fp8(x, *ws)
    csa.device_status()
    assert all(torch.isfinite(o).all() for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,dm,d,r", [(1, 16, 1024, 128, 4), (2, 300, 272, 512, 4)])
def test_compress_projections_with_a_nan_token(cuda_lib, B, T, dm, d, r):
    """C and Z of compress() with FP8 weights: the token's rows are NaN, all others finite and within the bound."""
    csa = cuda_lib
    G = gen(T + 1)
    x = normal((B, T, dm), 1.0, G)
    x[0, 5, 100] = NAN
    wk, wg = normal((d, dm), dm ** -0.5, G), normal((d, dm), dm ** -0.5, G)
    Wk, Wg = csa.quant_fp8(wk.to(DEV), block_rows=128), csa.quant_fp8(wg.to(DEV), block_rows=128)
    _, _, C, Z = csa.compress(x=x.to(DEV), W_kv=Wk, W_g=Wg, b_pos=torch.zeros((r, d), device=DEV), ratio=r)
    csa.device_status()
    xc, xs = O.quant_fp8(f64(x.reshape(B * T, dm)), 1)
    for got, w in ((C, wk), (Z, wg)):
        ref, mag = O.gemm_fp8(xc, xs, *O.quant_fp8(f64(w), 128))
        assert np.isnan(ref[5]).all() and np.isfinite(np.delete(ref, 5, 0)).all()
        check_finite_product(f64(got).reshape(B * T, d), ref, mag, dm)
