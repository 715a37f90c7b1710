"""GPU parity of the FP8 projections: block quantisation (bit-exact), the block-scaled product for one and two
weights over its tile arrangements, and the compressor fed by them, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from csa_workloads import gen, normal
from oracle import csa_oracle as O
from tests.cmp_utils import OUT_ATOL, OUT_RTOL, assert_close, f64, np_u8

pytestmark = pytest.mark.gpu
DEV = "cuda"

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2          # 2^-8: the output's rounding, relative


def product_bound(ref, mag, K):
    """The output's bf16 rounding plus the fp32 sums: K products and ceil(K/128) scaled blocks are added (with two
    roundings of each scale product), every addition off by at most one unit of 2^-23 of the terms' magnitudes
    (the tensor cores may truncate where fp32 arithmetic rounds)."""
    terms = K + -(-K // 128) + 4
    return BF16_HALF * np.abs(ref) + terms * 2.0 ** -23 * mag * (1 + BF16_HALF)


def check_product(got, ref, mag, K, what=""):
    err = np.abs(f64(got) - ref)
    bad = err > product_bound(ref, mag, K)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err - product_bound(ref, mag, K))}"


def quantised(csa, x, block_rows):
    q = csa.quant_fp8(x.to(DEV), block_rows=block_rows)
    return q, np_u8(q.codes), f64(q.scales)


@pytest.mark.parametrize("rows,K,block", [(1, 16, 1), (1, 128, 1), (3, 144, 1), (37, 2064, 1), (130, 4096, 1), (1, 16, 128),
                                          (128, 128, 128), (129, 272, 128), (300, 1040, 128), (1000, 400, 128)])
def test_quant_bit_exact(cuda_lib, rows, K, block):
    x = (normal((rows, K), 1.0, gen(rows + K), dtype=torch.float32) *
         torch.exp(3 * torch.randn((1, K), generator=gen(5)))).to(torch.bfloat16)
    _, codes, scales = quantised(cuda_lib, x, block)
    rc, rs = O.quant_fp8(f64(x), block)
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, rc)


@pytest.mark.parametrize("exponent", [-126, -70, -55, 0, 60, 75, 126])
def test_quant_every_mantissa_by_every_mantissa(cuda_lib, exponent):
    """Blocks whose largest value has each of the 128 bf16 mantissas, over all mantissas and twelve binades below it: the
    quotients fall on both sides of, and on, every rounding border of E4M3.  Scales inside and outside the range
    where the quotient is computed with a reciprocal, and scales that are subnormal."""
    lead = (1 + torch.arange(128) / 128.0) * 2.0 ** exponent
    tail = (1 + torch.arange(128) / 128.0)[:, None] * 2.0 ** (exponent - 0.0 - torch.arange(12))[None, :]
    tail = tail.reshape(-1)                                                   # 1536 values
    blocks = []
    for a in lead:
        v = torch.where(tail <= a, tail, tail / 2)
        v = torch.nn.functional.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
        blocks.append(torch.cat([a.expand(len(v), 1), v * torch.where(torch.arange(127) % 3 == 0, -1.0, 1.0)], 1))
    x = torch.cat(blocks).to(torch.bfloat16)
    _, codes, scales = quantised(cuda_lib, x, 1)
    x64 = f64(x)
    s = (np.abs(x64).max(1).astype(np.float32) / np.float32(448.0))
    q = (x64.astype(np.float32) / s[:, None]).astype(np.float64)
    v = O.e4m3_rne_satfinite(q)
    want = O.e4m3_encode(np.abs(v)) | np.where(v < 0, 0x80, 0).astype(np.uint8)
    assert np.array_equal(scales[:, 0], s.astype(np.float64))
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("block", [1, 128])
def test_quant_special_values(cuda_lib, block):
    """Zero blocks, -0, the type's smallest and largest values, values that all fall on E4M3 midpoints, infinities and
    NaN, each in a block of its own and next to ordinary blocks."""
    rows, K = 16 * block, 512
    x = normal((rows, K), 1.0, gen(3)).float()
    r = [slice(i * block, (i + 1) * block) for i in range(16)]
    x[r[0], :128] = 0.0
    x[r[1], :128] = -0.0
    x[r[2], 128:256] = 2.0 ** -133                       # the smallest bf16: the scale is a subnormal fp32
    x[r[3], 128:256] = torch.finfo(torch.bfloat16).max
    x[r[4], 256:384] = 0.0
    x[r[4], 300] = float("nan")
    x[r[5], 260] = float("inf")
    x[r[6], 261] = -float("inf")
    x[r[6], 262] = float("nan")
    grid = torch.arange(128, dtype=torch.float32) * 3.5 + 0.25
    x[r[7], 384:] = grid
    x[r[7], 384] = 448.0
    x[r[8], 384:] = torch.where(torch.arange(128) % 2 == 0, -(2.0 ** -10) * torch.arange(128), torch.tensor(1.0))
    x = x.to(torch.bfloat16)
    _, codes, scales = quantised(cuda_lib, x, block)
    rc, rs = O.quant_fp8(f64(x), block)
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, rc)
    assert not (codes == 0x80).any()                     # no -0


# one token; each arrangement's edges; rows, channels and K that end inside a tile; parts of K of different length
SIZES = [(1, 8, 16, False), (1, 512, 4096, True), (16, 128, 1024, True), (17, 136, 144, False), (32, 640, 1152, True),
         (33, 200, 272, True), (64, 1024, 896, False), (65, 264, 128, False), (100, 648, 2064, True), (128, 128, 1920, False),
         (129, 8, 4096, True), (257, 1032, 272, True), (700, 1000, 784, False), (2500, 1288, 400, True),
         # pairs of CTAs: one block of K or a part of one, more tiles than pairs, the last tile almost empty
         (2500, 1000, 128, True), (2305, 1040, 16, True), (5000, 2056, 144, False)]


@pytest.mark.parametrize("M,N,K,pair", SIZES)
def test_product_against_the_oracle(cuda_lib, M, N, K, pair):
    csa = cuda_lib
    G = gen(M + N + K)
    x, xc, xs = quantised(csa, normal((M, K), 1.0, G), 1)
    ws = [quantised(csa, normal((N, K), K ** -0.5, G), 128) for _ in range(2 if pair else 1)]
    # rows behind the last one are left as they were
    full = [torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in ws]
    outs = csa.gemm_fp8(x, *[w[0] for w in ws], **dict(zip(("out", "out2"), [f[:M] for f in full])))
    csa.device_status()
    assert len(outs) == len(ws)
    for i, (o, w) in enumerate(zip(outs, ws)):
        ref, mag = O.gemm_fp8(xc, xs, w[1], w[2])
        check_product(o, ref, mag, K, f"weight {i}")
        assert (full[i][M:] == 7.0).all()
    again = csa.gemm_fp8(x, *[w[0] for w in ws])
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


def test_product_of_a_prefill_chunk(cuda_lib):
    """A chunk of 4096 tokens through both projections: every row against an fp32 product of the dequantised operands,
    sampled rows against the oracle."""
    csa = cuda_lib
    M, N, K = 4096, 512, 4096
    G = gen(9)
    x, xc, xs = quantised(csa, normal((M, K), 1.0, G), 1)
    ws = [quantised(csa, normal((N, K), K ** -0.5, G), 128) for _ in range(2)]
    outs = csa.gemm_fp8(x, ws[0][0], ws[1][0])
    csa.device_status()
    rows = np.r_[0:2, 127:130, 2047:2050, 4094:4096]
    for o, w in zip(outs, ws):
        ref, mag = O.gemm_fp8(xc[rows], xs[rows], w[1], w[2])
        check_product(o[torch.as_tensor(rows, device=DEV)], ref, mag, K)
        xd = torch.as_tensor(O.dequant_fp8(xc, xs, 1), device=DEV)
        wd = torch.as_tensor(O.dequant_fp8(w[1], w[2], 128), device=DEV)
        check_product(o, f64(xd @ wd.T), f64(xd.abs() @ wd.abs().T), K)


@pytest.mark.parametrize("M", [5, 300])
def test_product_keeps_nan_and_zero_blocks(cuda_lib, M):
    """A NaN in a token makes that token's outputs NaN and no other's; a block of zeros (scale 0) adds nothing."""
    csa = cuda_lib
    N, K = 256, 640
    G = gen(2)
    xb = normal((M, K), 1.0, G)
    xb[3, 200] = float("nan")
    xb[1, 128:256] = 0.0
    wb = normal((N, K), K ** -0.5, G)
    wb[:128, 256:384] = 0.0
    x, xc, xs = quantised(csa, xb, 1)
    w, wc, wsc = quantised(csa, wb, 128)
    out, = csa.gemm_fp8(x, w)
    csa.device_status()
    assert torch.isnan(out[3]).all()
    keep = np.arange(M) != 3
    ref, mag = O.gemm_fp8(xc[keep], xs[keep], wc, wsc)
    check_product(out[torch.as_tensor(keep, device=DEV)], ref, mag, K)


@pytest.mark.parametrize("B,T,dm,d,r", [(1, 16, 1024, 128, 4), (2, 300, 272, 512, 4), (1, 256, 256, 512, 128)])
def test_compress_with_fp8_weights(cuda_lib, B, T, dm, d, r):
    """compress() with FP8 weights: C and Z are the products, the entries those of the pooling mode on them, and both
    agree with the oracle's pooling of the oracle's projections."""
    csa = cuda_lib
    G = gen(T)
    d_r = 64 if d == 512 else 32
    x = normal((B, T, dm), 1.0, G)
    wk, wg = normal((d, dm), dm ** -0.5, G), normal((d, dm), dm ** -0.5, G)
    b_pos = normal((r, d), 0.1, G, dtype=torch.float32).to(DEV)
    Wk, Wg = csa.quant_fp8(wk.to(DEV), block_rows=128), csa.quant_fp8(wg.to(DEV), block_rows=128)
    c, _, C, Z = csa.compress(x=x.to(DEV), W_kv=Wk, W_g=Wg, b_pos=b_pos, ratio=r, d_rope=d_r, rope_theta=10000.0)
    c2, _, _, _ = csa.compress(C=C, Z=Z, b_pos=b_pos, ratio=r, d_rope=d_r, rope_theta=10000.0)
    csa.device_status()
    assert torch.equal(c, c2)
    xc, xs = O.quant_fp8(f64(x.reshape(B * T, dm)), 1)
    for got, w in ((C, wk), (Z, wg)):
        ref, mag = O.gemm_fp8(xc, xs, *O.quant_fp8(f64(w), 128))
        check_product(got.reshape(B * T, d), ref, mag, dm)
    for b in range(B):
        ref = O.compress_pool(f64(C[b]), f64(Z[b]), f64(b_pos), r, d_r, 10000.0, 0)
        assert_close(f64(c[b]), ref, OUT_ATOL, OUT_RTOL)
    if B == 1:
        c3, _, C3, _ = csa.compress(x=csa.quant_fp8(x[0].to(DEV)), W_kv=Wk, W_g=Wg, b_pos=b_pos, ratio=r, d_rope=d_r,
                                    rope_theta=10000.0, C=torch.empty_like(C))
        assert torch.equal(C3, C) and torch.equal(c3, c)


def test_captured_and_replayed_on_another_stream(cuda_lib):
    """Quantisation and product captured into a graph on a side stream and replayed with new inputs."""
    csa = cuda_lib
    M, N, K = 48, 256, 512
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    w = csa.quant_fp8(normal((N, K), K ** -0.5, gen(1)).to(DEV), block_rows=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, = csa.gemm_fp8(csa.quant_fp8(x, stream=s), w, stream=s)        # once before the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, = csa.gemm_fp8(csa.quant_fp8(x), w)
    for seed in (4, 5):
        new = normal((M, K), 1.0, gen(seed)).to(DEV)
        x.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, csa.gemm_fp8(csa.quant_fp8(new), w)[0])
    csa.device_status()
