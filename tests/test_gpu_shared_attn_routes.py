"""GPU parity of the shared-prefix attention where the own keys are attended query by query: the per-query and the persistent
kernel over the entries behind the prefix, in slots of their own, with several queries a sequence, pages, options and global
scales, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from tests.cmp_utils import LSE_ATOL, OUT_ATOL, assert_close, f64, np_u8
from tests.test_gpu_shared_attn import D, DEV, DR, W, Case

pytestmark = pytest.mark.gpu

# 180 queries and a bf16 window: the persistent kernel, in units of one and of several splits; fewer, or an FP8 window: the
# per-query kernel.  The long window buffers keep the own keys out of the prefix kernel.
SHAPES = [(180, 1, 2, 300, 900, 128, False), (60, 3, 8, 300, 300, 2000, False), (60, 3, 8, 300, 300, 2000, True),
          (40, 2, 16, 129, 70, 3000, False), (200, 1, 4, 300, 500, 128, False), (200, 1, 4, 300, 500, 128, True)]


def widen(csa, c, Wn, fp8):
    """The window's rows inside a buffer of Wn, the others ones."""
    B, rows = c.win.shape[0], c.win.shape[1]
    before = (Wn - rows) // 2
    if before <= 0:
        return
    if fp8:
        wide = csa.Fp8Window(B, Wn, D, DR, DEV)
        wide.scales.fill_(1.0), wide.codes.fill_(0x38), wide.rope.fill_(1.0)
        for name in ("codes", "scales", "rope"):
            getattr(wide, name)[:, before:before + rows] = getattr(c.win, name)
    else:
        wide = torch.ones((B, Wn, D), dtype=torch.bfloat16, device=DEV)
        wide[:, before:before + rows] = c.win
    c.win = wide
    c.args = c.args[:5] + (wide, c.args[6] - before)


def case(csa, B, Nq, H, n_p, own, Wn, fp8, **kw):
    """Lengths all over the own entries: none, one, a full cache; positions that rise by one."""
    rng = np.random.default_rng(B + own)
    n_c = n_p + rng.integers(0, own + 1, B)
    n_c[0], n_c[1], n_c[2] = n_p + own, n_p, n_p + 1
    t0 = 128 * n_c.astype(np.int64) + rng.integers(0, 129 - Nq, B)
    c = Case(csa, B, Nq, H, n_p, own, fp8=fp8, n_c=n_c, t=t0[:, None] + np.arange(Nq), seed=B + H, **kw)
    widen(csa, c, Wn, fp8)
    # the own keys are attended query by query: a longer buffer asks for no more workspace
    size = csa.shared_attn_workspace_size(*c.args, ratio=c.r, window=W)
    longer = c.args[:5] + (csa.Fp8Window(B, Wn + 2 * Nq, D, DR, DEV) if fp8 else c.win.new_zeros((B, Wn + 2 * Nq, D)), c.args[6])
    assert csa.shared_attn_workspace_size(*longer, ratio=c.r, window=W) == size
    return c


@pytest.mark.parametrize("B,Nq,H,n_p,own,Wn,fp8", SHAPES)
def test_against_the_oracle(cuda_lib, B, Nq, H, n_p, own, Wn, fp8):
    csa = cuda_lib
    c = case(csa, B, Nq, H, n_p, own, Wn, fp8)
    out, lse = c.run(csa)
    c.check(out, lse, rows=(0, 1, 2, B // 2, B - 1))
    again = c.run(csa)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,call", [(dict(page=128), {}), (dict(page=256), {}), (dict(), dict(out_rope_theta=10000.0)),
                                     (dict(), dict(softmax_scale=0.02))], ids=str)
def test_layouts_and_options(cuda_lib, kw, call, fp8):
    csa = cuda_lib
    c = case(csa, 60, 3, 8, 300, 300, 2000, fp8, **kw)
    out, lse = c.run(csa, **call)
    c.check(out, lse, scale=call.get("softmax_scale", D ** -0.5), theta=call.get("out_rope_theta", 0.0), rows=(0, 1, 2, 31, 59))


@pytest.mark.parametrize("fp8", [False, True])
def test_positions_that_see_part_or_nothing(cuda_lib, fp8):
    """Positions that hide own entries, part of the prefix or all of it, and the window at the start of a sequence."""
    csa = cuda_lib
    B, H, n_p, own, r = 160, 2, 300, 500, 128
    n_c = [n_p + own] * B
    t = [[r * (n_p + own)]] * B
    t[0], t[1], t[2], t[3], t[4] = [r * n_p - 1], [r * n_p + r - 1], [r * (n_p + 130) + 5], [r * 77 + 3], [40]
    n_c[5], n_c[6] = 0, 17
    c = Case(csa, B, 1, H, n_p, own, fp8=fp8, n_c=n_c, t=t, seed=31)
    out, lse = c.run(csa)
    c.check(out, lse, rows=range(8))


@pytest.mark.parametrize("g", [0.25, 4.0, 0.3])
@pytest.mark.parametrize("B,Nq,H,n_p,own,Wn,fp8", [(200, 1, 4, 300, 500, 128, False), (130, 1, 1, 300, 500, 128, True),
                                                   (6, 2, 16, 300, 40, 129, False)])
def test_global_scales(cuda_lib, B, Nq, H, n_p, own, Wn, fp8, g):
    """Global scales of the cache on each route (the last shape's own keys go with the prefix).  A scale that is no power of
    two costs an entry two bf16 roundings (of scale x g, and of the product), 2^-8 of an element: a logit moves by at most
    scale 2^-8 sum |q_e k_e|, an output by twice that times the largest value and 2^-8 of it."""
    csa = cuda_lib
    rng = np.random.default_rng(7)
    n_c = n_p + rng.integers(1, own + 1, B)
    t = [[128 * int(n) + 3 + j for j in range(Nq)] for n in n_c]
    c = Case(csa, B, Nq, H, n_p, own, fp8=fp8, n_c=n_c, t=t, seed=12)
    c.cache.g = g
    out, lse = c.run(csa)
    for b in (0, 1, B - 1):
        rows = O.entry_kv(np_u8(c.cache.codes[b, n_p:]), np_u8(c.cache.scales[b, n_p:]), f64(c.cache.rope[b, n_p:]), D - DR, g)
        rows = np.concatenate([f64(c.prefix), rows])[: int(c.n_c[b])]
        ro, rl = O.hca_attention(f64(c.q[b]), c.t[b], rows, int(c.n_c[b]), c.r, c.win_rows[b], int(c.p0[b]), W, D ** -0.5)
        own_rows, move = np.abs(rows[n_p:]), 0.0
        if g == 0.3:
            move = D ** -0.5 * 2.0 ** -8 * np.max(np.abs(f64(c.q[b])).reshape(-1, D) @ own_rows.T)
        top = max(np.abs(rows).max(), np.abs(c.win_rows[b]).max())
        assert_close(f64(lse[b]), rl, LSE_ATOL + move, 1e-4, f"lse b={b}")
        # unit-scale entries have the tolerance OUT_ATOL for values of up to 5
        assert_close(f64(out[b]), ro, OUT_ATOL * max(1.0, top / 5) + (2 * move + (2.0 ** -8 if move else 0.0)) * top, 2e-2,
                     f"out b={b}")
