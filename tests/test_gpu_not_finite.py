"""Keys that are not finite: a NaN or an infinity in an entry or window row makes NaN of every result of the queries that
see it, and changes nothing for the others, bit for bit, on each route of the attention: the shared-prefix call with the
sequences' own keys in the per-query and in the persistent kernel and without a prefix, and the plain attentions."""
import pytest
import torch

from csa_workloads import gen, normal
from tests.test_gpu_shared_attn import D, DEV, DR, W, Case

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# own keys in the per-query kernel (bf16 and FP8 windows), in the persistent kernel (more than 148 queries, bf16 window);
# without a prefix: several splits merged, whole queries, persistent
SHAPES = [(130, 1, 1, 300, 500, False), (130, 1, 1, 300, 500, True), (200, 1, 4, 300, 500, False), (200, 1, 4, 300, 500, True),
          (5, 2, 16, 0, 40, False), (5, 2, 16, 0, 40, True), (200, 1, 4, 0, 300, False)]


def copies_own_rows(csa, c):
    """Whether the call writes the own keys as bf16 rows (they are then part of its workspace)."""
    B, own = len(c.n_c), c.cache.n_max - c.n_p + (c.win.shape[1] if c.win is not None else 0)
    return csa.shared_attn_workspace_size(*c.args, ratio=c.r, window=W) >= B * own * 1024


def lengths(B, n_p, own):
    return [n_p + own - 7 * b % 37 for b in range(B)]


def positions(B, Nq, n_p, own):
    return [[128 * n + 41 + j for j in range(Nq)] for n in lengths(B, n_p, own)]


def check_hits(got, want, hit):
    (o2, l2), (out, lse) = got, want
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])


@pytest.mark.parametrize("B,Nq,H,n_p,own,fp8", SHAPES)
def test_nan_entry_reaches_its_readers(cuda_lib, B, Nq, H, n_p, own, fp8):
    """A NaN in the first, a middle and the last entry that a sequence sees, and in the entry behind it (nobody's)."""
    csa = cuda_lib
    c = Case(csa, B, Nq, H, n_p, own, fp8=fp8, n_c=lengths(B, n_p, own), t=positions(B, Nq, n_p, own), seed=B + H)
    assert n_p == 0 or not copies_own_rows(csa, c)
    want = c.run(csa)
    hit = torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
    for b, i in ((0, n_p), (1, n_p + own // 2), (2, int(c.n_c[2]) - 1), (B - 1, int(c.n_c[B - 1]) - 3)):
        c.cache.rope[b, i, 5] = NAN
        hit[b] = True
    c.cache.rope[3, int(c.n_c[3]), 0] = NAN
    check_hits(c.run(csa), want, hit)


@pytest.mark.parametrize("B,H,n_p", [(130, 1, 300), (200, 4, 300), (5, 16, 0), (200, 4, 0)])
def test_the_only_key_is_nan(cuda_lib, B, H, n_p):
    """A sequence whose one own key is NaN, without a window: its split has no finite score at all.  Beside it one that
    has no own key."""
    csa = cuda_lib
    own = 500
    n_c = lengths(B, n_p, own)
    n_c[1], n_c[2] = n_p + 1, n_p
    c = Case(csa, B, 1, H, n_p, own, win=False, n_c=n_c, seed=B)
    out, lse = c.run(csa)
    c.cache.rope[1, n_p] = NAN
    o2, l2 = c.run(csa)
    assert torch.isnan(o2[1]).all() and torch.isnan(l2[1]).all()
    keep = torch.arange(B, device=DEV) != 1
    assert torch.equal(o2[keep], out[keep]) and torch.equal(l2[keep], lse[keep])
    if n_p == 0:
        assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("early,cluster", [(False, False), (True, False), (False, True), (True, True)])
def test_selected_entry_with_a_nan(cuda_lib, early, cluster):
    """Sparse attention in splits merged through the workspace or inside a cluster, with and without the early window."""
    csa = cuda_lib
    B, H, n, k = 6, 64, 700, 384
    G = gen(7)
    kv = csa.PackedCache(B, n, D, DR, DEV)
    csa.pack_fp4(normal((B, n, D), 1.0, G).to(DEV), kv)
    q = normal((B, 1, H, D), 1.0, G).to(DEV)
    win = normal((B, W, D), 1.0, G).to(DEV)
    idx = torch.stack([torch.randperm(n - 1, generator=G)[:k] for _ in range(B)]).view(B, 1, k).int().to(DEV)
    n_c = torch.full((B,), n, dtype=torch.int32, device=DEV)
    t = torch.full((B, 1), 4 * n - 1, dtype=torch.int64, device=DEV)

    def run():
        r = csa.sparse_attn(q, t, kv, n_c, idx, win, t[:, 0] - W + 1, ratio=4, window=W, early_start=early, cluster=cluster)
        csa.device_status()
        return r
    want = run()
    for b, j in ((0, 0), (3, 200), (5, k - 1)):
        kv.rope[b, int(idx[b, 0, j]), 9] = NAN
    kv.rope[:, n - 1] = NAN                                 # never selected
    win[4, 77, 100] = NAN
    hit = torch.tensor([True, False, False, True, True, True], device=DEV)[:, None]
    check_hits(run(), want, hit)


@pytest.mark.parametrize("Nq,n", [(1, 60), (1, 700), (200, 60)])
def test_small_head_attention_with_a_nan(cuda_lib, Nq, n):
    """The 128-wide heads' kernel, in one part and in several: a NaN entry, and one that is a query's only key."""
    csa = cuda_lib
    B, H = 3, 16
    G = gen(8)
    kv = csa.PackedCache(B, n, 128, 32, DEV)
    csa.pack_fp4(normal((B, n, 128), 1.0, G).to(DEV), kv)
    q = normal((B, Nq, H, 128), 1.0, G).to(DEV)
    n_c = torch.tensor([n, n, 1], dtype=torch.int32, device=DEV)
    t = torch.full((B, Nq), 4 * n - 1, dtype=torch.int64, device=DEV)

    def run():
        r = csa.hca_attn(q, t, kv, n_c, ratio=4, window=W)
        csa.device_status()
        return r
    want = run()
    kv.rope[0, n // 2, 3] = NAN
    kv.rope[2, 0] = NAN
    kv.rope[2, 1] = NAN                                     # behind n_c
    check_hits(run(), want, torch.tensor([True, False, True], device=DEV)[:, None].expand(B, Nq))


@pytest.mark.parametrize("B,Nq,H,n_p,own,fp8", SHAPES + [(3, 5, 8, 0, 333, False), (60, 3, 8, 0, 333, False)])
def test_window_rows_that_a_query_does_not_see(cuda_lib, B, Nq, H, n_p, own, fp8):
    """A window buffer longer than the window, NaN in all its rows that nobody sees; then also in the rows of a sequence's
    later queries, which reach those alone."""
    csa = cuda_lib
    c = Case(csa, B, Nq, H, n_p, own, fp8=fp8, n_c=lengths(B, n_p, own), t=positions(B, Nq, n_p, own),
             seed=B + H + 1)
    before, behind = 17, 41                                 # rows that end the window inside a block of 32 at many places
    rows = W + Nq - 1
    if fp8:
        wide = csa.Fp8Window(B, before + rows + behind, D, DR, DEV)
        for name in ("codes", "scales", "rope"):
            getattr(wide, name)[:, before:before + rows] = getattr(c.win, name)
        wide.rope[:, :before] = wide.rope[:, before + rows:] = 1.0
        edge = wide.rope
    else:
        wide = edge = torch.ones((B, before + rows + behind, D), dtype=torch.bfloat16, device=DEV)
        wide[:, before:before + rows] = c.win
    c.win = wide
    c.args = c.args[:5] + (wide, c.args[6] - before)
    want = c.run(csa)
    edge[:, :before] = NAN
    edge[:, before + rows:] = NAN
    hit = torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
    check_hits(c.run(csa), want, hit)
    if Nq > 1:
        for b in range(0, B, 2):
            edge[b, before + W, 3 + b % 7] = NAN            # the row of the second query: all but the first see it
            hit[b, 1:] = True
        check_hits(c.run(csa), want, hit)


@pytest.mark.parametrize("B,Nq,H,n_p,own,fp8", SHAPES)
def test_infinite_keys_reach_every_result_of_their_readers(cuda_lib, B, Nq, H, n_p, own, fp8):
    """A row with an infinity scores +inf, -inf or NaN by the sign of the head's query there; all its readers' heads,
    channels and lse are NaN, whichever it is."""
    csa = cuda_lib
    c = Case(csa, B, Nq, H, n_p, own, fp8=fp8, n_c=lengths(B, n_p, own), t=positions(B, Nq, n_p, own),
             seed=B + H)
    want = c.run(csa)
    hit = torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
    for b, i, v in ((0, n_p, INF), (1, n_p + own // 2, -INF), (2, int(c.n_c[2]) - 1, INF), (B - 1, int(c.n_c[B - 1]) - 3, -INF)):
        c.cache.rope[b, i, 5] = v
        hit[b] = True
    (c.win.rope if fp8 else c.win)[3, W - 1, 11] = -INF     # a row that every query of sequence 3 sees
    hit[3] = True
    check_hits(c.run(csa), want, hit)
