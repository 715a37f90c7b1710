"""GPU parity of HCA attention with a shared prefix: against the 64-bit oracle over batches, heads, prefix lengths,
own entries, windows and layouts; the cases where rows see part of the prefix or nothing; scores that keep rising;
and the whole path from FP8 projections to attention over the read-back prefix."""
import numpy as np
import pytest
import torch

from csa_workloads import gen, normal
from oracle import csa_oracle as O
from tests.cmp_utils import LSE_ATOL, LSE_RTOL, OUT_ATOL, OUT_RTOL, assert_close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, DR, W = 512, 64, 128


class Case:
    """Inputs of one call: a prefix, caches whose rows behind it are packed (the rows of the prefix hold garbage), a window."""

    def __init__(self, csa, B, Nq, H, n_p, own, r=128, page=0, win=True, fp8=False, n_c=None, t=None, seed=0, q_std=1.0,
                 prefix=None):
        G = gen(seed)
        self.r, self.n_p, n_max = r, n_p, n_p + own
        rng = np.random.default_rng(seed)
        if n_c is None:
            n_c = [n_p + int(v) for v in rng.integers(0, own + 1, B)]
            n_c[-1] = n_max
        self.n_c = np.asarray(n_c, np.int32)
        if t is None:
            t = [[r * int(n) + int(rng.integers(0, r - Nq + 1)) + j for j in range(Nq)] for n in self.n_c]
        self.t = np.asarray(t, np.int64)
        self.q = normal((B, Nq, H, D), q_std, G).to(DEV)
        self.prefix = (normal((n_p, D), 1.0, G) if prefix is None else prefix).to(DEV)
        rows = normal((B, own, D), 1.0, G).to(DEV)
        if page:
            width = -(-n_max // page)
            table = torch.as_tensor(rng.permutation(B * width).reshape(B, width).astype(np.int32))
            self.cache = csa.PagedCache(B, n_max, D, DR, DEV, page, B * width, table)
        else:
            self.cache = csa.PackedCache(B, n_max, D, DR, DEV)
        self.cache.codes.fill_(0x77)
        self.cache.scales.fill_(0x7F)                       # E4M3 NaN: the prefix's rows are not read
        self.cache.rope.fill_(float("nan"))
        if own:
            csa.pack_fp4(rows, self.cache, row0=torch.full((B,), n_p, dtype=torch.int32, device=DEV))
        self.own = lambda b: O.entry_kv(*O.pack_fp4(f64(rows[b]), DR, 1.0), D - DR, 1.0) if own else np.zeros((0, D))
        self.win = self.win_pos0 = None
        self.win_rows = np.zeros((B, 0, D))
        p0 = self.t[:, 0] - W + 1
        self.p0 = p0
        if win:
            w = normal((B, W + Nq - 1, D), 1.0, G).to(DEV)
            self.win_rows = f64(w)
            self.win = w
            if fp8:
                self.win = csa.Fp8Window(B, W + Nq - 1, D, DR, DEV)
                csa.pack_fp8_window(w, self.win)
                self.win_rows = f64(csa.unpack_fp8_window(self.win))     # the bf16 rows the attention reads
            self.win_pos0 = torch.as_tensor(p0, device=DEV)
        self.args = (self.q, torch.as_tensor(self.t, device=DEV), self.cache, torch.as_tensor(self.n_c, device=DEV),
                     self.prefix, self.win, self.win_pos0)

    def run(self, csa, **kw):
        out, lse = csa.hca_shared_attn(*self.args, ratio=self.r, window=W, **kw)
        csa.device_status()
        return out, lse

    def check(self, out, lse, scale=D ** -0.5, theta=0.0, rows=None, atol=OUT_ATOL, rtol=OUT_RTOL):
        pre = f64(self.prefix)
        for b in (range(len(self.n_c)) if rows is None else rows):
            kv = np.concatenate([pre, self.own(b)])
            ro, rl = O.hca_attention(f64(self.q[b]), self.t[b], kv, int(self.n_c[b]), self.r, self.win_rows[b], int(self.p0[b]), W,
                                     scale, out_rope_theta=theta, d_rope=DR)
            assert_close(f64(out[b]), ro, atol, rtol, f"out b={b}")
            assert_close(f64(lse[b]), rl, LSE_ATOL, LSE_RTOL, f"lse b={b}")


@pytest.mark.parametrize("B,Nq,H,n_p,own", [
    (1, 1, 1, 1, 0), (1, 1, 64, 128, 0), (2, 1, 16, 260, 3), (3, 2, 24, 127, 40), (1, 1, 96 - 32, 129, 1),
    (3, 1, 32, 1000, 0), (5, 5, 64, 300, 70), (7, 1, 40, 640, 130), (13, 3, 64, 515, 5), (2, 1, 64, 8192, 64)])
def test_against_the_oracle(cuda_lib, B, Nq, H, n_p, own):
    c = Case(cuda_lib, B, Nq, H, n_p, own, seed=B + n_p)
    c.check(*c.run(cuda_lib))


@pytest.mark.parametrize("kw,call", [
    (dict(page=128), {}), (dict(page=256), {}), (dict(win=False), {}), (dict(fp8=True), {}), (dict(r=4), {}),
    (dict(), dict(out_rope_theta=10000.0)), (dict(), dict(softmax_scale=0.02))], ids=str)
def test_layouts_and_options(cuda_lib, kw, call):
    c = Case(cuda_lib, 3, 2, 24, 300, 37, seed=11, **kw)
    out, lse = c.run(cuda_lib, **call)
    c.check(out, lse, scale=call.get("softmax_scale", D ** -0.5), theta=call.get("out_rope_theta", 0.0))


def test_rows_that_see_part_of_the_prefix_or_nothing(cuda_lib):
    """Sequences that have only some of the shared entries yet, whose position hides others, and that see no key at all;
    without a window the last ones give zero rows and lse = -inf."""
    csa = cuda_lib
    n_p, r = 700, 128
    n_c = [0, 5, 128, 400, 700, 700, 700, 731]
    t = [[50], [r * 5], [r * 128], [r * 400 + 3], [r * 300 + 126], [r * 300 + 127], [60], [r * 740]]
    for win in (False, True):
        c = Case(csa, 8, 1, 24, n_p, 31, win=win, n_c=n_c, t=t, seed=3)
        out, lse = c.run(csa)
        c.check(out, lse)
        if not win:
            for b in (0, 6):
                assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_scores_that_move_from_tile_to_tile(cuda_lib, order):
    """Prefix rows along the queries' common direction with a growing (falling) weight: the running reference moves in
    every tile (never again after the first), by far more than its slack.  The scores reach about 60, so the weights
    of a tile are those of its last few keys; out keeps the tolerance of unit-scale rows times the rows' scale."""
    csa = cuda_lib
    n_p, B, H = 1400, 2, 48
    G = gen(6)
    base = normal((D,), 1.0, G).float()
    w = torch.linspace(-3.0, 3.0, n_p)
    if order == "falling":
        w = w.flip(0)
    prefix = (w[:, None] * base + 0.3 * torch.randn((n_p, D), generator=G)).to(torch.bfloat16)
    c = Case(csa, B, 1, H, n_p, 20, prefix=prefix, seed=6)
    c.q.copy_((base.to(DEV) + 0.1 * torch.randn(c.q.shape, device=DEV, generator=gen(1, DEV))).to(torch.bfloat16))
    out, lse = c.run(csa)
    c.check(out, lse, atol=OUT_ATOL * float(prefix.abs().max()) / 5)


def test_same_as_the_unshared_attention(cuda_lib):
    """With the read-back rows of a cache as the prefix, the result is hca_attn's on that cache: more query rows and
    blocks than SMs, sequences of different length."""
    csa = cuda_lib
    B, H, n_p, own, r = 96, 64, 384, 20, 128
    c = Case(csa, B, 2, H, n_p, own, seed=9)
    src = normal((1, n_p, D), 1.0, gen(4)).to(DEV)
    one = csa.PackedCache(1, n_p, D, DR, DEV)
    csa.pack_fp4(src, one)
    csa.pack_fp4(src.expand(B, -1, -1).contiguous(), c.cache)
    args = list(c.args)
    args[4] = csa.unpack_fp4(one)[0]
    out, lse = csa.hca_shared_attn(*args, ratio=r, window=W)
    ro, rl = csa.hca_attn(*args[:4], *args[5:], ratio=r, window=W)
    csa.device_status()
    assert_close(f64(out), f64(ro), OUT_ATOL, OUT_RTOL)
    assert_close(f64(lse), f64(rl), LSE_ATOL, LSE_RTOL)
    c.prefix = args[4]
    c.check(out, lse, rows=(0, 41, 95))


@pytest.mark.parametrize("B,Nq,H,n_p,own,fp8", [(40, 1, 16, 200, 3000, False), (40, 1, 16, 200, 3000, True),
                                                (3, 1, 64, 300, 600, False), (130, 1, 1, 300, 9, False), (9, 3, 7, 300, 50, True),
                                                (130, 1, 1, 300, 500, False), (130, 1, 1, 300, 500, True)])
def test_own_keys_long_and_many(cuda_lib, B, Nq, H, n_p, own, fp8):
    """Own entries that outnumber the prefix in many sequences (attended query by query), several tiles of them in few
    sequences, and blocks of rows that touch many sequences or cut them at odd places."""
    c = Case(cuda_lib, B, Nq, H, n_p, own, fp8=fp8, seed=B)
    out, lse = c.run(cuda_lib)
    c.check(out, lse, rows=(0, B // 2, B - 1))


@pytest.mark.parametrize("fp8,page", [(False, 0), (True, 128)])
def test_own_rows_that_are_not_finite_stay_with_their_readers(cuda_lib, fp8, page):
    """Sequences share blocks of query rows: a NaN or infinity in one's cache or window makes NaN of the queries that see
    it, and changes nothing for the others, bit for bit."""
    csa = cuda_lib
    n_p, own, B, Nq = 300, 40, 5, 2
    n_c = [n_p + own - 1, n_p + 7, n_p, n_p + own, n_p + 1]
    c = Case(csa, B, Nq, 16, n_p, own, fp8=fp8, page=page, n_c=n_c, t=[[128 * n + 5 + j for j in range(Nq)] for n in n_c],
             seed=11)
    out, lse = c.run(csa)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    win = c.win.rope if fp8 else c.win                      # [B, W + Nq - 1, ..]: query j sees rows j .. j + W - 1
    win[1, 0, -1] = float("nan")                            # query 0 alone
    win[2, W, 3] = float("inf")                             # query 1 alone
    rope = c.cache.rope.view(-1, DR)
    def row(b, i):
        return int(c.cache.table[b, i // page]) * page + i % page if page else b * (n_p + own) + i
    rope[row(3, n_p + own - 1), 0] = float("-inf")          # both of sequence 3
    rope[row(0, n_p + own - 1), 0] = float("nan")           # entry n_c[0]: nobody
    o2, l2 = c.run(csa)
    hit = torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
    hit[1, 0] = hit[2, 1] = hit[3, 0] = hit[3, 1] = True
    assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], out[~hit]) and torch.equal(l2[~hit], lse[~hit])


def test_parts_that_follow_one_another(cuda_lib):
    """More blocks of query rows than pairs of CTAs, each of few tiles: a pair stores one block's partial while the next
    block's scores are there already.  The same result at every run, and the unshared attention's."""
    csa = cuda_lib
    B, Nq, H, n_p, own = 130, 3, 34, 257, 900
    c = Case(csa, B, Nq, H, n_p, own, r=4, seed=59, q_std=4.0)
    out, lse = c.run(csa)
    c.check(out, lse, rows=(0, 4, 77, B - 1))
    for _ in range(5):
        o2, l2 = c.run(csa)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_no_prefix_is_the_plain_attention(cuda_lib):
    csa = cuda_lib
    c = Case(csa, 3, 1, 16, 0, 200, seed=2)
    out, lse = c.run(csa)
    ro, rl = csa.hca_attn(*c.args[:4], *c.args[5:], ratio=c.r, window=W)
    assert torch.equal(out, ro) and torch.equal(lse, rl)


def test_workspace_contents_and_repeats(cuda_lib):
    """The result does not depend on what the workspace and outputs held, is the same at every run, and rows behind the
    outputs stay as they were."""
    csa = cuda_lib
    c = Case(csa, 5, 1, 24, 900, 33, seed=8)
    out, lse = c.run(csa)
    n = csa.shared_attn_workspace_size(*c.args, ratio=c.r, window=W)
    for fill in (0, 0xFF):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        o2 = torch.full((6, 1, 24, D), 5.0, dtype=torch.bfloat16, device=DEV)
        l2 = torch.full((6, 1, 24), 5.0, device=DEV)
        csa.hca_shared_attn(*c.args, ratio=c.r, window=W, ws=ws[:n], out=o2[:5], lse=l2[:5])
        csa.device_status()
        assert torch.equal(o2[:5], out) and torch.equal(l2[:5], lse)
        assert (o2[5] == 5.0).all() and (l2[5] == 5.0).all() and (ws[n:] == fill).all()
    with pytest.raises(csa.CSAError, match="CSA_ERR_WORKSPACE"):
        csa.hca_shared_attn(*c.args, ratio=c.r, window=W, ws=ws[: n - 1])
    with pytest.raises(csa.CSAError, match="CSA_ERR_UNSUPPORTED"):
        csa.hca_shared_attn(*c.args, ratio=c.r, window=W, ws=ws[8: 8 + n])


def test_captured_and_replayed(cuda_lib):
    """A captured call (its workspace in the graph's pool) replayed after the queries and lengths changed."""
    csa = cuda_lib
    c = Case(csa, 4, 1, 16, 500, 30, seed=5)
    d = Case(csa, 4, 1, 16, 500, 30, seed=55)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    csa.hca_shared_attn(*c.args, ratio=c.r, window=W, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, lse = csa.hca_shared_attn(*c.args, ratio=c.r, window=W)
    for i in (0, 1, 3):
        c.args[i].copy_(d.args[i])
    c.cache.codes.copy_(d.cache.codes), c.cache.scales.copy_(d.cache.scales), c.cache.rope.copy_(d.cache.rope)
    c.prefix.copy_(d.prefix), c.win.copy_(d.win), c.win_pos0.copy_(d.win_pos0)
    g.replay()
    d.check(out, lse)
    csa.device_status()


def test_two_graphs_and_an_eager_call_interleaved(cuda_lib):
    """Two captured calls of different sizes, and eager calls of both between their replays on two streams: each keeps its
    workspace, so each result stays its own."""
    csa = cuda_lib
    cs = [Case(csa, 4, 1, 16, 500, 30, seed=5), Case(csa, 2, 5, 64, 1300, 90, seed=6)]
    want = [c.run(csa) for c in cs]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cs], [], []
    for c, s in zip(cs, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(csa.hca_shared_attn(*c.args, ratio=c.r, window=W))
        graphs.append(g)
    for _ in range(3):
        eager = []
        for c, s, g in zip(cs, streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                eager.append(csa.hca_shared_attn(*c.args, ratio=c.r, window=W))
        for s in streams:
            s.synchronize()
        for got in (outs, eager):
            for (o, l), (wo, wl) in zip(got, want):
                assert torch.equal(o, wo) and torch.equal(l, wl)
    csa.device_status()


def test_prompt_to_shared_attention(cuda_lib):
    """The operators together, as a shared prompt is served: its hidden states through FP8 projections into compressed
    entries, packed to FP4 once, read back once, and attended by a batch whose own entries went the same way."""
    csa = cuda_lib
    G = gen(21)
    r, dm, n_p, own, B, H = 16, 256, 40, 3, 4, 16
    wk, wg = (csa.quant_fp8(normal((D, dm), dm ** -0.5, G).to(DEV), block_rows=128) for _ in range(2))
    b_pos = normal((r, D), 0.1, G, dtype=torch.float32).to(DEV)
    x = normal((1, n_p * r, dm), 1.0, G).to(DEV)
    one = csa.PackedCache(1, n_p, D, DR, DEV)
    c, _, _, _ = csa.compress(x=x, W_kv=wk, W_g=wg, b_pos=b_pos, ratio=r, d_rope=DR, rope_theta=10000.0, kv_cache=one)
    prefix = csa.unpack_fp4(one)[0]
    cache = csa.PackedCache(B, n_p + own, D, DR, DEV)
    row0 = torch.full((B,), n_p, dtype=torch.int32, device=DEV)
    xo = normal((B, own * r, dm), 1.0, G).to(DEV)
    co, _, Co, _ = csa.compress(x=xo, W_kv=wk, W_g=wg, b_pos=b_pos, ratio=r, d_rope=DR, rope_theta=10000.0,
                                pos0=torch.full((B,), n_p * r, dtype=torch.int64, device=DEV), kv_cache=cache, row0=row0)
    n_c = torch.full((B,), n_p + own, dtype=torch.int32, device=DEV)
    q_pos = torch.full((B, 1), (n_p + own) * r - 1, dtype=torch.int64, device=DEV)
    q = normal((B, 1, H, D), 1.0, G).to(DEV)
    win, p0 = Co.contiguous(), torch.full((B,), n_p * r, dtype=torch.int64, device=DEV)
    out, lse = csa.hca_shared_attn(q, q_pos, cache, n_c, prefix, win, p0, ratio=r, window=32)
    csa.device_status()
    pre = O.entry_kv(*O.pack_fp4(f64(c[0]), DR, 1.0), D - DR, 1.0)
    assert np.array_equal(f64(prefix), pre)
    for b in range(B):
        kv = np.concatenate([pre, O.entry_kv(*O.pack_fp4(f64(co[b]), DR, 1.0), D - DR, 1.0)])
        ro, rl = O.hca_attention(f64(q[b]), np.full(1, (n_p + own) * r - 1), kv, n_p + own, r, f64(win[b]),
                                 n_p * r, 32, D ** -0.5)
        assert_close(f64(out[b]), ro, OUT_ATOL, OUT_RTOL)
        assert_close(f64(lse[b]), rl, LSE_ATOL, LSE_RTOL)
