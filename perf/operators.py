"""What the operators around the compressor's projections and the shared prefix are measured on.

Four operators of the CSA layer, each in its plain form (elementary torch operations in 32 bits) and as a user
calls it:

  quant      bf16 rows to E4M3 codes with one fp32 scale per 128 channels (activations) or per 128 x 128 block (weights)
  product    out[m][n] = sum_k x[m][k] W[n][k] of two such operands, for one weight or the compressor's two
  readback   entries of the FP4 cache, or rows of the FP8 window, back as bf16 rows: ranges or lists of ids
  shared     HCA attention of a batch whose sequences begin with the same prefix: the prefix's rows are read once for
             all, each sequence adds its own entries and its window

`own` is set from outside: false runs the plain forms, true the framework's entry points.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
D, DR = 512, 64                      # head width of the caches and its RoPE slice
DN = D - DR
RATIO, WINDOW = 128, 128             # HCA: tokens per entry, sliding window


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a prefill chunk's hidden states on their way into the compressor's FP8 projection
        dict(name="quant chunk 4096x4096", op="quant", rows=4096, K=4096, block=1),
        # a weight of odd height whose last blocks are cut off in both directions
        dict(name="quant weight 1000x2064", op="quant", rows=1000, K=2064, block=128),
        # the small layer's two projections (d_model 1024, d 128) for 16 tokens: latency
        dict(name="product small 16", op="product", M=16, N=128, K=1024, pair=True),
        # one decode step's tokens of 32 sequences through both projections: the weights are the traffic
        dict(name="product decode 32", op="product", M=32, N=512, K=4096, pair=True),
        # a prefill chunk through both projections
        dict(name="product chunk 4096", op="product", M=4096, N=512, K=4096, pair=True),
        # a ragged batch of tokens against a weight whose sides end inside a block
        dict(name="product ragged 1111", op="product", M=1111, N=648, K=2064, pair=False),
        # one prefix of 128 entries expanded for sharing: latency
        dict(name="readback fp4 prefix 128", op="readback", fmt="fp4", B=1, n=128, n_max=128, ids=False, page=0, gpow=0),
        # the ids that 16 sequences selected, gathered from a paged cache (absent ids are -1)
        dict(name="readback fp4 ids paged", op="readback", fmt="fp4", B=16, n=2048, n_max=8192, ids=True, page=256, gpow=-4),
        # every window of a large batch
        dict(name="readback fp8 window", op="readback", fmt="fp8", B=512, n=128, n_max=128, ids=False, page=0, gpow=0),
        # two short conversations over a prompt of 33 K tokens, few heads: latency
        dict(name="shared decode 2x260", op="shared", B=2, Nq=1, H=16, prefix=260, own=3),
        # five draft positions of 8 sequences over half a million tokens, an odd number of heads
        dict(name="shared drafts 8x5x4099", op="shared", B=8, Nq=5, H=24, prefix=4099, own=70),
        # one decode step of 64 sequences over a prefix of a million tokens
        dict(name="shared decode 64x8192", op="shared", B=64, Nq=1, H=64, prefix=8192, own=64),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(lo, min(hi, int(round(v / step)) * step))

    op = rng.choice(("quant", "product", "readback", "shared"))
    if op == "quant":
        return dict(op=op, rows=size(1, 4096), K=size(128, 4096, 16), block=rng.choice((1, 1, 128)))
    if op == "product":
        return dict(op=op, M=size(1, 4096), N=size(64, 512, 8), K=size(128, 4096, 16), pair=rng.random() < 0.6)
    if op == "readback":
        fmt = rng.choice(("fp4", "fp4", "fp8"))
        if fmt == "fp8":
            n_max = size(128, 256)
            return dict(op=op, fmt=fmt, B=size(1, 128), n=rng.randint(1, n_max), n_max=n_max, ids=rng.random() < 0.5, page=0, gpow=0)
        n_max = size(128, 8192)
        return dict(op=op, fmt=fmt, B=size(1, 16), n=min(n_max, size(1, 2048)), n_max=n_max, ids=rng.random() < 0.5,
                    page=rng.choice((0, 128, 256)), gpow=rng.choice((0, -4, 1)))
    H = rng.choice((8, 16, 24, 40, 64))
    Nq = rng.choice((1, 1, 1, 2, 5))
    return dict(op=op, B=size(1, 64 // Nq), Nq=Nq, H=H, prefix=size(128, 8192), own=rng.randint(0, 64))


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _block_quant(x, block):
    """E4M3 codes and fp32 scales of x [rows, K] for blocks of `block` rows x 128 channels."""
    rows, K = x.shape
    R, C = -(-rows // block), -(-K // 128)
    p = torch.zeros((R * block, C * 128), dtype=torch.float32, device=x.device)
    p[:rows, :K] = x.float()
    p = p.view(R, block, C, 128)
    s = p.abs().amax(dim=(1, 3)) / 448.0
    q = torch.where(s[:, None, :, None] > 0, p / s[:, None, :, None], torch.zeros_like(p))
    q = q.view(R * block, C * 128)[:rows, :K].clamp(-448.0, 448.0) + 0.0
    return q.to(torch.float8_e4m3fn).contiguous(), s


def _pack_fp4(x, g):
    """FP4 cache bytes of rows x [..., D]: codes, scales (padded to a multiple of 4), RoPE slice."""
    lead = x.shape[:-1]
    v = x[..., :DN].float().reshape(*lead, DN // 32, 32)
    s8 = (v.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = s8.float() * g
    q = torch.where(den[..., None] > 0, v / den[..., None], torch.zeros_like(v))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(q.abs(), edges).to(torch.uint8)
    code = torch.where((q < 0) & (code > 0), code | 8, code).reshape(*lead, DN)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    pad = (DN // 32 + 3) // 4 * 4
    scales = torch.zeros((*lead, pad), dtype=torch.uint8, device=x.device)
    scales[..., : DN // 32] = s8.view(torch.uint8)
    return codes.contiguous(), scales, x[..., DN:].contiguous()


def _pack_fp8(x):
    lead = x.shape[:-1]
    v = x[..., :DN].float().reshape(*lead, DN // 64, 64)
    s = v.abs().amax(-1) / 448.0
    q = torch.where(s[..., None] > 0, v / s[..., None], torch.zeros_like(v)).clamp(-448.0, 448.0) + 0.0
    codes = q.reshape(*lead, DN).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.zeros((*lead, (DN // 64 + 3) // 4 * 4), dtype=torch.float32, device=x.device)
    scales[..., : DN // 64] = s
    return codes.contiguous(), scales, x[..., DN:].contiguous()


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quant":
        x = _normal(g, case["rows"], case["K"])
        # channels of different strength, as hidden states and trained weights have them
        x *= torch.exp(0.5 * _normal(g, 1, case["K"]))
        return dict(x=x.to(torch.bfloat16))
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        xq, xs = _block_quant(_normal(g, M, K).to(torch.bfloat16), 1)
        w = [_block_quant((_normal(g, N, K) * K ** -0.5).to(torch.bfloat16), 128) for _ in range(2 if case["pair"] else 1)]
        return dict(xq=xq, xs=xs, w=w)
    if op == "readback":
        B, n, n_max = case["B"], case["n"], case["n_max"]
        rows = _normal(g, B, n_max, D).to(torch.bfloat16)
        gs = 2.0 ** case["gpow"] if case["gpow"] <= 0 else 0.05      # a power of two, or a scale that rounds
        d = dict(g=gs, idx=None, row0=None, table=None)
        if case["fmt"] == "fp4":
            codes, scales, rope = _pack_fp4(rows, gs)
            if case["page"]:
                ps = case["page"]
                width = -(-n_max // ps)
                perm = torch.randperm(B * width, generator=g, device="cuda").view(B, width)
                d["table"] = perm.to(torch.int32)

                def paged(t):
                    p = torch.zeros((B * width, ps, t.shape[-1]), dtype=t.dtype, device="cuda")
                    padded = torch.zeros((B, width * ps, t.shape[-1]), dtype=t.dtype, device="cuda")
                    padded[:, :n_max] = t
                    p[perm.view(-1)] = padded.view(B * width, ps, -1)
                    return p.view(B * width * ps, -1)
                codes, scales, rope = paged(codes), paged(scales), paged(rope)
        else:
            codes, scales, rope = _pack_fp8(rows)
        d.update(codes=codes, scales=scales, rope=rope)
        if case["ids"]:
            idx = torch.randint(0, n_max, (B, n), generator=g, device="cuda", dtype=torch.int32)
            drop = torch.rand((B, n), generator=g, device="cuda") < 0.05
            d["idx"] = torch.where(drop, torch.full_like(idx, -1), idx)
        else:
            d["row0"] = torch.randint(0, n_max - n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        return d
    B, Nq, H, P = case["B"], case["Nq"], case["H"], case["prefix"]
    n_max = P + case["own"]
    own_n = torch.randint(0, case["own"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    own_n[0] = case["own"]
    n_c = own_n + P
    t0 = RATIO * n_c.long() + torch.randint(0, RATIO - Nq + 1, (B,), generator=g, device="cuda")
    codes = torch.zeros((B, n_max, DN // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((B, n_max, 16), dtype=torch.uint8, device="cuda")
    rope = torch.zeros((B, n_max, DR), dtype=torch.bfloat16, device="cuda")
    c, s, r = _pack_fp4(_normal(g, B, case["own"], D).to(torch.bfloat16), 1.0)
    codes[:, P:], scales[:, P:], rope[:, P:] = c, s, r
    pc, ps, pr = _pack_fp4(_normal(g, P, D).to(torch.bfloat16), 1.0)
    prefix = torch.cat([_fp4_rows(pc, ps, 1.0).to(torch.bfloat16), pr], -1).contiguous()
    return dict(q=_normal(g, B, Nq, H, D).to(torch.bfloat16), q_pos=t0[:, None] + torch.arange(Nq, device="cuda"), n_c=n_c,
                codes=codes, scales=scales, rope=rope, prefix=prefix,
                win=_normal(g, B, WINDOW + Nq - 1, D).to(torch.bfloat16), win_pos0=t0 - WINDOW + 1)


def _fp4_rows(codes, scales, g):
    """fp32 values of the FP4 channels: E2M1 * E4M3 scale * global scale."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    lo, hi = lut[(codes & 15).long()], lut[(codes >> 4).long()]
    v = torch.stack([lo, hi], -1).reshape(*codes.shape[:-1], -1)
    s = scales[..., : DN // 32].contiguous().view(torch.float8_e4m3fn).float()
    return (v.view(*v.shape[:-1], -1, 32) * s[..., None] * g).reshape(v.shape)


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = dict(case)
    if not own:
        return d
    import compressed_sparse_attention_18_b200 as csa
    op = case["op"]
    if op == "product":
        d["x8"] = csa.Fp8Blocks(d["xq"].view(torch.uint8), d["xs"], 1)
        d["w8"] = [csa.Fp8Blocks(q.view(torch.uint8), s, 128) for q, s in d["w"]]
    elif op == "readback":
        B, n_max = case["B"], case["n_max"]
        if case["fmt"] == "fp8":
            cache = csa.Fp8Window(B, n_max, D, DR, "cuda")
        elif case["page"]:
            cache = csa.PagedCache(B, n_max, D, DR, "cuda", case["page"], d["table"].numel(), d["table"], d["g"])
        else:
            cache = csa.PackedCache(B, n_max, D, DR, "cuda", d["g"])
        cache.codes, cache.scales, cache.rope = d["codes"], d["scales"], d["rope"]
        d["cache"] = cache
    elif op == "shared":
        cache = csa.PackedCache(case["B"], d["codes"].shape[1], D, DR, "cuda", 1.0)
        cache.codes, cache.scales, cache.rope = d["codes"], d["scales"], d["rope"]
        d["cache"] = cache
    return d


# ------------------------------------------------------------------------------------------ passes

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(d):
    import compressed_sparse_attention_18_b200 as csa
    case = d["case"]
    op = case["op"]
    if op == "quant":
        q = csa.quant_fp8(d["x"], block_rows=case["block"])
        return dict(values=q.codes.view(torch.float8_e4m3fn), scales=q.scales)
    if op == "product":
        return list(csa.gemm_fp8(d["x8"], *d["w8"]))
    if op == "readback":
        read = csa.unpack_fp4 if case["fmt"] == "fp4" else csa.unpack_fp8_window
        return read(d["cache"], n=case["n"], row0=d["row0"], idx=d["idx"])
    out, lse = csa.hca_shared_attn(d["q"], d["q_pos"], d["cache"], d["n_c"], d["prefix"], d["win"], d["win_pos0"],
                                   ratio=RATIO, window=WINDOW)
    return dict(out=out, lse=lse)


def _run_plain(d):
    case = d["case"]
    op = case["op"]
    if op == "quant":
        q, s = _block_quant(d["x"], case["block"])
        return dict(values=q, scales=s)
    if op == "product":
        K = case["K"]
        x = d["xq"].float() * d["xs"].repeat_interleave(128, 1)[:, :K]
        outs = []
        for q, s in d["w"]:
            w = q.float() * s.repeat_interleave(128, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, :K]
            outs.append((x @ w.T).to(torch.bfloat16))
        return outs
    if op == "readback":
        return _readback_plain(d, case)
    return _shared_plain(d, case)


def _pick(t, rows, valid):
    out = t.reshape(-1, t.shape[-1])[rows.clamp(min=0)]
    return torch.where(valid[..., None], out, torch.zeros_like(out))


def _readback_plain(d, case):
    B, n, n_max = case["B"], case["n"], case["n_max"]
    if d["idx"] is not None:
        i = d["idx"].long()
    else:
        i = d["row0"].long()[:, None] + torch.arange(n, device="cuda")
    valid = i >= 0
    b = torch.arange(B, device="cuda")[:, None]
    if d["table"] is not None:
        ps = case["page"]
        rows = d["table"].long()[b, i.clamp(min=0) // ps] * ps + i.clamp(min=0) % ps
    else:
        rows = b * n_max + i.clamp(min=0)
    codes, scales, rope = (_pick(d[k], rows, valid) for k in ("codes", "scales", "rope"))
    if case["fmt"] == "fp4":
        v = _fp4_rows(codes, scales, d["g"])
    else:
        c = codes.view(torch.float8_e4m3fn).float()
        v = (c.view(B, n, -1, 64) * scales[..., : DN // 64, None]).view(B, n, DN)
    return torch.cat([v.to(torch.bfloat16), rope], -1)


def _shared_plain(d, case):
    B, Nq, H, P = case["B"], case["Nq"], case["H"], case["prefix"]
    q = d["q"].float().view(B, Nq * H, D)
    pre = d["prefix"].float()
    own_rows = torch.cat([_fp4_rows(d["codes"][:, P:], d["scales"][:, P:], 1.0), d["rope"][:, P:].float()], -1)
    win = d["win"].float()
    t = d["q_pos"]
    scale = D ** -0.5
    zp = (q.reshape(-1, D) @ pre.T).view(B, Nq, H, P)
    zo = (q @ own_rows.transpose(1, 2)).view(B, Nq, H, -1)
    zw = (q @ win.transpose(1, 2)).view(B, Nq, H, -1)
    i = torch.arange(P + own_rows.shape[1], device="cuda")
    vis = (i < d["n_c"][:, None, None]) & (RATIO * i + RATIO - 1 <= t[..., None])
    pos = d["win_pos0"][:, None, None] + torch.arange(win.shape[1], device="cuda")
    wvis = (pos >= 0) & (pos <= t[..., None]) & (pos > t[..., None] - WINDOW)
    mask = torch.cat([vis, wvis], -1)[:, :, None]
    z = torch.cat([zp, zo, zw], -1) * scale
    z = torch.where(mask, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    n_own = own_rows.shape[1]
    o = (p[..., :P].reshape(-1, P) @ pre).view(B, Nq * H, D)
    o = o + p[..., P:P + n_own].reshape(B, Nq * H, n_own) @ own_rows
    o = o + p[..., P + n_own:].reshape(B, Nq * H, -1) @ win
    out = o.view(B, Nq, H, D) / l
    return dict(out=out.to(torch.bfloat16), lse=(m + torch.log(l)).squeeze(-1))


# ------------------------------------------------------------------------------------------- costs

def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["K"]
        blocks = -(-case["rows"] // case["block"]) * -(-case["K"] // 128)
        return dict(bytes=3 * n + 4 * blocks, flops=2 * n)
    if op == "product":
        M, N, K, w = case["M"], case["N"], case["K"], 2 if case["pair"] else 1
        kb = -(-K // 128)
        return dict(bytes=M * K + 4 * M * kb + w * (N * K + 4 * -(-N // 128) * kb + 2 * M * N), flops=2 * w * M * N * K)
    if op == "readback":
        rows = case["B"] * case["n"]
        entry = 2 * DR + (DN // 2 + DN // 32 if case["fmt"] == "fp4" else DN + 4 * (DN // 64))
        ids = 4 * rows if case["ids"] else 4 * case["B"]
        return dict(bytes=rows * (entry + 2 * D) + ids, flops=rows * DN)
    B, Nq, H, P = case["B"], case["Nq"], case["H"], case["prefix"]
    rows = B * Nq * H
    entry = DN // 2 + DN // 32 + 2 * DR
    own_n = case["own"] * (B + 1) / (2 * B) if B else 0            # every count in 0 .. own is as likely; one is full
    keys = P + own_n + WINDOW
    return dict(bytes=int(rows * (4 * D + 4) + P * 2 * D + B * (own_n * entry + (WINDOW + Nq - 1) * 2 * D)),
                flops=int(4 * D * rows * keys))


# -------------------------------------------------------------------------- the definition in 64 bits

def _e4m3_64(byte):
    """The value of an E4M3 byte from its fields: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = byte.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.pow(2.0, (e - 10).double()))
    return torch.where(b >= 128, -v, v)


def _e2m1_64(nib):
    """The value of an E2M1 code from its fields: sign, 2 exponent bits (bias 1), 1 mantissa bit."""
    n = nib.long()
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    return torch.where(n >= 8, -v, v)


def _near_e4m3(x):
    """x (64 bits) rounded to the nearest E4M3 value, ties to even, at most 448."""
    a = x.abs().clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _entry64(codes, scales, rope, g):
    """64-bit rows [.., D] of FP4 entries."""
    out = torch.empty((*codes.shape[:-1], D), dtype=torch.float64, device=codes.device)
    sc = _e4m3_64(scales[..., : DN // 32]).repeat_interleave(32, -1) * g
    out[..., 0:DN:2] = _e2m1_64(codes & 15) * sc[..., 0::2]
    out[..., 1:DN:2] = _e2m1_64(codes >> 4) * sc[..., 1::2]
    out[..., DN:] = rope.double()
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "quant":
        x, blk = d["x"].double(), case["block"]
        scales = torch.stack([torch.stack([c.abs().max() for c in r.split(128, 1)]) for r in x.split(blk, 0)]) / 448.0 \
            if blk > 1 else torch.stack([c.abs().amax(1) for c in x.split(128, 1)], 1) / 448.0
        full = scales.repeat_interleave(blk, 0)[: x.shape[0]].repeat_interleave(128, 1)[:, : x.shape[1]]
        return dict(values=_near_e4m3(torch.nan_to_num(x / full)), scales=scales)
    if op == "product":
        K, outs = case["K"], []
        for q, s in d["w"]:
            acc = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
            for kb, k0 in enumerate(range(0, K, 128)):
                part = _e4m3_64(d["xq"][:, k0:k0 + 128].view(torch.uint8)) @ _e4m3_64(q[:, k0:k0 + 128].view(torch.uint8)).T
                sw = s[:, kb].double()[torch.arange(case["N"], device="cuda") // 128]
                acc += part * d["xs"][:, kb].double()[:, None] * sw[None, :]
            outs.append(acc)
        return outs
    if op == "readback":
        B, n, n_max, ps = case["B"], case["n"], case["n_max"], case["page"]
        out = torch.zeros((B, n, D), dtype=torch.float64, device="cuda")
        for b in range(B):
            i = d["idx"][b].long() if d["idx"] is not None else d["row0"][b].long() + torch.arange(n, device="cuda")
            at = (i >= 0).nonzero()[:, 0]
            i = i[at]
            if ps:
                j = d["table"][b].long()[i // ps] * ps + i % ps
                codes, scales, rope = d["codes"][j], d["scales"][j], d["rope"][j]
            else:
                codes, scales, rope = d["codes"][b, i], d["scales"][b, i], d["rope"][b, i]
            if case["fmt"] == "fp4":
                out[b, at] = _entry64(codes, scales, rope, d["g"])
            else:
                out[b, at, :DN] = _e4m3_64(codes) * scales[:, : DN // 64].double().repeat_interleave(64, 1)
                out[b, at, DN:] = rope.double()
        return out
    B, Nq, H, P = case["B"], case["Nq"], case["H"], case["prefix"]
    out = torch.empty((B, Nq, H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, Nq, H), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(d["n_c"][b])
        ent = torch.cat([d["prefix"].double(), _entry64(d["codes"][b, P:n], d["scales"][b, P:n], d["rope"][b, P:n], 1.0)])
        for j in range(Nq):
            t = int(d["q_pos"][b, j])
            see = min(n, (t + 1) // RATIO)
            w0 = int(d["win_pos0"][b])
            lo, hi = max(0, t - WINDOW + 1, w0), min(t, w0 + d["win"].shape[1] - 1)
            keys = torch.cat([ent[:see], d["win"][b, lo - w0:hi - w0 + 1].double()])
            z = (d["q"][b, j].double() @ keys.T) / math.sqrt(D)
            lse[b, j] = torch.logsumexp(z, -1)
            out[b, j] = torch.exp(z - lse[b, j][:, None]) @ keys
    return dict(out=out, lse=lse)
