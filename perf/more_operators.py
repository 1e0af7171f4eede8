"""Cases of the grouped-attention operators: what they compute in plain form, and the calls of this package.

The softmax attention layer of a hybrid, with Hq query heads that share Hk heads of keys and values:

  prologue      RMS norm of every query and key head, and the rotation by its token's position, from raw projections
  prologue_bwd  its gradients: of the raw projections, and of the two norm weights (sums over tokens and heads)
  fwd           causal attention over packed sequences of different lengths, whole prompts or the last rows of longer ones
  bwd           its gradients, of the queries and of the shared keys and values
  append        new tokens into a paged cache of 8-bit values with one scale for 16 tokens of a head
  step          one token a sequence over that cache
"""
import math

import torch

own = False

BLOCK = 16    # tokens that share a scale
TOP = 448.0   # largest e4m3 value


def listed():
    return [
        # One decode step of a serving batch at far positions: latency counts.
        dict(name="prologue decode batch", op="prologue", lens=" ".join(["1"] * 64), Hq=32, Hk=8, D=128, R=128, far=262144, dtype="bf16"),
        # Prompts of several users, cut out of one fused projection.
        dict(name="prologue prompts", op="prologue", lens="9001 4096 2047 1240", Hq=32, Hk=8, D=128, R=128, far=0, dtype="bf16"),
        # Gradients in full precision at a size where launches count, half of the channels rotated.
        dict(name="prologue_bwd fp32 small", op="prologue_bwd", lens="257 31", Hq=8, Hk=2, D=64, R=32, far=0, dtype="fp32"),
        # A training step on a packed batch.
        dict(name="prologue_bwd training batch", op="prologue_bwd", lens="4999 1763 801 402 177 49 1", Hq=32, Hk=8, D=128, R=64,
             far=0, dtype="bf16"),
        # Short prompts in full precision, as a numerical check of a model runs them.
        dict(name="fwd fp32 short prompts", op="fwd", lens="401 130 64 17 1", past=0, Hq=8, Hk=2, D=64, dtype="fp32"),
        # Prefill of a packed batch: one long prompt among shorter ones, down to a single token.
        dict(name="fwd packed prompts", op="fwd", lens="4999 1763 801 402 177 49 1", past=0, Hq=32, Hk=8, D=128, dtype="bf16"),
        # Gradients of one short sequence: latency counts.
        dict(name="bwd short sequence", op="bwd", lens="333", past=0, Hq=16, Hk=4, D=64, dtype="bf16"),
        # A training step on a packed batch.
        dict(name="bwd packed batch", op="bwd", lens="4999 1763 801 402 177 49 1", past=0, Hq=16, Hk=4, D=128, dtype="bf16"),
        # One new token of every sequence of a serving batch.
        dict(name="append tokens", op="append", N=64, new=1, len=2100, Hk=8, D=128, page=64, dtype="bf16"),
        # Whole prompts and chunks of them.
        dict(name="append prompts", op="append", N=6, new=2731, len=4100, Hk=8, D=128, page=64, dtype="bf16"),
        # One user, one token: the smallest call.
        dict(name="step one user", op="step", N=1, len=300, Hq=32, Hk=8, D=128, page=64, dtype="bf16"),
        # A serving batch with long contexts, ragged, small pages.
        dict(name="step serving batch", op="step", N=64, len=16384, Hq=32, Hk=4, D=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total):
    """A packed batch: up to nine sequences of very different lengths, empty ones among them."""
    lens = []
    while total > 0 and len(lens) < 8:
        lens.append(_log(rng, 1, total))
        total -= lens[-1]
    if rng.random() < 0.3:
        lens.insert(rng.randrange(len(lens) + 1), 0)
    return " ".join(map(str, lens))


def draw(rng):
    op = rng.choice(("prologue", "prologue_bwd", "fwd", "bwd", "append", "step"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    D = rng.choice((64, 128, 128))
    Hk = rng.choice((1, 2, 3, 4, 8, 16))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    while Hk * G > 64:
        G = rng.choice((1, 2, 3, 4))
    c = dict(op=op, Hk=Hk, D=D, dtype=dtype)
    if op in ("prologue", "prologue_bwd"):
        most = 16384 * 40 * 128 // (2 if op == "prologue_bwd" else 1) // (2 if dtype == "fp32" else 1)
        c.update(Hq=Hk * G, lens=_split(rng, _log(rng, 1, most // ((Hk * G + Hk) * D))), R=rng.choice((D, D, D // 2, 16)),
                 far=rng.choice((0, 0, 4096, 1000000)))
        return c
    if op in ("fwd", "bwd"):
        most = (32 if op == "fwd" else 16) * 4999 * 4999 // (16 if dtype == "fp32" else 1)
        total = _log(rng, 1, min(8192, math.isqrt(most // (Hk * G))))
        past = _log(rng, 1, 500) if op == "fwd" and rng.random() < 0.3 else 0
        c.update(Hq=Hk * G, lens=_split(rng, total), past=past)
        return c
    page = rng.choice((16, 32, 48, 64, 128, 256))
    if op == "append":
        while True:
            new = 1 if rng.random() < 0.4 else _log(rng, 1, 4096)
            c.update(N=_log(rng, 1, 128), new=new, len=new + _log(rng, 1, 2048), page=page)
            if c["N"] * new * Hk * D <= 6 * 2731 * 8 * 128 and c["N"] * c["len"] * Hk * D <= 64 * 2100 * 8 * 128:
                return c
    while True:
        c.update(N=_log(rng, 1, 256), len=_log(rng, 1, 65536), Hq=Hk * G, page=page)
        if c["N"] * c["len"] * Hk * D <= 64 * 16384 * 4 * 128 and c["N"] * c["len"] * c["Hq"] <= 64 * 16384 * 32:
            return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _seqs(case):
    """Lengths of a packed batch."""
    return [int(n) for n in case["lens"].split()]


def _starts(lens):
    """Row offsets of packed sequences, int32."""
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _lens(case):
    """Cached lengths of a batch: from the full length down to half of it (no fewer than its new tokens), spread evenly."""
    N, full = case["N"], case["len"]
    return [max(full - (i * full) // (2 * N), _news(case)[i]) for i in range(N)]


def _news(case):
    """New tokens of each sequence: the full number down to half of it."""
    N, new = case["N"], case.get("new", 1)
    return [new - (i * new) // (2 * N) for i in range(N)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, D, Hk, op = _dtype(case), case["D"], case["Hk"], case["op"]
    Hq = case.get("Hq", 0)

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    s = dict(op=op)
    if op in ("prologue", "prologue_bwd"):
        lens, R = _seqs(case), case["R"]
        T = sum(lens)
        # queries, keys and values come out of one projection
        fused = normal(T, Hq + 2 * Hk, D)
        starts = torch.cat([torch.full((n,), 0 if not case["far"] else (case["far"] * (i + 1)) // len(lens) - 1)
                            for i, n in enumerate(lens)])
        within = torch.cat([torch.arange(n) for n in lens])
        s.update(q_raw=fused[:, :Hq], k_raw=fused[:, Hq:Hq + Hk], eps=1e-6,
                 w_q=1 + 0.2 * normal(D, dtype=torch.float32), w_k=1 + 0.2 * normal(D, dtype=torch.float32),
                 inv_freq=(10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda(),
                 pos=(starts + within).to(torch.int32).cuda())
        if op == "prologue_bwd":
            s.update(d_q=normal(T, Hq, D), d_k=normal(T, Hk, D))
        return s
    s["scale"] = 1.0 / math.sqrt(D)
    if op in ("fwd", "bwd"):
        keys = [n + case["past"] if n else 0 for n in _seqs(case)]
        T, Tk = sum(_seqs(case)), sum(keys)
        s.update(q=normal(T, Hq, D), k=normal(Tk, Hk, D), v=normal(Tk, 2 * Hk, D)[:, Hk:], cu_q=_starts(_seqs(case)),
                 cu_k=_starts(keys) if case["past"] else None)
        if op == "bwd":
            # what the forward pass of the same step left in hand
            s["o"], s["lse"] = _attention(s)
            s["d_o"] = normal(T, Hq, D)
        return s
    N, page = case["N"], case["page"]
    width = -(-case["len"] // page)
    pages = N * width + 3
    lens, news = _lens(case), _news(case)
    order = torch.randperm(N, generator=g, device="cuda").tolist()
    lens, news = [lens[i] for i in order], [news[i] for i in order]

    def stored(*shape):
        # values as an earlier append left them: scaled into e4m3's range
        return (normal(*shape, dtype=torch.bfloat16) * 70).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)

    def scales():
        return torch.exp2(torch.randint(-7, -4, (pages, Hk, page // BLOCK), generator=g, device="cuda").float())

    s.update(k_cache=stored(pages, Hk, page, D), v_cache=stored(pages, Hk, page // BLOCK, D, BLOCK), k_scale=scales(), v_scale=scales(),
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             table=torch.randperm(pages, generator=g, device="cuda")[:N * width].reshape(N, width).to(torch.int32))
    if op == "append":
        T = sum(news)
        s.update(k=normal(T, Hk, D), v=normal(T, 2 * Hk, D)[:, Hk:], cu=None if case["new"] == 1 else _starts(news))
    else:
        s["q"] = normal(N, Hq, D)
    return s


def _angles(s):
    """Cosines and sines [T, 1, R / 2]: far positions need the angle in 64 bits."""
    a = s["pos"].double()[:, None, None] * s["inv_freq"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def _rotated(x, cos, sin):
    h = cos.shape[-1]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]), -1)


def _prologue(s):
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q_raw"], s["w_q"]), (s["k_raw"], s["w_k"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w
        out.append(_rotated(y, cos, sin).to(x.dtype))
    return tuple(out)


def _prologue_gradients(s):
    cos, sin = _angles(s)
    out = {}
    for n, x, w, d in (("q", s["q_raw"], s["w_q"], s["d_q"]), ("k", s["k_raw"], s["w_k"], s["d_k"])):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + s["eps"])
        z = _rotated(d.float(), cos, -sin)   # the rotation's transpose
        xn = x32 * r
        wz = z * w
        out["d%s_raw" % n] = (r * (wz - xn * (wz * xn).mean(-1, keepdim=True))).to(x.dtype)
        out["dw_" + n] = (z * xn).sum((0, 1), dtype=torch.float64).float()
    return out


def _visible(s):
    """[Tq, Tk]: which keys a packed query row sees."""
    cu_q = s["cu_q"].long()
    cu_k = cu_q if s["cu_k"] is None else s["cu_k"].long()
    i, j = torch.arange(s["q"].shape[0], device="cuda"), torch.arange(s["k"].shape[0], device="cuda")
    bi, bj = torch.searchsorted(cu_q[1:], i, right=True), torch.searchsorted(cu_k[1:], j, right=True)
    place = i + (cu_k[bi + 1] - cu_q[bi + 1])   # a row's own key
    return (bi[:, None] == bj) & (j <= place[:, None])


def _heads(s):
    """q, k, v as [Hq, T, D] in 32 bits, keys and values repeated for the heads that share them."""
    q, k, v = s["q"].float().transpose(0, 1), s["k"].float().transpose(0, 1), s["v"].float().transpose(0, 1)
    G = q.shape[0] // k.shape[0]
    return q, k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)


def _attention(s):
    q, k, v = _heads(s)
    a = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).masked_fill_(~_visible(s), -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p / torch.where(total == 0, 1.0, total), v)
    return o.transpose(0, 1).to(s["q"].dtype).contiguous(), (top + torch.log(total))[..., 0].T.contiguous()


def _gradients(s):
    q, k, v = _heads(s)
    Hk, dt = s["k"].shape[1], s["q"].dtype
    d_o = s["d_o"].float().transpose(0, 1)
    a = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    p = torch.exp(a - s["lse"].T[..., None]).masked_fill_(~_visible(s), 0.0)
    del a
    ds = torch.matmul(d_o, v.transpose(1, 2))
    ds = p * (ds - (p * ds).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k).transpose(0, 1).to(dt)

    def shared(x):   # the sum over the query heads of a group
        return x.reshape(Hk, -1, *x.shape[1:]).sum(1).transpose(0, 1).to(dt)

    return dict(dq=dq, dk=shared(torch.matmul(ds.transpose(1, 2), q)), dv=shared(torch.matmul(p.transpose(1, 2), d_o)))


def _scale_of(amax):
    """The smallest power of two (2^-126 or more) that takes amax to 448 or less: 448 is 0.875 2^9."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e - 9 + (m > 0.875), -126).clamp_(min=-126))


def _append(s):
    """New tokens into their blocks.  A block that a larger value joins takes a larger scale, and what it holds moves to it."""
    page = s["k_cache"].shape[2]
    bpp = page // BLOCK
    N, T = s["lens"].shape[0], s["k"].shape[0]
    lens = s["lens"].long()
    cu = torch.arange(N + 1, device="cuda") if s["cu"] is None else s["cu"].long()
    t = torch.arange(T, device="cuda")
    n = torch.searchsorted(cu[1:], t, right=True)
    first = lens - (cu[1:] - cu[:-1])      # positions of the first new tokens
    at = first[n] + t - cu[n]
    pg = s["table"].long()[n, at // page]
    block = pg * bpp + at % page // BLOCK  # of all blocks of the cache
    # blocks that begin with older tokens: one a sequence at most
    old = torch.where(first % BLOCK > 0, first, 0)
    opg = s["table"].long()[torch.arange(N, device="cuda"), old // page]
    oblk, kept = old % page // BLOCK, first % BLOCK
    slots = torch.arange(BLOCK, device="cuda")
    for x, cache, scale, transposed in ((s["k"], s["k_cache"], s["k_scale"], False), (s["v"], s["v_cache"], s["v_scale"], True)):
        x = x.float()
        Hk, D = x.shape[1:]
        flat = scale.transpose(1, 2).reshape(-1, Hk)   # [blocks, Hk]
        amax = torch.zeros_like(flat).index_reduce_(0, block, x.abs().amax(-1), "amax")
        want = torch.zeros_like(flat).index_copy_(0, block, _scale_of(amax)[block])
        before = flat[opg * bpp + oblk]
        grown = torch.where((kept > 0)[:, None], torch.maximum(before, want[opg * bpp + oblk]), want[opg * bpp + oblk])
        want[opg * bpp + oblk] = torch.where((kept > 0)[:, None], grown, want[opg * bpp + oblk])
        scale.copy_(torch.where(want > 0, want, flat).reshape(scale.shape[0], bpp, Hk).transpose(1, 2))
        bits = cache.view(torch.uint8)
        view = bits.reshape(bits.shape[0], Hk, bpp, D, BLOCK).transpose(3, 4) if transposed else bits.reshape(bits.shape[0], Hk, bpp, BLOCK, D)
        held = view[opg, :, oblk]           # [N, Hk, BLOCK, D]
        moved = (held.view(torch.float8_e4m3fn).float() * (before / torch.where(grown > 0, grown, 1.0))[:, :, None, None]).to(torch.float8_e4m3fn)
        mine = (slots < kept[:, None])[:, None, :, None]
        view[opg, :, oblk] = torch.where(mine, moved.view(torch.uint8), held)
        view[pg, :, at % page // BLOCK, at % BLOCK] = (x / want[block][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _step(s):
    q = s["q"].float()
    N, Hq, D = q.shape
    pages, Hk, page, _ = s["k_cache"].shape
    table = s["table"].long()
    k = s["k_cache"][table].float().reshape(N, -1, Hk, page // BLOCK, BLOCK, D) * s["k_scale"][table][..., None, None]
    v = s["v_cache"][table].float().reshape(N, -1, Hk, page // BLOCK, D, BLOCK) * s["v_scale"][table][..., None, None]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(N, Hk, -1, D)
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(N, Hk, -1, D)
    a = torch.matmul(q.reshape(N, Hk, -1, D), k.transpose(2, 3)) * s["scale"]
    see = torch.arange(k.shape[2], device="cuda") < s["lens"].long()[:, None]
    a = a.masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(a - a.amax(-1, keepdim=True))
    return torch.matmul(p / p.sum(-1, keepdim=True), v).reshape(N, Hq, D).to(s["q"].dtype)


def run(s):
    op = s["op"]
    if own:
        import gated_deltanet_layer_amd as gdn
        if op == "prologue":
            return gdn.attn_prologue(s["q_raw"], s["k_raw"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"], eps=s["eps"])
        if op == "prologue_bwd":
            return gdn.attn_prologue_bwd(s["q_raw"], s["k_raw"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"], s["d_q"], s["d_k"], eps=s["eps"])
        if op == "fwd":
            return gdn.attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"])
        if op == "bwd":
            return gdn.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["d_o"], s["cu_q"], s["cu_k"], scale=s["scale"])
        if op == "append":
            gdn.attn_append_(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], cu=s["cu"])
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return gdn.attn_step(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"], scale=s["scale"])
    plain = dict(prologue=_prologue, prologue_bwd=_prologue_gradients, fwd=_attention, bwd=_gradients, append=_append, step=_step)
    return plain[op](s)


def work(case):
    es, D, Hk, Hq, op = 2 if case["dtype"] == "bf16" else 4, case["D"], case["Hk"], case.get("Hq", 0), case["op"]
    if op in ("prologue", "prologue_bwd"):
        T = sum(_seqs(case))
        values = T * (Hq + Hk) * D
        ways = 2 if op == "prologue" else 3
        return dict(bytes=ways * values * es + 4 * T + (ways - 1) * 8 * D + 2 * case["R"], flops=(9 if op == "prologue" else 18) * values)
    if op in ("fwd", "bwd"):
        T, past = sum(_seqs(case)), case["past"]
        keys = sum(n + past for n in _seqs(case) if n)
        pairs = sum(n * past + n * (n + 1) // 2 for n in _seqs(case))
        q, kv, lse = T * Hq * D * es, 2 * keys * Hk * D * es, 4 * T * Hq
        if op == "fwd":
            return dict(bytes=2 * q + kv + lse, flops=4 * D * Hq * pairs)
        return dict(bytes=4 * q + 2 * kv + lse, flops=10 * D * Hq * pairs)
    N, page, live = case["N"], case["page"], sum(_lens(case))
    if op == "append":
        T = sum(_news(case))
        return dict(bytes=T * 2 * Hk * D * (es + 1) + T * 2 * Hk * 4 // BLOCK + 8 * N, flops=6 * T * Hk * D)
    return dict(bytes=live * Hk * (2 * D + 8 / BLOCK) + 2 * N * Hq * D * es + 4 * live // page + 4 * N, flops=4 * D * Hq * live)


def exact(case, seed):
    """The definitions in 64 bits, one sequence (and one head) at a time; gradients by differentiating."""
    s = prepare(case, seed)
    f, op = torch.float64, case["op"]
    if op in ("prologue", "prologue_bwd"):
        R = case["R"]
        out = {}
        turn = torch.polar(torch.ones((), dtype=f, device="cuda"), torch.outer(s["pos"].to(f), s["inv_freq"].to(f)))[:, None]
        for n in ("q", "k"):
            x, w = s[n + "_raw"].to(f).requires_grad_(), s["w_" + n].to(f).requires_grad_()
            with torch.set_grad_enabled(op == "prologue_bwd"):
                y = w * x / torch.sqrt(x.square().mean(-1, keepdim=True) + s["eps"])
                z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
                y = torch.cat((z.real, z.imag, y[..., R:]), -1)
            if op == "prologue":
                out[n] = y
            else:
                out["d%s_raw" % n], out["dw_" + n] = torch.autograd.grad(y, (x, w), s["d_" + n].to(f))
        return (out["q"], out["k"]) if op == "prologue" else out
    if op in ("fwd", "bwd"):
        Hq, G, D = case["Hq"], case["Hq"] // case["Hk"], case["D"]
        cu_q = s["cu_q"].tolist()
        cu_k = cu_q if s["cu_k"] is None else s["cu_k"].tolist()
        o, lse = torch.zeros(s["q"].shape, dtype=f, device="cuda"), torch.zeros(s["q"].shape[:2], dtype=f, device="cuda")
        d = {n: torch.zeros(s[n].shape, dtype=f, device="cuda") for n in "qkv"}
        for a, b, c, e in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
            if a == b:
                continue
            hidden = torch.ones(b - a, e - c, dtype=torch.bool, device="cuda").triu((e - c) - (b - a) + 1)
            for h in range(Hq):
                q, k, v = (x.to(f).requires_grad_(op == "bwd") for x in (s["q"][a:b, h], s["k"][c:e, h // G], s["v"][c:e, h // G]))
                x = (q @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                y = torch.exp(x - z[:, None]) @ v
                if op == "fwd":
                    o[a:b, h], lse[a:b, h] = y, z
                else:
                    gq, gk, gv = torch.autograd.grad(y, (q, k, v), s["d_o"][a:b, h].to(f))
                    d["q"][a:b, h] = gq
                    d["k"][c:e, h // G] += gk
                    d["v"][c:e, h // G] += gv
                    del gq, gk, gv
                del x, y, z
        return (o, lse) if op == "fwd" else dict(dq=d["q"], dk=d["k"], dv=d["v"])
    page, D = case["page"], case["D"]
    if op == "append":
        # block by block: real values over the block's scale (what is stored is these, rounded to e4m3)
        lens, table = s["lens"].tolist(), s["table"].tolist()
        cu = list(range(case["N"] + 1)) if s["cu"] is None else s["cu"].tolist()
        out = {}
        for n, turned in (("k", False), ("v", True)):
            scale = s[n + "_scale"].to(f)
            cache = s[n + "_cache"].to(f)
            x = s[n].to(f)
            for i, live in enumerate(lens):
                first = live - (cu[i + 1] - cu[i])
                for b in range(first // BLOCK, -(-live // BLOCK)):
                    lo, hi = max(first, b * BLOCK), min(live, (b + 1) * BLOCK)
                    if lo >= hi:
                        continue
                    p, j = table[i][b * BLOCK // page], b * BLOCK % page // BLOCK
                    rows = x[cu[i] + lo - first:cu[i] + hi - first]   # [tokens, Hk, D]
                    need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((0, 2)) / TOP)).clamp(min=-126))
                    held = cache[p, :, j].transpose(1, 2) if turned else cache[p, :, j * BLOCK:(j + 1) * BLOCK]   # [Hk, BLOCK, D]
                    if lo > b * BLOCK:
                        need = torch.maximum(need, scale[p, :, j])
                        held[:, :lo - b * BLOCK] *= (scale[p, :, j] / need)[:, None, None]
                    held[:, lo - b * BLOCK:hi - b * BLOCK] = rows.transpose(0, 1) / need[:, None, None]
                    scale[p, :, j] = need
            out[n + "_cache"], out[n + "_scale"] = cache, scale
        return out
    out, G = [], case["Hq"] // case["Hk"]
    for n, live in enumerate(s["lens"].tolist()):
        used = s["table"][n, :-(-live // page)].long()
        rows = []
        for h in range(case["Hk"]):
            k = s["k_cache"][used, h].to(f).reshape(-1, D)[:live] * s["k_scale"][used, h].to(f).reshape(-1).repeat_interleave(BLOCK)[:live, None]
            v = s["v_cache"][used, h].to(f).transpose(2, 3).reshape(-1, D)[:live]
            v = v * s["v_scale"][used, h].to(f).reshape(-1).repeat_interleave(BLOCK)[:live, None]
            rows.append(torch.softmax(s["q"][n, h * G:(h + 1) * G].to(f) @ k.T * s["scale"], -1) @ v)
        out.append(torch.cat(rows))
    return torch.stack(out)
