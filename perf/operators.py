"""Cases of the latent-attention operators: what they compute in plain form, and the calls of this package.

Latent attention keeps one latent vector and one rotary key a token for all heads.  It has two forms.  The
expanded form (prefill, training) works on the per-head keys and values that the up-projection makes of the
latents; the absorbed form (decode) works on the latents themselves, the up-projections folded into the query
and the output.

  fwd    expanded forward, causal, padded batches and chunked prefill
  bwd    its gradients: of q, of the expanded keys and values, of the rotary key that all heads share
  step   absorbed, one token a sequence over a paged cache
  steps  absorbed, M drafted tokens a sequence (a tree) over a paged cache and over each other
"""
import math

import torch

own = False

ROPE = 64  # width of the rotary part, in every case


def listed():
    return [
        # A short prompt of one user: latency counts.
        dict(name="fwd short prompt", op="fwd", B=1, Tq=333, Tk=333, H=16, dn=128, dv=128, dtype="bf16", ragged=False),
        # A padded batch in full precision, as a numerical check of a model runs it.
        dict(name="fwd fp32 padded batch", op="fwd", B=2, Tq=1021, Tk=1021, H=8, dn=64, dv=64, dtype="fp32", ragged=True),
        # Prefill of a long prompt, or the forward half of a training step on a long sequence.
        dict(name="fwd long prompt", op="fwd", B=1, Tq=8192, Tk=8192, H=16, dn=128, dv=128, dtype="bf16", ragged=False),
        # Gradients in full precision at a size where launches count.
        dict(name="bwd fp32 small", op="bwd", B=1, Tq=257, Tk=257, H=4, dn=64, dv=64, dtype="fp32", ragged=False),
        # A padded training batch.
        dict(name="bwd padded batch", op="bwd", B=4, Tq=1531, Tk=1531, H=16, dn=64, dv=128, dtype="bf16", ragged=True),
        # A training step on one long sequence.
        dict(name="bwd long sequence", op="bwd", B=1, Tq=8192, Tk=8192, H=16, dn=128, dv=128, dtype="bf16", ragged=False),
        # One user, one token: the smallest call.
        dict(name="step one user", op="step", N=1, H=16, r=512, len=300, page=64, dtype="bf16"),
        # A small batch in full precision with a narrower latent.
        dict(name="step fp32", op="step", N=8, H=16, r=256, len=2000, page=32, dtype="fp32"),
        # A serving batch with the heads of one of eight tensor-parallel ranks, ragged, small pages.
        dict(name="step serving batch", op="step", N=64, H=16, r=512, len=4100, page=16, dtype="bf16"),
        # A large data-parallel batch with all heads on one card, long contexts.
        dict(name="step large batch", op="step", N=128, H=128, r=512, len=8192, page=64, dtype="bf16"),
        # A small tree of drafts for two users.
        dict(name="steps small tree", op="steps", N=2, M=5, H=16, r=512, len=700, page=64, dtype="bf16"),
        # Wide trees for a batch: the verification step of speculative decoding.
        dict(name="steps batch of trees", op="steps", N=16, M=32, H=32, r=512, len=4096, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "bwd", "step", "steps"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op in ("fwd", "bwd"):
        most = 16 * 8192 * 8192 // (32 if dtype == "fp32" else 1)
        while True:
            Tk = _log(rng, 1, 8192)
            Tq = Tk if op == "bwd" or rng.random() < 0.6 else _log(rng, 1, Tk)
            c = dict(op=op, B=_log(rng, 1, 8), Tq=Tq, Tk=Tk, H=_log(rng, 1, 48), dn=rng.choice((64, 128)),
                     dv=rng.choice((64, 128)), dtype=dtype, ragged=rng.random() < 0.5)
            if c["B"] * c["H"] * Tq * Tk <= most:
                return c
    r = rng.choice((256, 512, 512))
    page = rng.choice((1, 16, 17, 32, 64, 100, 256))
    while True:
        c = dict(op=op, N=_log(rng, 1, 256), H=rng.choice((1, 4, 8, 16, 24, 40, 64, 128)), r=r, len=_log(rng, 1, 16384),
                 page=page, dtype=dtype)
        if op == "steps":
            c["M"] = _log(rng, 1, 64)
        rows = c["H"] * c.get("M", 1)
        if c["N"] * c["len"] <= (1 << 20) // (4 if dtype == "fp32" else 1) and \
                c["N"] * c["len"] * rows <= (1 << 26) // (8 if dtype == "fp32" else 1):
            return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    """Live lengths of a batch: from the full length down to half of it, spread evenly."""
    if case["op"] in ("fwd", "bwd"):
        n, full = case["B"], case["Tk"]
        if not case["ragged"]:
            return [full] * n
    else:
        n, full = case["N"], case["len"]
    return [full - (i * full) // (2 * n) for i in range(n)]


def _scale(case):
    return 1.0 / math.sqrt(case.get("dn", 128) + ROPE)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    s = dict(case=case, op=case["op"], scale=_scale(case))
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(len(lens), generator=g, device="cuda")]
    if case["op"] in ("fwd", "bwd"):
        B, Tq, Tk, H, dn, dv = (case[k] for k in ("B", "Tq", "Tk", "H", "dn", "dv"))
        s.update(q=normal(B, Tq, H, dn + ROPE), kv=normal(B, Tk, H, dn + dv), k_rope=normal(B, Tk, ROPE),
                 lens=lens if case["ragged"] else None)
        if case["op"] == "bwd":
            # what the forward pass of the same step left in hand
            s["o"], s["lse"] = _expanded(s)
            s["d_o"] = normal(B, Tq, H, dv)
        return s
    N, H, r, page = (case[k] for k in ("N", "H", "r", "page"))
    width = -(-case["len"] // page)
    pages = N * width + 3
    s.update(cache=normal(pages, page, r + ROPE), lens=lens,
             table=torch.randperm(pages, generator=g, device="cuda")[:N * width].reshape(N, width).to(torch.int32))
    if case["op"] == "step":
        s["q"] = normal(N, H, r + ROPE)
    else:
        M = case["M"]
        s["q"] = normal(N, M, H, r + ROPE)
        s["draft"] = normal(N, M, r + ROPE)
        # every node hangs from an earlier one, or from the last cached token
        parent = torch.floor(torch.rand(N, M, generator=g, device="cuda") * (torch.arange(M, device="cuda") + 1)).long() - 1
        tree = torch.zeros(N, M, dtype=torch.int64, device="cuda")
        for i in range(M):
            up = tree.gather(1, parent[:, i:i + 1].clamp(min=0))[:, 0] * (parent[:, i] >= 0)
            tree[:, i] = up | (1 << i if i < 63 else -(1 << 63))
        s["tree"] = tree
    return s


def _visible(s):
    """[B or 1, 1, Tq, Tk]: which keys a query row sees."""
    Tq, Tk = s["q"].shape[1], s["kv"].shape[1]
    pos = torch.arange(Tq, device="cuda")[:, None] + (Tk - Tq)
    key = torch.arange(Tk, device="cuda")
    see = (key <= pos)[None]
    if s["lens"] is not None:
        n = s["lens"].long()[:, None, None]
        see = see & (key < n) & (pos < n)
    return see[:, None]


def _heads(s):
    """q, k, v as [B, H, T, D] in 32 bits, the shared rotary key repeated for every head."""
    q, kv, k_rope = s["q"].float(), s["kv"].float(), s["k_rope"].float()
    dn = q.shape[-1] - k_rope.shape[-1]
    k = torch.cat((kv[..., :dn], k_rope[:, :, None].expand(-1, -1, kv.shape[2], -1)), -1)
    return q.transpose(1, 2), k.transpose(1, 2), kv[..., dn:].transpose(1, 2)


def _weights(score, see):
    """Softmax of the visible scores, zero for a row that sees none, and the log of its sum."""
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (top + torch.log(total))[..., 0]


def _expanded(s):
    q, k, v = _heads(s)
    p, lse = _weights(torch.matmul(q, k.transpose(2, 3)) * s["scale"], _visible(s))
    return torch.matmul(p, v).transpose(1, 2).to(s["q"].dtype).contiguous(), lse.transpose(1, 2).contiguous()


def _gradients(s):
    q, k, v = _heads(s)
    dn = q.shape[-1] - s["k_rope"].shape[-1]
    d_o = s["d_o"].float().transpose(1, 2)
    see = _visible(s)
    lse = s["lse"].transpose(1, 2)[..., None]
    p = torch.exp(torch.matmul(q, k.transpose(2, 3)) * s["scale"] - torch.where(lse == -math.inf, 0.0, lse)).masked_fill(~see, 0.0)
    dp = torch.matmul(d_o, v.transpose(2, 3))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    dv = torch.matmul(p.transpose(2, 3), d_o)
    dt = s["q"].dtype
    return dict(dq=dq.transpose(1, 2).to(dt), dkv=torch.cat((dk[..., :dn], dv), -1).transpose(1, 2).to(dt),
                dk_rope=dk[..., dn:].sum(1).to(dt))


def _absorbed(s):
    """Rows of one token or of M drafted tokens over the cache (and the drafts)."""
    q = s["q"].float()
    N, H, D = q.shape[0], q.shape[-2], q.shape[-1]
    M = q.shape[1] if q.dim() == 4 else 1
    r = D - ROPE
    page = s["cache"].shape[1]
    at = torch.arange(s["table"].shape[1] * page, device="cuda")
    keys = s["cache"].reshape(-1, D)[s["table"].long()[:, at // page] * page + at % page].float()
    see = (at < s["lens"].long()[:, None])[:, None].expand(-1, M, -1)
    if s["op"] == "steps":
        keys = torch.cat((keys, s["draft"].float()), 1)
        see = torch.cat((see, (s["tree"][:, :, None] >> torch.arange(M, device="cuda")) & 1 == 1), -1)
    score = torch.matmul(q.reshape(N, M * H, D), keys.transpose(1, 2)) * s["scale"]
    p, _ = _weights(score, see.repeat_interleave(H, 1))
    return torch.matmul(p, keys[..., :r]).reshape(*q.shape[:-1], r).to(s["q"].dtype)


def run(s):
    if own:
        import gated_deltanet_layer_amd as gdn
        if s["op"] == "fwd":
            return gdn.latent_fwd(s["q"], s["kv"], s["k_rope"], lens=s["lens"], scale=s["scale"])
        if s["op"] == "bwd":
            return gdn.latent_bwd(s["q"], s["kv"], s["k_rope"], s["o"], s["lse"], s["d_o"], lens=s["lens"], scale=s["scale"])
        if s["op"] == "step":
            return gdn.latent_step(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])
        return gdn.latent_steps(s["q"], s["draft"], s["tree"], s["cache"], s["table"], s["lens"], scale=s["scale"])
    if s["op"] == "fwd":
        return _expanded(s)
    if s["op"] == "bwd":
        return _gradients(s)
    return _absorbed(s)


def _pairs(case):
    """Visible (query, key) pairs of all sequences, one head."""
    n = 0
    off = case["Tk"] - case["Tq"]
    for live in _lens(case):
        rows = max(0, live - off)  # query rows that are no padding: positions off .. live - 1
        n += rows * (off + 1) + rows * (rows - 1) // 2
    return n


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("fwd", "bwd"):
        B, Tq, Tk, H, dn, dv = (case[k] for k in ("B", "Tq", "Tk", "H", "dn", "dv"))
        dk = dn + ROPE
        q, kv, kr, o, lse = B * Tq * H * dk * es, B * Tk * H * (dn + dv) * es, B * Tk * ROPE * es, B * Tq * H * dv * es, B * Tq * H * 4
        if case["op"] == "fwd":
            return dict(bytes=q + kv + kr + o + lse, flops=2 * H * _pairs(case) * (dk + dv))
        return dict(bytes=2 * (q + kv + kr + o) + lse, flops=2 * H * _pairs(case) * (3 * dk + 2 * dv))
    N, H, r, M = case["N"], case["H"], case["r"], case.get("M", 1)
    drafts = M if case["op"] == "steps" else 0
    live = sum(_lens(case))
    rows = live + N * drafts
    return dict(bytes=rows * (r + ROPE) * es + N * M * H * (2 * r + ROPE) * es + live * 4 // case["page"] + N * (4 + 8 * drafts),
                flops=2 * M * H * (rows if drafts else live) * (2 * r + ROPE))


def exact(case, seed):
    """The definitions in 64 bits, one sequence (and one head) at a time; gradients by differentiating the forward."""
    s = prepare(case, seed)
    f = torch.float64
    out = []
    if case["op"] in ("fwd", "bwd"):
        B, Tq, Tk, H, dn = (case[k] for k in ("B", "Tq", "Tk", "H", "dn"))
        o = torch.zeros(B, Tq, H, case["dv"], dtype=f, device="cuda")
        lse = torch.full((B, Tq, H), -math.inf, dtype=f, device="cuda")
        dq, dkv = torch.zeros(s["q"].shape, dtype=f, device="cuda"), torch.zeros(s["kv"].shape, dtype=f, device="cuda")
        dkr = torch.zeros(s["k_rope"].shape, dtype=f, device="cuda")
        for b in range(B):
            n = Tk if s["lens"] is None else int(s["lens"][b])
            rows = max(0, n - (Tk - Tq))
            if not rows:
                continue
            hidden = torch.ones(rows, n, dtype=torch.bool, device="cuda").triu(n - rows + 1)
            for h in range(H):
                q, kv, kr = (x.to(f).requires_grad_(case["op"] == "bwd")
                             for x in (s["q"][b, :rows, h], s["kv"][b, :n, h], s["k_rope"][b, :n]))
                a = (q[:, :dn] @ kv[:, :dn].T + q[:, dn:] @ kr.T) * s["scale"]
                a = a.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(a, 1)
                y = torch.exp(a - z[:, None]) @ kv[:, dn:]
                if case["op"] == "fwd":
                    o[b, :rows, h], lse[b, :rows, h] = y, z
                else:
                    gq, gkv, gkr = torch.autograd.grad(y, (q, kv, kr), s["d_o"][b, :rows, h].to(f))
                    dq[b, :rows, h], dkv[b, :n, h] = gq, gkv
                    dkr[b, :n] += gkr
                    del gq, gkv, gkr
                del a, z, y
        return (o, lse) if case["op"] == "fwd" else dict(dq=dq, dkv=dkv, dk_rope=dkr)
    r, page = case["r"], case["page"]
    for n, live in enumerate(s["lens"].tolist()):
        used = s["table"][n, :-(-live // page)].long()
        x = s["cache"][used].reshape(-1, r + ROPE)[:live].to(f)
        q = s["q"][n].to(f)
        if case["op"] == "step":
            out.append(torch.softmax(q @ x.T * s["scale"], -1) @ x[:, :r])
            continue
        M, H = q.shape[:2]
        x = torch.cat((x, s["draft"][n].to(f)))
        shut = torch.zeros(M, live + M, dtype=torch.bool)
        for i, bits in enumerate(s["tree"][n].tolist()):
            for j in range(M):
                shut[i, live + j] = not (bits >> j) & 1
        a = torch.matmul(q.reshape(M * H, -1), x.T).reshape(M, H, -1) * s["scale"]
        a = a.masked_fill(shut.cuda()[:, None], -math.inf)
        out.append((torch.softmax(a, -1).reshape(M * H, -1) @ x[:, :r]).reshape(M, H, r))
    return torch.stack(out)
