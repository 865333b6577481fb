"""What is measured of the operators that adapting a language model needs beside cross entropy: the
log-probabilities of given tokens over a large vocabulary, the clipped policy loss with a KL term and
the preference loss of paired answers with their gradients, layer norm with its gradient, and the
global gradient norm with clipping.

Tensors are row-major; T tokens, H hidden size, V vocabulary.  `run` computes an operator in its plain
form (elementary torch operations) or, where `own` is set, through this repository's entry points;
`exact` is the operator's definition in 64 bits.

A token whose target is -1 (a prompt's, padding) is not counted: log-probability 0, no gradient.
The 8-bit format of layer norm's checkpoint: blocks of 32 along a row share a power-of-two scale,
E = max(floor(log2 amax), -120) kept as the byte E + 127; elements q = round(x / 2^(E - 6)) within
[-127, 127].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CLIP = (0.2, 0.28)
BETA = 0.1


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # scoring one short answer: bound by reading the weights
        {"name": "token logp 64 tokens", "op": "logp", "dtype": "bf16", "T": 64, "V": 32000, "H": 2048, "masked": 0.0},
        # the reference model's log-probabilities of a batch, float32 with odd sizes; a fifth are prompts
        {"name": "token logp odd f32", "op": "logp", "dtype": "f32", "T": 2003, "V": 32003, "H": 1001, "masked": 0.2},
        # a policy step on sampled answers against a large vocabulary, half of the tokens prompts
        {"name": "policy 8k tokens 128k", "op": "policy", "dtype": "bf16", "T": 8192, "V": 131072, "H": 2048,
         "masked": 0.5, "kl": 0.04, "weighted": False},
        # odd sizes in float32, every sequence with the same weight, no reference model
        {"name": "policy odd f32", "op": "policy", "dtype": "f32", "T": 1000, "V": 50021, "H": 1001, "masked": 0.3,
         "kl": 0.0, "weighted": True},
        # one pair of short answers: a micro-batch of one
        {"name": "preference 1 pair", "op": "preference", "dtype": "bf16", "T": 96, "V": 32000, "H": 2048,
         "masked": 0.25, "pairs": 1, "average": False, "smoothing": 0.0},
        # a batch of pairs with a shared prompt each
        {"name": "preference 16 pairs", "op": "preference", "dtype": "bf16", "T": 6000, "V": 128256, "H": 2048,
         "masked": 0.4, "pairs": 16, "average": True, "smoothing": 0.1},
        # a decoding step's norm: launch latency; its checkpoint is read back
        {"name": "layernorm 32 tokens", "op": "layernorm", "dtype": "bf16", "T": 32, "H": 2048, "residual": True,
         "bias": True, "keep": True},
        # a whole batch (32 sequences of 2048 tokens) through one residual norm
        {"name": "layernorm 64k tokens", "op": "layernorm", "dtype": "bf16", "T": 65536, "H": 2048, "residual": True,
         "bias": True, "keep": False},
        # its gradient, from the 8-bit checkpoint
        {"name": "layernorm grad 64k tokens", "op": "layernorm_grad", "dtype": "bf16", "T": 65536, "H": 2048,
         "kept": True},
        # a wide, odd row in float32, from the residual sums themselves
        {"name": "layernorm grad odd f32", "op": "layernorm_grad", "dtype": "f32", "T": 2051, "H": 4100, "kept": False},
        # low-rank adapters' gradients: many small tensors, launch latency
        {"name": "clip 130 small", "op": "clip", "dtype": "bf16", "tensors": 130, "elements": 2000003},
        # the gradients of 16 blocks of a 2048-wide model (112 matrices), written beside them for the optimizer
        {"name": "clip 112 matrices f32", "op": "clip", "dtype": "f32", "tensors": 112, "elements": 973078528},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; half of them whole multiples of 64 where they can be."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 128:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["logp", "policy", "preference", "layernorm", "layernorm_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = {"op": op, "dtype": dtype}
    if op in ("logp", "policy", "preference"):
        c |= {"T": _size(rng, 1, 8192), "V": _size(rng, 1000, 131072), "H": _size(rng, 64, 4096),
              "masked": rng.choice([0.0, round(rng.uniform(0.05, 0.7), 2)])}
        if op == "policy":
            # (of a few tokens float32 log-probabilities do not tell the mean KL: its terms are near 0)
            c |= {"kl": rng.choice([0.0, 0.04]) if c["T"] >= 512 else 0.0, "weighted": rng.random() < 0.5}
        if op == "preference":
            c["T"] = max(4, c["T"])
            c |= {"pairs": rng.randint(1, max(1, min(32, c["T"] // 4))), "average": rng.random() < 0.5,
                  "smoothing": rng.choice([0.0, 0.1])}
        while c["T"] * c["V"] * c["H"] > (1 << 41 if dtype == "bf16" else 1 << 38):
            c["T" if c["T"] > 1024 else "V"] //= 2
    elif op in ("layernorm", "layernorm_grad"):
        c |= {"T": _size(rng, 1, 65536), "H": _size(rng, 64, 8192)}
        while c["T"] * c["H"] > 1 << 27:
            c["T"] //= 2
        if op == "layernorm":
            c |= {"residual": rng.random() < 0.7, "bias": rng.random() < 0.7, "keep": rng.random() < 0.5}
        else:
            c["kept"] = rng.random() < 0.5
    else:
        c |= {"tensors": _size(rng, 1, 400), "elements": _size(rng, 1000, 1 << 29)}
    return c


def _counted(case):
    """Counted tokens: exact, as the inputs are cut by the same numbers."""
    return case["T"] - int(case["masked"] * case["T"])


def work(case):
    s = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "clip":  # each gradient read, each clipped one written
        return {"bytes": 2 * s * case["elements"], "flops": 3 * case["elements"]}
    T, H = case["T"], case["H"]
    blocks = -(-H // 32)
    if op == "layernorm":  # x (and the residual) -> h, y, statistics, and the checkpoint written and read back
        b = T * H * s * (4 if case["residual"] else 2) + 8 * T + 2 * H * s
        if case["keep"]:
            b += T * (H + blocks) + T * (H + blocks + 2 * H)
        return {"bytes": b, "flops": 8 * T * H}
    if op == "layernorm_grad":  # dy, dh, the normalised rows or h -> dx and the weights' gradients
        return {"bytes": T * (3 * H * s + 4 + (H + blocks if case["kept"] else H * s + 4)) + H * s + 8 * H,
                "flops": 12 * T * H}
    n, V = _counted(case), case["V"]
    if op == "logp":
        return {"bytes": s * (n * H + V * H) + 12 * T, "flops": 2 * n * V * H}
    b = s * (n * H + T * H + 2 * V * H) + T * (8 + 4 + (20 if op == "policy" else 4))
    return {"bytes": b, "flops": 6 * n * V * H}


# ---- inputs ---------------------------------------------------------------------------------

def _ids(g, T, V, dev):
    """Token ids with p(rank) ~ 1 / rank over a shuffled vocabulary."""
    u = torch.rand(T, generator=g, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    return torch.randperm(V, generator=g, device=dev)[rank]


def _starts(g, T, n, dev):
    """Starts of n sequences of at least one token each that fill T tokens, and the end."""
    cuts = torch.randperm(T - 1, generator=g, device=dev)[:n - 1].add_(1).sort().values
    return torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])


def _prompts(starts, share, T):
    """Which tokens are their sequence's prompt: its first ones, `share` of all tokens in the sum."""
    t = torch.arange(T, device=starts.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    before = (starts.double() * share).floor().long()
    before[-1] = int(share * T)
    return t - starts[seq] < (before[1:] - before[:-1])[seq], seq


def _plain_logp(h, W, tgt):
    """Log-probabilities of the targets (0 where there is none), logits and their log-sum-exp, in float32."""
    logits = h.float() @ W.float().t()
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp_().sum(1, keepdim=True).log_()
    logp = (logits.gather(1, tgt.clamp(min=0)[:, None]) - lse).squeeze(1)
    return torch.where(tgt >= 0, logp, torch.zeros_like(logp)), logits, lse


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std)

    st = {"case": case}
    if op == "clip":
        # one buffer for all gradients, as a step's all-reduce has it; tensors of sizes a factor of 30 apart
        n, k = case["elements"], case["tensors"]
        part = torch.exp(torch.rand(k, generator=g, device=dev, dtype=torch.float64) * math.log(30.0))
        unit = 2048 if n // k > 1 << 20 else 1  # large ones are matrices of whole rows
        ends = ((part.cumsum(0) / part.sum() * (n // unit)).long() * unit).tolist()
        ends[-1] = n
        flat = torch.empty(n, dtype=dt, device=dev)
        for at in range(0, n, 1 << 26):
            flat[at:at + (1 << 26)] = normal(min(1 << 26, n - at), std=1e-3).to(dt)
        out = torch.empty_like(flat)
        begins = [0] + ends[:-1]
        return st | {"flat": flat, "out": out, "max_norm": 0.3e-3 * math.sqrt(n),
                     "grads": [flat[a:b] for a, b in zip(begins, ends)],
                     "outs": [out[a:b] for a, b in zip(begins, ends)]}
    T, H = case["T"], case["H"]
    if op in ("layernorm", "layernorm_grad"):
        loud = 1 + 15 * (torch.rand(H, generator=g, device=dev) < 0.005)  # a few loud channels
        st["gain"] = (1 + normal(H, std=0.2)).to(dt)
        rows = normal(T, H) * loud + normal(T, 1, std=0.5)
        if op == "layernorm":
            st |= {"x": rows.to(dt), "residual": normal(T, H, std=0.5).to(dt) if case["residual"] else None,
                   "bias": normal(H, std=0.1).to(dt) if case["bias"] else None}
            return st
        h = rows.to(dt)
        mean = h.float().mean(1, keepdim=True)
        rstd = torch.rsqrt((h.float() - mean).square().mean(1, keepdim=True) + EPS)
        st |= {"dy": normal(T, H, std=1e-3).to(dt), "dh": normal(T, H, std=1e-3).to(dt),
               "rstd": rstd.reshape(T).contiguous()}
        if case["kept"]:
            q, e = _pack((h.float() - mean) * rstd)
            st |= {"q": q, "e": e}
        else:
            st |= {"h": h, "mean": mean.reshape(T).contiguous()}
        return st
    V = case["V"]
    tgt = _ids(g, T, V, dev)
    W = normal(V, H, std=0.02)
    # a trained model's states lean towards their targets' rows, some little, some far
    lean = torch.rand(T, 1, generator=g, device=dev) * (10 / (0.02 * H))
    h = (normal(T, H) + lean * W[tgt] / 0.02).to(dt)
    W = W.to(dt)
    n = 2 * case["pairs"] if op == "preference" else max(1, min(16, T // 64))
    starts = _starts(g, T, n, dev)
    prompt, seq = _prompts(starts, case["masked"], T)
    tgt = torch.where(prompt, torch.full_like(tgt, -1), tgt)
    st |= {"h": h, "W": W, "targets": tgt}
    if op == "logp":
        return st
    logp = _plain_logp(h, W, tgt)[0]
    if op == "policy":
        # answers sampled from a policy some updates older; no ratio within 1e-3 of the clip, where
        # the gradient jumps and the last bits of a log-probability would decide
        d = normal(T, std=0.15)
        for edge in (math.log1p(-CLIP[0]), math.log1p(CLIP[1])):
            d = torch.where((d - edge).abs() < 1e-3, d + 2e-3, d)
        st |= {"old": logp - d, "advantages": normal(n)[seq].contiguous(),
               "ref": logp + normal(T, std=0.2) if case["kl"] else None, "weights": None}
        if case["weighted"]:  # the mean over the sequences of each one's mean
            count = torch.zeros(n, device=dev).index_add_(0, seq, (tgt >= 0).float())
            st["weights"] = (1 / (count.clamp(min=1) * n))[seq].contiguous()
    else:
        # a policy that has begun to learn: chosen answers above the reference model's, rejected ones below
        shift = (0.4 + normal(n, std=0.2).abs()) * (1 - 2 * ((torch.arange(n, device=dev) + 1) % 2))
        st |= {"starts": starts, "ref": logp + normal(T, std=0.2) + shift[seq]}
    return st


# ---- plain forms ----------------------------------------------------------------------------

def _pack(x):
    """The 8-bit blocks of a float32 matrix: q int8 [T, H], e uint8 [T, ceil(H / 32)]."""
    T, H = x.shape
    nb = -(-H // 32)
    p = torch.nn.functional.pad(x, (0, 32 * nb - H)).reshape(T, nb, 32)
    E = torch.frexp(p.abs().amax(2))[1].sub_(1).clamp_(-120, 127)
    q = torch.round(torch.ldexp(p, (6 - E).unsqueeze(2))).clamp_(-127, 127)
    return q.reshape(T, 32 * nb)[:, :H].to(torch.int8).contiguous(), (E + 127).to(torch.uint8)


def _unpack(q, e):
    return q.float() * torch.exp2(e.float() - 133).repeat_interleave(32, 1)[:, :q.shape[1]]


def _plain_policy(st, logp, counted):
    """Losses, their weighted sum, mean KL, clipped share, and the coefficients of softmax - onehot."""
    lp, A, zero = logp.double(), st["advantages"].double(), torch.zeros((), dtype=torch.float64, device=logp.device)
    count = counted.sum().clamp(min=1)
    w = counted / count if st["weights"] is None else st["weights"].double()
    w = torch.where(counted, w.double(), zero)
    r = torch.exp(lp - st["old"].double())
    full, cut = r * A, r.clamp(1 - CLIP[0], 1 + CLIP[1]) * A
    free = full <= cut
    loss = -torch.minimum(full, cut)
    c = torch.where(free, full, zero)
    kl = None
    if st["ref"] is not None:
        x = st["ref"].double() - lp
        k3 = torch.expm1(x) - x
        loss = loss + st["case"]["kl"] * k3
        c = c + st["case"]["kl"] * torch.expm1(x)
        kl = (torch.where(counted, k3, zero).sum() / count).float()
    loss = torch.where(counted, loss, zero)
    return {"loss": loss.float(), "total": (w * loss).sum().float(), "kl": kl,
            "clipped": ((counted & ~free).sum() / count).float()}, c * w


def _plain_preference(st, logp, counted):
    """Pair losses, their mean, rewards, and the coefficients of softmax - onehot."""
    case, starts, T = st["case"], st["starts"], logp.shape[0]
    n = starts.shape[0] - 1
    seq = torch.searchsorted(starts, torch.arange(T, device=logp.device), right=True) - 1
    diff = torch.where(counted, logp.double() - st["ref"].double(), torch.zeros((), dtype=torch.float64, device=logp.device))
    total = torch.zeros(n, dtype=torch.float64, device=logp.device).index_add_(0, seq, diff)
    share = torch.ones_like(total)
    if case["average"]:
        share = 1 / torch.zeros_like(total).index_add_(0, seq, counted.double()).clamp(min=1)
    rewards = (BETA * total * share).reshape(-1, 2)
    z, e = rewards[:, 0] - rewards[:, 1] - 0.25, case["smoothing"]
    loss = (1 - e) * torch.log1p(torch.exp(-z)) + e * torch.log1p(torch.exp(z))
    c = ((1 - e) * torch.sigmoid(-z) - e * torch.sigmoid(z)) * BETA / (n // 2)
    return {"loss": loss.float(), "mean": loss.mean().float(), "rewards": rewards.float()}, \
        torch.where(counted, (torch.stack([c, -c], 1).reshape(-1) * share)[seq], torch.zeros_like(diff))


def _plain(st):
    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "clip":
        x = st["flat"].float()
        norm = (x * x).sum(dtype=torch.float64).sqrt()
        scale = (st["max_norm"] / (norm + 1e-6)).clamp(max=1).float()
        return {"norm": norm.float(), "scale": scale, "clipped": (x * scale).to(dt)}
    if op == "layernorm":
        h = st["x"].float()
        h = h if st["residual"] is None else h + st["residual"].float()
        mean = h.mean(1, keepdim=True)
        rstd = torch.rsqrt((h - mean).square().mean(1, keepdim=True) + EPS)
        n = (h - mean) * rstd
        y = n * st["gain"].float()
        y = y if st["bias"] is None else y + st["bias"].float()
        return {"h": h.to(dt), "y": y.to(dt), "mean": mean.squeeze(1), "rstd": rstd.squeeze(1),
                "kept": _unpack(*_pack(n)).to(torch.bfloat16) if case["keep"] else None}
    if op == "layernorm_grad":
        rstd = st["rstd"][:, None]
        n = _unpack(st["q"], st["e"]) if case["kept"] else (st["h"].float() - st["mean"][:, None]) * rstd
        dy = st["dy"].float()
        a = dy * st["gain"].float()
        dx = st["dh"].float() + rstd * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgain": (dy * n).sum(0), "dbias": dy.sum(0)}
    h, W, tgt = st["h"], st["W"], st["targets"]
    logp, logits, lse = _plain_logp(h, W, tgt)
    if op == "logp":
        return logp
    counted = tgt >= 0
    out, c = (_plain_policy if op == "policy" else _plain_preference)(st, logp, counted)
    c = c.float()[:, None]
    d = logits.sub_(lse).exp_().mul_(c)
    d.scatter_add_(1, tgt.clamp(min=0)[:, None], -c)
    return out | {"logp": logp, "dh": (d @ W.float()).to(dt), "dW": (d.t() @ h.float()).to(dt)}


def run(state):
    if not own:
        return _plain(state)
    import spectral_correction_optimizer_amd as sco
    st, case = state, state["case"]
    op = case["op"]
    if op == "clip":
        r = sco.clip_grads(st["grads"], st["max_norm"], out=st["outs"])
        return {"norm": r.norm, "scale": r.scale, "clipped": st["out"]}
    if op == "layernorm":
        r = sco.layernorm(st["x"], st["gain"], bias=st["bias"], residual=st["residual"], eps=EPS, keep=case["keep"])
        return {"h": r.h, "y": r.y, "mean": r.mean, "rstd": r.rstd,
                "kept": sco.act_unpack(r.kept, torch.bfloat16) if case["keep"] else None}
    if op == "layernorm_grad":
        if case["kept"]:
            rows = sco.ActCheckpoint(st["q"], st["e"])
            dx, dgain, dbias = sco.layernorm_grad(st["dy"], st["gain"], st["rstd"], kept=rows, dh=st["dh"])
        else:
            dx, dgain, dbias = sco.layernorm_grad(st["dy"], st["gain"], st["rstd"], h=st["h"], mean=st["mean"],
                                                  dh=st["dh"])
        return {"dx": dx, "dgain": dgain, "dbias": dbias}
    if op == "logp":
        return sco.token_logp(st["h"], st["W"], st["targets"])
    if op == "policy":
        r = sco.policy_loss(st["h"], st["W"], st["targets"], st["old"], st["advantages"], ref_logp=st["ref"],
                            clip=CLIP, kl=case["kl"], weights=st["weights"])
        return {"loss": r.loss, "total": r.total, "kl": r.kl, "clipped": r.clipped, "logp": r.logp, "dh": r.dh,
                "dW": r.dW}
    r = sco.preference_loss(st["h"], st["W"], st["targets"], st["starts"], ref_logp=st["ref"], beta=BETA, margin=0.25,
                            smoothing=case["smoothing"], average=case["average"])
    return {"loss": r.loss, "mean": r.mean, "rewards": r.rewards, "logp": r.logp, "dh": r.dh, "dW": r.dW}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "clip":
        total = math.fsum(float(torch.linalg.vecdot(g.to(f64), g.to(f64))) for g in st["grads"])
        scale = min(1.0, st["max_norm"] / (math.sqrt(total) + 1e-6))
        one = torch.ones((), dtype=f64, device=st["flat"].device)
        return {"norm": one * math.sqrt(total), "scale": one * scale, "clipped": st["flat"].to(f64).mul_(scale)}
    T, H = case["T"], case["H"]
    if op == "layernorm":
        h = st["x"].to(f64)
        if st["residual"] is not None:
            h += st["residual"].to(f64)
        mu = h.sum(1) / H
        n = h - mu[:, None]
        rstd = 1 / ((n * n).sum(1) / H + EPS).sqrt()
        n *= rstd[:, None]
        y = n * st["gain"].to(f64)
        if st["bias"] is not None:
            y += st["bias"].to(f64)
        kept = None
        if case["keep"]:
            kept = torch.empty_like(n)
            for b in range(0, H, 32):
                x = n[:, b:b + 32]
                amax = x.abs().max(1, keepdim=True).values
                E = torch.log2(amax.clamp(min=2.0 ** -120)).floor()
                E = torch.where(torch.pow(2.0, E + 1) <= amax, E + 1, E)
                E = torch.where(torch.pow(2.0, E) > amax, E - 1, E).clamp(min=-120)
                unit = torch.pow(2.0, E) / 64
                kept[:, b:b + 32] = (x / unit).round().clamp(-127, 127) * unit
        return {"h": h, "y": y, "mean": mu, "rstd": rstd, "kept": kept}
    if op == "layernorm_grad":
        rs = st["rstd"].to(f64)
        if case["kept"]:
            unit = torch.pow(2.0, st["e"].to(f64) - 127) / 64
            n = st["q"].to(f64) * unit[:, torch.arange(H, device=unit.device) // 32]
        else:
            n = (st["h"].to(f64) - st["mean"].to(f64)[:, None]) * rs[:, None]
        dn = st["dy"].to(f64) * st["gain"].to(f64)
        dx = dn - dn.sum(1, keepdim=True) / H - n * (torch.linalg.vecdot(dn, n)[:, None] / H)
        return {"dx": dx * rs[:, None] + st["dh"].to(f64), "dgain": torch.linalg.vecdot(st["dy"].to(f64), n, dim=0),
                "dbias": st["dy"].to(f64).sum(0)}
    tgt = st["targets"]
    dev = tgt.device
    real = (tgt >= 0).nonzero().squeeze(1)
    k, y = real.numel(), tgt[real]
    at = torch.arange(k, device=dev)
    h, W = st["h"][real].to(f64), st["W"].to(f64)
    s = h @ W.t()
    lse = torch.logsumexp(s, 1)
    lp = s[at, y] - lse
    logp = torch.zeros(T, dtype=f64, device=dev)
    logp[real] = lp
    if op == "logp":
        return logp
    g = torch.zeros(k, dtype=f64, device=dev)  # derivative of the loss by each log-probability
    if op == "policy":
        A, ratio = st["advantages"][real].to(f64), torch.exp(lp - st["old"][real].to(f64))
        w = torch.full_like(lp, 1 / max(k, 1)) if st["weights"] is None else st["weights"][real].to(f64)
        stopped = ((A > 0) & (ratio > 1 + CLIP[1])) | ((A < 0) & (ratio < 1 - CLIP[0]))
        bound = torch.where(A > 0, 1 + CLIP[1], 1 - CLIP[0])
        each = -A * torch.where(stopped, bound, ratio)
        g -= torch.where(stopped, 0.0, A * ratio)
        out = {"kl": None}
        if st["ref"] is not None:
            q = torch.exp(st["ref"][real].to(f64) - lp)
            k3 = q - 1 - (st["ref"][real].to(f64) - lp)
            each = each + case["kl"] * k3
            g += case["kl"] * (1 - q)
            out["kl"] = k3.sum() / max(k, 1)
        g *= w
        loss = torch.zeros(T, dtype=f64, device=dev)
        loss[real] = each
        out |= {"loss": loss, "total": (w * each).sum(), "clipped": stopped.to(f64).sum() / max(k, 1)}
    else:
        b, P, e = st["starts"].tolist(), case["pairs"], case["smoothing"]
        where = torch.bucketize(real, st["starts"][1:], right=True)
        rewards = torch.zeros(P, 2, dtype=f64, device=dev)
        length = torch.ones(2 * P, dtype=f64, device=dev)
        for i in range(2 * P):
            m = (real >= b[i]) & (real < b[i + 1])
            if case["average"]:
                length[i] = max(1, int(m.sum()))
            rewards[i // 2, i % 2] = BETA * (lp[m] - st["ref"][real[m]].to(f64)).sum() / length[i]
        z = rewards[:, 0] - rewards[:, 1] - 0.25
        soft = torch.nn.functional.softplus
        each = (1 - e) * soft(-z) + e * soft(z)
        dz = (e - 1) / (1 + torch.exp(z)) + e / (1 + torch.exp(-z))
        g = BETA / P * torch.stack([dz, -dz], 1).reshape(-1)[where] / length[where]
        out = {"loss": each, "mean": each.sum() / P, "rewards": rewards}
    d = torch.exp(s.sub_(lse[:, None])).mul_(-g[:, None])
    d[at, y] += g
    dh = torch.zeros(T, H, dtype=f64, device=dev)
    dh[real] = d @ W
    return out | {"logp": logp, "dh": dh, "dW": d.t() @ h}
