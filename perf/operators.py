"""Cases, inputs and plain forms of the scoring operators and of the 8-bit output projection.

Five operators, each with its cases:

* ``score``      : ``token_logprobs`` - log-probabilities of given tokens, entropy and top
  alternatives of logits that are at hand.
* ``score_grad`` : ``token_logprobs_backward`` - the gradient of those log-probabilities and of
  the entropy with respect to the logits.
* ``head``       : ``projected_logprobs`` - log-probabilities and entropy straight from hidden
  states and the output matrix, without the logits.
* ``head_train`` : ``fused_token_logprobs`` - the same with gradients of the hidden states and
  of the output matrix.
* ``e4m3``       : ``block_quantize`` and ``block_scaled_projection`` - an output projection in
  8-bit floating point with a scale for each block of 128.

With z the logits of a position, q = softmax(z) and tokens t (an id of -1 is an empty slot):

    logp_t  = z_t - log sum_v exp(z_v)                      (empty slot: 0)
    entropy = - sum_v q_v log q_v                            (0 log 0 = 0)
    norm    = (max z, log sum_v exp(z_v - max z))
    top     = the k largest logits, equal ones by lowest id, and their log-probabilities
    dz_v    = sum_t g_t [v = t] - q_v (sum_t g_t + g_e (log q_v + entropy))

A position whose mask leaves nothing (all logits -inf) has norm (-inf, 0), log-probabilities
-inf, entropy 0, the ids 0..k-1 as alternatives and a zero gradient.

``own`` chooses between the plain form (False) and the package's operators (True).
"""
import math

import torch

own = False

EMPTY = -1
BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence being decoded: its sampled token's log-probability and 20 alternatives
        {"name": "score 1x201088 top20", "op": "score", "N": 1, "V": 201088, "type": "bf16", "T": 1, "top": 20,
         "mask": "none"},
        # a constrained decoding batch: an odd vocabulary in 32 bits, most tokens masked with
        # -inf and one sequence with nothing left, three candidate tokens each
        {"name": "score 257x50001 masked", "op": "score", "N": 257, "V": 50001, "type": "fp32", "T": 3, "top": 5,
         "mask": "inf"},
        # a chunk of a teacher's logits turned into cache entries: the top 100 of every position
        {"name": "score 4096x128256 top100", "op": "score", "N": 4096, "V": 128256, "type": "bf16", "T": 1,
         "top": 100, "mask": "none"},
        # gradient for a short answer, half-precision logits of an odd vocabulary masked with the
        # type's lowest value
        {"name": "score_grad 301x50001", "op": "score_grad", "N": 301, "V": 50001, "type": "fp16", "T": 2,
         "mask": "lowest"},
        # gradient for a training batch of sequences
        {"name": "score_grad 4096x128256", "op": "score_grad", "N": 4096, "V": 128256, "type": "bf16", "T": 1,
         "mask": "none"},
        # one decoded position scored from its hidden state
        {"name": "head 1x2880x201088", "op": "head", "N": 1, "d": 2880, "V": 201088, "T": 1, "chunk": 2048},
        # evaluation: the log-probabilities of whole texts
        {"name": "head 8192x2880x201088", "op": "head", "N": 8192, "d": 2880, "V": 201088, "T": 1, "chunk": 2048},
        # a training step of a small student on a few answers, four candidate tokens each
        {"name": "head_train 777x1024x32000", "op": "head_train", "N": 777, "d": 1024, "V": 32000, "T": 4,
         "chunk": 512},
        # a training step at the size of the distillation workloads
        {"name": "head_train 4096x2880x201088", "op": "head_train", "N": 4096, "d": 2880, "V": 201088, "T": 1,
         "chunk": 2048},
        # 16 sequences decoded together by a teacher whose head is stored in 8 bits
        {"name": "e4m3 16x2880x201088", "op": "e4m3", "what": "project", "N": 16, "d": 2880, "V": 201088,
         "out": "fp32"},
        # that teacher scoring texts for the cache
        {"name": "e4m3 8192x2880x201088", "op": "e4m3", "what": "project", "N": 8192, "d": 2880, "V": 201088,
         "out": "bf16"},
        # bringing a teacher's head into 8 bits, once per checkpoint
        {"name": "e4m3 weights 201088x2880", "op": "e4m3", "what": "quantize", "N": 201088, "d": 2880,
         "type": "bf16", "rows": 128},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score_grad", "head", "head_train", "e4m3"])
    c = {"op": op}
    if op in ("score", "score_grad"):
        c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        c["V"] = _log_uniform(rng, 1000, 201088)
        room = 4096 * 128256 * 2 // (c["V"] * (4 if c["type"] == "fp32" else 2))
        c["N"] = _log_uniform(rng, 1, min(4096, room))
        c["T"] = rng.randint(1, 8)
        c["mask"] = rng.choice(["none", "none", "inf", "lowest"])
        if op == "score":
            c["top"] = rng.choice([0, 1, rng.randint(2, 128)])
    elif op in ("head", "head_train"):
        c["V"] = _log_uniform(rng, 1000, 201088)
        c["d"] = 8 * _log_uniform(rng, 8, 360)
        c["N"] = _log_uniform(rng, 1, 8192) if op == "head" else _log_uniform(rng, 16, 4096)
        c["T"] = rng.randint(1, 4)
        c["chunk"] = rng.choice([512, 1024, 2048])
    else:
        c["what"] = rng.choice(["project", "project", "quantize"])
        c["V"] = _log_uniform(rng, 1000, 201088)
        c["d"] = 8 * _log_uniform(rng, 8, 360)
        c["N"] = _log_uniform(rng, 1, 8192)
        if c["what"] == "quantize":
            c["rows"] = rng.choice([1, 128])
            c["N"] = c.pop("V") if c["rows"] == 128 else c["N"]
            c.pop("V", None)
            c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        else:
            c["out"] = rng.choice(["bf16", "fp32"])
    return c


def work(case):
    N = case["N"]
    if case["op"] in ("score", "score_grad"):
        V, T = case["V"], case["T"]
        e = 4 if case["type"] == "fp32" else 2
        if case["op"] == "score":
            return {"bytes": N * (V * e + 8 * T + 12 + 8 * case["top"]), "flops": 6 * N * V}
        return {"bytes": N * (2 * V * e + 8 * T + 16), "flops": 6 * N * V}
    if case["op"] in ("head", "head_train"):
        V, d, T = case["V"], case["d"], case["T"]
        if case["op"] == "head":
            return {"bytes": 2 * (N + V) * d + N * (8 * T + 8), "flops": 2 * N * d * V}
        return {"bytes": 4 * (N + V) * d + N * (12 * T + 8), "flops": 6 * N * d * V}
    d = case["d"]
    if case["what"] == "quantize":
        e = 4 if case["type"] == "fp32" else 2
        kb = -(-d // BLOCK)
        return {"bytes": N * d * (e + 1) + 4 * kb * -(-N // case["rows"]), "flops": 3 * N * d}
    V = case["V"]
    o = 4 if case["out"] == "fp32" else 2
    return {"bytes": 2 * N * d + V * d + o * N * V + 4 * -(-V // BLOCK) * -(-d // BLOCK), "flops": 2 * N * d * V}


# ------------------------------------------------------------------ inputs
def _hidden(g, N, d):
    """Hidden states after a final norm: unit scale, a few channels much larger."""
    loud = torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 6.0, 1.0)
    return (torch.randn(N, d, generator=g, device="cuda") * loud).to(torch.bfloat16)


def _output_matrix(g, V, d):
    return (torch.randn(V, d, generator=g, device="cuda") / math.sqrt(d)).to(torch.bfloat16)


def _tokens(g, N, V, T):
    t = torch.randint(0, V, (N, T), generator=g, device="cuda", dtype=torch.int32)
    if T > 1:  # ragged candidate lists: some of the later slots are empty
        drop = torch.rand(N, T, generator=g, device="cuda") < 0.15
        drop[:, 0] = False
        t = torch.where(drop, torch.full_like(t, EMPTY), t)
    return t


def _logits(g, case):
    """A bulk of unlikely tokens and a few likely ones, as a trained model gives; masked ones keep
    a set of allowed tokens, position 0 (of several) none."""
    N, V, T = case["N"], case["V"], case["T"]
    z = torch.randn(N, V, generator=g, device="cuda") * 2.2
    likely = torch.randint(0, V, (N, 12), generator=g, device="cuda")
    z.scatter_add_(1, likely, 4 + 6 * torch.rand(N, 12, generator=g, device="cuda"))
    tokens = _tokens(g, N, V, T)
    if case["mask"] != "none":
        left = torch.randint(0, V, (N, max(64, 2 * case.get("top", 0))), generator=g, device="cuda")
        keep = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, left, True)
        if N > 1:
            keep[0] = False
        low = -math.inf if case["mask"] == "inf" else torch.finfo(TYPES[case["type"]]).min
        z = z.masked_fill(~keep, low)
        tokens = torch.where(tokens == EMPTY, tokens, left[:, :T].to(torch.int32))
    return z.to(TYPES[case["type"]]), tokens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    N = case["N"]
    if case["op"] in ("score", "score_grad"):
        s["logits"], s["tokens"] = _logits(g, case)
        if case["op"] == "score_grad":  # what the forward pass left, and the upstream gradients
            _, s["entropy"], s["norm"], _, _ = _plain_score(s["logits"], s["tokens"], 0)
            s["g_logp"] = torch.randn(N, case["T"], generator=g, device="cuda")
            s["g_entropy"] = 0.3 * torch.randn(N, generator=g, device="cuda")
        return s
    if case["op"] in ("head", "head_train"):
        s["H"] = _hidden(g, N, case["d"])
        s["W"] = _output_matrix(g, case["V"], case["d"])
        s["tokens"] = _tokens(g, N, case["V"], case["T"])
        if case["op"] == "head_train":
            s["g_logp"] = torch.randn(N, case["T"], generator=g, device="cuda")
            s["g_entropy"] = 0.3 * torch.randn(N, generator=g, device="cuda")
            s["H"].requires_grad_()
            s["W"].requires_grad_()
        return s
    if case["what"] == "quantize":
        x = _output_matrix(g, N, case["d"]) if case["rows"] == BLOCK else _hidden(g, N, case["d"])
        s["x"] = x.to(TYPES[case["type"]])
        return s
    s["H"] = _hidden(g, N, case["d"])
    s["W8"], s["scale"] = _plain_quantize(_output_matrix(g, case["V"], case["d"]), BLOCK, pad=True)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_score(logits, tokens, top):
    z = logits.float()
    m = z.amax(1, keepdim=True)
    some = m > -math.inf
    d = torch.where(some, z - m, torch.full_like(z, -math.inf))
    e = d.exp()
    l = torch.where(some, e.sum(1, keepdim=True), torch.ones_like(m))
    log_l = l.log()
    t = torch.where(e > 0, d * e, torch.zeros_like(e)).sum(1, keepdim=True)
    entropy = torch.where(some, log_l - t / l, torch.zeros_like(m))[:, 0]
    norm = torch.cat([m, log_l], 1)
    at = d.gather(1, tokens.clamp(min=0).long())
    logp = torch.where(tokens == EMPTY, torch.zeros_like(at), at - log_l)
    if top:
        order = (z + 0.0).sort(dim=1, descending=True, stable=True)[1][:, :top]  # stable: equal logits stay by id
        return logp, entropy, norm, order.to(torch.int32), d.gather(1, order) - log_l
    none = torch.empty(z.shape[0], 0, device=z.device)
    return logp, entropy, norm, none.to(torch.int32), none


def _plain_dense_grad(z, m, log_l, tokens, entropy, g_logp, g_entropy):
    """dz in 32 bits."""
    g = torch.where(tokens == EMPTY, torch.zeros_like(g_logp), g_logp)
    log_q = z - m - log_l
    q = log_q.exp()
    dz = -q * (g.sum(1, keepdim=True) + g_entropy[:, None] * (log_q + entropy[:, None]))
    dz = torch.where(q > 0, dz, torch.zeros_like(dz))
    dz.scatter_add_(1, tokens.clamp(min=0).long(), g)
    return torch.where(m > -math.inf, dz, torch.zeros_like(dz))


def _plain_head(H, W, tokens):
    z = H.float() @ W.float().t()
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    l = e.sum(1, keepdim=True)
    lse = m + l.log()
    entropy = (l.log() - ((z - m) * e).sum(1, keepdim=True) / l)[:, 0]
    at = z.gather(1, tokens.clamp(min=0).long())
    logp = torch.where(tokens == EMPTY, torch.zeros_like(at), at - lse)
    return z, logp, entropy, lse


def _plain_quantize(x, rows, pad=False):
    """(e4m3 values, scales): one scale per `rows` x 128 block. With pad the rows of the values lie
    a multiple of 16 bytes apart."""
    R, C = x.shape
    rb, cb = -(-R // rows), -(-C // BLOCK)
    full = torch.zeros(rb * rows, cb * BLOCK, device=x.device)
    full[:R, :C] = x.float()
    amax = full.view(rb, rows, cb, BLOCK).abs().amax((1, 3))
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=2.0 ** -126)  # a true quotient
    q = (full.view(rb, rows, cb, BLOCK) / scale[:, None, :, None]).view(rb * rows, cb * BLOCK)[:R]
    q = q.to(torch.float8_e4m3fn)
    if pad:
        return q[:, :-(-C // 16) * 16].contiguous()[:, :C], scale
    return q[:, :C].contiguous(), scale


def _plain_values(q, scale, rows):
    s = scale.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "score":
        return _plain_score(s["logits"], s["tokens"], s["top"])
    if s["op"] == "score_grad":
        return _plain_dense_grad(s["logits"].float(), s["norm"][:, :1], s["norm"][:, 1:], s["tokens"], s["entropy"],
                                 s["g_logp"], s["g_entropy"]).to(s["logits"].dtype)
    if s["op"] == "head":
        _, logp, entropy, lse = _plain_head(s["H"], s["W"], s["tokens"])
        return logp, entropy, lse[:, 0]
    if s["op"] == "head_train":
        H, W = s["H"].detach(), s["W"].detach()
        z, logp, entropy, lse = _plain_head(H, W, s["tokens"])
        dz = _plain_dense_grad(z, lse, 0.0, s["tokens"], entropy, s["g_logp"], s["g_entropy"])
        return logp, entropy, (dz @ W.float()).to(H.dtype), (dz.t() @ H.float()).to(W.dtype)
    if s["what"] == "quantize":
        return _plain_quantize(s["x"], s["rows"])
    h = _plain_values(*_plain_quantize(s["H"], 1), 1)
    return (h @ _plain_values(s["W8"], s["scale"], BLOCK).t()).to(TYPES[s["out"]])


def _run_own(s):
    import chunked_kl_loss_gb300 as fckl
    if s["op"] == "score":
        return fckl.token_logprobs(s["logits"], s["tokens"], top=s["top"])
    if s["op"] == "score_grad":
        return fckl.token_logprobs_backward(s["logits"], s["tokens"], s["norm"], s["entropy"], s["g_logp"],
                                            s["g_entropy"])
    if s["op"] == "head":
        return fckl.projected_logprobs(s["H"], s["W"], s["tokens"], s["chunk"])
    if s["op"] == "head_train":
        logp, entropy = fckl.fused_token_logprobs(s["H"], s["W"], s["tokens"], s["chunk"])
        dH, dW = torch.autograd.grad((logp, entropy), (s["H"], s["W"]), (s["g_logp"], s["g_entropy"]))
        return logp.detach(), entropy.detach(), dH, dW
    if s["what"] == "quantize":
        return fckl.block_quantize(s["x"], rows=s["rows"])
    return fckl.block_scaled_projection(s["H"], s["W8"], s["scale"], out_dtype=TYPES[s["out"]])


# ------------------------------------------------------------------ 64 bits
def _exact_top(logits, top):
    """Largest first by one whole-number key per entry: the value's order, then the lower id."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits - 1, bits)  # sign-magnitude to an ordered number
    key = order * (1 << 31) + (1 << 31) - 1 - torch.arange(logits.shape[1], device=logits.device)
    return key.topk(top, 1)[1].to(torch.int32)


def _exact_score(logits, tokens, top):
    z = logits.double()
    some = torch.isfinite(z).any(1, keepdim=True)
    lq = torch.where(some, torch.log_softmax(z, 1), torch.full_like(z[:, :1], -math.inf))
    entropy = torch.special.entr(lq.exp()).sum(1)
    m = z.max(1, keepdim=True)[0]
    norm = torch.cat([m, torch.where(some, torch.logsumexp(z - torch.where(some, m, 0.0), 1, keepdim=True), 0.0)], 1)
    pick = torch.take_along_dim(lq, tokens.long().clamp_min(0), 1)
    logp = torch.where(tokens < 0, 0.0, pick)
    if not top:
        none = torch.empty(z.shape[0], 0, device=z.device, dtype=torch.float64)
        return logp, entropy, norm, none.to(torch.int32), none
    ids = _exact_top(logits, top)
    return logp, entropy, norm, ids, torch.take_along_dim(lq, ids.long(), 1)


def _exact_grad(lq, tokens, g_logp, g_entropy):
    """Gradient of sum g_t logp_t + g_e entropy through softmax, from log q in 64 bits."""
    q = lq.exp()
    g = torch.where(tokens < 0, 0.0, g_logp.double())
    entropy = torch.special.entr(q).sum(1, keepdim=True)
    dz = q * g.sum(1, keepdim=True) - torch.special.entr(q) * g_entropy.double()[:, None]
    dz += q * (entropy * g_entropy.double()[:, None])
    dz.neg_()
    return dz.scatter_add(1, tokens.long().clamp_min(0), g)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "score":
        return _exact_score(s["logits"], s["tokens"], s["top"])
    if case["op"] == "score_grad":
        z = s["logits"].double()
        some = torch.isfinite(z).any(1, keepdim=True)
        lq = torch.log_softmax(torch.where(some, z, 0.0), 1)
        return torch.where(some, _exact_grad(lq, s["tokens"], s["g_logp"], s["g_entropy"]), 0.0)
    if case["op"] in ("head", "head_train"):
        N, step = case["N"], 512
        with torch.no_grad():
            H, W = s["H"].detach().double(), s["W"].detach().double()
            out = [[], [], [], []]
            dW = torch.zeros_like(W) if case["op"] == "head_train" else None
            for a in range(0, N, step):
                h, tok = H[a:a + step], s["tokens"][a:a + step]
                z = h @ W.t()
                lq = torch.log_softmax(z, 1)
                out[0].append(torch.where(tok < 0, 0.0, torch.take_along_dim(lq, tok.long().clamp_min(0), 1)))
                out[1].append(torch.special.entr(lq.exp()).sum(1))
                if case["op"] == "head":
                    out[2].append(torch.logsumexp(z, 1))
                    continue
                dz = _exact_grad(lq, tok, s["g_logp"][a:a + step], s["g_entropy"][a:a + step])
                out[2].append(dz @ W)
                dW += dz.t() @ h
            got = [torch.cat(x) for x in out if x]
        return (*got, dW) if dW is not None else tuple(got)
    if case["what"] == "quantize":
        return _exact_quantize(s["x"], case["rows"])
    q, scale = _exact_quantize(s["H"], 1)
    h = q.double() * scale.double().repeat_interleave(BLOCK, 1)[:, :case["d"]]
    w = s["W8"].double() * s["scale"].double().repeat_interleave(BLOCK, 0)[:case["V"]].repeat_interleave(
        BLOCK, 1)[:, :case["d"]]
    return torch.cat([h[a:a + 512] @ w.t() for a in range(0, case["N"], 512)])


def _exact_quantize(x, rows):
    """The scale is by definition the 32-bit number nearest to amax / 448, and the 8-bit value the
    one nearest to the 32-bit quotient."""
    R, C = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -C % BLOCK, 0, -R % rows))
    tiles = v.unfold(0, rows, rows).unfold(1, BLOCK, BLOCK)  # [row blocks, column blocks, rows, 128]
    scale = torch.clamp_min(tiles.abs().amax((2, 3)) / E4M3_MAX, 2.0 ** -126).float()
    spread = scale.double().repeat_interleave(rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :C]
    return (x.double() / spread).float().to(torch.float8_e4m3fn), scale
