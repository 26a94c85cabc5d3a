"""The training end of the packed head: what is measured of it, on which cases.

Three operators that follow each other in one training step through a frozen
packed head:

  policy      the clipped policy loss with a KL term over rows of logits, with
              its gradient with respect to the logits
  preference  the preference loss over pairs of sequences (log ratios of a
              chosen and a rejected answer), with the same gradient
  backward    the gradient of the hidden states from that of the logits,
              dH = dY W_hat, through the packed bytes

`run` computes a case in its plain form (elementary torch operations in fp32,
per-row numbers in fp64) or, where `own` is true, by the framework's entry
points.  `exact` is the definition in fp64.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
CLIP_LOW, CLIP_HIGH, KL_COEF, INV_TEMPERATURE = 0.2, 0.28, 0.04, 0.75
BETA, SMOOTHING = 0.1, 0.05

# The largest work of a case: rows times vocabulary of a loss, and that times
# the hidden size for the backward.
_MOST_LOGITS = 4096 * 151936
_MOST_MACS = 4096 * 151936 * 4096


def _policy(name, N, V, y, dy, keep):
    return dict(name=name, op="policy", N=N, V=V, y=y, dy=dy, keep=keep)


def _preference(name, B, N, V, y, dy, keep):
    return dict(name=name, op="preference", B=B, N=N, V=V, y=y, dy=dy, keep=keep)


def _backward(name, N, V, D, r_c, r_r, g, dy):
    return dict(name=name, op="backward", N=N, V=V, D=D, r_c=r_c, r_r=r_r, g=g, dy=dy)


def listed():
    return [
        # a unit-test-sized vocabulary, a handful of tokens: nothing but latency
        _policy("policy_few_small_vocab", 4, 1024, BF16, BF16, 1.0),
        # one token of a full vocabulary: token-by-token online updates
        _policy("policy_one_token", 1, 151936, BF16, BF16, 1.0),
        # a micro-batch of a rollout, a quarter of whose rows are prompt or padding
        _policy("policy_microbatch", 512, 151936, BF16, BF16, 0.75),
        # fp32 logits of a vocabulary of odd size (rows at every alignment), gradient
        # in bf16 for the head's backward
        _policy("policy_f32_odd_vocab", 257, 100003, F32, BF16, 0.9),
        # a long rollout's 4096 rows at once
        _policy("policy_rollout", 4096, 151936, BF16, BF16, 0.9),
        # one pair of short answers, fp32 all through
        _preference("preference_short_pair", 1, 12, 1000, F32, F32, 1.0),
        # four pairs, half of whose rows are the prompts in front of the answers
        _preference("preference_pairs", 4, 480, 151936, BF16, BF16, 0.5),
        # eight pairs of long answers of the larger head's vocabulary
        _preference("preference_long_pairs", 8, 4096, 128256, BF16, BF16, 0.8),
        # the smallest head: latency
        _backward("backward_few_small_head", 4, 1024, 256, 16, 8, 64, BF16),
        # one token: the packed head is streamed once
        _backward("backward_one_token", 1, 151936, 4096, 32, 32, 128, BF16),
        # a 70B-class head, one short sequence
        _backward("backward_large_head", 256, 128256, 8192, 64, 64, 128, BF16),
        # the rollout's rows at once
        _backward("backward_rollout", 4096, 151936, 4096, 64, 64, 128, BF16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "preference", "backward"])
    V = _log_int(rng, 1000, 152000)
    if op == "backward":
        g = rng.choice([32, 64, 128, 256])
        D = 256 * _log_int(rng, 1, 32)
        N = _log_int(rng, 1, max(1, min(4096, _MOST_MACS // (V * D))))
        return dict(op=op, N=N, V=V, D=D, r_c=8 * rng.randint(0, 8), r_r=8 * rng.randint(0, 8), g=g,
                    dy=rng.choice([BF16, BF16, F32]))
    N = _log_int(rng, 1 if op == "policy" else 4, min(4096, _MOST_LOGITS // V))
    y = rng.choice([BF16, BF16, F32])
    dy = rng.choice([BF16, F32])
    keep = rng.choice([1.0, 0.9, 0.75, 0.5])
    if op == "policy":
        return dict(op=op, N=N, V=V, y=y, dy=dy, keep=keep)
    return dict(op=op, B=rng.randint(1, max(1, min(16, N // 4))), N=N, V=V, y=y, dy=dy, keep=keep)


def _kept(case):
    """Rows that count in the loss."""
    return max(1, round(case["N"] * case["keep"]))


def work(case):
    N, V = case["N"], case["V"]
    size = {BF16: 2, F32: 4}
    if case["op"] == "backward":
        D, r = case["D"], case["r_c"] + case["r_r"]
        n_a = (case["r_c"] > 0) + (case["r_r"] > 0)
        head = V * (D // 2 + D // case["g"] + 2 + r + 2 * n_a) + r * (D + 2 * (D // case["g"]))
        return {"bytes": head + N * V * size[case["dy"]] + N * D * 2, "flops": 2 * N * V * (D + r) + 2 * N * r * D}
    # logits of the rows that count read once, the gradient of every row written once
    rows = _kept(case) * V * size[case["y"]] + N * V * size[case["dy"]]
    return {"bytes": rows + N * 24, "flops": 10 * _kept(case) * V}


# ------------------------------------------------------------------ inputs ---

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(gen, N, V, dtype):
    """Logits of a language model's kind: spread of a few units, one likely
    token per row that is the row's label; returns (Y, labels)."""
    Y = (torch.randn((N, V), generator=gen, device="cuda") * 2.5).to(dtype)
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda")
    rows = torch.arange(N, device="cuda")
    lift = torch.rand(N, generator=gen, device="cuda") * 14.0
    Y[rows, labels] = (Y[rows, labels].float() + lift).to(dtype)
    return Y, labels


def _label_logp(Y, labels, scale):
    z = Y.double() * scale
    return z.gather(1, labels[:, None])[:, 0] - torch.logsumexp(z, 1)


def _weights(gen, N, kept):
    """1/kept for the rows that count, 0 for the others, in a random order."""
    w = torch.zeros(N, device="cuda")
    w[torch.randperm(N, generator=gen, device="cuda")[:kept]] = 1.0 / kept
    return w


def _layout(V, D, r_c, r_r, g):
    """Section offsets of a packed head (format version 1) and its size."""
    V16, r, n_a, ng = -(-V // 16) * 16, r_c + r_r, (r_c > 0) + (r_r > 0), D // g
    sizes = [("header", 64), ("r_codes", V16 * D // 2), ("r_gcodes", V16 * ng), ("r_rowscale", 2 * V16),
             ("a_codes", V16 * r), ("a_scales", 2 * V16 * n_a), ("b_codes", r * D), ("b_scales", 2 * r * ng)]
    at, out = 0, {}
    for name, size in sizes:
        out[name] = (at, size)
        at += -(-size // 256) * 256
    return out, at, V16


def _packed_head(gen, V, D, r_c, r_r, g):
    """A packed head's bytes: uniform codes, half-normal scales."""
    where, total, V16 = _layout(V, D, r_c, r_r, g)
    r, n_a, ng = r_c + r_r, (r_c > 0) + (r_r > 0), D // g
    buf = torch.zeros(total, dtype=torch.uint8, device="cuda")

    def put(name, t):
        at, size = where[name]
        buf[at:at + size] = t.contiguous().view(torch.uint8).reshape(-1)

    def scales(shape, sigma):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).abs().half()

    def codes(shape):
        return torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)

    put("header", torch.tensor([0x48435241, 1, V, 0, D, 0, r_c, r_r, g] + [0] * 7, dtype=torch.int32, device="cuda"))
    tiles = torch.randint(0, 256, (D // 128, V16 // 16, 64, 16), generator=gen, device="cuda", dtype=torch.uint8)
    gcodes = torch.randint(1, 256, (V16, ng), generator=gen, device="cuda", dtype=torch.uint8)
    s_R, A, s_A = scales((V16,), 1e-3), codes((V16, r)), scales((V16, n_a), 1e-2)
    if V16 > V:  # rows past the vocabulary are zero
        past = torch.arange(64, device="cuda") % 16 + V16 - 16 >= V
        tiles[:, -1, past] = 0
        gcodes[V:], s_R[V:], A[V:], s_A[V:] = 0, 0, 0, 0
    put("r_codes", tiles)
    put("r_gcodes", gcodes)
    put("r_rowscale", s_R)
    if r:
        put("a_codes", A)
        put("a_scales", s_A)
        put("b_codes", codes((r, D)))
        put("b_scales", scales((r, ng), 1e-2))
    return buf


def prepare(case, seed):
    gen, N, V = _generator(seed), case["N"], case["V"]
    state = dict(case=dict(case))
    if case["op"] == "backward":
        dims = (V, case["D"], case["r_c"], case["r_r"], case["g"])
        state["packed"] = _packed_head(gen, *dims)
        # the gradient a loss leaves: a coefficient times (one-hot - softmax), a few rows zero
        dY, labels = _logits(gen, N, V, _DTYPES[case["dy"]])
        coef = torch.randn(N, generator=gen, device="cuda") / N
        if N > 8:
            coef[torch.rand(N, generator=gen, device="cuda") < 0.1] = 0.0
        p = torch.softmax(dY.float(), 1)
        p[torch.arange(N, device="cuda"), labels] -= 1.0
        state["dY"] = (p * -coef[:, None]).to(dY.dtype)
        if own:
            import compressed_output_head_amd as ah
            state["head"] = ah.PackedHead(*dims, state["packed"])
        return state
    Y, labels = _logits(gen, N, V, _DTYPES[case["y"]])
    logp = _label_logp(Y, labels, INV_TEMPERATURE)
    w = _weights(gen, N, _kept(case))
    # prompt and padding rows carry no label
    state.update(Y=Y, labels=torch.where(w != 0, labels, -100).int(), weight=w)
    state["ref_logp"] = (logp + 0.2 * torch.randn(N, generator=gen, device="cuda")).float()
    if case["op"] == "policy":
        delta = 0.25 * torch.randn(N, generator=gen, device="cuda", dtype=torch.float64)
        # a ratio on a border of the clip range is decided by the last bit: none is within 1e-3 of one
        for border in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
            delta = torch.where((delta - border).abs() < 1e-3, border + 2e-3, delta)
        state["old_logp"] = (logp - delta).float()
        # rewards of 0 or 1 against a baseline
        state["advantage"] = (torch.rand(N, generator=gen, device="cuda") < 0.5).float() - 0.3
    else:
        # rows dealt out to 2 B sequences of at least one row
        cuts = torch.randperm(N - 1, generator=gen, device="cuda")[:2 * case["B"] - 1].sort()[0] + 1
        ends = torch.tensor([N], device="cuda")
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts, ends]).int()
        # the model has moved from the reference towards the chosen answers (even sequences)
        seq = torch.searchsorted(cuts, torch.arange(N, device="cuda"), right=True)
        state["ref_logp"] += torch.where(seq % 2 == 0, -0.1, 0.1)
    return state


# -------------------------------------------------------------- plain forms ---

def _plain_rows(Y, labels):
    """exp(z - max z), its row sums (fp64) and the labels' log-probabilities
    (fp64) of z = Y * INV_TEMPERATURE; rows without a label take column 0."""
    at = labels.long().clamp(min=0)[:, None]
    top = Y.amax(1, keepdim=True)
    e = torch.exp((Y.float() - top.float()) * INV_TEMPERATURE)
    total = e.sum(1, dtype=torch.float64)
    below = Y.gather(1, at).double() - top.double()
    return e, total, below[:, 0] * INV_TEMPERATURE - torch.log(total), at


def _plain_gradient(e, total, logp, at, coef, dtype):
    """coef_n * INV_TEMPERATURE * (one-hot - softmax), zero rows where coef is zero."""
    coef = coef * INV_TEMPERATURE
    grad = e * (-coef / total).float()[:, None]
    grad.scatter_(1, at, (-coef * torch.expm1(logp)).float()[:, None])
    return torch.where((coef != 0)[:, None], grad, 0.0).to(dtype)


def _plain_policy(s):
    e, total, logp, at = _plain_rows(s["Y"], s["labels"])
    w, adv = s["weight"].double(), s["advantage"].double()
    on = w != 0
    ratio = torch.exp(logp - s["old_logp"].double())
    clipped = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    d = s["ref_logp"].double() - logp
    row = torch.where(on, KL_COEF * (torch.expm1(d) - d) - torch.minimum(ratio * adv, clipped * adv), 0.0)
    slope = -torch.expm1(d) * KL_COEF - torch.where(ratio * adv <= clipped * adv, ratio * adv, 0.0)
    dY = _plain_gradient(e, total, logp, at, torch.where(on, w * slope, 0.0), _DTYPES[s["case"]["dy"]])
    return {"loss": (w * row).sum().float(), "logp": torch.where(on, logp, 0.0).float(), "row_loss": row.float(), "dY": dY}


def _plain_preference(s):
    e, total, logp, at = _plain_rows(s["Y"], s["labels"])
    w, N, B = s["weight"].double(), s["case"]["N"], s["case"]["B"]
    on = w != 0
    seq = torch.searchsorted(s["offsets"].long(), torch.arange(N, device="cuda"), right=True) - 1
    sums = torch.zeros(2 * B, dtype=torch.float64, device="cuda")
    sums.index_add_(0, seq, torch.where(on, w * (logp - s["ref_logp"].double()), 0.0))
    chosen, rejected = sums[0::2], sums[1::2]
    margin = BETA * (chosen - rejected)
    losses = (1 - SMOOTHING) * torch.log1p(torch.exp(-margin)) + SMOOTHING * torch.log1p(torch.exp(margin))
    slope = BETA * (SMOOTHING - 1 / (1 + torch.exp(margin)))
    coef = torch.where(on, torch.stack([slope, -slope], 1).reshape(-1)[seq] * w, 0.0)
    dY = _plain_gradient(e, total, logp, at, coef, _DTYPES[s["case"]["dy"]])
    return {"loss": losses.sum().float(), "logp": torch.where(on, logp, 0.0).float(),
            "chosen_reward": (BETA * chosen).float(), "rejected_reward": (BETA * rejected).float(), "dY": dY}


def _plain_w_hat(buf, V, D, r_c, r_r, g):
    """W_hat = R + A_c B_c + A_w B_w in fp32 from the packed bytes."""
    where, _, V16 = _layout(V, D, r_c, r_r, g)
    r, n_a, ng = r_c + r_r, (r_c > 0) + (r_r > 0), D // g

    def get(name, dtype, *shape):
        at, size = where[name]
        return buf[at:at + size].view(dtype).reshape(shape)

    # tile byte 16 l + 4 s + c: row l % 16, columns 32 s + 8 (l / 16) + 2 c and the next
    t = get("r_codes", torch.uint8, D // 128, V16 // 16, 4, 16, 4, 4).permute(1, 3, 0, 4, 2, 5)
    nibbles = torch.stack([t & 15, t >> 4], -1).reshape(V16, D).view(torch.int8)
    W = torch.where(nibbles > 7, nibbles - 16, nibbles).float()
    scale = get("r_gcodes", torch.uint8, V16, ng).float() * get("r_rowscale", torch.float16, V16, 1).float()
    W = (W.view(V16, ng, g) * scale[:, :, None]).view(V16, D)
    if r:
        A = get("a_codes", torch.int8, V16, r).float()
        s_A = get("a_scales", torch.float16, V16, n_a).float()
        A *= torch.cat([s_A[:, i:i + 1].expand(V16, n) for i, n in enumerate(n for n in (r_c, r_r) if n)], 1)
        B = get("b_codes", torch.int8, r, ng, g).float() * get("b_scales", torch.float16, r, ng, 1).float()
        W += A @ B.view(r, D)
    return W[:V]


def _plain_backward(s):
    c = s["case"]
    W = _plain_w_hat(s["packed"], c["V"], c["D"], c["r_c"], c["r_r"], c["g"])
    return {"dH": (s["dY"].float() @ W).to(torch.bfloat16)}


_PLAIN = {"policy": _plain_policy, "preference": _plain_preference, "backward": _plain_backward}


def run(state):
    case = state["case"]
    if not own:
        return _PLAIN[case["op"]](state)
    import compressed_output_head_amd as ah
    if case["op"] == "backward":
        return {"dH": ah.archead_logits_backward(state["dY"], state["head"])}
    if case["op"] == "policy":
        return ah.archead_policy_loss(state["Y"], state["labels"], state["advantage"], old_logp=state["old_logp"],
                                      ref_logp=state["ref_logp"], weight=state["weight"], clip_low=CLIP_LOW,
                                      clip_high=CLIP_HIGH, kl_coef=KL_COEF, inv_temperature=INV_TEMPERATURE,
                                      dY_dtype=_DTYPES[case["dy"]])
    return ah.archead_preference_loss(state["Y"], state["labels"], state["offsets"], ref_logp=state["ref_logp"],
                                      weight=state["weight"], beta=BETA, label_smoothing=SMOOTHING,
                                      inv_temperature=INV_TEMPERATURE, dY_dtype=_DTYPES[case["dy"]])


# --------------------------------------------------- the definitions in fp64 ---

def _exact_head(buf, V, D, r_c, r_r, g):
    """(R, [A_c | A_w], [B_c ; B_w]) in fp64, element by element from the layout."""
    where, _, V16 = _layout(V, D, r_c, r_r, g)
    raw = {k: buf[a:a + n] for k, (a, n) in where.items()}
    v, k = torch.arange(V, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    tile = (k // 128 * (V16 // 16) + v // 16) * 1024
    code = raw["r_codes"][tile + 16 * (v % 16 + 16 * (k % 32 // 8)) + 4 * (k % 128 // 32) + k % 8 // 2].short()
    code = (code >> (4 * (k % 2)).short()) % 16
    R = (code - 16 * (code >= 8)).double()
    R *= raw["r_gcodes"][v * (D // g) + k // g].double()
    R *= raw["r_rowscale"].view(torch.float16)[:V].double()[:, None]
    if r_c + r_r == 0:
        return R, None, None
    part = (torch.arange(r_c + r_r, device="cuda") >= (r_c or r_c + r_r)).long()
    s_A = raw["a_scales"].view(torch.float16).view(V16, -1)[:V].double()
    A = raw["a_codes"].view(torch.int8).view(V16, r_c + r_r)[:V].double() * s_A[:, part]
    B = raw["b_codes"].view(torch.int8).view(r_c + r_r, D).double()
    B = B * raw["b_scales"].view(torch.float16).view(r_c + r_r, D // g).double().repeat_interleave(g, 1)
    return R, A, B


def _softplus(x):
    return torch.logaddexp(torch.zeros_like(x), x)


def exact(case, seed):
    s = prepare(case, seed)
    N = case["N"]
    if case["op"] == "backward":
        R, A, B = _exact_head(s["packed"], case["V"], case["D"], case["r_c"], case["r_r"], case["g"])
        out = torch.empty((N, case["D"]), dtype=torch.float64, device="cuda")
        for a in range(0, N, 1024):
            G = s["dY"][a:a + 1024].double()
            out[a:a + 1024] = G @ R if A is None else G @ R + (G @ A) @ B
        return {"dH": out}
    w, ref = s["weight"].double(), s["ref_logp"].double()
    rows = torch.nonzero(w)[:, 0]
    label = s["labels"][rows].long()
    logp = torch.zeros(N, dtype=torch.float64, device="cuda")
    dY = torch.zeros((N, case["V"]), dtype=torch.float64, device="cuda")
    for a in range(0, len(rows), 512):
        n = rows[a:a + 512]
        q = torch.log_softmax(s["Y"][n].double() * INV_TEMPERATURE, 1)
        logp[n] = q.gather(1, label[a:a + 512, None])[:, 0]
        dY[n] = -torch.exp(q)
    out = {}
    slope = torch.zeros(N, dtype=torch.float64, device="cuda")
    if case["op"] == "policy":
        lp = logp[rows].clone().requires_grad_()
        adv = s["advantage"][rows].double()
        ratio = (lp - s["old_logp"][rows].double()).exp()
        gain = torch.min(ratio * adv, torch.clip(ratio, 1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
        d = ref[rows] - lp
        row = -gain + KL_COEF * (d.exp() - d - 1)
        (w[rows] * row).sum().backward()
        slope[rows] = lp.grad
        out["loss"] = (w[rows] * row).sum().detach()
        out["row_loss"] = torch.zeros(N, dtype=torch.float64, device="cuda").index_copy(0, rows, row.detach())
    else:
        ends = s["offsets"].tolist()
        lp = logp.clone().requires_grad_()
        terms = w * (lp - ref)
        sums = torch.stack([terms[a:b].sum() for a, b in zip(ends, ends[1:])])
        h = BETA * (sums[0::2] - sums[1::2])
        loss = ((1 - SMOOTHING) * _softplus(-h) + SMOOTHING * _softplus(h)).sum()
        loss.backward()
        slope = lp.grad
        out["loss"] = loss.detach()
        out["chosen_reward"], out["rejected_reward"] = (BETA * sums[0::2]).detach(), (BETA * sums[1::2]).detach()
    out["logp"] = logp
    dY[rows, label] += 1.0
    dY *= (slope * INV_TEMPERATURE)[:, None]
    out["dY"] = dY
    return out
