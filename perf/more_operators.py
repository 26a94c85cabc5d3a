"""From the residual stream to logits or a loss: what is measured of it, on which cases.

Operators in front of a packed head and through it, as a model's last layers
call them:

  norm           the residual's addition and the root-mean-square norm, with the
                 hidden states in 8 bits and a scale for each token (serving),
                 or in bf16 with what its gradient needs (training)
  norm_backward  the norm's gradient, with the gradient that reaches the sum by
                 the residual stream
  int8           logits of INT8 hidden states through a row-INT8 head: a product
                 in 8-bit integers with scales for each token and channel
  xent           cross entropy of next tokens through a packed ARCHead head, the
                 vocabulary in pieces, with the hidden states' gradient and
                 without the logits

`run` computes a case in its plain form (elementary torch operations in fp32 or
fp64) or, where `own` is true, by the framework's entry points.  `exact` is the
definition in fp64.
"""
import math

import torch

own = False

BF16, F32, INT8 = "bf16", "f32", "int8"
_DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6

# The largest work of a case: elements of a norm, and multiplications of a product.
_MOST_ELEMENTS = 4096 * 8192
_MOST_MACS = 4096 * 151936 * 4096


def _norm(name, N, D, residual, out):
    return dict(name=name, op="norm", N=N, D=D, residual=residual, out=out)


def _norm_backward(name, N, D, through):
    return dict(name=name, op="norm_backward", N=N, D=D, through=through)


def _int8(name, N, V, D, y):
    return dict(name=name, op="int8", N=N, V=V, D=D, y=y)


def _xent(name, N, V, D, r_c, r_r, g, keep):
    return dict(name=name, op="xent", N=N, V=V, D=D, r_c=r_c, r_r=r_r, g=g, keep=keep)


def listed():
    return [
        # the final norm of one token's decoding step, for the INT8 head
        _norm("norm_one_token", 1, 4096, True, INT8),
        # a long prompt's rows of a 70B-class model, for the INT8 head
        _norm("norm_prefill", 4096, 8192, True, INT8),
        # a small model of odd width: rows at every alignment, no residual stream behind it
        _norm_backward("norm_backward_odd", 257, 1001, False),
        # a training step's rows, a gradient arriving by the residual stream as well
        _norm_backward("norm_backward_rows", 4096, 4096, True),
        # one token: the head is streamed once
        _int8("int8_one_token", 1, 151936, 4096, F32),
        # a serving batch on a vocabulary of odd size
        _int8("int8_batch", 61, 100003, 4096, F32),
        # a 70B-class head, one short sequence's perplexity
        _int8("int8_large_head", 256, 128256, 8192, BF16),
        # a long prompt's rows at once
        _int8("int8_prefill", 4096, 151936, 4096, BF16),
        # the smallest head: latency
        _xent("xent_few_small_head", 4, 1024, 256, 16, 8, 64, 1.0),
        # token-by-token adaptation on a full vocabulary
        _xent("xent_one_token", 1, 151936, 4096, 32, 32, 128, 1.0),
        # a 70B-class head, an instruction with its answer: a quarter of the rows is the prompt
        _xent("xent_large_head", 250, 128256, 8192, 64, 64, 128, 0.75),
        # a micro-batch of full sequences, a tenth of whose rows is padding
        _xent("xent_rows", 4096, 151936, 4096, 64, 64, 128, 0.9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "int8", "xent"])
    if op in ("norm", "norm_backward"):
        D = _log_int(rng, 64, 16384)
        D -= D % rng.choice([1, 8, 128]) if D > 128 else 0
        N = _log_int(rng, 1, min(16384, _MOST_ELEMENTS // D))
        if op == "norm":
            return dict(op=op, N=N, D=D, residual=rng.choice([True, True, False]), out=rng.choice([INT8, INT8, BF16]))
        return dict(op=op, N=N, D=D, through=rng.choice([True, False]))
    V = _log_int(rng, 1000, 152000)
    D = 512 * _log_int(rng, 1, 16)
    N = _log_int(rng, 1, max(1, min(4096, _MOST_MACS // (V * D))))
    if op == "int8":
        return dict(op=op, N=N, V=V, D=D, y=rng.choice([F32, BF16]))
    g = rng.choice([g for g in (32, 64, 128, 256) if D // g <= 64])
    return dict(op=op, N=N, V=V, D=D, r_c=8 * rng.randint(0, 8), r_r=8 * rng.randint(0, 8), g=g,
                keep=rng.choice([1.0, 0.9, 0.75, 0.5]))


def _kept(case):
    """Rows that count in the loss."""
    return max(1, round(case["N"] * case["keep"]))


def work(case):
    N, D = case["N"], case["D"]
    if case["op"] == "norm":
        # x, the residual stream and its sum; codes and a scale, or bf16 and the factor
        row = D * (2 + 4 * case["residual"] + (1 if case["out"] == INT8 else 2)) + 4
        return {"bytes": N * row + 2 * D, "flops": 8 * N * D}
    if case["op"] == "norm_backward":
        return {"bytes": N * (D * (6 + 2 * case["through"]) + 4) + 6 * D, "flops": 9 * N * D}
    V = case["V"]
    if case["op"] == "int8":
        size = {BF16: 2, F32: 4}[case["y"]]
        return {"bytes": V * (D + 2) + N * (D + 4) + N * V * size, "flops": 2 * N * V * D}
    K, r = _kept(case), case["r_c"] + case["r_r"]
    n_a = (case["r_c"] > 0) + (case["r_r"] > 0)
    head = V * (D // 2 + D // case["g"] + 2 + r + 2 * n_a) + r * (D + 2 * (D // case["g"]))
    # the packed head and the rows that count read once, every row's gradient written
    return {"bytes": head + (K + N) * D * 2 + N * 12, "flops": 4 * K * (V * (D + r) + r * D)}


# ------------------------------------------------------------------ inputs ---

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _hidden(gen, N, D):
    """Activations: normal, with a few channels that are much larger, as a
    trained model's residual stream has them."""
    x = _randn(gen, N, D)
    x[:, torch.randperm(D, generator=gen, device="cuda")[:max(1, D // 512)]] *= 8.0
    return x


def _layout(V, D, r_c, r_r, g, int8=False):
    """Section offsets of a packed head (format version 1) and its size."""
    V16, r, n_a, ng = -(-V // 16) * 16, r_c + r_r, (r_c > 0) + (r_r > 0), D // g
    codes, groups = (V16 * D, 0) if int8 else (V16 * D // 2, V16 * ng)
    sizes = [("header", 64), ("r_codes", codes), ("r_gcodes", groups), ("r_rowscale", 2 * V16),
             ("a_codes", V16 * r), ("a_scales", 2 * V16 * n_a), ("b_codes", r * D), ("b_scales", 2 * r * ng)]
    at, out = 0, {}
    for name, size in sizes:
        out[name] = (at, size)
        at += -(-size // 256) * 256
    return out, at, V16


def _packed_head(gen, V, D, r_c, r_r, g, int8=False):
    """A packed head's bytes: uniform codes, and scales of which logits of unit
    hidden states spread by about two."""
    where, total, V16 = _layout(V, D, r_c, r_r, g, int8)
    r, ng = r_c + r_r, D // g
    buf = torch.zeros(total, dtype=torch.uint8, device="cuda")
    target = 1.5 / math.sqrt(D)  # of an element of the residual, and of each low-rank part

    def put(name, t):
        at, size = where[name]
        buf[at:at + size] = t.contiguous().view(torch.uint8).reshape(-1)

    def scales(shape, sigma):
        return (_randn(gen, *shape) * sigma).abs().half()

    def codes(shape):
        return torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)

    put("header", torch.tensor([0x48435241, 1, V, 0, D, 0, r_c, r_r, g, 2 * int8] + [0] * 6, dtype=torch.int32,
                               device="cuda"))
    past = torch.arange(64, device="cuda") % 16 + V16 - 16 >= V  # rows past the vocabulary are zero
    if int8:
        tiles = codes((D // 128, V16 // 16, 64, 32))
        tiles[:, -1, past] = 0
        s_R = scales((V16,), target / 73)
        s_R[V:] = 0
        put("r_codes", tiles)
        put("r_rowscale", s_R)
        return buf
    tiles = torch.randint(0, 256, (D // 128, V16 // 16, 64, 16), generator=gen, device="cuda", dtype=torch.uint8)
    gcodes = torch.randint(1, 256, (V16, ng), generator=gen, device="cuda", dtype=torch.uint8)
    s_R, A = scales((V16,), target / (4.6 * 148)), codes((V16, r))
    tiles[:, -1, past] = 0
    gcodes[V:], s_R[V:], A[V:] = 0, 0, 0
    put("r_codes", tiles)
    put("r_gcodes", gcodes)
    put("r_rowscale", s_R)
    if r:
        ranks = [n for n in (r_c, r_r) if n]
        sigma = [math.sqrt(target / math.sqrt(n)) / 73 for n in ranks]
        s_A = torch.cat([scales((V16, 1), s) for s in sigma], 1)
        s_A[V:] = 0
        put("a_codes", A)
        put("a_scales", s_A)
        put("b_codes", codes((r, D)))
        put("b_scales", torch.cat([scales((n, ng), s) for n, s in zip(ranks, sigma)], 0))
    return buf


def _head_rows(buf, dims, v):
    """Rows v of W_hat in fp64, element by element from the layout."""
    V, D, r_c, r_r, g = dims
    where, _, V16 = _layout(*dims)
    raw = {k: buf[a:a + n] for k, (a, n) in where.items()}
    v, k = v[:, None], torch.arange(D, device="cuda")[None, :]
    tile = (k // 128 * (V16 // 16) + v // 16) * 1024
    code = raw["r_codes"][tile + 16 * (v % 16 + 16 * (k % 32 // 8)) + 4 * (k % 128 // 32) + k % 8 // 2].short()
    code = (code >> (4 * (k % 2)).short()) % 16
    W = (code - 16 * (code >= 8)).double()
    W *= raw["r_gcodes"][v * (D // g) + k // g].double()
    W *= raw["r_rowscale"].view(torch.float16)[v].double()
    if r_c + r_r == 0:
        return W
    part = (torch.arange(r_c + r_r, device="cuda") >= (r_c or r_c + r_r)).long()
    A = raw["a_codes"].view(torch.int8).view(V16, -1)[v[:, 0]].double()
    A = A * raw["a_scales"].view(torch.float16).view(V16, -1)[v[:, 0]].double()[:, part]
    B = raw["b_codes"].view(torch.int8).view(-1, D).double()
    return W + A @ (B * raw["b_scales"].view(torch.float16).view(-1, D // g).double().repeat_interleave(g, 1))


def _dims(case):
    return case["V"], case["D"], case.get("r_c", 0), case.get("r_r", 0), case.get("g", 128)


def prepare(case, seed):
    gen, N, D = _generator(seed), case["N"], case["D"]
    state = dict(case=dict(case))
    if case["op"] in ("norm", "norm_backward"):
        state["x"] = (_hidden(gen, N, D) * (0.5 + _randn(gen, N, 1).abs())).bfloat16()
        state["weight"] = (1.0 + 0.2 * _randn(gen, D)).bfloat16()
        if case["op"] == "norm":
            state["residual"] = (_hidden(gen, N, D) * 2.0).bfloat16() if case["residual"] else None
            return state
        # what the forward pass keeps, and the gradients that arrive
        square = state["x"].double().square().mean(1)
        state["inv_rms"] = torch.rsqrt(square + EPS).float()
        state["dh"] = (_randn(gen, N, D) / N).bfloat16()
        state["dsum"] = (_randn(gen, N, D) / N).bfloat16() if case["through"] else None
        return state
    dims = _dims(case)
    state["packed"] = _packed_head(gen, *dims, int8=case["op"] == "int8")
    if case["op"] == "int8":
        # hidden states as a norm leaves them, rounded to 8 bits by their row's largest
        h = _hidden(gen, N, D)
        state["scale"] = h.abs().amax(1) / 127
        state["codes"] = torch.round(h / state["scale"][:, None]).to(torch.int8)
    else:
        # hidden states that point to their label's row by more or less
        labels = torch.randint(0, case["V"], (N,), generator=gen, device="cuda")
        rows = _head_rows(state["packed"], dims, labels).float()
        lift = torch.rand((N, 1), generator=gen, device="cuda") * 14.0 / rows.square().sum(1, keepdim=True)
        state["H"] = (_hidden(gen, N, D) + lift * rows).bfloat16()
        weight = torch.zeros(N, device="cuda")
        weight[torch.randperm(N, generator=gen, device="cuda")[:_kept(case)]] = 1.0 / _kept(case)
        # prompt and padding rows carry no label
        state.update(labels=torch.where(weight != 0, labels, -100).int(), weight=weight)
    if own:
        import compressed_output_head_amd as ah
        fmt = ah.ARCHEAD_FMT_ROW_INT8 if case["op"] == "int8" else ah.ARCHEAD_FMT_ARCHEAD
        state["head"] = ah.PackedHead(*dims, state["packed"], fmt=fmt)
    return state


# -------------------------------------------------------------- plain forms ---

def _plain_norm(s):
    total, out = s["x"], {}
    if s["residual"] is not None:
        total = out["sum"] = (s["x"].float() + s["residual"].float()).bfloat16()
    inv = torch.rsqrt(total.double().square().mean(1) + EPS)
    # significands of 8 bits each: the product is exact
    t = total.float() * s["weight"].float()
    if s["case"]["out"] == INT8:
        top = t.abs().amax(1)
        scale = (top.double() * inv / 127).float()
        # a value next to a border between two codes is decided in fp64
        codes = torch.round(127 * t.double() / top.clamp(min=1e-30).double()[:, None])
        out.update(h=codes.float() * scale[:, None], scale=scale)
    else:
        out.update(h=(t.double() * inv[:, None]).bfloat16(), inv_rms=inv.float())
    return out


def _plain_norm_backward(s):
    x, dh, inv = s["x"].float(), s["dh"].float(), s["inv_rms"][:, None]
    g = dh * s["weight"].float()
    c = (g * x).sum(1, keepdim=True) * inv * inv / s["case"]["D"]
    dx = inv * (g - x * c)
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.bfloat16(), "dweight": (dh * x * inv).sum(0)}


def _get(buf, where, name, dtype, *shape):
    at, size = where[name]
    return buf[at:at + size].view(dtype).reshape(shape)


def _plain_int8(s):
    V, D = s["case"]["V"], s["case"]["D"]
    where, _, V16 = _layout(*_dims(s["case"]), int8=True)
    # tile byte 32 l + 8 s + p: row l % 16, columns 32 s + 8 (l / 16) and the p-th of 0 1 4 5 2 3 6 7
    t = _get(s["packed"], where, "r_codes", torch.int8, D // 128, V16 // 16, 4, 16, 4, 2, 2, 2)
    W = t.permute(1, 3, 0, 4, 2, 6, 5, 7).reshape(V16, D)[:V].float()
    rows = _get(s["packed"], where, "r_rowscale", torch.float16, V16)[:V].float()
    # sums of whole numbers, most of them below 2^24
    Y = s["codes"].float() @ W.T
    return {"Y": (Y * (s["scale"][:, None] * rows)).to(_DTYPES[s["case"]["y"]])}


def _plain_w_hat(buf, V, D, r_c, r_r, g):
    """W_hat = R + A_c B_c + A_w B_w in fp32 from the packed bytes."""
    where, _, V16 = _layout(V, D, r_c, r_r, g)
    r, n_a, ng = r_c + r_r, (r_c > 0) + (r_r > 0), D // g
    # tile byte 16 l + 4 s + c: row l % 16, columns 32 s + 8 (l / 16) + 2 c and the next
    t = _get(buf, where, "r_codes", torch.uint8, D // 128, V16 // 16, 4, 16, 4, 4).permute(1, 3, 0, 4, 2, 5)
    nibbles = torch.stack([t & 15, t >> 4], -1).reshape(V16, D).view(torch.int8)
    W = torch.where(nibbles > 7, nibbles - 16, nibbles).float()
    scale = _get(buf, where, "r_gcodes", torch.uint8, V16, ng).float()
    scale = scale * _get(buf, where, "r_rowscale", torch.float16, V16, 1).float()
    W = (W.view(V16, ng, g) * scale[:, :, None]).view(V16, D)
    if r:
        A = _get(buf, where, "a_codes", torch.int8, V16, r).float()
        s_A = _get(buf, where, "a_scales", torch.float16, V16, n_a).float()
        A *= torch.cat([s_A[:, i:i + 1].expand(V16, n) for i, n in enumerate(n for n in (r_c, r_r) if n)], 1)
        B = _get(buf, where, "b_codes", torch.int8, r, ng, g).float()
        B = B * _get(buf, where, "b_scales", torch.float16, r, ng, 1).float()
        W += A @ B.view(r, D)
    return W[:V]


def _plain_xent(s):
    W = _plain_w_hat(s["packed"], *_dims(s["case"]))
    at, w = s["labels"].long().clamp(min=0)[:, None], s["weight"]
    Y = s["H"].float() @ W.T
    top = Y.amax(1, keepdim=True)
    below = Y.gather(1, at).double() - top.double()
    P = torch.exp(Y.sub_(top))
    # the label's own term apart: 1 - p of a sure row keeps its digits
    label = P.gather(1, at)
    P.scatter_(1, at, 0.0)
    rest = P.sum(1, keepdim=True, dtype=torch.float64)
    logp = -torch.log1p(rest * torch.exp(-below))[:, 0]
    total = rest + label.double()
    P *= (w[:, None] / total).float()
    P.scatter_(1, at, (-w.double()[:, None] * rest / total).float())
    dH = (P @ W).bfloat16()
    on = w != 0
    logp = torch.where(on, logp, 0.0)
    return {"loss": -(w.double() * logp).sum().float(), "logp": logp.float(), "dH": dH}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "int8": _plain_int8, "xent": _plain_xent}


def run(state):
    case = state["case"]
    if not own:
        return _PLAIN[case["op"]](state)
    import compressed_output_head_amd as ah
    if case["op"] == "norm":
        wanted = ("codes", "scale") if case["out"] == INT8 else ("h", "inv_rms")
        out = ah.archead_rmsnorm(state["x"], weight=state["weight"], residual=state["residual"], eps=EPS, outputs=wanted)
        if case["out"] == INT8:  # as the values that they stand for
            out["h"] = out.pop("codes").float() * out["scale"][:, None]
        return out
    if case["op"] == "norm_backward":
        return ah.archead_rmsnorm_backward(state["dh"], state["x"], state["inv_rms"], weight=state["weight"],
                                           dsum=state["dsum"])
    if case["op"] == "int8":
        return {"Y": ah.archead_logits_int8(state["codes"], state["scale"], state["head"], out_dtype=_DTYPES[case["y"]])}
    return ah.archead_cross_entropy(state["H"], state["labels"], state["head"], weight=state["weight"])


# --------------------------------------------------- the definitions in fp64 ---

def exact(case, seed):
    s = prepare(case, seed)
    N, D, out = case["N"], case["D"], {}
    if case["op"] == "norm":
        total = s["x"].double()
        if s["residual"] is not None:  # the stream is kept in bf16, and that is what is normalised
            total = out["sum"] = (total + s["residual"].double()).bfloat16().double()
        inv = (total.pow(2).sum(1, keepdim=True) / D + EPS) ** -0.5
        h = total * s["weight"].double()
        if case["out"] == INT8:
            step = h.abs().max(1, keepdim=True)[0] / 127
            codes = torch.where(step > 0, torch.round(h / step), 0.0)
            return {**out, "h": codes * step * inv, "scale": (step * inv)[:, 0]}
        return {**out, "h": h * inv, "inv_rms": inv[:, 0]}
    if case["op"] == "norm_backward":
        x, dh, w, inv = s["x"].double(), s["dh"].double(), s["weight"].double(), s["inv_rms"].double()[:, None]
        unit = x * inv
        dx = inv * (dh * w - unit * torch.mean(dh * w * unit, 1, keepdim=True))
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return {"dx": dx, "dweight": torch.sum(dh * unit, 0)}
    V = case["V"]
    if case["op"] == "int8":
        where, _, V16 = _layout(*_dims(case), int8=True)
        raw = {k: s["packed"][a:a + n] for k, (a, n) in where.items()}
        Y = torch.empty((N, V), dtype=torch.float64, device="cuda")
        k = torch.arange(D, device="cuda")[None, :]
        slot = torch.tensor([0, 1, 4, 5, 2, 3, 6, 7], device="cuda")[k % 8]  # its own inverse
        for a in range(0, V, 16384):
            v = torch.arange(a, min(V, a + 16384), device="cuda")
            row = v[:, None]
            at = (k // 128 * (V16 // 16) + row // 16) * 2048 + 32 * (row % 16 + 16 * (k % 32 // 8)) + 8 * (k % 128 // 32)
            W = raw["r_codes"].view(torch.int8)[at + slot].double()
            W *= raw["r_rowscale"].view(torch.float16)[row].double()
            Y[:, a:a + len(v)] = (s["codes"].double() * s["scale"].double()[:, None]) @ W.T
        return {"Y": Y}
    W = torch.cat([_head_rows(s["packed"], _dims(case), torch.arange(a, min(V, a + 16384), device="cuda"))
                   for a in range(0, V, 16384)])
    rows = torch.nonzero(s["weight"])[:, 0]
    logp = torch.zeros(N, dtype=torch.float64, device="cuda")
    dH = torch.zeros((N, D), dtype=torch.float64, device="cuda")
    for a in range(0, len(rows), 1024):
        n = rows[a:a + 1024]
        label = s["labels"][n].long()
        q = torch.log_softmax(s["H"][n].double() @ W.T, 1)
        logp[n] = q[torch.arange(len(n), device="cuda"), label]
        P = torch.exp(q)
        P[torch.arange(len(n), device="cuda"), label] = torch.expm1(logp[n])
        dH[n] = (s["weight"][n].double()[:, None] * P) @ W
    return {"loss": -(s["weight"].double() * logp).sum(), "logp": logp, "dH": dH}
