"""GPU parity of archead_logits_backward with the fp64 oracle, dH = dY W_hat.

Tolerance, from the kernels' arithmetic.  With e(n) the power of two that
brings a row's largest |dY s| to [2^14, 2^15), every dY s is rounded to fp16
once: 2^-11 of itself, or half a subnormal step, 2^-25, which is less than
2^-39 of the row's largest.  The integers q4 c8 and the INT8 codes are exact;
an fp32 sum of m terms in any order is off by less than m 2^-24 of the sum of
their absolute values (m <= V / 8 here: an MFMA adds 8 or 16 products at
once, plus at most 64 + 64 partial sums).  With
    T[n, d] = sum_v |dY s_R| |q4 c8|,   Y[n, j] = sum_v |dY s_A| |code|
the residual's part is off by (2^-11 + m 2^-24) T + 2^-39 max|dY s_R| sum_v
|q4 c8|, Z by the same with its own terms, and dH by these, |Z's error| |B|,
r 2^-23 |Z| |B| (products and sums of the last step; of many rows 3 * 2^-18
more, as Z and B are pairs of bf16 numbers there whose smallest product is
left out), and the rounding to bf16, 2^-8 |dH|.
"""
import ctypes

import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


def _head(seed, V, D, r_c, r_r, g):
    h = synth.draw_head(np.random.default_rng(seed), V, D, r_c, r_r, g)
    return h, ah_mod().PackedHead.from_components(h)


def _gradient(rng, N, V):
    """A loss's gradient: coefficients times (one-hot - softmax), some rows zero."""
    z = rng.normal(0, 2.5, (N, V))
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    p[np.arange(N), rng.integers(0, V, N)] -= 1.0
    coef = rng.normal(0, 1, N) * 10.0 ** rng.integers(-6, 3, N)
    if N > 3:
        coef[rng.random(N) < 0.15] = 0.0
    return p * coef[:, None]


def _run(head, dY, **kw):
    torch = torch_mod()
    dH = torch.full((dY.shape[0], head.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ah_mod().archead_logits_backward(dY, head, dH, **kw)
    torch.cuda.synchronize()
    return dH.double().cpu().numpy()


def _bound(dY, h, want):
    V, D = h.V, h.D
    m = (V / 8 + 128) * 2.0 ** -24
    codes = np.abs(h.q4.astype(np.float64)) * np.repeat(h.c8.astype(np.float64), h.g, axis=1)
    parts = [(np.abs(dY) * h.s_R.astype(np.float64), codes, None, None)]
    for A, s_A, B, s_B in ((h.A_c, h.s_Ac, h.B_c, h.s_Bc), (h.A_w, h.s_Aw, h.B_w, h.s_Bw)):
        if A.shape[1]:
            parts.append((np.abs(dY) * s_A.astype(np.float64), np.abs(A.astype(np.float64)),
                          np.abs(B.astype(np.float64)) * np.repeat(s_B.astype(np.float64), h.g, axis=1), A.shape[1]))
    tol = np.zeros_like(want)
    for x, w, B, r in parts:
        S = x @ w
        err = (2.0 ** -11 + m) * S + 2.0 ** -39 * x.max(1, keepdims=True) * w.sum(0)
        tol += err if B is None else err @ B + (r * 2.0 ** -23 + 3 * 2.0 ** -18) * (S @ B)
    return tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -120


def _check(head, h, dY_dev, what):
    dY = dY_dev.double().cpu().numpy()
    got, want = _run(head, dY_dev), oracle.logits_backward(dY, h)
    tol = _bound(dY, h, want)
    worst = np.max(np.abs(got - want) / tol)
    norm = np.linalg.norm(want)
    rel = np.linalg.norm(got - want) / norm if norm else 0.0
    log(f"  {what}: worst error / bound {worst:.3f}, norm of the error {rel:.2e}")
    assert not np.isnan(got).any() and worst <= 1.0, what
    # bf16 rounding alone is at most 2^-8 of every element, so of the norm
    assert rel <= 2.0 ** -8, what
    zero = ~dY.any(1)
    assert not got[zero].any()


CASES = [  # V, D, r_c, r_r, g, N: the four token tiles, ragged everything
    (1, 128, 0, 0, 32, 1),
    (16, 128, 8, 8, 128, 3),
    (1000, 512, 16, 8, 64, 1),
    (777, 256, 8, 0, 32, 16),
    (2048, 1024, 32, 32, 128, 32),
    (1031, 384, 0, 24, 64, 33),
    (530, 512, 40, 72, 256, 64),
    (999, 640, 64, 64, 128, 65),
    (4099, 256, 0, 0, 256, 128),
    (1000, 512, 16, 8, 32, 130),
    (3001, 896, 32, 64, 128, 257),
    (515, 512, 8, 152, 64, 300),
    (33000, 256, 16, 16, 64, 40),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V,D,r_c,r_r,g,N", CASES)
def test_backward_matches_oracle(V, D, r_c, r_r, g, N, dtype):
    torch = torch_mod()
    log(f"backward V={V} D={D} r_c={r_c} r_r={r_r} g={g} N={N} {dtype}")
    h, head = _head(V + N, V, D, r_c, r_r, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N), N, V), device="cuda").to(getattr(torch, dtype))
    _check(head, h, dY, f"V={V} N={N}")


@pytest.mark.parametrize("N", [1, 5, 31])
@pytest.mark.parametrize("V,D,r_c,r_r,g", [(1031, 512, 40, 72, 256), (2500, 768, 0, 40, 256), (999, 640, 72, 0, 128),
                                           (640, 384, 24, 8, 64), (1234, 256, 32, 136, 32)])
def test_few_tokens_of_every_group_size(V, D, r_c, r_r, g, N):
    """The few-token kernels: shared and several group codes a tile, rank tiles
    that end early, rows of fewer tokens than an operand holds."""
    torch = torch_mod()
    h, head = _head(V + g, V, D, r_c, r_r, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N + V), N, V), device="cuda").bfloat16()
    _check(head, h, dY, f"V={V} D={D} r={r_c}+{r_r} g={g} N={N}")


@pytest.mark.parametrize("V,D,r_c,r_r,g,N", [(200, 1152, 24, 0, 128, 2100), (333, 1152, 8, 16, 32, 1999),
                                             (3001, 4096, 40, 24, 64, 500), (150, 1024, 0, 0, 256, 2048)])
def test_many_rows_of_wide_heads(V, D, r_c, r_r, g, N):
    """The last kernel of many rows: ranks that end in a half step, columns and
    rows that end inside a workgroup and a tile, several parts."""
    torch = torch_mod()
    h, head = _head(V + g, V, D, r_c, r_r, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(N), N, V), device="cuda").bfloat16()
    _check(head, h, dY, f"V={V} D={D} r={r_c}+{r_r} g={g} N={N}")


def _dequant(h):
    return (h.q4.astype(np.float64) * np.repeat(h.c8.astype(np.float64), h.g, axis=1)
            * h.s_R.astype(np.float64)[:, None])


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -90])
@pytest.mark.parametrize("V,D,g,N", [(700, 512, 32, 32), (350, 256, 64, 64), (333, 384, 128, 128), (900, 512, 256, 900)])
def test_one_hot_rows_give_the_residual_rows_exactly(V, D, g, N, scale):
    """dY one-hot: no sum rounds, so dH is the head's row rounded to bf16, also
    where the row's scale is a subnormal fp16 and the gradient tiny."""
    torch = torch_mod()
    h, head = _head(g, V, D, 0, 0, g)
    W = _dequant(h)
    rng = np.random.default_rng(V)
    for first in range(0, V, N):
        v = (first + rng.permutation(N)) % V
        dY = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
        dY[torch.arange(N), torch.as_tensor(v)] = scale
        got = _run(head, dY)
        want = torch.as_tensor(W[v] * scale).to(torch.bfloat16).double().numpy()
        assert np.array_equal(got, want), (first, np.argwhere(got != want)[:4])


@pytest.mark.parametrize("N", [3, 40])
def test_large_values_of_entries_of_scale_zero(N):
    """A row whose products with the scales are tiny, next to a value that only
    meets a scale of 0: nothing overflows, and the tiny row is still exact."""
    torch = torch_mod()
    V, D, g = 96, 256, 64
    h = synth.draw_head(np.random.default_rng(11), V, D, 0, 0, g)
    h.s_R[5] = 0
    head = ah_mod().PackedHead.from_components(h)
    W = _dequant(h)
    dY = torch.zeros((N, V), dtype=torch.float32, device="cuda")
    v = [i % V for i in range(6, 6 + N)]
    dY[torch.arange(N), torch.as_tensor(v)] = 2.0 ** -95
    dY[:, 5] = 1e30
    got = _run(head, dY)
    want = torch.as_tensor(W[v] * 2.0 ** -95).to(torch.bfloat16).double().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("N", [5, 4096])
def test_backward_of_the_largest_ranks(N):
    """r_c + r_r = 1024, with few and with many rows."""
    torch = torch_mod()
    V, D, g = 70, 1024, 128
    h, head = _head(12, V, D, 512, 512, g)
    dY = torch.as_tensor(_gradient(np.random.default_rng(12), N, V), device="cuda").bfloat16()
    _check(head, h, dY, f"r=512+512 N={N}")


def test_calls_on_two_streams_at_once():
    """Losses and gradients of two streams that run at the same time, each call
    with a workspace of its own: the results of calls alone."""
    torch = torch_mod()
    ah = ah_mod()
    V, D = 5000, 512
    h, head = _head(13, V, D, 16, 8, 64)
    jobs = []
    for N in (24, 700):
        gen = torch.Generator(device="cuda").manual_seed(N)
        Y = torch.randn((N, V), generator=gen, device="cuda").bfloat16()
        labels = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
        adv = torch.randn((N,), generator=gen, device="cuda")
        offsets = torch.tensor([0, N // 3, N // 2, N - 1, N], dtype=torch.int32, device="cuda")
        jobs.append((Y, labels, adv, offsets, torch.cuda.Stream()))

    def step(Y, labels, adv, offsets, stream=None):
        p = ah.archead_policy_loss(Y, labels, adv, stream=stream)
        q = ah.archead_preference_loss(Y, labels, offsets, stream=stream)
        return [p["loss"], p["logp"], p["dY"], q["loss"], q["dY"],
                ah.archead_logits_backward(p["dY"], head, stream=stream),
                ah.archead_logits_backward(q["dY"], head, stream=stream)]

    want = [[t.clone() for t in step(*j[:4])] for j in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [step(*j[:4], stream=j[4]) for j in jobs]
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, x))


def test_backward_strided_and_unaligned():
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(5, 1003, 512, 16, 8, 64)
    for dtype in (torch.bfloat16, torch.float32):
        dY = torch.as_tensor(_gradient(np.random.default_rng(1), 50, 1003), device="cuda").to(dtype)
        want = ah.archead_logits_backward(dY, head)
        for pad, first in ((0, 0), (5, 1), (13, 3)):
            buf = torch.full((50 * (1003 + pad) + first,), float("nan"), dtype=dtype, device="cuda")
            view = buf[first:].view(50, 1003 + pad)[:, :1003]
            view.copy_(dY)
            out = torch.full((50 * (512 + pad) + first,), 3.0, dtype=torch.bfloat16, device="cuda")
            dH = out[first:].view(50, 512 + pad)[:, :512]
            ah.archead_logits_backward(view, head, dH)
            torch.cuda.synchronize()
            assert torch.equal(dH, want), (dtype, pad)
            dH.fill_(3.0)
            assert (out == 3.0).all(), "written beside the rows"


def test_backward_rows_are_independent():
    """Rows that are not finite leave the others alone; a row's result does not
    depend on its place or its neighbours (the same token tile)."""
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(6, 600, 256, 8, 8, 64)
    g = _gradient(np.random.default_rng(2), 40, 600)
    dY = torch.as_tensor(g, device="cuda").bfloat16()
    base = ah.archead_logits_backward(dY, head)
    bad = dY.clone()
    bad[3, 17] = float("nan")
    bad[20, 599] = float("inf")
    got = ah.archead_logits_backward(bad, head)
    torch.cuda.synchronize()
    keep = [i for i in range(40) if i not in (3, 20)]
    assert torch.equal(got[keep], base[keep])
    assert not torch.isfinite(got[[3, 20]].float()).any()
    flipped = ah.archead_logits_backward(dY.flip(0).contiguous(), head)
    assert torch.equal(flipped.flip(0), base)


def test_backward_of_many_rows_in_chunks():
    """More rows than one pass takes: the rows of each pass as in a call of their own."""
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(7, 130, 128, 8, 8, 32)
    g = torch.as_tensor(_gradient(np.random.default_rng(3), 8192 + 70, 130), device="cuda").bfloat16()
    got = ah.archead_logits_backward(g, head)
    for a, b in ((0, 4096), (4096, 8192), (8192, 8262)):
        assert torch.equal(got[a:b], ah.archead_logits_backward(g[a:b].contiguous(), head))
    rows = [0, 31, 4095, 4096, 8191, 8192, 8261]
    want = oracle.logits_backward(g[rows].double().cpu().numpy(), h)
    assert np.all(np.abs(got[rows].double().cpu().numpy() - want) <= _bound(g[rows].double().cpu().numpy(), h, want))
    assert ah.archead_logits_backward(g[:0], head).shape == (0, 128)


def test_backward_in_a_graph_and_on_another_stream():
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(8, 5000, 512, 32, 32, 128)
    rng = np.random.default_rng(4)
    dY = torch.as_tensor(_gradient(rng, 48, 5000), device="cuda").bfloat16()
    want = ah.archead_logits_backward(dY, head)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = ah.archead_logits_backward(dY, head, stream=s)
        side.synchronize()
        assert torch.equal(got, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ah.archead_logits_backward(dY, head)
        graphs.append((g, out))
    for i in range(4):
        dY.copy_(torch.as_tensor(_gradient(rng, 48, 5000)))
        want = ah.archead_logits_backward(dY, head).clone()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs), i


def test_training_step_through_the_head():
    """Logits, loss with the gradient over them, and the hidden states' gradient:
    against the oracle's chain, and against differences of the loss along a
    direction of H."""
    torch = torch_mod()
    ah = ah_mod()
    N, V, D = 24, 1500, 512
    inp = synth.make("tiny", seed=31, V=V, D=D, N=N, r_c=16, r_r=16, g=64, n_outlier=0)
    inp.head.s_R = (inp.head.s_R * np.float16(0.05)).astype(np.float16)  # logits of a few units
    for k in ("s_Ac", "s_Aw"):
        setattr(inp.head, k, (getattr(inp.head, k) * np.float16(0.005)).astype(np.float16))
    head = ah.PackedHead.from_components(inp.head)
    H = torch.from_numpy(inp.H_bits.view(np.int16)).view(torch.bfloat16).cuda()
    rng = np.random.default_rng(1)
    labels = rng.integers(0, V, N)
    W = oracle.w_hat(inp.head)
    H64 = H.double().cpu().numpy()
    weight = np.where(np.arange(N) % 5 == 0, 0.0, 1.0 / N).astype(np.float32)
    dev = lambda x, t=torch.float32: torch.as_tensor(x, dtype=t, device="cuda")
    ref = -ah.archead_logits_stats(H, head, targets=dev(labels, torch.int32))["ce"]  # log p of this very policy
    old = ref - dev(rng.normal(0, 0.05, N))
    A = rng.normal(0, 1, N).astype(np.float32)
    off = np.array([0, 6, 12, 20, 24])

    def oracle_policy(h64):
        return oracle.policy_loss(h64 @ W.T, labels, A, old_logp=old.double().cpu().numpy(),
                                  ref_logp=ref.double().cpu().numpy(), weight=weight, kl_coef=0.25)

    def oracle_preference(h64):
        return oracle.preference_loss(h64 @ W.T, labels, off, ref_logp=ref.double().cpu().numpy(), beta=0.5)

    direction = rng.normal(0, 1, H64.shape)
    for name, f in (("policy", oracle_policy), ("preference", oracle_preference)):
        Y = ah.logits(H, head)
        if name == "policy":
            out = ah.archead_policy_loss(Y, dev(labels, torch.int32), dev(A), old_logp=old, ref_logp=ref,
                                         weight=dev(weight), kl_coef=0.25, dY=Y)
        else:
            out = ah.archead_preference_loss(Y, dev(labels, torch.int32), dev(off, torch.int32), ref_logp=ref, beta=0.5,
                                             dY=Y)
        dH = ah.archead_logits_backward(out["dY"], head)
        torch.cuda.synchronize()
        want = f(H64)
        want_dH = want["dY"] @ W
        got = dH.double().cpu().numpy()
        assert abs(out["loss"].item() - want["loss"]) <= 1e-5 * max(1.0, np.abs(want["logp"]).max())
        # 2^-8 for dH's rounding; the logits' error (1e-5 of their size, the forward's bound) moves dY by as much
        rel = np.linalg.norm(got - want_dH) / np.linalg.norm(want_dH)
        assert rel <= 2.0 ** -8 + 1e-5 * 2 * np.abs(H64 @ W.T).max(), (name, rel)
        step = 1e-4
        slope = (f(H64 + step * direction)["loss"] - f(H64 - step * direction)["loss"]) / (2 * step)
        along = (got * direction).sum()
        spread = 2.0 ** -8 * np.linalg.norm(want_dH) * np.linalg.norm(direction) + 1e-5 * abs(slope)
        assert abs(along - slope) <= spread, (name, along, slope)
        log(f"  {name}: dH error {rel:.2e}, along a direction {along:.6f} against differences {slope:.6f}")


def test_backward_binding_refusals():
    torch = torch_mod()
    ah = ah_mod()
    h, head = _head(9, 100, 128, 0, 0, 64)
    dY = torch.zeros((4, 100), device="cuda")
    for f in (lambda: ah.archead_logits_backward(dY.cpu(), head), lambda: ah.archead_logits_backward(dY.t(), head),
              lambda: ah.archead_logits_backward(dY, head, workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    for f, status in ((lambda: ah.archead_logits_backward(dY[:, :99], head), 5),
                      (lambda: ah.archead_logits_backward(dY.half(), head), 4),
                      (lambda: ah.archead_logits_backward(dY, head, torch.zeros((4, 128), device="cuda")), 4),
                      (lambda: ah.archead_logits_backward(dY, head, torch.zeros((3, 128), dtype=torch.bfloat16,
                                                                                device="cuda")), 5),
                      (lambda: ah.archead_logits_backward(dY, head, workspace=torch.zeros(256, dtype=torch.uint8,
                                                                                          device="cuda")), 7)):
        with pytest.raises(ah.ArcheadError) as e:
            f()
        assert e.value.status == status
