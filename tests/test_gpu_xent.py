"""GPU parity of archead_cross_entropy with the fp64 oracle.

Tolerances, from the kernels' arithmetic.  A logit is an fp32 sum of D / 16 +
ranks / 16 steps (an MFMA adds 16 products at once) and a few roundings of its
parts: off by
    eps = (D / 16 + r / 16 + 32) 2^-24 sum_k |h_k| |W|_vk
at most, |W| the residual's and the factors' magnitudes.  Exponentials: their
argument by 2^-24 of itself (up to 40 here), 2^x by the hardware 2^-22, sums in
short fp32 runs: 2^-18 of a probability in all, and tau eps twice (its own and
the sum's).  In the product they are rounded to fp16, 2^-11, and so is the
residual's operand of many rows: 2^-10.  The row's largest operand is at least
2^10 (at most 2^14, less 3 powers of two of room for later pieces, and it is
above half of that), and below 2^-14 the half step is 2^-25, twice where an
operand is brought to another exponent: 2^-34 of the largest.  Sums over the vocabulary are fp32 sums of
V / 16 + 128 terms, Z B as in the backward (r 2^-23 + 3 2^-18).  With
    T = sum_{v != l} p_v |W|_v + (1 - p_l) |W|_l
dH is off by the sum of these times |w| tau T, and by its rounding, 2^-8; log p
by (1 - p)(2 tau eps + 2^-18) and its rounding, 2^-24.
"""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu


def _head(seed, V, D, r_c, r_r, g, spread=2.0):
    """A head whose logits of unit hidden states spread by about `spread`."""
    h = synth.draw_head(np.random.default_rng(seed), V, D, r_c, r_r, g)
    W = oracle.w_hat(h)
    f = spread / max(np.sqrt((W ** 2).sum(1).mean()), 1e-6)
    for s in (h.s_R, h.s_Ac, h.s_Aw):
        s[...] = (s.astype(np.float64) * f).astype(np.float16)
    return h, ah_mod().PackedHead.from_components(h)


def _hidden(seed, N, D, W, labels, lift=8.0):
    """bf16 hidden states; half of the rows point to their label's row."""
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    H = rng.normal(0, 1, (N, D))
    rows = W[labels]
    sure = (rng.random(N) < 0.5) * rng.random(N) * lift
    H += (sure / np.maximum((rows ** 2).sum(1), 1e-9))[:, None] * rows
    return torch.from_numpy(H.astype(np.float32)).cuda().bfloat16()


def _magnitudes(h):
    R = np.abs(h.q4.astype(np.float64)) * np.repeat(h.c8.astype(np.float64), h.g, 1) * np.abs(h.s_R.astype(np.float64))[:, None]
    low, r = np.zeros_like(R), 0
    for A, s_A, B, s_B in ((h.A_c, h.s_Ac, h.B_c, h.s_Bc), (h.A_w, h.s_Aw, h.B_w, h.s_Bw)):
        if A.shape[1]:
            low += (np.abs(A.astype(np.float64)) * np.abs(s_A.astype(np.float64))[:, None]) @ (
                np.abs(B.astype(np.float64)) * np.repeat(np.abs(s_B.astype(np.float64)), h.g, 1))
            r += A.shape[1]
    return R, low, r


def _check(got, H, labels, w, h, tau, what):
    torch = torch_mod()
    H64, labels = H.double().cpu().numpy(), np.asarray(labels)
    w64 = np.ones(len(H64)) if w is None else w.double().cpu().numpy()
    on = w64 != 0
    W = oracle.w_hat(h)
    want = oracle.cross_entropy(np.where(on[:, None], H64, 0), np.where(on, labels, 0), h, w64, tau, W=W)
    R, low, r = _magnitudes(h)
    Wabs, V, D = R + low, h.V, h.D
    logp, dH = got["logp"].double().cpu().numpy(), got["dH"].double().cpu().numpy()
    assert not logp[~on].any() and not dH[~on].any()
    eps = (D / 16 + r / 16 + 32) * 2.0 ** -24 * (np.abs(H64) @ Wabs.T).max(1)
    q = -np.expm1(want["logp"])
    tol_p = q * (2 * tau * eps + 2.0 ** -18) + 2.0 ** -24 * np.abs(want["logp"]) + 2.0 ** -149
    err_p = np.abs(logp - want["logp"])
    assert (err_p <= tol_p)[on].all(), (what, (err_p / tol_p)[on].max())
    z = np.where(on[:, None], H64, 0) @ W.T * tau
    z[np.arange(len(z)), np.where(on, labels, 0)] = -np.inf
    top = z.max(1, keepdims=True) if V > 1 else np.zeros((len(z), 1))
    e = np.exp(z - top)
    S = np.maximum(e.sum(1, keepdims=True), 1e-300)
    T = q[:, None] * (e / S @ Wabs + Wabs[np.where(on, labels, 0)])
    rel = 2.0 ** -10 + 4 * tau * eps[:, None] + 2.0 ** -17 + (V / 16 + 128) * 2.0 ** -24 + r * 2.0 ** -23 + 3 * 2.0 ** -18
    tol = np.abs(w64)[:, None] * tau * (rel * T + 2.0 ** -34 * q[:, None] / S * Wabs.sum(0))
    tol = tol + 2.0 ** -8 * (np.abs(want["dH"]) + tol) + 2.0 ** -134
    err = np.abs(dH - want["dH"])
    assert (err <= tol)[on].all(), (what, (err / tol)[on].max())
    size = np.linalg.norm(want["dH"])
    if size:
        rel_norm = np.linalg.norm(dH - want["dH"]) / size
        log(f"  {what}: log p error / bound {(err_p / tol_p)[on].max():.3f}, dH {(err / tol)[on].max():.3f}, norm {rel_norm:.2e}")
        assert rel_norm <= 2.0 ** -8
    loss = (np.abs(w64) * tol_p)[on].sum() + 2.0 ** -23 * abs(want["loss"])
    assert abs(got["loss"].item() - want["loss"]) <= loss


CASES = [  # V, D, r_c, r_r, g, N
    (1, 128, 0, 0, 32, 1), (2, 128, 0, 0, 64, 3), (17, 128, 8, 8, 128, 5), (1000, 512, 16, 8, 64, 1),
    (777, 256, 8, 0, 32, 16), (2048, 1024, 32, 32, 128, 17), (1031, 384, 0, 24, 64, 32), (5000, 512, 40, 72, 256, 9),
    (999, 640, 64, 64, 128, 33), (4099, 256, 0, 0, 256, 64), (1000, 512, 16, 8, 32, 65), (3001, 896, 32, 64, 128, 130),
    (515, 512, 8, 152, 64, 200), (9000, 256, 16, 16, 64, 257), (256, 512, 8, 8, 64, 300), (300, 128, 0, 8, 32, 513),
]


@pytest.mark.parametrize("tau,weighted", [(1.0, True), (0.7, False)])
@pytest.mark.parametrize("V,D,r_c,r_r,g,N", CASES)
def test_cross_entropy_matches_oracle(V, D, r_c, r_r, g, N, tau, weighted):
    log(f"xent V={V} D={D} r_c={r_c} r_r={r_r} g={g} N={N} tau={tau}")
    torch, ah = torch_mod(), ah_mod()
    h, head = _head(V + N, V, D, r_c, r_r, g)
    rng = np.random.default_rng(N)
    labels = rng.integers(0, V, N)
    H = _hidden(N, N, D, oracle.w_hat(h), labels)
    w = None
    if weighted:
        w = torch.from_numpy((rng.normal(0, 1, N) * (rng.random(N) < 0.7)).astype(np.float32)).cuda()
        labels = np.where(w.cpu().numpy() != 0, labels, -100)
    got = ah.archead_cross_entropy(H, torch.from_numpy(labels).int().cuda(), head, weight=w, inv_temperature=tau)
    _check(got, H, labels, w, h, float(np.float32(tau)), f"V={V} N={N}")


def test_log_probabilities_of_the_same_logits():
    """Few rows: log p against fp64 sums over archead_logits' own fp32 logits,
    also where the label holds nearly all of the probability."""
    torch, ah = torch_mod(), ah_mod()
    V, D, N = 20011, 512, 32
    h, head = _head(1, V, D, 16, 16, 128)
    labels = np.random.default_rng(1).integers(0, V, N)
    H = _hidden(2, N, D, oracle.w_hat(h), labels, lift=200.0)
    lab = torch.from_numpy(labels).int().cuda()
    got = ah.archead_cross_entropy(H, lab, head)["logp"].double()
    Y = ah.logits(H, head).double()
    yl = Y.gather(1, lab.long()[:, None])
    Y.scatter_(1, lab.long()[:, None], -float("inf"))
    want = -torch.log1p(torch.exp(torch.logsumexp(Y, 1) - yl[:, 0]))
    q = -torch.expm1(want)
    assert q.min() < 1e-9  # rows that are sure
    assert ((got - want).abs() <= q * 2.0 ** -18 + want.abs() * 2.0 ** -24).all()


ROWS = [4, 32, 40, 200]


@pytest.mark.parametrize("N", ROWS)
def test_rows_that_do_not_count_and_rows_that_are_bad(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 1000, 512
    h, head = _head(3, V, D, 16, 8, 64)
    rng = np.random.default_rng(N)
    labels = rng.integers(0, V, N)
    H = _hidden(4, N, D, oracle.w_hat(h), labels)
    lab = torch.from_numpy(labels).int().cuda()
    w = torch.full((N,), 0.5, device="cuda")
    w[1] = 0.0
    want = ah.archead_cross_entropy(H, lab, head, weight=w)
    assert torch.isfinite(want["dH"]).all()
    B, blab = H.clone(), lab.clone()
    B[1] = float("nan")
    blab[1] = 1 << 30
    got = ah.archead_cross_entropy(B, blab, head, weight=w)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert got["logp"][1] == 0 and not got["dH"][1].any()
    for change in ("label", "low", "nan", "inf"):
        B, blab = H.clone(), lab.clone()
        if change == "label":
            blab[2] = V
        elif change == "low":
            blab[2] = -1
        else:
            B[2, 7] = float(change)
        got = ah.archead_cross_entropy(B, blab, head, weight=w)
        assert torch.isnan(got["logp"][2]) and torch.isnan(got["dH"][2]).all() and torch.isnan(got["loss"]), change
        keep = torch.arange(N, device="cuda") != 2
        assert torch.equal(got["logp"][keep], want["logp"][keep]), change
        assert torch.equal(got["dH"][keep], want["dH"][keep]), change
    none = ah.archead_cross_entropy(B, blab, head, weight=torch.zeros(N, device="cuda"))
    assert none["loss"] == 0 and not none["logp"].any() and not none["dH"].any()


@pytest.mark.parametrize("N", ROWS)
def test_strides_outputs_and_workspace(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 1500, 512
    h, head = _head(5, V, D, 8, 16, 128)
    labels = np.random.default_rng(N).integers(0, V, N)
    H = _hidden(6, N, D, oracle.w_hat(h), labels)
    lab = torch.from_numpy(labels).int().cuda()
    want = ah.archead_cross_entropy(H, lab, head)
    again = ah.archead_cross_entropy(H, lab, head)
    big = torch.zeros((N, D + 64), dtype=torch.bfloat16, device="cuda")
    big[:, 8:8 + D] = H
    out = torch.full((N, D + 7), 3.0, dtype=torch.bfloat16, device="cuda")
    need = ah.archead_cross_entropy_workspace_bytes(V, D, 8, 16, 128, N)
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    got = ah.archead_cross_entropy(big[:, 8:8 + D], lab, head, dH=out[:, 3:3 + D], workspace=ws[:need])
    for k in want:
        assert torch.equal(got[k], want[k]) and torch.equal(again[k], want[k]), k
    assert (out[:, :3] == 3).all() and (out[:, 3 + D:] == 3).all() and (ws[need:] == 7).all()
    alone = ah.archead_cross_entropy(H, lab, head, with_gradient=False)
    assert "dH" not in alone
    for k in alone:
        assert torch.equal(alone[k], want[k]), k
    none = ah.archead_cross_entropy(H[:0], lab[:0], head)
    assert none["loss"] == 0 and none["dH"].shape == (0, D)


@pytest.mark.parametrize("N", ROWS)
def test_in_graphs_and_on_streams(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 2500, 512
    h, head = _head(7, V, D, 8, 8, 64)
    W = oracle.w_hat(h)
    labels = np.random.default_rng(N).integers(0, V, N)
    H, lab = _hidden(8, N, D, W, labels), torch.from_numpy(labels).int().cuda()
    w = torch.rand(N, device="cuda")
    ah.archead_cross_entropy(H, lab, head, weight=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ah.archead_cross_entropy(H, lab, head, weight=w)
    for k in range(4):
        H.copy_(_hidden(20 + k, N, D, W, labels))
        w.copy_((torch.rand(N, device="cuda") < 0.3 * k).float())
        graph.replay()
        torch.cuda.synchronize()
        want = ah.archead_cross_entropy(H, lab, head, weight=w)
        for name in want:
            assert torch.equal(held[name], want[name]), (k, name)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [ah.archead_cross_entropy(H, lab, head, weight=w, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        for name in want:
            assert torch.equal(g[name], want[name]), name


@pytest.mark.parametrize("N", [3, 90])
def test_gradient_against_differences(N):
    """The kernels' gradient against differences of the kernels' own loss, along
    a direction whose steps bf16 holds exactly."""
    torch, ah = torch_mod(), ah_mod()
    V, D = 800, 256
    h, head = _head(9, V, D, 8, 8, 64)
    labels = np.random.default_rng(N).integers(0, V, N)
    H, lab = _hidden(10, N, D, oracle.w_hat(h), labels), torch.from_numpy(labels).int().cuda()
    step = torch.where(torch.rand((N, D), device="cuda") < 0.5, -1.0, 1.0) * H.abs().float() * 2.0 ** -7
    up, down = (H.float() + step).bfloat16(), (H.float() - step).bfloat16()
    move = (up.double() - down.double())
    a, b = (ah.archead_cross_entropy(x, lab, head)["logp"].double() for x in (up, down))
    dH = ah.archead_cross_entropy(H, lab, head)["dH"].double()
    want = (dH * move).sum(1)
    # per row: dH by 2^-8 of each term, log p by its digits, the curve's third derivative along the step
    noise = 2.0 ** -7 * (dH.abs() * move.abs()).sum(1) + 2.0 ** -17 + 0.1 * want.abs() + move.square().sum(1)
    assert ((b - a) - want).abs().le(noise).all()


def test_a_training_step_from_the_stream_to_its_gradient():
    """Norm, cross entropy through the packed head, the norm's gradient, as a
    training step calls them; against the oracle's own chain."""
    torch, ah = torch_mod(), ah_mod()
    V, D, N = 1200, 512, 70
    h, head = _head(11, V, D, 16, 8, 64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn((N, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    g = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    f = ah.archead_rmsnorm(x, weight=g, residual=r, outputs=("h", "inv_rms"))
    loss = ah.archead_cross_entropy(f["h"], labels, head, weight=torch.full((N,), 1 / N, device="cuda"))
    back = ah.archead_rmsnorm_backward(loss["dH"], f["sum"], f["inv_rms"], weight=g)
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    of = oracle.rmsnorm(n64(x), n64(r), n64(g))
    ol = oracle.cross_entropy(n64(f["h"]), labels.cpu().numpy(), h, np.full(N, 1 / N))
    ob = oracle.rmsnorm_backward(ol["dH"], of["sum"], of["inv_rms"], n64(g))
    assert abs(loss["loss"].item() - ol["loss"]) <= 1e-5 * abs(ol["loss"])
    for k in ("dx", "dweight"):  # two roundings to bf16 and the product's
        assert np.linalg.norm(n64(back[k]) - ob[k]) <= 2.0 ** -7 * np.linalg.norm(ob[k]), k


# V, D, r_c, r_r, g, N, share of the rows that count: every number of row tiles
# that a workgroup takes, chosen by the rows that count or by the call's; passes
# of 4096 rows, the last of them without a row that counts; ranks behind the
# first 64 of either kind, and factors of one kind alone
SHARES = [
    (700, 256, 8, 8, 64, 100, 0.1), (700, 256, 8, 8, 64, 300, 0.3), (700, 256, 8, 8, 64, 300, 0.9),
    (650, 384, 16, 0, 128, 500, 0.7), (650, 128, 0, 16, 64, 900, 0.95), (650, 512, 8, 8, 256, 1024, 0.02),
    (333, 128, 8, 8, 128, 1100, 0.5), (1500, 256, 160, 0, 64, 70, 0.8), (1500, 256, 0, 104, 64, 70, 1.0),
    (1500, 512, 72, 136, 32, 90, 1.0), (200, 128, 8, 8, 64, 4097, 1.0), (200, 128, 8, 8, 64, 8300, 0.4),
    (300, 256, 8, 8, 64, 1500, 0.8), (260, 256, 8, 0, 256, 4500, 0.95), (20000, 256, 8, 8, 64, 500, 0.5),
]


@pytest.mark.parametrize("V,D,r_c,r_r,g,N,share", SHARES)
def test_shares_of_the_rows(V, D, r_c, r_r, g, N, share):
    log(f"xent V={V} D={D} r_c={r_c} r_r={r_r} g={g} N={N} share={share}")
    torch, ah = torch_mod(), ah_mod()
    h, head = _head(V + N, V, D, r_c, r_r, g)
    rng = np.random.default_rng(N)
    labels = rng.integers(0, V, N)
    H = _hidden(N, N, D, oracle.w_hat(h), labels)
    on = rng.random(N) < share
    w = torch.from_numpy((rng.uniform(0.5, 1.5, N) * on).astype(np.float32)).cuda()
    labels = np.where(on, labels, -100)
    H[torch.from_numpy(~on).cuda()] = float("nan")
    need = ah.archead_cross_entropy_workspace_bytes(V, D, r_c, r_r, g, N)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    got = ah.archead_cross_entropy(H, torch.from_numpy(labels).int().cuda(), head, weight=w, workspace=ws[:need])
    assert (ws[need:] == 255).all()
    H[torch.from_numpy(~on).cuda()] = 0.0
    _check(got, H, labels, w, h, 1.0, f"V={V} N={N}")


@pytest.mark.parametrize("V,r_c,r_r,N", [(150000, 16, 8, 1000), (120000, 0, 0, 1200), (1000000, 8, 0, 150)])
def test_rows_whose_maximum_rises_along_the_vocabulary(V, r_c, r_r, N):
    """A vocabulary in several pieces, and rows whose logits rise from one to
    the next, also by more than an exponent of fp32 holds."""
    torch, ah = torch_mod(), ah_mod()
    D, g = 128, 64
    h, head = _head(21, V, D, r_c, r_r, g)
    W = oracle.w_hat(h)
    rng = np.random.default_rng(1)
    labels = rng.integers(0, V, N)
    H = rng.normal(0, 1, (N, D))
    late = rng.integers(V // 2, V, N)
    rise = rng.choice([0.0, 5.0, 20.0, 60.0, 200.0], N)
    H += (rise / (W[late] ** 2).sum(1))[:, None] * W[late]
    labels = np.where(rng.random(N) < 0.3, late, labels)
    H = torch.from_numpy(H.astype(np.float32)).cuda().bfloat16()
    got = ah.archead_cross_entropy(H, torch.from_numpy(labels).int().cuda(), head)
    _check(got, H, labels, None, h, 1.0, "rising")


@pytest.mark.parametrize("N", ROWS)
def test_flat_and_huge_logits(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 1501, 256
    for spread, H in ((2.0, torch.zeros((N, D), device="cuda").bfloat16()),
                      (2000.0, torch.randn((N, D), device="cuda").bfloat16())):
        h, head = _head(31, V, D, 8, 8, 64, spread=spread)
        labels = np.random.default_rng(N).integers(0, V, N)
        labels[-1] = V - 1
        got = ah.archead_cross_entropy(H, torch.from_numpy(labels).int().cuda(), head)
        _check(got, H, labels, None, h, 1.0, f"spread {spread} N={N}")


def test_graphs_that_share_a_workspace():
    """Few and many rows captured on one workspace, replayed in turn between
    eager calls."""
    torch, ah = torch_mod(), ah_mod()
    V, D = 3000, 512
    h, head = _head(41, V, D, 8, 8, 64)
    W = oracle.w_hat(h)
    sets = []
    for N in (20, 150, 700):
        labels = np.random.default_rng(N).integers(0, V, N)
        sets.append((_hidden(N, N, D, W, labels), torch.from_numpy(labels).int().cuda(), torch.rand(N, device="cuda")))
    need = max(ah.archead_cross_entropy_workspace_bytes(V, D, 8, 8, 64, len(H)) for H, _, _ in sets)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    run = lambda i: ah.archead_cross_entropy(*sets[i][:2], head, weight=sets[i][2], workspace=ws)  # noqa: E731
    want = [run(i) for i in range(3)]
    torch.cuda.synchronize()
    graphs, held = [], []
    for i in range(3):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(run(i))
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        for t in held[i].values():
            t.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        for k in want[i]:
            assert torch.equal(held[i][k], want[i][k]), (i, k)
        run((i + 1) % 3)
