"""GPU parity of archead_rmsnorm and archead_rmsnorm_backward with the fp64 oracle.

Tolerances, from the kernels' arithmetic: the sum is bf16(fp32(x + residual))
bit for bit; codes are equal; scale and inv_rms are fp64 rounded once to fp32,
2^-24, with some fp64 roundings before (2^-23 allowed); h has two fp32 roundings
(the factor, the product) and the one to bf16, 2^-8.  Of the gradient every fp32
step rounds 2^-24 of a term: at most 16 of them for an element of dx (nine in
the sum of eight products, three in the sum's factor, four in the element),
each of the size of inv |g|, inv |s| sum_d|g s| inv^2 / D or |dsum|; and for
dweight one for each row that a thread adds (rows / parts + 1) and three more.
Where bf16 is subnormal its half step is 2^-134.
"""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -134


def _bf16(gen, *shape, sigma=1.0):
    torch = torch_mod()
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).bfloat16()


def _np(t):
    return t.double().cpu().numpy()


def _gen(seed):
    return torch_mod().Generator(device="cuda").manual_seed(seed)


ALL = ("sum", "h", "codes", "scale", "inv_rms")


def _check_forward(got, x, residual, weight, eps=1e-6):
    want = oracle.rmsnorm(_np(x), None if residual is None else _np(residual), None if weight is None else _np(weight), eps)
    assert np.array_equal(_np(got["sum"]), want["sum"])
    assert np.array_equal(got["codes"].cpu().numpy(), want["codes"])
    fine = ~np.isnan(want["scale"])  # rows with a product past fp32's range are not
    assert np.array_equal(fine, ~np.isnan(_np(got["scale"])))
    for k in ("scale", "inv_rms"):
        assert (np.abs(_np(got[k]) - want[k]) <= 2.0 ** -23 * np.abs(want[k]))[fine].all(), k
    err = np.abs(_np(got["h"])[fine] - want["h"][fine])
    assert (err <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want["h"][fine]) + TINY).all()


# one and several rows a workgroup, every width of a thread's share, ends inside an octet
SHAPES = [(1, 1), (3, 7), (1, 64), (5, 129), (9, 511), (2, 512), (7, 1001), (300, 1024), (11, 1537), (1, 2048), (4, 2049),
          (130, 4096), (3, 4100), (2, 8191), (5, 8192), (3, 12001), (2, 16384), (2, 16385), (1, 32768)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("N,D", SHAPES)
def test_norm_matches_oracle(N, D, residual):
    log(f"norm N={N} D={D} residual={residual}")
    gen = _gen(N * D)
    x, w = _bf16(gen, N, D, sigma=3.0), _bf16(gen, D)
    r = _bf16(gen, N, D) if residual else None
    got = ah_mod().archead_rmsnorm(x, weight=w, residual=r, outputs=ALL)
    _check_forward(got, x, r, w)
    again = ah_mod().archead_rmsnorm(x, weight=w, residual=r, outputs=ALL)
    for k in ALL:
        assert (got[k] == again[k]).all()


def test_norm_of_halves_zeros_and_extremes():
    """Exact ties between codes, rows of zeros, rows whose squares leave fp32,
    a weight of one, large and small eps."""
    torch = torch_mod()
    gen = _gen(5)
    x = _bf16(gen, 12, 96)
    x[:, 48:] = x[:, :48] * 0.5
    x[1] = 0
    x[2] = 0
    x[2, 17] = -2.0 ** -120
    x[3] *= 2.0 ** 90   # squares above fp32's range
    x[4] *= 2.0 ** -100  # and below it
    x[5, 3] = 3e38
    w = _bf16(gen, 96)
    w[48:] = w[:48]
    for weight in (w, None):
        for eps in (1e-6, 0.5, 1e-30):
            _check_forward(ah_mod().archead_rmsnorm(x, weight=weight, outputs=ALL + ("sum",), eps=eps), x, None, weight,
                           float(np.float32(eps)))
    assert torch.equal(x[1], torch.zeros_like(x[1]))


def test_norm_of_rows_that_are_not_finite():
    torch = torch_mod()
    gen = _gen(6)
    x, w = _bf16(gen, 6, 300), _bf16(gen, 300)
    good = ah_mod().archead_rmsnorm(x, weight=w, outputs=ALL)
    bad = x.clone()
    bad[1, 7], bad[3, 299], bad[4, 0] = float("nan"), float("inf"), -float("inf")
    got = ah_mod().archead_rmsnorm(bad, weight=w, outputs=ALL)
    for n in (0, 2, 5):
        for k in ALL:
            assert torch.equal(got[k][n], good[k][n])
    for n in (1, 3, 4):
        assert torch.isnan(got["scale"][n]) and not got["codes"][n].any()
        assert torch.isnan(got["h"][n]).any()


def test_norm_strides_places_and_outputs():
    """Rows of larger tensors at odd elements, written in place, each output
    alone, nothing written beside the rows."""
    torch, ah = torch_mod(), ah_mod()
    gen = _gen(7)
    N, D = 37, 333
    big, rbig, w = _bf16(gen, N, D + 13), _bf16(gen, N, D + 5), _bf16(gen, D)
    x, r = big[:, 3:3 + D], rbig[:, 1:1 + D]
    want = ah.archead_rmsnorm(x.contiguous(), weight=w, residual=r.contiguous(), outputs=ALL)
    obig = torch.full((N, D + 9), 7, dtype=torch.int8, device="cuda")
    hbig = torch.full((N, D + 9), 7, dtype=torch.bfloat16, device="cuda")
    x0, r0 = big.clone(), rbig.clone()
    got = ah.archead_rmsnorm(x, weight=w, residual=r, outputs=ALL, codes=obig[:, 5:5 + D], h=hbig[:, 2:2 + D], sum=r)
    for k in ALL:
        assert torch.equal(got[k], want[k]), k
    assert (obig[:, :5] == 7).all() and (obig[:, 5 + D:] == 7).all()
    assert (hbig[:, :2] == 7).all() and (hbig[:, 2 + D:] == 7).all()
    assert torch.equal(big, x0) and torch.equal(rbig[:, 0], r0[:, 0]) and torch.equal(rbig[:, 1 + D:], r0[:, 1 + D:])
    y = x.clone()  # h over x
    assert torch.equal(ah.archead_rmsnorm(y, weight=w, h=y)["h"], ah.archead_rmsnorm(x, weight=w)["h"])
    for k in ("h", "inv_rms", "codes"):
        alone = ah.archead_rmsnorm(x.contiguous(), weight=w, residual=r0[:, 1:1 + D], outputs=(k,))
        assert torch.equal(alone[k], want[k]) and torch.equal(alone["sum"], want["sum"])
    none = ah.archead_rmsnorm(x[:0], weight=w, outputs=ALL)
    assert none["h"].shape == (0, D)


def _check_backward(got, dh, s, inv, w, ds, parts):
    g64, s64, inv64 = _np(dh), _np(s), _np(inv)[:, None]
    want = oracle.rmsnorm_backward(g64, s64, inv64[:, 0], None if w is None else _np(w), None if ds is None else _np(ds))
    g = np.abs(g64 * (1.0 if w is None else _np(w)))
    size = inv64 * (g + np.abs(s64) * inv64 ** 2 * np.mean(g * np.abs(s64), 1, keepdims=True))
    size = size + (0 if ds is None else np.abs(_np(ds)))
    tol = 2.0 ** -20 * size
    tol = tol + 2.0 ** -8 * (np.abs(want["dx"]) + tol) + TINY
    err = np.abs(_np(got["dx"]) - want["dx"])
    assert (err <= tol).all(), (err / tol).max()
    terms = np.abs(g64 * s64 * inv64).sum(0)
    tol = (len(s64) / parts + 4) * 2.0 ** -24 * terms + 2.0 ** -24 * np.abs(want["dweight"]) + 2.0 ** -149
    err = np.abs(_np(got["dweight"]) - want["dweight"])
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("through", [True, False])
@pytest.mark.parametrize("N,D", SHAPES + [(2500, 520), (1300, 2304), (777, 9000)])
def test_norm_backward_matches_oracle(N, D, through):
    log(f"norm backward N={N} D={D} through={through}")
    gen = _gen(N + D)
    x, w, dh = _bf16(gen, N, D, sigma=2.0), _bf16(gen, D), _bf16(gen, N, D)
    ds = _bf16(gen, N, D) if through else None
    inv = ah_mod().archead_rmsnorm(x, weight=w, outputs=("inv_rms",))["inv_rms"]
    got = ah_mod().archead_rmsnorm_backward(dh, x, inv, weight=w, dsum=ds)
    parts = min(N, 128)  # at least: a thread adds N / parts rows and one at most
    _check_backward(got, dh, x, inv, w, ds, parts)
    again = ah_mod().archead_rmsnorm_backward(dh, x, inv, weight=w, dsum=ds)
    assert (got["dx"] == again["dx"]).all() and (got["dweight"] == again["dweight"]).all()


def test_norm_backward_in_place_strided_and_without_parts():
    torch, ah = torch_mod(), ah_mod()
    gen = _gen(8)
    N, D = 41, 777
    s, dh, ds = (_bf16(gen, N, D + k)[:, k:] for k in (1, 4, 7))
    w = _bf16(gen, D)
    inv = ah.archead_rmsnorm(s, outputs=("inv_rms",))["inv_rms"]
    want = ah.archead_rmsnorm_backward(dh.contiguous(), s.contiguous(), inv, weight=w, dsum=ds.contiguous())
    _check_backward(want, dh, s, inv, w, ds, N)
    got = ah.archead_rmsnorm_backward(dh, s, inv, weight=w, dsum=ds)
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dweight"], want["dweight"])
    only = ah.archead_rmsnorm_backward(dh, s, inv, weight=w, dsum=ds, with_dweight=False)
    assert torch.equal(only["dx"], want["dx"]) and "dweight" not in only
    for name in ("dh", "sum", "dsum"):  # dx in an input's place
        t = dict(dh=dh.clone(), sum=s.clone(), dsum=ds.clone())
        got = ah.archead_rmsnorm_backward(t["dh"], t["sum"], inv, weight=w, dsum=t["dsum"], dx=t[name])
        assert torch.equal(t[name], want["dx"]) and torch.equal(got["dweight"], want["dweight"])
    one = ah.archead_rmsnorm_backward(dh, s, inv)  # no weight, nothing by the residual stream
    _check_backward(one, dh, s, inv, None, None, N)
    none = ah.archead_rmsnorm_backward(dh[:0], s[:0], inv[:0], weight=w)
    assert not none["dweight"].any() and none["dx"].shape == (0, D)


def test_norm_backward_of_a_row_that_is_not_finite():
    torch, ah = torch_mod(), ah_mod()
    gen = _gen(9)
    s, dh = _bf16(gen, 4, 200), _bf16(gen, 4, 200)
    inv = ah.archead_rmsnorm(s, outputs=("inv_rms",))["inv_rms"]
    want = ah.archead_rmsnorm_backward(dh, s, inv)
    dh[2, 5] = float("nan")
    got = ah.archead_rmsnorm_backward(dh, s, inv)
    assert torch.isnan(got["dx"][2]).all() and torch.isnan(got["dweight"][5])
    keep = [0, 1, 3]
    assert torch.equal(got["dx"][keep], want["dx"][keep])
    assert torch.isfinite(got["dweight"][:5]).all()


def test_norm_gradient_against_differences():
    """The kernels' own gradient against differences of the kernels' own h, in
    steps that bf16 holds exactly (the rounding of h bounds the precision)."""
    torch, ah = torch_mod(), ah_mod()
    gen = _gen(10)
    D = 64
    x, dh = _bf16(gen, 1, D), _bf16(gen, 1, D)
    inv = ah.archead_rmsnorm(x, outputs=("inv_rms",))["inv_rms"]
    dx = _np(ah.archead_rmsnorm_backward(dh, x, inv)["dx"])[0]
    X = x.repeat(2 * D, 1)
    i = torch.arange(D, device="cuda")
    up, down = X[0].float() * 1.25, X[0].float() * 0.75
    X[i, i], X[D + i, i] = up.bfloat16(), down.bfloat16()
    f = _np(ah.archead_rmsnorm(X)["h"]) @ _np(dh)[0]
    step = _np(X[i, i] - X[D + i, i])
    # h is off by 2^-8 of itself; the curve's third derivative over the step, (x / 4)^2 / D, is below that
    noise = 2 * 2.0 ** -8 * (np.abs(_np(ah.archead_rmsnorm(X)["h"])) @ np.abs(_np(dh)[0])).max()
    assert (np.abs((f[:D] - f[D:]) - dx * step) <= noise + 0.02 * np.abs(dx * step)).all()


def test_norm_in_graphs_and_on_streams():
    """Captured forward and backward, replayed on new contents between eager
    calls; two streams at once."""
    torch, ah = torch_mod(), ah_mod()
    gen = _gen(11)
    N, D = 600, 1500
    x, r, w, dh = _bf16(gen, N, D), _bf16(gen, N, D), _bf16(gen, D), _bf16(gen, N, D)

    def step():
        f = ah.archead_rmsnorm(x, weight=w, residual=r, outputs=ALL)
        return {**f, **ah.archead_rmsnorm_backward(dh, f["sum"], f["inv_rms"], weight=w, dsum=dh)}

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(_bf16(gen, N, D, sigma=1.0 + k))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        for name in want:
            assert torch.equal(held[name], want[name]), (k, name)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[] for _ in streams]
    for _ in range(5):
        for s, o in zip(streams, outs):
            f = ah.archead_rmsnorm(x, weight=w, residual=r, outputs=ALL, stream=s)
            o.append({**f, **ah.archead_rmsnorm_backward(dh, f["sum"], f["inv_rms"], weight=w, dsum=dh, stream=s)})
    torch.cuda.synchronize()
    for o in outs:
        for got in o:
            for name in want:
                assert torch.equal(got[name], want[name]), name


# widths of every number of threads a row, and either side of where it changes
WIDTHS = [(1, 40), (128, 33), (129, 70), (256, 17), (257, 9), (513, 300), (1025, 40), (2049, 700), (4097, 300), (8193, 300),
          (16385, 300), (20480, 600), (32761, 260), (32768, 300)]


@pytest.mark.parametrize("D,N", WIDTHS)
def test_gradient_of_many_rows_in_place(D, N):
    """More rows than are worked on at a time, dx over dsum or over dh."""
    torch, ah = torch_mod(), ah_mod()
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, dh, dsum = (torch.randn((N, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = (1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
    inv = ah.archead_rmsnorm(x, weight=w, outputs=("inv_rms",))["inv_rms"]
    want = ah.archead_rmsnorm_backward(dh, x, inv, weight=w, dsum=dsum)
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    exact = oracle.rmsnorm_backward(n64(dh), n64(x), n64(inv), n64(w), n64(dsum))
    # dx: fp32 sums of eight and few roundings (2^-20 of the terms), then bf16; dweight: a part's
    # fp32 sum of its rows and two roundings of each term
    s, g, i64 = n64(x), np.abs(n64(w) * n64(dh)), n64(inv)[:, None]
    terms = np.abs(n64(dsum)) + i64 * (g + np.abs(s) * i64 ** 2 * (g * np.abs(s)).mean(1, keepdims=True))
    assert (np.abs(n64(want["dx"]) - exact["dx"]) <= 2.0 ** -8 * np.abs(exact["dx"]) + 2.0 ** -19 * terms).all()
    size = (np.abs(n64(dh) * s) * i64).sum(0)
    assert (np.abs(n64(want["dweight"]) - exact["dweight"]) <= (N + 4) * 2.0 ** -24 * size + 2.0 ** -140).all()
    for k in ("dsum", "dh"):
        args = {"dsum": dsum.clone(), "dh": dh.clone()}
        got = ah.archead_rmsnorm_backward(args["dh"], x, inv, weight=w, dsum=args["dsum"], dx=args[k])
        assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dweight"], want["dweight"]), k


def test_offsets_past_32_bits():
    """2^31 elements and more: the last rows as in a call of their own."""
    torch, ah = torch_mod(), ah_mod()
    N, D, last = (1 << 21) + 5, 1030, 7
    gen = torch.Generator(device="cuda").manual_seed(1)
    block = torch.randn((4096, D), generator=gen, device="cuda").bfloat16()
    x = block.repeat((N + 4095) // 4096, 1)[:N]
    x[-last:] = torch.randn((last, D), generator=gen, device="cuda").bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
    got = ah.archead_rmsnorm(x, weight=w, residual=x, outputs=("codes", "scale", "inv_rms"))
    want = ah.archead_rmsnorm(x[-last:].clone(), weight=w, residual=x[-last:].clone(), outputs=("codes", "scale", "inv_rms"))
    for k in want:
        assert torch.equal(got[k][-last:], want[k]), k
    del got["codes"]
    dx = ah.archead_rmsnorm_backward(x, got["sum"], got["inv_rms"], weight=w, dx=x, with_dweight=False)["dx"]
    assert torch.equal(dx[:4096], dx[4096:8192])  # the rows of the block, first and again
    alone = ah.archead_rmsnorm_backward(want["sum"] * 0.5, want["sum"], want["inv_rms"], weight=w, with_dweight=False)["dx"]
    assert torch.equal(dx[-last:], alone)  # x + x is twice x, exactly
