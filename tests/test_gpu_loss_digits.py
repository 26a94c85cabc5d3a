"""Digits of log p and of the gradient in rows whose label has almost all of the
probability: relative bounds, where test_gpu_loss.py's are absolute.

With q = sum of exp(s (y_j - y_label)) over the other columns, log p = -log1p(q),
the label's element is -w s A q / (1 + q) = w s A expm1(log p) and another's is
w s A exp(s (y_j - y_label)) / (1 + q).  The kernels hold q's sum in fp32 terms and
add the rest in fp64.  With u = 2^-24 and x a term's octaves below the number it
is taken by, at most the others' spread: the exponential has 2u, its argument's
two roundings 2u x ln 2, the trees of up to 32 terms 5u, rescaling a piece, a wave
or a lane 2u + 2u x ln 2 of which at most 74 follow each other (and of their x,
which are steps of a maximum that rises, the sum is at most the spread), and
storing u:
    rel = u (2 + 2 spread ln 2 + 5 + 74 * 2 + 2 spread ln 2 + 1) < u (3 spread + 160).
An element of the gradient has its own exponential besides, u (2 + 2 spread ln 2),
and three roundings: 2 rel covers it; bf16 adds 2^-8, fp32 2^-126 times the
coefficient, as smaller exponentials are 0.
"""
import numpy as np
import pytest

from tests.gpu_helpers import torch_mod
from tests.test_gpu_loss import _make_Y, _run_policy, _run_preference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# one workgroup; a few long rows; rows cut into pieces; one launch that holds all of a row, and part of it
WAYS = [(6, 900), (6, 30011), (40, 30011), (260, 60001), (257, 100003)]
LIFTS = [12.0, 20.0, 25.0, 30.0, 35.0, 40.0, 60.0, 80.0]


def _confident(rng, N, V, dtype):
    """Rows with a label far above the rest, at the ends, in the middle and behind column 8192, every
    other one with the next largest logit beside it (in the same 16 bytes)."""
    Y, _ = _make_Y(rng, N, V, dtype)
    labels = rng.integers(0, V, N)
    labels[:6] = 0, V - 1, V // 2, V - 2, min(8200, V - 9), V // 8 * 8 - 1
    for n in range(N):
        Y[n, int(labels[n])] = LIFTS[n % 8]
        if n % 2:
            Y[n, int(labels[n]) ^ 1 if labels[n] ^ 1 < V else int(labels[n]) - 1] = LIFTS[n % 8] - 16.0
    return Y, Y.double().cpu().numpy(), labels


def _want(Y64, labels, s):
    """(others' exp(s (y - y_label)) with 0 at the label, q, relative bound) of each row."""
    n = np.arange(len(Y64))
    e = np.exp(s * (Y64 - Y64[n, labels][:, None]))
    e[n, labels] = 0.0
    others = Y64.copy()
    others[n, labels] = np.nan
    spread = np.minimum((np.nanmax(others, 1) - np.nanmin(others, 1)) * s / np.log(2), 150.0)
    return e, e.sum(1), U * (3 * spread + 160)


def _relative(got, want, rel, least, what):
    worst = np.max(np.abs(got - want) / (rel * np.abs(want) + least))
    print(f"  {what}: worst error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1.0, what


@pytest.mark.parametrize("s", [0.75, 0.9])
@pytest.mark.parametrize("y,dy", [("bfloat16", "float32"), ("bfloat16", "bfloat16"), ("float32", "float32")])
@pytest.mark.parametrize("N,V", WAYS)
def test_policy_of_confident_rows_keeps_its_digits(N, V, y, dy, s):
    torch = torch_mod()
    print(f"N={N} V={V} {y} {dy} s={s}", flush=True)
    rng = np.random.default_rng(V + N)
    Y, Y64, labels = _confident(rng, N, V, getattr(torch, y))
    A = rng.uniform(0.2, 1, N).astype(np.float32)
    got = _run_policy(Y, labels, A, inv_temperature=s, dY_dtype=getattr(torch, dy))
    s = float(np.float32(s))
    e, q, rel = _want(Y64, labels, s)
    _relative(got["logp"], -np.log1p(q), rel, 0.0, "logp")
    coef = A.astype(np.float64) * s
    want = coef[:, None] * e / (1 + q)[:, None]
    want[np.arange(N), labels] = -coef * q / (1 + q)
    _relative(got["dY"], want, (2 * rel + (2.0 ** -8 if dy == "bfloat16" else 0.0))[:, None], 2.0 ** -126, "dY")


@pytest.mark.parametrize("N,V", WAYS[:3])
def test_preference_of_confident_rows_keeps_its_digits(N, V):
    torch = torch_mod()
    rng = np.random.default_rng(V + N)
    Y, Y64, labels = _confident(rng, N, V, torch.bfloat16)
    got = _run_preference(Y, labels, [0, N // 3, N], dY_dtype=torch.float32)
    e, q, rel = _want(Y64, labels, 1.0)
    logp = -np.log1p(q)
    _relative(got["logp"], logp, rel, 0.0, "logp")
    h = logp[:N // 3].sum() - logp[N // 3:].sum()
    slope = 0.1 * (-1 / (1 + np.exp(0.1 * h)))  # moves by less than 0.1 of h's error, relative to itself
    coef = np.where(np.arange(N) < N // 3, slope, -slope)
    want = -coef[:, None] * e / (1 + q)[:, None]
    want[np.arange(N), labels] = coef * q / (1 + q)
    moved = 0.1 * np.sum(rel * np.abs(logp))
    _relative(got["dY"], want, (2 * rel + moved)[:, None], 2.0 ** -126, "dY")


@pytest.mark.parametrize("s", [0.1, 1.0, 10.0])
@pytest.mark.parametrize("y", ["bfloat16", "float32"])
@pytest.mark.parametrize("N,V", WAYS[:4] + [(4, 1)])
def test_rows_where_only_the_label_is_left(N, V, y, s):
    """Everything but the label is -inf: p = 1 whatever the label's logit, in the plain row too."""
    torch = torch_mod()
    rng = np.random.default_rng(N + V)
    dtype = getattr(torch, y)
    Y = torch.full((N, V), -float("inf"), dtype=dtype, device="cuda")
    labels = rng.integers(0, V, N)
    least = torch.finfo(dtype).min
    values = [0.0, 1000.0, -1000.0, least, -least, 1e-30, 90.0, -90.0]
    for n in range(N):
        Y[n, int(labels[n])] = values[n % 8]
    got = _run_policy(Y, labels, np.ones(N), inv_temperature=s)
    assert not got["logp"].any() and got["loss"] == -N and not got["dY"].any()
    got = _run_preference(Y, labels, [0, N // 2, N], inv_temperature=s)
    assert not got["logp"].any() and not got["dY"].any() and abs(got["loss"] - np.log(2)) < 1e-7


@pytest.mark.parametrize("y", ["bfloat16", "float32"])
@pytest.mark.parametrize("N,V", WAYS[:4])
def test_labels_of_lowest_and_infinite_logits(N, V, y):
    """A label far below the rest keeps its log p, one at -inf has log p -inf, one at +inf NaN."""
    torch = torch_mod()
    rng = np.random.default_rng(N + V)
    Y, Y64 = _make_Y(rng, N, V, getattr(torch, y))
    labels = rng.integers(0, V, N)
    for n, v in ((0, -1e4), (1, -float("inf")), (2, float("inf")), (3, -700.0)):
        Y[n, int(labels[n])] = v
    Y64 = Y.double().cpu().numpy()
    got = _run_policy(Y, labels, np.ones(N), old_logp=np.zeros(N), clip_low=float("inf"), clip_high=float("inf"))
    assert got["logp"][1] == -np.inf and np.isnan(got["logp"][2]) and np.isnan(got["dY"][2]).all()
    for n in (0, 3):
        others = np.delete(Y64[n], labels[n])
        top = others.max()
        want = Y64[n, labels[n]] - top - np.log(np.exp(others - top).sum())
        assert abs(got["logp"][n] - want) <= 1e-4 + U * abs(want)
    assert not got["dY"][1].any() and got["row_loss"][1] == 0  # r = 0


@pytest.mark.parametrize("y,dy", [("bfloat16", "float32"), ("float32", "float32"), ("float32", "bfloat16")])
@pytest.mark.parametrize("N,V", WAYS)
def test_rows_whose_first_columns_are_far_below_the_rest(N, V, y, dy):
    """A vocabulary whose first columns are pushed down by a finite number, 40 to 95 units, and
    small weights: no element of the gradient that is a normal number loses its digits."""
    torch = torch_mod()
    rng = np.random.default_rng(V - N)
    Y, _ = _make_Y(rng, N, V, getattr(torch, y))
    first = min(V // 2, 9000)
    Y[:, :first] -= torch.as_tensor(40.0 + 5.0 * (np.arange(N) % 12), dtype=Y.dtype, device="cuda")[:, None]
    Y64 = Y.double().cpu().numpy()
    labels = rng.integers(0, V, N)
    w = np.full(N, 1e-5, np.float32)
    got = _run_policy(Y, labels, np.ones(N), weight=w, dY_dtype=getattr(torch, dy))
    e, q, rel = _want(Y64, labels, 1.0)
    _relative(got["logp"], -np.log1p(q), rel, 0.0, "logp")
    coef = w.astype(np.float64)
    p = np.exp(np.where(e > 0, np.log(np.maximum(e, 1e-300)) - np.log1p(q)[:, None], -np.inf))
    want = coef[:, None] * p
    want[np.arange(N), labels] = -coef * q / (1 + q)
    _relative(got["dY"], want, (2 * rel + (2.0 ** -8 if dy == "bfloat16" else 0.0))[:, None], 2.0 ** -126, "dY")


@pytest.mark.parametrize("N,V", WAYS[:4])
def test_own_policy_of_a_label_at_minus_infinity(N, V):
    """Without old_logp the ratio is 1 in every row that has a log p, -inf among them."""
    torch = torch_mod()
    rng = np.random.default_rng(N + V)
    Y, _ = _make_Y(rng, N, V, torch.float32)
    labels = rng.integers(0, V, N)
    Y[1, int(labels[1])] = -float("inf")
    got = _run_policy(Y, labels, np.full(N, 2.0))
    assert got["logp"][1] == -np.inf and (got["row_loss"] == -2.0).all() and got["loss"] == -2.0 * N
    p = np.exp(Y[1].double().cpu().numpy())
    want = 2.0 * p / p.sum()
    want[labels[1]] = -2.0
    _relative(got["dY"][1], want, 2 * U * (3 * 50 + 160), 2.0 ** -125, "dY")  # the spread is below 50 octaves


@pytest.mark.parametrize("what", ["finite mask", "mask", "one column"])
@pytest.mark.parametrize("y,dy", [("bfloat16", "float32"), ("float32", "bfloat16")])
@pytest.mark.parametrize("N,V", WAYS[3:])
def test_rows_whose_largest_logits_are_in_their_last_columns(N, V, y, dy, what):
    """Nine tenths of the columns 14 to 95 units below the rest, or at -inf; or one column, which is
    not the label's, so far above all others."""
    torch = torch_mod()
    rng = np.random.default_rng(V + N)
    Y, _ = _make_Y(rng, N, V, getattr(torch, y))
    first = V - V // 10
    by = torch.as_tensor(np.array([14.0, 20.0, 30.0, 50.0, 70.0, 80.0, 88.0, 95.0])[np.arange(N) % 8], dtype=Y.dtype,
                         device="cuda")
    if what == "one column":
        Y[:, V - 3] = by
    else:
        Y[:, :first] -= by[:, None]
        if what == "mask":
            Y[:, :first] = -float("inf")
    Y64 = Y.double().cpu().numpy()
    labels = rng.integers(first, V - 3, N)
    w = np.full(N, 1e-5, np.float32)
    got = _run_policy(Y, labels, np.ones(N), weight=w, dY_dtype=getattr(torch, dy))
    top = Y64.max(1, keepdims=True)
    e = np.exp(Y64 - top)
    p = e / e.sum(1, keepdims=True)
    n = np.arange(N)
    logp = (Y64 - top)[n, labels] - np.log(e.sum(1))
    finite = np.where(np.isfinite(Y64), Y64, np.nan)
    rel = U * (3 * np.minimum((np.nanmax(finite, 1) - np.nanmin(finite, 1)) / np.log(2), 150.0) + 160)
    _relative(got["logp"], logp, U, rel, "logp")
    want = w[:, None].astype(np.float64) * p
    want[n, labels] -= w
    _relative(got["dY"], want, (2 * rel + (2.0 ** -8 if dy == "bfloat16" else 0.0))[:, None], 2.0 ** -126, "dY")
