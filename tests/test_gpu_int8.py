"""GPU parity of archead_logits_int8 with the fp64 oracle.

The sums are exact whole numbers.  An element has three fp32 roundings (the sum
where it is above 2^24, the product of the scales, their product), 2^-24 each:
2^-22 allowed; and 2^-8 for bf16.  Scales of one and of powers of two make
every sum below 2^24 come out exactly.
"""
import numpy as np
import pytest

import oracle
import synth
from tests.gpu_helpers import ah_mod, log, torch_mod

pytestmark = pytest.mark.gpu

R8 = 2


def _head(seed, V, D, g=64):
    h = synth.draw_alt_head(np.random.default_rng(seed), R8, V, D, g)
    return h, ah_mod().PackedHead.from_components(h)


def _codes(seed, N, D, lo=-128):
    torch = torch_mod()
    X = torch.from_numpy(np.random.default_rng(seed).integers(lo, 128, (N, D), dtype=np.int8)).cuda()
    s = torch.from_numpy(np.random.default_rng(seed + 1).lognormal(-3, 1, N).astype(np.float32)).cuda()
    return X, s


def _check(Y, X, s, h, dtype):
    want = oracle.logits_int8(X.cpu().numpy(), s.double().cpu().numpy(), h)
    got = Y.double().cpu().numpy()
    tol = (2.0 ** -22 + (2.0 ** -8 if dtype == "bfloat16" else 0)) * np.abs(want) + 2.0 ** -134
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


CASES = [  # V, D, N: few tokens in LDS, the token tiles, ragged ends
    (1, 128, 1), (15, 128, 16), (1000, 256, 1), (777, 640, 3), (2003, 1024, 16), (4099, 512, 7),
    (300, 8192, 16), (200, 16384, 5), (64, 65536, 2),
    (1000, 128, 17), (333, 384, 32), (2003, 512, 33), (1031, 1152, 64), (999, 256, 65), (517, 640, 128),
    (4099, 256, 129), (530, 896, 257), (1000, 512, 700), (129, 128, 1100), (70, 16384, 40),
    (1000, 512, 8), (1000, 512, 9), (500, 16384, 8), (40, 32768, 8),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V,D,N", CASES)
def test_int8_matches_oracle(V, D, N, dtype):
    log(f"int8 V={V} D={D} N={N} {dtype}")
    torch, ah = torch_mod(), ah_mod()
    h, head = _head(V + N, V, D)
    X, s = _codes(N, N, D)
    Y = torch.full((N, V), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    ah.archead_logits_int8(X, s, head, Y)
    _check(Y, X, s, h, dtype)
    assert torch.equal(ah.archead_logits_int8(X, s, head, out_dtype=Y.dtype), Y)


@pytest.mark.parametrize("N", [1, 9, 32, 50, 100, 300])
def test_one_hot_rows_and_extreme_codes(N):
    """Unit codes give the head's codes bit for bit, in every column's place;
    rows of the lowest code against rows of the largest the largest sums."""
    torch, ah = torch_mod(), ah_mod()
    V, D = 300, 512
    h, _ = _head(N, V, D)
    h.scales[:] = 1.0
    h.codes[0], h.codes[1] = -127, 127
    head = ah.PackedHead.from_components(h)
    for k0 in range(0, D, N):
        k = torch.arange(k0, k0 + N, device="cuda") % D
        X = torch.zeros((N, D), dtype=torch.int8, device="cuda")
        X[torch.arange(N, device="cuda"), k] = -128
        Y = ah.archead_logits_int8(X, torch.full((N,), -1 / 128, device="cuda"), head)
        assert np.array_equal(Y.cpu().numpy(), h.codes[:, k.cpu().numpy()].T.astype(np.float32))
        if N < 100 and k0 > 2 * N:
            break
    X = torch.full((N, D), -128, dtype=torch.int8, device="cuda")
    Y = ah.archead_logits_int8(X, torch.ones(N, device="cuda"), head)
    assert (Y[:, 0] == 128 * 127 * D).all() and (Y[:, 1] == -128 * 127 * D).all()


@pytest.mark.parametrize("N", [4, 40, 200])
def test_sums_past_24_bits(N):
    """Sums that fp32 cannot hold while they grow: exact up to the last rounding."""
    torch, ah = torch_mod(), ah_mod()
    V, D = 40, 32768
    h, _ = _head(1, V, D)
    h.codes[:] = np.where(np.arange(D) % 2, 127, 126)
    h.scales[:] = 0.5
    head = ah.PackedHead.from_components(h)
    X = torch.full((N, D), 127, dtype=torch.int8, device="cuda")
    X[:, 5] = torch.arange(N, device="cuda") % 127
    s = torch.full((N,), 2.0, device="cuda")
    want = (X.cpu().numpy().astype(np.int64) @ h.codes.astype(np.int64).T).astype(np.float32)
    assert np.array_equal(ah.archead_logits_int8(X, s, head).cpu().numpy(), want)


@pytest.mark.parametrize("N", [3, 45, 150])
def test_strides_and_a_scale_that_is_not_finite(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 517, 384
    h, head = _head(2, V, D)
    big = torch.randint(-128, 128, (N, D + 48), device="cuda", dtype=torch.int8)
    X, s = big[:, 16:16 + D], _codes(3, N, D)[1]
    for dtype in (torch.float32, torch.bfloat16):
        want = ah.archead_logits_int8(X.contiguous(), s, head, out_dtype=dtype)
        Ybig = torch.full((N, V + 9), 5.0, dtype=dtype, device="cuda")
        ah.archead_logits_int8(X, s, head, Ybig[:, 3:3 + V])
        assert torch.equal(Ybig[:, 3:3 + V], want)
        assert (Ybig[:, :3] == 5).all() and (Ybig[:, 3 + V:] == 5).all()
        t = s.clone()
        t[1] = float("nan")
        got = ah.archead_logits_int8(X, t, head, out_dtype=dtype)
        assert torch.isnan(got[1]).all()
        keep = torch.arange(N, device="cuda") != 1
        assert torch.equal(got[keep], want[keep])
    assert ah.archead_logits_int8(X[:0], s[:0], head).shape == (0, V)


def test_more_rows_than_a_pass():
    torch, ah = torch_mod(), ah_mod()
    V, D, N = 33, 128, 16384 + 50
    h, head = _head(4, V, D)
    X, s = _codes(5, N, D)
    Y = torch.full((N, V), float("nan"), device="cuda")
    need = ah.archead_logits_int8_workspace_bytes(V, D, 64, N)
    ws = torch.full((need + 512,), 3, dtype=torch.uint8, device="cuda")
    ah.archead_logits_int8(X, s, head, Y, workspace=ws[:need])
    _check(Y, X, s, h, "float32")
    assert (ws[need:] == 3).all()


@pytest.mark.parametrize("N", [2, 64, 300])
def test_int8_in_graphs_and_on_streams(N):
    torch, ah = torch_mod(), ah_mod()
    V, D = 3001, 512
    _, head = _head(6, V, D)
    X, s = _codes(7, N, D)
    want = ah.archead_logits_int8(X, s, head)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ah.archead_logits_int8(X, s, head)
    for k in range(3):
        X.copy_(_codes(20 + k, N, D)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = ah.archead_logits_int8(X, s, head)
        assert torch.equal(held, want), k
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [ah.archead_logits_int8(X, s, head, stream=st) for _ in range(4) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("N", [1, 33, 260])
def test_from_the_residual_stream_to_logits(N, residual):
    """The norm's codes and scales through the INT8 head, as they are used:
    next to the logits of the norm's bf16 output through the same head."""
    torch, ah = torch_mod(), ah_mod()
    V, D = 1000, 512
    h, head = _head(8, V, D)
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, w = torch.randn((N, D), generator=gen, device="cuda").bfloat16(), torch.randn(D, generator=gen, device="cuda").bfloat16()
    r = torch.randn((N, D), generator=gen, device="cuda").bfloat16() if residual else None
    f = ah.archead_rmsnorm(x, weight=w, residual=r, outputs=("codes", "h"))
    Y = ah.archead_logits_int8(f["codes"], f["scale"], head)
    _check(Y, f["codes"], f["scale"], h, "float32")
    Y16 = ah.logits(f["h"], head)
    # codes are off by half a step of the row's scale, bf16 by 2^-8 of a value of at most 127 steps
    W = np.abs(oracle.w_hat_alt(h)).sum(1)
    bound = f["scale"].double().cpu().numpy()[:, None] * (0.5 + 127 * 2.0 ** -8) * W * 1.0001
    assert (np.abs((Y - Y16).double().cpu().numpy()) <= bound).all()


def test_offsets_past_32_bits():
    """Logits of more than 2^31 elements in two passes: the last rows as in a
    call of their own."""
    torch, ah = torch_mod(), ah_mod()
    V, D, N = 131071, 128, 16390
    h, head = _head(8, V, D)
    X, s = _codes(8, N, D)
    Y = ah.archead_logits_int8(X, s, head, out_dtype=torch.bfloat16)
    for rows in (slice(0, 3), slice(16380, 16384), slice(16384, N)):
        alone = ah.archead_logits_int8(X[rows].contiguous(), s[rows].contiguous(), head, out_dtype=torch.bfloat16)
        assert torch.equal(Y[rows], alone), rows
