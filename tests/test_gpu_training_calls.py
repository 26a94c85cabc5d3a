"""Calls that the header allows of the losses and the backward, on every way through the kernels:
a gradient over its logits, captured graphs in turn with eager calls, workspaces of exactly the size
asked for, rows 2^24 and 2^31 elements apart, no pairs.  All are compared bit by bit with the plain
call, whose results other tests compare with the oracle."""
import numpy as np
import pytest

import synth
from tests.gpu_helpers import ah_mod, torch_mod

pytestmark = pytest.mark.gpu

# one workgroup; a few long rows; rows cut into pieces; pieces of whole rounds of loads; one launch for many rows
LOSS = [(6, 900), (6, 30011), (40, 5003), (300, 16411), (260, 100003)]
# dims and rows: maxima within the first kernel, 16 x 16 and 32 x 32 operands of few rows, token tiles of 64, 128 and
# 256, several passes
BACKWARD = [((1000, 256, 8, 8, 64), 4), ((5000, 512, 16, 8, 128), 9), ((5000, 512, 16, 8, 32), 30),
            ((3001, 640, 40, 0, 128), 50), ((3001, 512, 16, 24, 64), 100), ((1031, 1024, 8, 64, 256), 700),
            ((130, 128, 8, 8, 32), 4096 + 33)]


def _inputs(N, V, dtype, seed):
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Y = (torch.randn((N, V), generator=gen, device="cuda") * 3).to(dtype)
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    vec = [torch.randn(N, generator=gen, device="cuda") for _ in range(3)]
    w = (torch.rand(N, generator=gen, device="cuda") < 0.7).float()
    offsets = torch.tensor([0, N // 6, N // 2, N - 1, N], dtype=torch.int32, device="cuda")
    return Y, labels, vec, w, offsets


def _both(Y, labels, vec, w, offsets, own=None, **kw):
    """Outputs of the policy and the preference loss; own: (workspace, dY) for each."""
    ah = ah_mod()
    more = own or [{}, {}]
    p = ah.archead_policy_loss(Y, labels, vec[0], old_logp=vec[1] * 0.1 - 9, ref_logp=vec[2] - 9, weight=w, kl_coef=0.1,
                               inv_temperature=0.9, **more[0], **kw)
    q = ah.archead_preference_loss(Y, labels, offsets, ref_logp=vec[2] - 9, weight=w, inv_temperature=0.9, **more[1], **kw)
    return [p[k] for k in sorted(p)] + [q[k] for k in sorted(q)]


def _same(a, b):
    torch = torch_mod()
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.isfinite(y.float()).all() and torch.equal(x, y), i


def _head(dims, seed=1):
    h = synth.draw_head(np.random.default_rng(seed), *dims)
    return ah_mod().PackedHead.from_components(h)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("N,V", LOSS)
def test_gradient_over_the_logits(N, V, dtype):
    torch = torch_mod()
    Y, *rest = _inputs(N, V, getattr(torch, dtype), V)
    want = _both(Y, *rest)
    over = [Y.clone(), Y.clone()]
    got = _both_over(over, rest)
    torch.cuda.synchronize()
    _same(got, want)


def _both_over(over, rest):
    ah = ah_mod()
    labels, vec, w, offsets = rest
    p = ah.archead_policy_loss(over[0], labels, vec[0], old_logp=vec[1] * 0.1 - 9, ref_logp=vec[2] - 9, weight=w,
                               kl_coef=0.1, inv_temperature=0.9, dY=over[0])
    q = ah.archead_preference_loss(over[1], labels, offsets, ref_logp=vec[2] - 9, weight=w, inv_temperature=0.9,
                                   dY=over[1])
    assert p["dY"] is over[0] and q["dY"] is over[1]
    return [p[k] for k in sorted(p)] + [q[k] for k in sorted(q)]


@pytest.mark.parametrize("N,V", LOSS)
def test_losses_in_graphs(N, V):
    """Two graphs of the same calls, replayed in turn with eager ones on inputs that change."""
    torch = torch_mod()
    Y, *rest = _inputs(N, V, torch.bfloat16, V)
    _both(Y, *rest)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _both(Y, *rest)
        graphs.append((g, outs))
    for i in range(4):
        fresh = _inputs(N, V, torch.bfloat16, 100 + i)
        Y.copy_(fresh[0])
        rest[2].copy_(fresh[3])  # the rows that count
        want = [t.clone() for t in _both(Y, *rest)]
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            _same(outs, want)


@pytest.mark.parametrize("dims,N", BACKWARD)
def test_backward_in_graphs(dims, N):
    torch = torch_mod()
    ah = ah_mod()
    head = _head(dims)
    gen = torch.Generator(device="cuda").manual_seed(N)
    dY = torch.randn((N, dims[0]), generator=gen, device="cuda").bfloat16()
    ah.archead_logits_backward(dY, head)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ah.archead_logits_backward(dY, head)
        graphs.append((g, out))
    for i in range(4):
        dY.copy_(torch.randn((N, dims[0]), generator=gen, device="cuda") * 10.0 ** (i - 2))
        want = ah.archead_logits_backward(dY, head).clone()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        _same([o for _, o in graphs], [want, want])


def _guarded(bytes_):
    """A workspace of exactly that size between two guards, filled with NaN patterns."""
    torch = torch_mod()
    buf = torch.full((bytes_ + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + bytes_]


@pytest.mark.parametrize("N,V", LOSS)
def test_losses_stay_in_their_workspace(N, V):
    torch = torch_mod()
    ah = ah_mod()
    Y, *rest = _inputs(N, V, torch.bfloat16, V)
    want = _both(Y, *rest)
    bufs, own = [], []
    for pairs in (0, 2):
        buf, ws = _guarded(ah.archead_loss_workspace_bytes(N, V, pairs))
        bufs.append(buf)
        own.append(dict(workspace=ws))
    for _ in range(2):  # what the first call left does not matter to the second
        _same(_both(Y, *rest, own=own), want)
        for buf in bufs:
            assert (buf[:256] == 0xFF).all() and (buf[-256:] == 0xFF).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("dims,N", BACKWARD)
def test_backward_stays_in_its_workspace(dims, N, dtype):
    torch = torch_mod()
    ah = ah_mod()
    head = _head(dims)
    gen = torch.Generator(device="cuda").manual_seed(N)
    dY = torch.randn((N, dims[0]), generator=gen, device="cuda").to(getattr(torch, dtype))
    want = ah.archead_logits_backward(dY, head)
    buf, ws = _guarded(ah.archead_logits_backward_workspace_bytes(*dims, N))
    for _ in range(2):
        out = torch.full((N + 2, dims[1]), 3.0, dtype=torch.bfloat16, device="cuda")
        _same([ah.archead_logits_backward(dY, head, out[1:N + 1], workspace=ws)], [want])
        assert (buf[:256] == 0xFF).all() and (buf[-256:] == 0xFF).all()
        assert (out[0] == 3).all() and (out[N + 1] == 3).all()


@pytest.mark.parametrize("N,V,stride", [(3, 900, 2 ** 31 + 3), (3, 30011, 2 ** 31 + 3), (40, 5003, 2 ** 27 + 1),
                                        (260, 100003, 2 ** 24 + 5)])
def test_rows_far_apart(N, V, stride):
    """Offsets past 2^32 elements, of the logits and of the gradient."""
    torch = torch_mod()
    Y, *rest = _inputs(N, V, torch.bfloat16, V)
    want = _both(Y, *rest)
    far = torch.empty((N - 1) * stride + V, dtype=torch.bfloat16, device="cuda").as_strided((N, V), (stride, 1))
    far.copy_(Y)
    ah = ah_mod()
    _same(_both(far, *rest), want)
    out = torch.empty((N - 1) * stride + V, dtype=torch.bfloat16, device="cuda").as_strided((N, V), (stride, 1))
    gradients = [t for t in want if t.dim() == 2]
    got = _both(Y, *rest, own=[dict(dY=out), {}])
    assert torch.equal(out, gradients[0])
    got = _both(Y, *rest, own=[{}, dict(dY=out)])
    assert torch.equal(out, gradients[1]) and torch.equal(got[-1], want[-1])
    del out, got
    for r in (0, 8):
        head = _head((V, 256, r, 8, 64))
        w = ah.archead_logits_backward(Y, head)
        dH = torch.empty((N - 1) * stride + 256, dtype=torch.bfloat16, device="cuda").as_strided((N, 256), (stride, 1))
        ah.archead_logits_backward(far, head, dH)
        _same([dH.contiguous()], [w])


@pytest.mark.parametrize("N,V", LOSS)
def test_no_pairs_and_nothing_that_counts(N, V):
    torch = torch_mod()
    ah = ah_mod()
    Y, labels, vec, w, _ = _inputs(N, V, torch.bfloat16, V)
    Y[:] = float("nan")
    none = torch.tensor([N // 2], dtype=torch.int32, device="cuda")
    q = ah.archead_preference_loss(Y, labels, none)
    assert q["loss"].item() == 0 and q["chosen_reward"].shape == (0,) and not q["dY"].any() and not q["logp"].any()
    p = ah.archead_policy_loss(Y, labels, vec[0], weight=0 * w)
    assert p["loss"].item() == 0 and not p["dY"].any() and not p["logp"].any() and not p["row_loss"].any()
