"""The learning operators together: the router's training step (learn.py)
against float64 autograd of the layer's definition, with the step's own picks
and expert rows, and AdamW on its gradient."""
import numpy as np
import pytest
import torch

import learn_ref as ref
from learn_ref import U, UB
from mixture_experts_layer_28_b200 import build as mb
from mixture_experts_layer_28_b200 import learn
from mixture_experts_layer_28_b200 import moe_zc as mz

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    mb.build()
    mz.lib()


def layer(N, Z, K, d, I, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()
    W_r, x, dout = r(N + Z, d), r(T, d, std=1.0), r(T, d, std=0.1)
    b = (torch.rand(N + Z, generator=g) * 0.02).cuda()
    return W_r, b, r(N, I, d), r(N, I, d), r(N, d, I), x, dout


@pytest.mark.parametrize("N,Z,K,T,seq,masked,offset", [
    (8, 4, 3, 70, None, False, False),
    (6, 0, 2, 33, [0, 10, 10, 29], True, True),
    (5, 6, 4, 300, [0, 100, 300], True, False),
    (1, 1, 1, 1, None, False, False),
])
def test_router_step(N, Z, K, T, seq, masked, offset):
    d, I, E = 256, 128, N + Z
    W_r, b, Wg, Wu, Wd, x, dout = layer(N, Z, K, d, I, T, seed=N + T)
    mask = (torch.arange(T) % 5 != 2).cuda() if masked else None
    if masked:
        dout[~mask] = 0.0        # (padding has no loss, so no gradient)
    s = None if seq is None else torch.tensor(seq, dtype=torch.int32, device="cuda")
    off = torch.linspace(-0.5, 0.5, E).cuda() if offset else None
    W0 = W_r.clone()
    st = learn.RouterStep(N, Z, K, W_r, b, Wg, Wu, Wd, lr=1e-2, balance=0.5)
    out = st.forward(x, mask, s, off)
    _, logits, idx, gate, slot, y = st._saved[:6]
    if off is None:
        assert torch.equal(out, mz.forward(x, W_r, b, Wg, Wu, Wd, N, Z, K))
    grad = st.backward(dout)

    # float64, with autograd through the softmax
    W = W0.double().cpu().requires_grad_()
    xc, ic, sc = x.double().cpu(), idx.long().cpu(), slot.long().cpu()
    z = xc @ W.t() + (0 if off is None else off.double().cpu())
    p = torch.softmax(z, 1)
    gates = p.gather(1, ic)
    row = torch.where((sc >= 0)[..., None], y.double().cpu()[sc.clamp(min=0)] if y.shape[0] else torch.zeros(T, K, d).double(), xc[:, None])
    main = ((gates[..., None] * row).sum(1) * dout.double().cpu()).sum()
    losses = []
    for rows in ref.sequences(T, s, mask):
        n = max(len(rows), 1)
        c = torch.bincount(ic[rows].reshape(-1), minlength=E).double()
        losses.append((c * E / (K * n) * p[rows].sum(0) / n).sum())
    total = main + 0.5 * sum(losses) / len(losses)
    total.backward()
    # Relative error of a probability, and of sums of them: the fp32 logits' own
    # error (2 u a step of d products, of at most |x||W|, once in l and once in the
    # softmax's sum), then exp, sums over E and over the tokens.
    reach = float((xc.abs() @ W0.double().cpu().abs().t()).max())
    slack = 4 * U * d * reach + (E + T + 64) * 4 * U
    want = torch.stack(losses).detach()
    assert ((grad.balance.loss.cpu().double() - want).abs() <= slack * want).all()

    # bf16 logits' gradients (2^-8 each), their products with x exact, the result
    # rounded once more; the probabilities' error (twice: in p and in the dot, and
    # the dots' d products) on top
    coef, dl = grad.balance.coef, torch.full((len(losses),), 0.5 / len(losses))
    dlog, size = ref.route_backward(logits, idx, (dout.double().cpu()[:, None] * row).sum(2), coef, dl, offset=off, mask=mask, seq=s)
    bound = ((UB * dlog.abs() + (2 * slack + 2 * d * U) * size).t() @ xc.abs()) + UB * W.grad.abs() + 1e-30
    assert ((grad.W_r.double().cpu() - W.grad).abs() <= bound).all()

    # and the step on that gradient
    master = st.opt.master[0].clone()
    zero = torch.zeros_like(master)
    st.step(grad.W_r)
    (w1, _, _), (werr, _, _) = ref.adamw(master, grad.W_r, zero, zero, 1, 1e-2, (0.9, 0.95), 1e-8, 0.1)
    assert ((st.opt.master[0].double().cpu() - w1).abs() <= werr).all()
    assert torch.equal(W_r, st.opt.master[0].to(torch.bfloat16))
    mz.synchronize()


def test_router_step_twice_is_reproducible():
    def run():
        W_r, b, Wg, Wu, Wd, x, dout = layer(8, 4, 3, 256, 128, 200, seed=3)
        st = learn.RouterStep(8, 4, 3, W_r, b, Wg, Wu, Wd, lr=1e-2, state_bits=8)
        for _ in range(3):
            st.forward(x)
            st.step(st.backward(dout).W_r)
        return W_r
    assert torch.equal(run(), run())


def test_rows_gradient_and_dx_by_combine():
    """combine_backward's dy, and dx's part through dispatch and combine as
    moe_zc_combine of dout with gates of 1: against float64."""
    N, Z, K, d, T = 6, 3, 3, 256, 40
    W_r, b, Wg, Wu, Wd, x, dout = layer(N, Z, K, d, 128, T, seed=5)
    logits, idx, gate, zsum, counts = mz.route_logits(x, W_r, b, N, Z, K)
    rows = int(counts[:N].sum())
    slot, send, expert = mz.dispatch(x, idx, counts, N, rows)
    y = mz.experts(send, expert, 0, Wg, Wu, Wd)
    _, dy = mz.combine_backward(dout, x, y, slot, gate)
    _, _, wdy = ref.combine_backward(dout, x, y, slot, gate)
    assert ((dy.double().cpu() - wdy).abs() <= (UB + 2 * U) * wdy.abs() + 1e-40).all()
    # as if the experts' own backward had turned dy into dXrows = dy
    dx = mz.combine(dout, dy, slot, torch.ones_like(gate), zsum).double().cpu()
    want = zsum.double().cpu()[:, None] * dout.double().cpu()
    mag = want.abs()
    for k in range(K):
        sc = slot[:, k].long().cpu()
        part = torch.where((sc >= 0)[:, None], dy.double().cpu()[sc.clamp(min=0)], 0.0)
        want, mag = want + part, mag + part.abs()
    assert ((dx - want).abs() <= UB * want.abs() + (K + 2) * U * mag).all()


def test_bias_follows_the_load():
    N, Z, K = 8, 4, 3
    W_r, b, Wg, Wu, Wd, x, dout = layer(N, Z, K, 256, 128, 128, seed=7)
    st = learn.RouterStep(N, Z, K, W_r, b, Wg, Wu, Wd, lr=1e-2)
    c = mz.BiasController(b.cpu().numpy(), N, Z, K, target_zero_frac=0.3, kp=0.01, ki=0.0)
    twin = mz.BiasController(b.cpu().numpy(), N, Z, K, target_zero_frac=0.3, kp=0.01, ki=0.0)
    st.forward(x)
    r = st.backward(dout).balance
    st.follow_load(c, r.counts, 128)
    assert np.array_equal(b.cpu().numpy(), twin.step(r.counts.sum(0).cpu().numpy(), 128))


def test_a_batch_without_tokens():
    W_r, b, Wg, Wu, Wd, x, dout = layer(4, 2, 2, 256, 128, 0)
    st = learn.RouterStep(4, 2, 2, W_r, b, Wg, Wu, Wd, lr=1e-2)
    assert st.forward(x).shape == (0, 256)
    g = st.backward(dout)
    assert (g.W_r == 0).all() and (g.balance.loss == 0).all()


def test_backward_needs_a_forward():
    W_r, b, Wg, Wu, Wd, x, dout = layer(2, 1, 1, 256, 128, 4)
    st = learn.RouterStep(2, 1, 1, W_r, b, Wg, Wu, Wd, lr=1e-2)
    with pytest.raises(RuntimeError):
        st.backward(dout)
    with pytest.raises(ValueError):
        learn.RouterStep(0, 3, 1, W_r, b, Wg, Wu, Wd, lr=1e-2)


@pytest.mark.parametrize("mask_type", [torch.bool, torch.uint8])
def test_padding_may_hold_anything(mask_type):
    """NaN in padding reaches its own output rows alone.  Without a bias both a
    row of NaN and one of zeros pick experts 0 .. K - 1, so the rest of the step
    is the same, bits included."""
    N, Z, K, T, d = 6, 3, 3, 90, 256
    W_r, b, Wg, Wu, Wd, x, dout = layer(N, Z, K, d, 128, T, seed=11)
    b.zero_()
    mask = (torch.arange(T) % 4 != 1).to(mask_type).cuda()
    got = []
    for fill in (0.0, float("nan")):
        x[mask == 0], dout[mask == 0] = fill, fill
        st = learn.RouterStep(N, Z, K, W_r, b, Wg, Wu, Wd, lr=1e-2)
        out = st.forward(x, mask)
        got.append((out[mask != 0], *st.backward(dout)))
    (o0, w0, r0), (o1, w1, r1) = got
    assert torch.isfinite(w1).all() and torch.equal(w0, w1) and torch.equal(o0, o1)
    for a, c in zip(r0, r1):
        assert torch.equal(a, c)


def test_all_picks_on_zero_experts():
    N, Z, K, T, d = 4, 5, 3, 40, 256
    W_r, b, Wg, Wu, Wd, x, dout = layer(N, Z, K, d, 128, T, seed=3)
    b[:N] = -10.0
    st = learn.RouterStep(N, Z, K, W_r, b, Wg, Wu, Wd, lr=1e-2)
    out = st.forward(x)
    idx, slot = st._saved[2], st._saved[4]
    assert (idx >= N).all() and (slot < 0).all()
    assert torch.equal(out, mz.forward(x, W_r, b, Wg, Wu, Wd, N, Z, K))
    g = st.backward(dout)
    assert g.balance.counts[0, :N].sum() == 0 and g.balance.counts.sum() == T * K
    # the gates' gradient is dout . x for every pick: with p the softmax,
    # dlogits_i = p_i (x . dout) ([i picked] - sum of the picks' p), and the loss's
    W = W_r.double().cpu()
    xc, dc = x.double().cpu(), dout.double().cpu()
    p = torch.softmax(xc @ W.t(), 1)
    on = torch.zeros(T, N + Z, dtype=torch.float64).scatter_(1, idx.long().cpu(), 1.0)
    a = on * (xc * dc).sum(1, keepdim=True) + 1e-2 * g.balance.coef.double().cpu()
    want = (p * (a - (p * a).sum(1, keepdim=True))).t() @ xc
    # roundings: the logits' fp32 sums (d terms) move p by d U |x| |W| relative,
    # dgate's the same way; dlogits and the product are rounded to bf16
    dl = p * ((a.abs() + (p * a.abs()).sum(1, keepdim=True)))
    rel = 4 * d * U * (1 + (xc.abs() @ W.abs().t()).max())
    err = ((UB + rel) * dl).t() @ xc.abs() + p.t() @ (xc.abs() * 4 * d * U * (xc * dc).abs().sum(1, keepdim=True)) * 2
    err = err + UB * want.abs() + T * U * (dl.t() @ xc.abs())
    assert ((g.W_r.double().cpu() - want).abs() <= err).all()


def test_inputs_of_an_autograd_graph():
    W_r, b, Wg, Wu, Wd, x, dout = layer(4, 2, 2, 256, 128, 30)
    want = learn.RouterStep(4, 2, 2, W_r.clone(), b, Wg, Wu, Wd, lr=1e-2)
    want.forward(x)
    w = want.backward(dout).W_r
    W_r.requires_grad_()
    st = learn.RouterStep(4, 2, 2, W_r, b, Wg, Wu, Wd, lr=1e-2)
    y = (x.requires_grad_() * 1.0)
    assert not st.forward(y).requires_grad
    g = st.backward(dout)
    assert torch.equal(g.W_r, w) and not g.W_r.requires_grad
    st.step(g.W_r)
    assert torch.equal(W_r.detach(), st.opt.master[0].to(torch.bfloat16))
