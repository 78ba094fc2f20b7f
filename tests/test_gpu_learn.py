"""The operators with which the router and the weights learn, on the GPU,
against their plain float64 forms (learn_ref.py, which derives the bounds)."""
import math

import pytest
import torch

import learn_ref as ref
from learn_ref import U, UB
from mixture_experts_layer_28_b200 import build as mb
from mixture_experts_layer_28_b200 import moe_zc as mz

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    mb.build()
    mz.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_case(T, E, K, seed=0, std=1.0):
    g = gen(seed)
    logits = (torch.randn(T, E, generator=g) * std).cuda()
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) if T else torch.zeros(0, K)
    return logits, idx.to(torch.int32).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_balance(r, logits, idx, **kw):
    loss, counts, prob, coef = ref.balance(logits, idx, **kw)
    offset, T = kw.get("offset"), logits.shape[0]
    assert torch.equal(r.counts.cpu().double(), counts)
    # P: positive terms, the softmax's relative error and one u for each addition
    # (at most T of them); coef: a handful of products of exact counts
    rel = (ref.softmax_steps(logits.cpu(), None if offset is None else offset.cpu()) + T + 8) * U
    assert ((r.prob.cpu().double() - prob).abs() <= rel * prob).all()
    assert ((r.coef.cpu().double() - coef).abs() <= 8 * U * coef.abs()).all()
    E = logits.shape[1]
    assert ((r.loss.cpu().double() - loss).abs() <= (rel + (E + 16) * U) * loss.abs()).all()


SEQS = [
    ("one", None), ("even", [0, 50, 100]), ("ragged", [0, 1, 1, 8, 77, 77, 90]),
    ("gap in front and rows behind", [5, 5, 40, 61]), ("none counts", [30, 30]),
]


@pytest.mark.parametrize("E,K", [(1, 1), (4, 2), (12, 3), (33, 32), (128, 12), (130, 5), (384, 8), (385, 1), (640, 6), (768, 12), (1021, 9), (1024, 32)])
@pytest.mark.parametrize("name,seq", SEQS)
def test_balance_loss(E, K, name, seq):
    T = 100
    logits, idx = rows_case(T, E, K, seed=E + K)
    masked = (torch.rand(T, generator=gen(E)) < 0.7).cuda()
    offset = torch.linspace(-3, 1, E).cuda()
    weight = torch.linspace(0.5, 2.0 * E, E).cuda()
    s = None if seq is None else ints(seq)
    check_balance(mz.balance_loss(logits, idx, seq_start=s), logits, idx, seq=s)
    r = mz.balance_loss(logits, idx, logit_offset=offset, mask=masked, seq_start=s, weight=weight)
    check_balance(r, logits, idx, offset=offset, mask=masked, seq=s, weight=weight)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 9, 2367, 2369, 5000])
def test_balance_loss_lengths(T):
    logits, idx = rows_case(T, 20, 3, seed=T)
    s = ints([0, T // 3, T // 3, T])
    check_balance(mz.balance_loss(logits, idx, seq_start=s), logits, idx, seq=s)


@pytest.mark.parametrize("E,K,T,seq", [
    (8, 2, 20000, None), (33, 3, 9000, [0, 4000, 9000]), (96, 6, 4096, None), (250, 4, 8192, [0, 3000, 3000, 8000]),
    (384, 5, 6000, None), (385, 5, 4736, None), (500, 3, 4800, [0, 100, 4000, 4790]), (640, 4, 4740, [3, 4, 4700]),
    (768, 12, 5003, [0, 1000, 1001, 2000, 3000, 4000, 4500, 5000, 5003]), (768, 12, 4735, None), (1021, 9, 4799, None), (1024, 32, 5000, [0, 0, 2500, 4990]),
])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss_many_rows_to_add(E, K, T, seq, masked):
    logits, idx = rows_case(T, E, K, seed=T)
    kw = dict(mask=(torch.rand(T, generator=gen(E)) < 0.7).cuda()) if masked else {}
    if seq is not None:
        kw["seq"] = ints(seq)
    r = mz.balance_loss(logits, idx, mask=kw.get("mask"), seq_start=kw.get("seq"))
    check_balance(r, logits, idx, **kw)


def test_balance_loss_a_sequence_per_token():
    T = 1500
    logits, idx = rows_case(T, 40, 4)
    s = ints(list(range(T + 1)))
    check_balance(mz.balance_loss(logits, idx, seq_start=s), logits, idx, seq=s)


def test_balance_loss_many_empty_sequences():
    T, S = 300, 5000
    logits, idx = rows_case(T, 8, 2)
    s = ints([0] + sorted(int(v) for v in torch.randint(0, T + 1, (S - 1,), generator=gen(1))) + [T])
    check_balance(mz.balance_loss(logits, idx, seq_start=s), logits, idx, seq=s)


def test_no_sequences():
    logits, idx = rows_case(20, 8, 2)
    r = mz.balance_loss(logits, idx, seq_start=ints([0]))
    assert r.loss.shape == (0,) and r.coef.shape == (0, 8)
    d = mz.route_backward(logits, idx, coef=r.coef, dloss=r.loss, seq_start=ints([0]))
    assert (d == 0).all()


def test_all_tokens_masked():
    logits, idx = rows_case(40, 96, 6)
    mask = torch.zeros(40, dtype=torch.uint8, device="cuda")
    r = mz.balance_loss(logits, idx, mask=mask)
    for v in r:
        assert (v == 0).all()
    d = mz.route_backward(logits, idx, dgate=torch.ones(40, 6, device="cuda"), coef=r.coef, dloss=torch.ones(1, device="cuda"), mask=mask)
    assert (d == 0).all()


def test_padding_may_hold_anything():
    """NaN, infinities and wild picks in masked rows reach nothing."""
    T, E, K = 64, 100, 5
    logits, idx = rows_case(T, E, K)
    mask = (torch.arange(T) % 3 != 1).cuda()
    dgate = torch.randn(T, K, generator=gen(3)).cuda()
    clean = mz.balance_loss(logits, idx, mask=mask)
    one = torch.ones(1, device="cuda")
    dclean = mz.route_backward(logits, idx, dgate=dgate, coef=clean.coef, dloss=one, mask=mask)
    logits[~mask] = float("nan")
    logits[1] = float("inf")
    dgate[~mask] = float("inf")
    idx[~mask] = 2 ** 30
    dirty = mz.balance_loss(logits, idx, mask=mask)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    assert torch.equal(dclean, mz.route_backward(logits, idx, dgate=dgate, coef=dirty.coef, dloss=one, mask=mask))


def test_experts_masked_out_of_the_softmax():
    """-inf and the type's lowest value as masks: p = 0 there, a row of nothing
    but the lowest value is even, and no NaN appears."""
    T, E, K = 30, 72, 4
    logits, idx = rows_case(T, E, K)
    logits[:, 10:20] = -math.inf
    logits[:, 30:40] = torch.finfo(torch.float32).min
    logits[5] = torch.finfo(torch.float32).min
    r = mz.balance_loss(logits, idx)
    check_balance(r, logits, idx)
    dgate = torch.randn(T, K, generator=gen(4)).cuda()
    d = mz.route_backward(logits, idx, dgate=dgate).cpu().double()
    want, size = ref.route_backward(logits, idx, dgate)
    assert torch.isfinite(d).all()
    assert ((d - want).abs() <= 2 * (ref.softmax_steps(logits.cpu()) + 40) * U * size).all()


def test_picks_outside_the_pool_and_repeated():
    T, E, K = 50, 30, 8
    logits, idx = rows_case(T, E, K)
    idx[::3, 2] = -1
    idx[1::3, 5] = E
    idx[2::3, 1] = idx[2::3, 7]
    idx[4] = 11
    check_balance(mz.balance_loss(logits, idx), logits, idx)
    dgate = torch.randn(T, K, generator=gen(5)).cuda()
    want, size = ref.route_backward(logits, idx, dgate)
    d = mz.route_backward(logits, idx, dgate=dgate).cpu().double()
    assert ((d - want).abs() <= 2 * (ref.softmax_steps(logits.cpu()) + 40) * U * size).all()


@pytest.mark.parametrize("E,K", [(1, 1), (4, 2), (33, 32), (128, 12), (250, 5), (384, 8), (511, 1), (640, 6), (768, 12), (1021, 9), (1024, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("what", ["gates", "loss", "both"])
def test_route_backward(E, K, dtype, what):
    T = 45
    logits, idx = rows_case(T, E, K, seed=E)
    g = gen(E + 1)
    mask = (torch.rand(T, generator=g) < 0.8).cuda()
    offset = torch.linspace(-2, 2, E).cuda()
    seq = ints([0, 10, 10, 31, 40])
    kw = {}
    if what != "loss":
        kw.update(idx=idx, dgate=torch.randn(T, K, generator=g).cuda())
    if what != "gates":
        kw.update(coef=torch.rand(4, E, generator=g).cuda(), dloss=torch.randn(4, generator=g).cuda())
    got = mz.route_backward(logits, logit_offset=offset, mask=mask, seq_start=seq, dtype=dtype, **kw)
    want, size = ref.route_backward(logits, offset=offset, mask=mask, seq=seq, **kw)
    assert got.dtype == dtype
    # p's error twice (p itself and in the dot), E additions in the dot, a few more
    bound = (2 * ref.softmax_steps(logits.cpu(), offset.cpu()) + E + 40) * U * size
    if dtype == torch.bfloat16:
        bound = bound + UB * want.abs() + 1e-40
    assert ((got.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("E", [4, 6, 12, 130, 768, 1021])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gradient_near_an_even_load(E, sign):
    """The softmax's gradient does not see what all coefficients have in common,
    so its error goes by what is left: nothing where all are equal."""
    T = 40
    logits, _ = rows_case(T, E, 1, seed=E)
    seq, dloss = ints([0, 13, 40]), torch.tensor([0.7, -1.3]).cuda()
    same = torch.full((2, E), 0.3 * sign).cuda()
    assert (mz.route_backward(logits, coef=same, dloss=dloss, seq_start=seq) == 0).all()
    coef = same + 1e-4 * torch.rand(2, E, generator=gen(E)).cuda()
    got = mz.route_backward(logits, coef=coef, dloss=dloss, seq_start=seq)
    least = coef.abs().min(1, keepdim=True).values * sign
    want, size = ref.route_backward(logits, coef=coef.double() - least.double(), dloss=dloss, seq=seq)
    bound = (2 * ref.softmax_steps(logits.cpu()) + E + 40) * U * size
    assert ((got.cpu().double() - want).abs() <= bound).all()


def test_an_even_load_has_no_gradient():
    # K == E: every expert is picked by every token
    for E in (1, 4, 6, 32):
        logits, idx = rows_case(50, E, E, seed=E)
        seq = ints([0, 20, 50])
        r = mz.balance_loss(logits, idx, seq_start=seq)
        assert (mz.route_backward(logits, idx, coef=r.coef, dloss=torch.ones(2, device="cuda"), seq_start=seq) == 0).all()


@pytest.mark.parametrize("T", [0, 1, 3, 8, 20000])
def test_route_backward_lengths(T):
    logits, idx = rows_case(min(T, 50), 16, 2, seed=T)
    dgate = torch.randn(min(T, 50), 2, generator=gen(6)).cuda()
    if T > 50:
        n = T // 50
        logits, idx, dgate = logits.repeat(n, 1), idx.repeat(n, 1), dgate.repeat(n, 1)
    d = mz.route_backward(logits, idx, dgate=dgate)
    want, size = ref.route_backward(logits[:50], idx[:50], dgate[:50])
    want, size = want.repeat(max(1, T // 50), 1), size.repeat(max(1, T // 50), 1)
    assert d.shape == (T, 16)
    assert ((d.cpu().double() - want).abs() <= (2 * ref.softmax_steps(logits.cpu()) + 56 if T else 1) * U * size).all()


def test_gradients_against_differences():
    """d loss / d logits of the balance loss plus a linear function of the gates,
    by central differences of the float64 definition: h = 1e-4 leaves an error
    of h^2/6 times a third derivative below 30 (6 times terms of at most 5) and
    1e-15 / h of rounding, under 1e-7 together; the kernel's own bound beside it."""
    T, E, K = 12, 20, 3
    logits, idx = rows_case(T, E, K, seed=9)
    seq = ints([0, 5, 11])
    dgate = torch.randn(T, K, generator=gen(10)).cuda()
    dloss = torch.tensor([0.7, -1.3], device="cuda")
    r = mz.balance_loss(logits, idx, seq_start=seq)
    got = mz.route_backward(logits, idx, dgate=dgate, coef=r.coef, dloss=dloss, seq_start=seq).cpu().double()
    _, size = ref.route_backward(logits, idx, dgate, r.coef, dloss, seq=seq)
    bound = (2 * ref.softmax_steps(logits.cpu()) + E + 48) * U * size
    ic, dg, dl = idx.cpu().long(), dgate.cpu().double(), dloss.cpu().double()

    def value(z):
        p = torch.softmax(z, 1)
        out = (p.gather(1, ic) * dg).sum()
        for s, (a, b) in enumerate([(0, 5), (5, 11)]):
            c = torch.bincount(ic[a:b].reshape(-1), minlength=E).double()
            out = out + dl[s] * (c * E / (K * (b - a)) * p[a:b].mean(0)).sum()
        return float(out)

    base, h = logits.cpu().double(), 1e-4
    for t, i in [(0, 0), (3, 7), (4, 19), (5, 2), (10, 11), (11, 6)]:
        up, dn = base.clone(), base.clone()
        up[t, i] += h
        dn[t, i] -= h
        assert abs((value(up) - value(dn)) / (2 * h) - got[t, i]) <= 1e-7 + bound[t, i]


def test_a_batch_wide_loss_of_two_halves():
    """Counts summed over two calls give the coefficients of the whole batch."""
    T, E, K = 200, 24, 3
    logits, idx = rows_case(T, E, K, seed=12)
    whole = mz.balance_loss(logits, idx)
    a, b = mz.balance_loss(logits[:90].contiguous(), idx[:90].contiguous()), mz.balance_loss(logits[90:].contiguous(), idx[90:].contiguous())
    counts = a.counts + b.counts
    assert torch.equal(counts, whole.counts)
    coef = counts * (E / (K * T)) / T
    assert torch.allclose(coef, whole.coef, rtol=8 * U, atol=0)


# ------------------------------------------------------------------ combine


def combine_case(T, d, K, zero, seed=0, spare=0):
    g = gen(seed)
    n = T * K
    P = max(0, min(n, round((1 - zero) * n)))
    slot = torch.full((n,), -1, dtype=torch.int32)
    slot[torch.randperm(n, generator=g)[:P]] = torch.randperm(P + spare, generator=g)[:P].to(torch.int32)
    bf = torch.bfloat16
    return (torch.randn(T, d, generator=g).to(bf).cuda(), torch.randn(T, d, generator=g).to(bf).cuda(), torch.randn(P + spare, d, generator=g).to(bf).cuda(),
            slot.view(T, K).cuda(), torch.rand(T, K, generator=g).cuda())


@pytest.mark.parametrize("T,d,K,zero", [
    (1, 8, 1, 0.0), (1, 64, 1, 1.0), (3, 72, 2, 0.5), (5, 2056, 4, 0.3), (7, 256, 5, 0.2), (4, 6144, 12, 0.4), (6, 1024, 13, 0.3), (3, 128, 17, 0.3), (2, 4104, 32, 0.25),
    (5, 512, 8, 0.0), (5, 512, 8, 1.0), (33, 320, 3, 0.4)])
@pytest.mark.parametrize("rows", [True, False])
def test_combine_backward(T, d, K, zero, rows):
    dout, x, y, slot, gate = combine_case(T, d, K, zero, seed=T + d, spare=3)
    dgate, dy = mz.combine_backward(dout, x, y, slot, gate, rows=rows)
    want, mag, wdy = ref.combine_backward(dout, x, y, slot, gate)
    # products of bf16 are exact in fp32; d of them are added
    assert ((dgate.cpu().double() - want).abs() <= (d + 4) * U * mag).all()
    if not rows:
        assert dy is None
        return
    named = ~torch.isnan(wdy[:, 0])
    err = (dy.cpu().double()[named] - wdy[named]).abs()
    assert (err <= (UB + 2 * U) * wdy[named].abs() + 1e-40).all()


def test_combine_backward_leaves_other_rows():
    """Rows no slot names keep what they held, in a call on the C ABI's terms;
    a slot past the rows is not followed."""
    dout, x, y, slot, gate = combine_case(9, 264, 4, 0.3, seed=2, spare=5)
    R = y.shape[0]
    slot[0, 0] = R
    slot[1, 1] = 2 ** 31 - 1
    dy = torch.full_like(y, 7.0)
    dgate = torch.empty(9, 4, device="cuda")
    st = mz.lib().moe_zc_combine_backward(dout.data_ptr(), x.data_ptr(), y.data_ptr(), slot.data_ptr(), gate.data_ptr(), 9, 264, 4, R, dgate.data_ptr(), dy.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
    assert st == mz.OK
    assert dgate[0, 0] == 0 and dgate[1, 1] == 0
    inside = torch.where(slot >= R, -1, slot)
    want, mag, wdy = ref.combine_backward(dout, x, y, inside, gate)
    want[0, 0] = want[1, 1] = 0
    assert ((dgate.cpu().double() - want).abs() <= 268 * U * mag).all()
    free = torch.isnan(wdy[:, 0])
    assert (dy.cpu()[free] == 7.0).all()
    assert ((dy.cpu().double() - wdy)[~free].abs() <= (UB + 2 * U) * wdy[~free].abs() + 1e-40).all()


def test_combine_backward_no_tokens_no_rows():
    bf = torch.bfloat16
    e = torch.empty(0, 64, dtype=bf, device="cuda")
    dgate, dy = mz.combine_backward(e, e, e, torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 3, device="cuda"))
    assert dgate.shape == (0, 3) and dy.shape == (0, 64)
    dout, x, _, slot, gate = combine_case(4, 64, 3, 1.0)
    dgate, dy = mz.combine_backward(dout, x, e, slot, gate)
    want, mag, _ = ref.combine_backward(dout, x, e, slot, gate)
    assert ((dgate.cpu().double() - want).abs() <= 68 * U * mag).all()


def test_combine_backward_against_combine():
    """<dout, combine(gates + h e) - combine(gates - h e)> / 2h on the forward's
    kernel: linear in the gates, so only its bf16 rounding (2^-8 of |out| a
    side) separates the two."""
    dout, x, y, slot, gate = combine_case(6, 512, 4, 0.4, seed=8)
    dgate, _ = mz.combine_backward(dout, x, y, slot, gate)
    d64 = dout.double()

    def out(gates):
        zsum = torch.where(slot < 0, gates, 0.0).sum(1)
        return mz.combine(x, y, slot, gates.contiguous(), zsum).double()

    h = 4.0
    for t, k in [(0, 0), (2, 3), (5, 1), (3, 2)]:
        e = torch.zeros_like(gate)
        e[t, k] = h
        up, dn = out(gate + e), out(gate - e)
        diff = float((d64 * (up - dn)).sum() / (2 * h))
        slack = float((d64.abs() * (up.abs() + dn.abs()))[t].sum() * (UB + 8 * U) / (2 * h))
        assert abs(diff - float(dgate[t, k])) <= slack


# ------------------------------------------------------------------ AdamW

HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def adam_case(sizes, p, g, seed=0):
    r = gen(seed)
    params = [(torch.randn(n, generator=r) * 0.05).to(p).cuda() for n in sizes]
    grads = [(torch.randn(n, generator=r) * 1e-3).to(g).cuda() for n in sizes]
    return params, grads


@pytest.mark.parametrize("sizes", [[1], [7], [8], [255], [256], [257], [2048], [2049], [5000, 0, 3, 256, 70001], [33] * 20, [1 + 37 * i for i in range(460)]])
@pytest.mark.parametrize("p,g", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_adamw_fp32_states(sizes, p, g):
    params, grads = adam_case(sizes, p, g)
    r = gen(1)
    m = [(torch.randn(n, generator=r) * 1e-3).cuda() for n in sizes]
    v = [(torch.rand(n, generator=r) * 1e-6).cuda() for n in sizes]
    before = [(a.clone(), c.clone(), e.clone()) for a, c, e in zip(params, m, v)]
    opt = mz.AdamW(params, **HYPER, exp_avg=m, exp_avg_sq=v, step=4)
    opt.step(grads, grad_scale=torch.tensor([0.5], device="cuda"))
    assert opt.step_count.tolist() == [5, 0]
    flat = [torch.cat([t.reshape(-1) for t in ts]) for ts in (zip(*before))]
    want, err = ref.adamw(flat[0], torch.cat(grads), flat[1], flat[2], 5, HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"], 0.5)
    got = [torch.cat(ts).cpu().double() for ts in (params, m, v)]
    perr = err[0] + (UB * want[0].abs() if p == torch.bfloat16 else 0)
    assert ((got[0] - want[0]).abs() <= perr).all()
    assert ((got[1] - want[1]).abs() <= err[1]).all()
    assert ((got[2] - want[2]).abs() <= err[2]).all()


@pytest.mark.parametrize("g", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_master_weights(g, bits):
    sizes = [300, 2000]
    params, grads = adam_case(sizes, torch.bfloat16, g)
    opt = mz.AdamW(params, **HYPER, state_bits=bits, master=True)
    start = [t.clone() for t in opt.master]
    for _ in range(3):
        opt.step(grads)
    for p, w, s in zip(params, opt.master, start):
        assert torch.equal(p, w.to(torch.bfloat16))
        assert not torch.equal(w, s)
    # the same weights in fp32 go the same way
    other = mz.AdamW([s.clone() for s in start], **HYPER, state_bits=bits)
    for _ in range(3):
        other.step(grads)
    for a, b in zip(other.params, opt.master):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 31, 256, 257, 4096, 5003])
@pytest.mark.parametrize("p,g", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)])
def test_adamw_8_bit_states(n, p, g):
    params, grads = adam_case([n], p, g, seed=n)
    opt = mz.AdamW(params, **HYPER, state_bits=8)
    for step in range(1, 4):
        m = ref.dequantise(*opt.exp_avg[0])
        root = ref.dequantise(*opt.exp_avg_sq[0])
        w0 = params[0].clone()
        opt.step(grads)
        (w, m1, v1), (perr, merr, verr) = ref.adamw(w0, grads[0], m, root * root, step, HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        if p == torch.bfloat16:
            perr = perr + UB * w.abs()
        # (the kernel's own decoding of m and of v = root^2 rounds twice more: 2 u)
        assert ((params[0].cpu().double() - w).abs() <= perr + 40 * U * (w0.cpu().double() - w).abs()).all()
        for _, bad, got, want in ref.check_codes(*opt.exp_avg[0], m1, merr + 2 * U * m.abs()):
            assert not bad.any()
        r1 = v1.sqrt()
        for _, bad, got, want in ref.check_codes(*opt.exp_avg_sq[0], r1, 8 * U * r1):
            # a positive root may be held as the smallest code although zero is nearer
            floor = (want > 0) & (got == 2.0 ** -9)
            assert not (bad & ~floor).any()
            assert (got[want > 0] > 0).all()


def test_adamw_8_bit_wide_blocks():
    """One large gradient in a block: the small ones' roots do not become zero, so
    their steps stay bounded, and a block of zeros stays at zero."""
    n = 512
    g = torch.full((n,), 1e-7, device="cuda")
    g[3] = 10.0
    g[256:] = 0.0
    w = torch.zeros(n, device="cuda")
    opt = mz.AdamW([w], lr=1e-2, betas=(0.9, 0.99), eps=1e-12, weight_decay=0.0, state_bits=8)
    for _ in range(5):
        opt.step([g])
        assert torch.isfinite(w).all()
        # |m / (1 - b1^n)| <= max|g| and the root is never below |g| / sqrt(...) rounded
        # down by more than half a step: a step moves a weight by at most 1.2 lr
    assert float(w.abs().max()) <= 5 * 1.2 * 1e-2
    codes, scales = opt.exp_avg_sq[0]
    assert (codes[:256] != 0).all()
    assert (codes[256:] == 0).all() and (w[256:] == 0).all()


def test_adamw_non_finite_gradients_stay_in_their_elements():
    """A NaN poisons its own element; its 8-bit block takes scale 1, the next
    block is untouched."""
    n = 512
    g = torch.full((n,), 1e-3, device="cuda")
    g[5] = float("nan")
    for bits in (32, 8):
        w = torch.zeros(n, device="cuda")
        opt = mz.AdamW([w], **HYPER, state_bits=bits)
        opt.step([g])
        assert torch.isnan(w[5]) and int(torch.isnan(w).sum()) == 1
        if bits == 8:
            assert opt.exp_avg[0].scales[0] == 1.0 and opt.exp_avg[0].scales[1] < 1.0
            assert int(opt.exp_avg[0].codes[5]) & 0x7F == 0x7F


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_tiny_and_huge_values(bits):
    """Gradients from 1e-15 to 1e15: every weight moves by about lr (the
    first step's m / sqrt(v) is 1 up to eps), none becomes NaN."""
    g = torch.cat([torch.full((256,), 10.0 ** e) for e in range(-15, 16, 3)]).cuda()
    w = torch.zeros_like(g)
    mz.AdamW([w], lr=1e-2, betas=(0.9, 0.99), eps=1e-30, weight_decay=0.0, state_bits=bits).step([g])
    assert torch.allclose(w, torch.full_like(w, -1e-2), rtol=1e-5)


def test_adamw_roots_at_the_edges():
    """sqrt(v) as the 8-bit state sees it (beta2 = 0, one element per block, so a
    block's scale is its root / 448): within 2 u of the exact root from the
    smallest normal float to the largest, and exactly the zero block's at v = 0."""
    e = torch.linspace(-62.5, 63.9, 1500, dtype=torch.float64)
    g = torch.zeros(1501, 256)
    g[1:, 0] = (2.0 ** e).float()
    w = torch.zeros(1501 * 256, device="cuda")
    opt = mz.AdamW([w], lr=1e-3, betas=(0.0, 0.0), eps=1e-30, weight_decay=0.0, state_bits=8)
    opt.step([g.view(-1).cuda()])
    scale = opt.exp_avg_sq[0].scales.cpu().double()
    v = (g[:, 0] * g[:, 0]).double()     # (rounded as the kernel rounds it)
    assert scale[0] == 2.0 ** -100 / 448 or abs(scale[0] * 448 / 2.0 ** -100 - 1) < 2 * U
    assert ((scale[1:] * 448 / v[1:].sqrt().clamp(min=2.0 ** -100) - 1).abs() <= 4 * U).all()


def test_adamw_step_count_and_scales():
    """Ten steps with a device-side schedule equal the float64 recurrence."""
    params, grads = adam_case([1000], torch.float32, torch.float32)
    w, m, v = params[0].cpu().double(), torch.zeros(1000).double(), torch.zeros(1000).double()
    opt = mz.AdamW(params, **HYPER)
    scale = torch.ones(1, device="cuda")
    drift = torch.zeros(1000).double()
    for n in range(1, 11):
        scale.fill_(1.0 / n)
        opt.step(grads, lr_scale=scale)
        lr = HYPER["lr"] * float(torch.tensor(1.0 / n))
        (w, m, v), (perr, _, _) = ref.adamw(w, grads[0], m, v, n, lr, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        # m and v are themselves off by at most 5 u and 7 u per step so far
        drift += perr + 12 * n * U * lr * 1.1
    assert ((params[0].cpu().double() - w).abs() <= drift).all()
    assert opt.step_count.tolist() == [10, 0]


# ------------------------------------------------------------------ streams, graphs, repeats


def calls():
    logits, idx = rows_case(700, 96, 6, seed=3)
    dgate = torch.randn(700, 6, generator=gen(4)).cuda()
    seq, dloss = ints([0, 100, 650]), torch.tensor([0.3, 0.6], device="cuda")
    c = combine_case(40, 1024, 6, 0.3, seed=5)

    def run(stream=None):
        r = mz.balance_loss(logits, idx, seq_start=seq, stream=stream)
        d = mz.route_backward(logits, idx, dgate=dgate, coef=r.coef, dloss=dloss, seq_start=seq, stream=stream)
        dg, dy = mz.combine_backward(*c, stream=stream)
        return [*r, d, dg, dy]
    return run, logits


def test_equal_bits_every_run():
    run, _ = calls()
    a = run()
    for _ in range(3):
        for x, y in zip(a, run()):
            assert torch.equal(x, y)


def test_another_stream():
    run, _ = calls()
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    raw = run(stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    default = run(stream=0)
    torch.cuda.synchronize()
    for a, b, c, d in zip(want, got, raw, default):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


def test_two_captured_graphs_replayed_together():
    run, logits = calls()
    run()
    want = [t.clone() for t in run()]
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(want, o):
            assert torch.equal(a, b)
    logits.mul_(0.5)
    fresh = run()
    graphs[0].replay()
    torch.cuda.synchronize()
    for a, b in zip(fresh, outs[0]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_replayed_steps_go_on_counting(bits):
    params, grads = adam_case([3000, 17], torch.float32, torch.float32)
    eager = mz.AdamW([p.clone() for p in params], **HYPER, state_bits=bits)
    opt = mz.AdamW(params, **HYPER, state_bits=bits)
    for _ in range(4):
        eager.step(grads)
    opt.step(grads)   # (also sets up what a first launch looks up)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step(grads)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert opt.step_count.tolist() == [4, 0] == eager.step_count.tolist()
    for a, b in zip(opt.params, eager.params):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ offsets past 32 bits


def test_rows_past_32_bit_offsets():
    """2.1 M rows of 1024 logits (8.6 GB): every thousandth row is the same, so the
    first thousand tell what all the others must be."""
    n, reps, E, K = 1000, 2100, 1024, 4
    small, idx = rows_case(n, E, K, seed=21)
    dgate = torch.randn(n, K, generator=gen(22)).cuda()
    logits = small.repeat(reps, 1)
    assert logits.numel() > 2 ** 31
    big, dbig = idx.repeat(reps, 1), dgate.repeat(reps, 1)
    want = mz.route_backward(small, idx, dgate=dgate, dtype=torch.bfloat16)
    got = mz.route_backward(logits, big, dgate=dbig, dtype=torch.bfloat16)
    assert torch.equal(got.view(reps, n, E)[-1], want) and torch.equal(got.view(reps, n, E)[reps // 2], want)
    del got
    seq = ints([0, n * (reps - 1), n * reps])
    r, one = mz.balance_loss(logits, big, seq_start=seq), mz.balance_loss(small, idx)
    assert torch.equal(r.counts[1], one.counts[0]) and torch.equal(r.counts[0], one.counts[0] * (reps - 1))
    # the same tokens' mean, summed in two orders
    rel = 2 * (ref.softmax_steps(small.cpu()) + 4 * n) * U
    assert torch.allclose(r.prob[1], one.prob[0], rtol=rel, atol=0)


def test_expert_rows_past_32_bit_offsets():
    """360 000 rows of 6144 features: a token's slots at the far end give what
    they give near the start."""
    d, K, R = 6144, 3, 360_000
    dout, x, y, _, gate = combine_case(4, d, K, 0.0, seed=23)
    rows = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    assert rows.numel() > 2 ** 31
    rows[R - 12:] = y
    near = torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3)
    want, wdy = mz.combine_backward(dout, x, y, near, gate)
    got, dy = mz.combine_backward(dout, x, rows, (near + (R - 12)).contiguous(), gate)
    assert torch.equal(got, want) and torch.equal(dy[R - 12:], wdy)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_past_32_bit_offsets(bits):
    """A tensor of 2^31 + 3000 elements whose last 4096 are those of a small one."""
    n, m = 2 ** 31 + 3000, 4096
    start = n // 256 * 256 - m + 256      # a block's start, so that both share their blocks
    m = n - start
    (w,), (g,) = adam_case([m], torch.bfloat16, torch.bfloat16, seed=24)
    big, bg = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    big[start:], bg[start:] = w, g
    for opt, gr in ((mz.AdamW([w], **HYPER, state_bits=bits), g), (mz.AdamW([big], **HYPER, state_bits=bits), bg)):
        opt.step([gr])
        opt.step([gr])
    assert torch.equal(big[start:], w)
    assert not big[:start].any()


def test_route_logits():
    """The logits route works on, with route's own results beside them, for
    batches whose router GEMM slices K and for those where it does not."""
    g = gen(7)
    N, Z, K, d = 40, 20, 4, 512
    W = (torch.randn(N + Z, d, generator=g) * 0.02).to(torch.bfloat16).cuda()
    b = (torch.rand(N + Z, generator=g) * 0.02).cuda()
    off = torch.linspace(-1, 1, N + Z).cuda()
    for T in (1, 64, 300, 40000):
        x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
        for o in (None, off):
            logits, idx, gate, zsum, counts = mz.route_logits(x, W, b, N, Z, K, logit_offset=o)
            for a, c in zip(mz.route(x, W, b, N, Z, K, logit_offset=o), (idx, gate, zsum, counts)):
                assert torch.equal(a, c)
            want = x.double() @ W.double().t()
            mag = x.double().abs() @ W.double().abs().t()
            # exact products; the tensor core's accumulation may truncate (2^-23 a step)
            assert ((logits.double() - want).abs() <= 2 * d * U * mag).all()
            p = ref.softmax64(logits.cpu(), None if o is None else o.cpu())
            assert torch.allclose(p.gather(1, idx.cpu().long()), gate.cpu().double(), rtol=1e-5)
    mz.synchronize()


def test_adamw_refuses_a_parameter_with_another_storage():
    params, grads = adam_case([300, 70], torch.float32, torch.float32)
    opt = mz.AdamW(params, **HYPER)
    opt.step(grads)
    old = params[1].data
    want = old.clone()
    params[1].data = torch.ones(70, device="cuda")
    with pytest.raises(ValueError, match="another storage"):
        opt.step(grads)
    assert torch.equal(old, want) and (params[1] == 1).all()
    assert opt.step_count.tolist() == [1, 0]
    params[1].data = old
    opt.step(grads)
    assert opt.step_count.tolist() == [2, 0]


def test_adamw_refuses_missing_gradients():
    params, grads = adam_case([300, 70], torch.float32, torch.float32)
    opt = mz.AdamW(params, **HYPER)
    for bad in ([None, grads[1]], [grads[0], None], grads[:1]):
        with pytest.raises(ValueError):
            opt.step(bad)
    assert opt.step_count.tolist() == [0, 0]


def test_adamw_keeps_its_states_storages():
    # a state whose .data is set elsewhere: the step still writes memory it holds
    params, grads = adam_case([4096], torch.float32, torch.float32)
    opt, twin = (mz.AdamW([p], **HYPER) for p in (params[0], params[0].clone()))
    opt.exp_avg[0].data = torch.empty(0, device="cuda")
    others = [torch.full((4096,), 7.0, device="cuda") for _ in range(4)]   # would take a freed one's place
    for _ in range(2):
        opt.step(grads)
        twin.step(grads)
    assert torch.equal(opt.params[0], twin.params[0])
    assert all((o == 7).all() for o in others)
