"""The loss operators on the GPU against their 64-bit forms.

Tolerances are bounds from the arithmetic, set before the first run:
  * rounding to BF16 is off by at most 2^-8 of the value;
  * a logit z = sum_i h_i W_i of exact products is summed in FP32 by the tensor
    cores, 16 products a step: off by at most (H / 8 + 2) 2^-23 max_v sum_i |h_i W_vi|;
  * FP32 exp, log and sums of n terms: 2^-20 relative for the sums here (pairwise
    over threads and warps, at most a few hundred terms in a row).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import host_memory_centric_gb300 as mt  # noqa: E402
from host_memory_centric_gb300 import ops  # noqa: E402
from tests import loss_reference as ref  # noqa: E402

BF = torch.bfloat16
HALF = 2.0 ** -8   # half a BF16 step, relative
F32 = 2.0 ** -20   # a few FP32 operations and a sum, relative


@pytest.fixture(autouse=True)
def _no_kernel_errors():
    ops.kernel_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert ops.kernel_error(clear=True) == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def behind(shape, dtype, fill=7.0):
    """A contiguous buffer with 64 sentinel values behind it."""
    n = int(np.prod(shape))
    big = torch.full((n + 64,), fill, dtype=dtype, device="cuda")
    return big[:n].view(*shape), big[n:]


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err.max()), float((err / tol.clamp(min=1e-300)).max()))


# ------------------------------------------------------------------ linear cross-entropy
def lce_inputs(T, H, V, seed, std=2.5):
    g = gen(seed)
    h = randn(g, T, H).to(BF)
    W = (randn(g, V, H) * (std / H ** 0.5)).to(BF)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return h, W, tgt


def run_lce(h, W, tgt, g, dh=True, dW=True, scratch=None):
    T, H = h.shape
    V = W.shape[0]
    loss, end = behind((T,), torch.float32)
    outs = [loss, behind((T, H), BF) if dh else None, behind((V, H), BF) if dW else None]
    if scratch is None:
        scratch = torch.empty(ops.linear_cross_entropy_scratch_bytes(T, H, V, dh or dW), dtype=torch.uint8, device="cuda")
        scratch.fill_(0xFF)  # nothing in it may need to start at zero
    ops.linear_cross_entropy(h, W, tgt, g, loss, outs[1] and outs[1][0], outs[2] and outs[2][0], scratch)
    torch.cuda.synchronize()
    for tail in [end] + [o[1] for o in outs[1:] if o]:
        assert bool((tail == 7.0).all())
    return loss, outs[1] and outs[1][0], outs[2] and outs[2][0]


def check_lce(h, W, tgt, g, got):
    loss, dh, dW = got
    H = h.shape[1]
    rl, rdh, rdW, mdh, mdW, mag = ref.linear_cross_entropy(h, W, tgt, g)
    ez = (H / 8 + 2) * 2.0 ** -23 * mag  # error of a logit of the row
    within(loss, rl, 2 * ez + F32 * (rl.abs() + mag), "loss")
    # a gradient element: two roundings (the exponential to 16 bits, the product with its piece's factor to BF16) and
    # the logits' errors in exp; then the FP32 sum over V or T, and the output's own rounding.  The exponential is
    # held as fp16(2^15 e), e <= 1: below the normal range its steps are 2^-24, so besides the relative error it is
    # off by at most 2^-25 2^-15 = 2^-40, which the piece's factor (at most 1) does not enlarge.
    rel, tiny = 2 * HALF + HALF ** 2 + 2 * float(ez.max()) + F32, 2.0 ** -40 * abs(g)
    if dh is not None:
        within(dh, rdh, rel * mdh + HALF * rdh.abs() + tiny * W.double().abs().sum(0) + 1e-30, "dh")
    if dW is not None:
        within(dW, rdW, rel * mdW + HALF * rdW.abs() + tiny * h.double().abs().sum(0) + 1e-30, "dW")


# one token, one column, ragged tiles and pieces in every dimension, a last piece of one column, V below a
# 64-wide box, several 256-row tiles; up to sixteen tokens (a path of their own), with H at its limits: one group of
# 32 columns and less, an even and an odd number of groups, wider than a block, the widest and one beyond
@pytest.mark.parametrize("T,H,V", [(1, 8, 1), (1, 64, 257), (5, 256, 1000), (130, 72, 515), (256, 256, 1024),
                                   (300, 264, 2050), (513, 128, 33), (1000, 520, 4099), (2, 296, 1258), (8, 24, 129),
                                   (3, 96, 40001), (8, 520, 20000), (7, 2056, 130), (4, 12768, 300), (4, 12776, 300),
                                   (9, 64, 600), (6, 1032, 9), (16, 6368, 200), (16, 6400, 200), (15, 256, 5000),
                                   (16, 136, 3001), (11, 520, 9000), (10, 64, 1), (17, 64, 700), (12, 40, 4111)])
def test_linear_cross_entropy(T, H, V):
    h, W, tgt = lce_inputs(T, H, V, 1)
    tgt[::5] = -1
    tgt[3::7] = V  # not a column either
    tgt[:1] = V - 1
    check_lce(h, W, tgt, 1.0 / T, run_lce(h, W, tgt, 1.0 / T))


@pytest.mark.parametrize("T", [6, 270])
@pytest.mark.parametrize("dh,dW", [(False, False), (True, False), (False, True)])
def test_linear_cross_entropy_parts_agree_with_the_whole(T, dh, dW):
    h, W, tgt = lce_inputs(T, 192, 3000, 2)
    full = run_lce(h, W, tgt, 0.01)
    part = run_lce(h, W, tgt, 0.01, dh, dW)
    assert torch.equal(full[0], part[0])
    for a, b in zip(full[1:], part[1:]):
        assert b is None or torch.equal(a, b)


def test_linear_cross_entropy_over_several_chunks():
    """More tokens than one chunk of exponentials holds: dW is summed over the chunks in FP32."""
    T, H, V = 3200, 64, 524288
    one = ops.linear_cross_entropy_scratch_bytes(T // 2, H, V)
    assert ops.linear_cross_entropy_scratch_bytes(T, H, V) > one + 4 * V * H  # it has the FP32 sum
    h, W, tgt = lce_inputs(T, H, V, 3)
    tgt[::9] = -1
    check_lce(h, W, tgt, 1.0 / T, run_lce(h, W, tgt, 1.0 / T))


@pytest.mark.parametrize("T", [3, 70])
def test_linear_cross_entropy_without_any_target(T):
    h, W, tgt = lce_inputs(T, 64, 300, 4)
    tgt.fill_(-1)
    loss, dh, dW = run_lce(h, W, tgt, 1.0)
    assert float(loss.abs().max()) == 0.0 and float(dh.abs().max()) == 0.0 and float(dW.abs().max()) == 0.0


@pytest.mark.parametrize("T", [8, 64])
@pytest.mark.parametrize("std", [0.0, 80.0])
def test_linear_cross_entropy_flat_and_large_logits(T, std):
    """Equal logits (loss = log V) and logits of some hundreds, where BF16 logits would be off by whole units."""
    h, W, tgt = lce_inputs(T, 128, 1500, 5, std)
    got = run_lce(h, W, tgt, 1.0)
    check_lce(h, W, tgt, 1.0, got)
    if std == 0.0:
        assert float((got[0] - np.log(1500)).abs().max()) < 1e-5


@pytest.mark.parametrize("T", [8, 64])
def test_linear_cross_entropy_confident_rows_keep_their_digits(T):
    """The target's logit leads by about 14: its gradient element p - 1 is about -1e-4 or smaller, and dh is small
    and comes from it; the bound of check_lce scales with that small gradient."""
    H, V = 64, 700
    h, W, tgt = lce_inputs(T, H, V, 6, 0.2)
    W = W.clone()
    tgt = torch.arange(T, dtype=torch.int32, device="cuda")
    W[:T] = h * (14.0 / H)  # z_target is about 14, the others' about 1.8 (14 / sqrt(H)) or less
    loss, dh, dW = run_lce(h, W.contiguous(), tgt, 1.0)
    assert float(loss.max()) < 0.1
    check_lce(h, W, tgt, 1.0, (loss, dh, dW))


@pytest.mark.parametrize("T", [8, 40])
def test_linear_cross_entropy_not_a_number_stays_in_its_row(T):
    h, W, tgt = lce_inputs(T, 64, 600, 7)
    want = run_lce(h, W, tgt, 1.0)
    bad = h.clone()
    bad[7, 3] = float("nan")
    loss, dh, _ = run_lce(bad, W, tgt, 1.0)
    assert bool(torch.isnan(loss[7])) and bool(torch.isnan(dh[7]).all())
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(loss[keep], want[0][keep]) and torch.equal(dh[keep], want[1][keep])


@pytest.mark.parametrize("T", [8, 40])
def test_linear_cross_entropy_padding_may_hold_anything(T):
    """Rows without a target hold NaN and infinities: they leave no trace in any output."""
    h, W, tgt = lce_inputs(T, 64, 600, 17)
    tgt[1::3] = -1
    clean = h.clone()
    clean[1::3] = 0
    h[1::3, ::2] = float("nan")
    h[4] = float("inf")
    for a, b in zip(run_lce(h, W, tgt, 0.5), run_lce(clean, W, tgt, 0.5)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [4, 33])
def test_linear_cross_entropy_gradient_matches_differences(T):
    h, W, tgt = lce_inputs(T, 64, 500, 8)
    g = gen(9)
    _, dh, dW = run_lce(h, W, tgt, 1.0)
    for x, d, f in ((h, dh, lambda t: ref.linear_cross_entropy(t, W, tgt, 1.0)[0].sum()),
                    (W, dW, lambda t: ref.linear_cross_entropy(h, t, tgt, 1.0)[0].sum())):
        a = randn(g, *x.shape).double()
        diff = float((f(x.double() + 1e-5 * a) - f(x.double() - 1e-5 * a)) / 2e-5)
        # rounding errors of independent sign along a random direction; at most the sum of their sizes
        assert abs(diff - float((d.double() * a).sum())) <= 4 * HALF * float((d.double().abs() * a.abs()).sum())


# every form of the pass over W that up to sixteen tokens take, at its narrowest and its widest row and just beyond,
# one stage of rows and less, stages that fill the ring exactly, more, and a last one that is not full
@pytest.mark.parametrize("T,H,V", [(8, 136, 7), (1, 512, 32), (16, 504, 65), (9, 136, 30001), (5, 520, 16), (8, 1024, 14593),
                                   (12, 1016, 777), (16, 1024, 9121), (8, 1032, 23), (3, 2048, 9121), (16, 2040, 3000),
                                   (9, 1032, 1), (1, 2056, 25), (8, 4096, 2432), (5, 4088, 4870), (16, 2056, 700),
                                   (8, 4104, 600)])
def test_linear_cross_entropy_of_few_tokens(T, H, V):
    h, W, tgt = lce_inputs(T, H, V, 16)
    W *= torch.linspace(0.2, 2.0, V, device="cuda")[:, None]  # the maximum keeps rising along V
    tgt[1::4] = -1
    tgt[2::7] = V
    full = run_lce(h, W, tgt, 1.0 / T)
    check_lce(h, W, tgt, 1.0 / T, full)
    for dh, dW in ((True, False), (False, True), (False, False)):
        part = run_lce(h, W, tgt, 1.0 / T, dh, dW)
        for a, b in zip(full, part):
            assert b is None or torch.equal(a, b)
    none = (tgt < 0) | (tgt >= V)
    h[none] = float("nan")  # padding may hold anything
    for a, b in zip(full, run_lce(h, W, tgt, 1.0 / T)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(4, 256), (12, 800), (8, 1200), (6, 3000)])
def test_linear_cross_entropy_of_few_tokens_masked_and_confident(T, H):
    """Rows of W that make logits of -inf and of some hundreds, and tokens whose target has all the probability."""
    h, W, tgt = lce_inputs(T, H, 5000, 17)
    h[:, 0] = 1.0
    W[100:300] = 0
    W[100:300, 0] = -float("inf")
    W[7] = 0
    W[7, 0] = 300.0
    tgt[:] = 400
    tgt[::2] = 7
    loss, dh, dW = run_lce(h, W, tgt, 1.0)
    z = h.double() @ W.double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, tgt.long()[:, None])[:, 0]
    # logits of at most 300 of H products, as in check_lce; lse and loss are FP32 of that size, 2^-23 300 < 1e-4
    assert float((loss.double() - want).abs().max()) <= 2 * (H / 8 + 2) * 2.0 ** -23 * 300 + 1e-4
    assert bool((dW[100:300] == 0).all()) and bool(torch.isfinite(dW).all())
    assert float(loss[::2].max()) == 0.0 and float(dW[7].float().abs().max()) > 0.5


@pytest.mark.parametrize("T", [5, 600])
def test_linear_cross_entropy_same_bits_twice_and_on_another_stream(T):
    h, W, tgt = lce_inputs(T, 256, 5000, 10)
    a = run_lce(h, W, tgt, 0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_lce(h, W, tgt, 0.5)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T", [4, 16])
def test_linear_cross_entropy_few_tokens_refilled_ring_under_load(T):
    h, W, tgt = lce_inputs(T, 2048, 100000, 15)
    want = run_lce(h, W, tgt, 0.5)
    for _ in range(20):
        for x, y in zip(run_lce(h, W, tgt, 0.5), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("T", [8, 520])
def test_linear_cross_entropy_two_graphs_replayed_at_once(T):
    """Two captured calls with a workspace each, replayed on two streams at the same time with new inputs."""
    H, V = 256, 6000
    cases, graphs = [lce_inputs(T, H, V, 20 + i) for i in range(2)], []
    static = [tuple(torch.empty_like(t) for t in c) for c in cases]
    outs = [(torch.empty(T, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda"),
             torch.empty(V, H, dtype=BF, device="cuda")) for _ in range(2)]
    sc = [torch.empty(ops.linear_cross_entropy_scratch_bytes(T, H, V), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [run_lce(*c, 1.0 / T) for c in cases]
    for i in range(2):
        for d, t in zip(static[i], cases[1 - i]):
            d.copy_(t)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ops.linear_cross_entropy(*static[i], 1.0 / T, *outs[i], sc[i])
        graphs.append(gr)
    for i in range(2):
        for d, t in zip(static[i], cases[i]):
            d.copy_(t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for x, y in zip(outs[i], want[i]):
            assert torch.equal(x, y)


def test_linear_cross_entropy_reports_a_wait_that_ran_out():
    """A product that gets no operands (injected on the host) ends by itself and is reported; the next call is right."""
    h, W, tgt = lce_inputs(300, 64, 700, 30)
    want = run_lce(h, W, tgt, 1.0)
    for nth in (1, 2):  # the logits' product, then the gradients' too
        mt.lib().mt_fault_inject(4, nth)
        run_lce(h, W, tgt, 1.0)
        assert ops.kernel_error(clear=True) != 0
        for a, b in zip(run_lce(h, W, tgt, 1.0), want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ distillation
def kd_inputs(R, V, K, seed, hard=True):
    g = gen(seed)
    z = (randn(g, R, V) * 2.5).to(BF)
    ids = torch.randint(0, V, (R, K), generator=g, device="cuda", dtype=torch.int32)  # repeats now and then
    y = randn(g, R, K) * 2
    tgt = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32) if hard else None
    return z, tgt, y, ids


def run_kd(z, tgt, y, ids, tau, w_ce, w_kd, grad=True, in_place=False):
    R, V = z.shape
    ce, ce_end = behind((R,), torch.float32)
    kd, kd_end = behind((R,), torch.float32)
    d, d_end = behind((R, V), BF)
    if in_place:
        d.copy_(z)
        z = d
    ops.distill_topk(z, tgt, y, ids, tau, w_ce, w_kd, ce if tgt is not None else None, kd, d if grad else None)
    torch.cuda.synchronize()
    for tail in (ce_end, kd_end, d_end):
        assert bool((tail == 7.0).all())
    return ce if tgt is not None else None, kd, d if grad else None


def check_kd(z, tgt, y, ids, tau, w_ce, w_kd, got):
    ce, kd, d = got
    rce, rkd, rdz, mag, kmag = ref.distill(z, tgt, y, ids, tau, w_ce, w_kd)
    zmax = z.double().abs().amax(1)
    # lse, logits over tau and their differences in FP32
    if ce is not None:
        within(ce, rce, F32 * (rce.abs() + zmax + 1), "ce")
    within(kd, rkd, F32 * (kmag + zmax / tau + 1), "kd")
    if d is not None:
        # p = exp(z / tau - lse): the exponent is off by 2^-23 of |z| / tau + |lse| a few times over
        rel = F32 * (1 + (zmax / min(tau, 1.0))[:, None] / 4)
        within(d, rdz, HALF * rdz.abs() + rel * mag + 1e-30, "dlogits")


# one row, one column, K above V, odd V (rows that start off a 16-byte boundary), K of one and of the most,
# vocabularies around the sizes where the row takes more threads or blocks
@pytest.mark.parametrize("R,V,K,tau,hard", [(1, 1, 1, 1.0, True), (3, 7, 9, 2.0, True), (17, 129, 8, 1.0, True),
                                            (5, 1000, 50, 0.7, False), (9, 1023, 33, 3.0, True), (4, 4096, 1024, 2.0, True),
                                            (6, 32000, 32, 2.0, True), (3, 50257, 64, 1.5, True), (2, 152064, 128, 1.0, True),
                                            (2, 201089, 5, 1.3, False), (3, 2047, 16, 1.0, False), (2, 16385, 16, 1.1, True),
                                            (2, 262145, 16, 1.1, True), (1, 524288, 16, 1.1, True), (9, 524287, 3, 1.0, True),
                                            (20, 5, 2, 1.2, True), (17, 9, 4, 1.0, True), (9, 14341, 40, 1.0, True)])
def test_distill(R, V, K, tau, hard):
    z, tgt, y, ids = kd_inputs(R, V, K, 30 + R, hard)
    check_kd(z, tgt, y, ids, tau, 0.4, 0.6 * tau, run_kd(z, tgt, y, ids, tau, 0.4, 0.6 * tau))


def test_distill_missing_slots_targets_and_rows():
    R, V, K = 24, 515, 6
    z, tgt, y, ids = kd_inputs(R, V, K, 40)
    tgt[::3] = -1
    tgt[1::6] = V
    ids[::2, 3:] = -1
    ids[3::4] = V + 5       # no slot of these rows is filled
    ids[4::8] = -1          # nor of these
    y[6] = -float("inf")    # a teacher without mass
    y[7, 1:] = -float("inf")
    ids[8] = ids[8, 0]      # the same id in every slot
    ids[9, 0] = int(tgt[9]) if 0 <= int(tgt[9]) < V else 0
    tgt[10] = ids[10, 2]
    none = ((tgt < 0) | (tgt >= V)) & (((ids < 0) | (ids >= V)).all(1) | (y == -float("inf")).all(1))
    z[none] = 0
    want = run_kd(z, tgt, y, ids, 1.5, 0.5, 1.0)
    check_kd(z, tgt, y, ids, 1.5, 0.5, 1.0, want)
    # padding may hold anything, and so may empty slots
    z[none] = float("nan")
    y[(ids < 0) | (ids >= V)] = float("nan")
    got = run_kd(z, tgt, y, ids, 1.5, 0.5, 1.0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert bool(none.any())
    assert float(got[2][none].abs().max()) == 0.0 and float(got[1][none].abs().max()) == 0.0


@pytest.mark.parametrize("V", [1024, 1031, 50257])
def test_distill_in_place_and_losses_alone(V):
    z, tgt, y, ids = kd_inputs(11, V, 12, 50)
    a = run_kd(z, tgt, y, ids, 2.0, 0.5, 2.0)
    b = run_kd(z, tgt, y, ids, 2.0, 0.5, 2.0, in_place=True)
    c = run_kd(z, tgt, y, ids, 2.0, 0.5, 2.0, grad=False)
    for x, y_ in zip(a, b):
        assert torch.equal(x, y_)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_distill_masked_columns_and_large_logits():
    """Columns of -inf (a vocabulary mask) take no probability; logits of some hundreds do not overflow."""
    z, tgt, y, ids = kd_inputs(8, 777, 5, 60)
    z[:, 700:] = -float("inf")
    tgt.clamp_(max=699)
    ids.clamp_(max=699)
    z[4:, :700] *= 100
    got = run_kd(z, tgt, y, ids, 2.0, 0.5, 2.0)
    rce, rkd, rdz, mag, kmag = ref.distill(z, tgt, y, ids, 2.0, 0.5, 2.0)
    top = z.double()[:, :700].abs().amax(1)
    within(got[0], rce, F32 * (rce.abs() + top + 1), "ce")
    within(got[1], rkd, F32 * (kmag + top + 1), "kd")
    within(got[2], rdz, HALF * rdz.abs() + F32 * (1 + top[:, None] / 4) * mag + 1e-30, "dlogits")
    assert float(got[2][:, 700:].abs().max()) == 0.0


def test_distill_matches_cross_entropy_and_vanishes_at_the_teacher():
    """With the hard part alone it is mt_cross_entropy; with the teacher's list the whole vocabulary and the
    student equal to it, loss and gradient vanish."""
    z, tgt, y, ids = kd_inputs(9, 1000, 4, 70)
    ce, _, d = run_kd(z, tgt, y, ids, 1.0, 0.25, 0.0)
    d2, rl = z.clone(), torch.empty(9, device="cuda")
    ops.cross_entropy(d2, tgt, 0.25, rl)
    assert float((ce - rl).abs().max()) < 1e-5
    assert float((d.float() - d2.float()).abs().max()) <= 2 ** -7 * 0.25
    z = z[:, :1000].contiguous()
    ids = torch.arange(1000, dtype=torch.int32, device="cuda").repeat(9, 1).contiguous()
    _, kd, d = run_kd(z, None, z.float().contiguous(), ids, 2.0, 0.0, 4.0)
    assert float(kd.abs().max()) < 1e-5 and float(d.abs().max()) < 1e-6


def test_distill_same_bits_twice_and_captured():
    z, tgt, y, ids = kd_inputs(40, 33000, 20, 80)
    want = run_kd(z, tgt, y, ids, 1.5, 0.5, 1.0)
    sz, sy = torch.zeros_like(z), torch.zeros_like(y)
    ce, kd, d = torch.empty(40, device="cuda"), torch.empty(40, device="cuda"), torch.empty_like(z)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ops.distill_topk(sz, tgt, sy, ids, 1.5, 0.5, 1.0, ce, kd, d)
    sz.copy_(z)
    sy.copy_(y)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(ce, want[0]) and torch.equal(kd, want[1]) and torch.equal(d, want[2])


# rows longer than each form's ring (1, 2, 4, 8 and 16 working warps), enough of them that every block takes several
# and the stores of the gradient are the limit: chunks are refilled while loads and stores wait in line
@pytest.mark.parametrize("R,V,tau,hard", [(16384, 7000, 1.0, True), (12288, 14000, 1.5, False), (8192, 32000, 2.0, True),
                                          (4096, 60000, 1.0, False), (2048, 152064, 1.3, True)])
def test_distill_refilled_rings_under_load(R, V, tau, hard):
    z, tgt, y, ids = kd_inputs(R, V, 32, 95, hard)
    got = run_kd(z, tgt, y, ids, tau, 0.4, 0.6)
    some = torch.arange(5, R, R // 256, device="cuda")
    check_kd(z[some], tgt[some] if hard else None, y[some], ids[some], tau, 0.4, 0.6,
             tuple(None if t is None else t[some] for t in got))
    for _ in range(10):
        for a, b in zip(run_kd(z, tgt, y, ids, tau, 0.4, 0.6), got):
            assert (a is None and b is None) or torch.equal(a, b)


# the gradient over the logits, row ends off the vectors, rows held by the ring and rows fetched a second time
@pytest.mark.parametrize("R,V,tau,hard", [(4096, 20001, 1.0, True), (4096, 32003, 2.0, True), (1024, 152067, 1.5, False)])
def test_distill_in_place_under_load(R, V, tau, hard):
    z, tgt, y, ids = kd_inputs(R, V, 40, 96, hard)
    want = run_kd(z, tgt, y, ids, tau, 0.4, 0.6)
    for _ in range(5):
        for a, b in zip(run_kd(z, tgt, y, ids, tau, 0.4, 0.6, in_place=True), want):
            assert (a is None and b is None) or torch.equal(a, b)


def test_distill_gradient_matches_differences():
    z, tgt, y, ids = kd_inputs(6, 300, 7, 90)
    _, _, d = run_kd(z, tgt, y, ids, 1.5, 0.5, 1.0)
    a = randn(gen(91), 6, 300).double()

    def total(x):
        ce, kd, *_ = ref.distill(x, tgt, y, ids, 1.5, 0.5, 1.0)
        return 0.5 * ce.sum() + kd.sum()

    diff = float((total(z.double() + 1e-5 * a) - total(z.double() - 1e-5 * a)) / 2e-5)
    assert abs(diff - float((d.double() * a).sum())) <= 2 * HALF * float((d.double().abs() * a.abs()).sum())


# ------------------------------------------------------------------ router balance
def bal_inputs(T, E, k, seed):
    g = gen(seed)
    z = randn(g, T, E) * 1.5 + randn(g, E)
    return z, torch.topk(z, k, dim=1).indices.to(torch.int32).contiguous()


def run_bal(z, idx, valid, S, alpha, zc, grad=True, scratch=None):
    T, E = z.shape
    G = T // S
    loss, e0 = behind((2,), torch.float32)
    counts, e1 = behind((G, E), torch.int32, 7)
    prob, e2 = behind((G, E), torch.float32)
    d, e3 = behind((T, E), BF)
    if scratch is None:
        scratch = torch.empty(ops.router_balance_scratch_bytes(T, S, E), dtype=torch.uint8, device="cuda")
        scratch.fill_(0xFF)
    ops.router_balance(z, idx, valid, S, alpha, zc, loss, counts, prob, d if grad else None, scratch)
    torch.cuda.synchronize()
    for tail in (e0, e1, e2, e3):
        assert bool((tail == 7).all())
    return loss, counts, prob, d if grad else None


def check_bal(z, idx, valid, S, alpha, zc, got):
    loss, counts, prob, d = got
    rl, rc, rp, rd, mag = ref.router_balance(z, idx, valid, S, alpha, zc)
    assert torch.equal(counts, rc)
    zmax = float(z.abs().max()) + 1
    n = max(1.0, S) ** 0.5  # sums over S tokens in a tree of blocks, warps and lanes, at most sqrt-ish deep in a row
    within(prob, rp, F32 * (1 + n / 16) * (rp + 1e-30), "prob")
    within(loss, rl, F32 * (1 + n / 16) * zmax * rl.abs() + 1e-30, "loss")
    if d is not None:
        within(d, rd, HALF * rd.abs() + F32 * zmax * mag + 1e-30, "dlogits")


@pytest.mark.parametrize("T,S,E,k", [(1, 1, 1, 1), (1, 1, 8, 2), (256, 128, 8, 2), (60, 12, 7, 3), (96, 32, 33, 8),
                                     (300, 300, 64, 4), (16, 1, 128, 8), (4096, 4096, 32, 4), (5000, 1000, 128, 8),
                                     (77, 77, 511, 8), (513, 171, 512, 9), (30000, 30000, 16, 2), (2000, 2, 24, 4)])
def test_router_balance(T, S, E, k):
    z, idx = bal_inputs(T, E, k, 100 + E)
    check_bal(z, idx, None, S, 0.01, 0.001, run_bal(z, idx, None, S, 0.01, 0.001))


def test_router_balance_padding_empty_groups_and_dropped_choices():
    T, S, E, k = 640, 64, 40, 4
    z, idx = bal_inputs(T, E, k, 110)
    g = gen(111)
    valid = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    valid[128:256] = 0      # two groups of padding alone
    valid[256:320] = 0
    valid[300] = 5          # one valid token; any value but 0 counts
    idx[::7, 2] = -1        # dropped
    idx[5::11, 1] = E
    z[3, 5:9] = -float("inf")  # experts this token may not take
    idx[3] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    z[valid == 0] = float("nan")  # what padding holds does not count
    got = run_bal(z, idx, valid, S, 0.02, 0.003)
    clean = torch.where(torch.isnan(z), torch.zeros_like(z), z)
    zmax = float(torch.where(torch.isinf(clean), torch.zeros_like(z), clean).abs().max()) + 1
    rl, rc, rp, rd, _ = ref.router_balance(clean, idx, valid, S, 0.02, 0.003)
    assert torch.equal(got[1], rc)
    within(got[2], rp, 2 * F32 * (rp + 1e-30), "prob")
    within(got[0], rl, 2 * F32 * zmax * rl.abs(), "loss")
    size = 0.02 * E / (T // S) + 2 * 0.003 * (zmax + 4) / (T // S)  # no term is larger than p times this (n >= 1)
    p = torch.softmax(clean.double(), 1)
    within(got[3], rd, HALF * rd.abs() + F32 * zmax * size * p + 1e-30, "dlogits")
    assert float(got[3][valid == 0].abs().max()) == 0.0
    assert float(got[3][3, 5:9].abs().max()) == 0.0


def test_router_balance_all_padding():
    z, idx = bal_inputs(64, 16, 2, 120)
    loss, counts, prob, d = run_bal(z, idx, torch.zeros(64, dtype=torch.uint8, device="cuda"), 32, 1.0, 1.0)
    for t in (loss, counts, prob, d):
        assert float(t.abs().max()) == 0.0


def test_router_balance_even_router_and_losses_alone():
    """A router that spreads evenly has the balance loss alpha, whatever E and k."""
    T, E, k = 512, 32, 4
    z = torch.zeros(T, E, device="cuda")
    idx = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k).contiguous()
    a = run_bal(z, idx, None, T, 0.01, 0.0)
    b = run_bal(z, idx, None, T, 0.01, 0.0, grad=False)
    assert abs(float(a[0][0]) - 0.01) < 1e-7 and float(a[0][1]) == 0.0 and float(a[3].abs().max()) == 0.0
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,S,E,k", [(256, 128, 8, 2), (24000, 6000, 64, 6)])
def test_router_balance_same_bits_twice_and_captured(T, S, E, k):
    z, idx = bal_inputs(T, E, k, 130)
    want = run_bal(z, idx, None, S, 0.01, 0.001)
    again = run_bal(z, idx, None, S, 0.01, 0.001)
    sz, si = torch.zeros_like(z), torch.zeros_like(idx)
    outs = (torch.empty(2, device="cuda"), torch.empty(T // S, E, dtype=torch.int32, device="cuda"),
            torch.empty(T // S, E, device="cuda"), torch.empty(T, E, dtype=BF, device="cuda"))
    sc = torch.empty(ops.router_balance_scratch_bytes(T, S, E), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ops.router_balance(sz, si, None, S, 0.01, 0.001, *outs, sc)
    sz.copy_(z)
    si.copy_(idx)
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    for x, y, o in zip(want, again, outs):
        assert torch.equal(x, y) and torch.equal(x, o)


# many rows, where a lane holds two vectors of a row, and just too few of them; a last block and chunk that are not full
@pytest.mark.parametrize("T,S,E,k", [(32768, 32768, 72, 4), (32767, 32767, 72, 4), (40000, 2500, 128, 8), (36000, 3600, 136, 2),
                                     (33000, 33000, 256, 8), (32768, 4096, 68, 3)])
def test_router_balance_many_rows(T, S, E, k):
    z, idx = bal_inputs(T, E, k, 136)
    valid = (torch.rand(T, generator=gen(137), device="cuda") > 0.1).to(torch.uint8)
    check_bal(z, idx, valid, S, 0.01, 0.001, run_bal(z, idx, valid, S, 0.01, 0.001))


def test_router_balance_refilled_ring_under_load():
    z, idx = bal_inputs(131072, 128, 8, 135)
    want = run_bal(z, idx, None, 32768, 0.01, 0.001)
    for _ in range(20):
        for x, y in zip(run_bal(z, idx, None, 32768, 0.01, 0.001), want):
            assert torch.equal(x, y)


def test_router_balance_gradient_matches_differences():
    z, idx = bal_inputs(48, 12, 3, 140)
    _, _, _, d = run_bal(z, idx, None, 16, 0.5, 0.1)
    a = randn(gen(141), 48, 12).double()
    f = lambda x: ref.router_balance(x, idx, None, 16, 0.5, 0.1)[0].sum()
    diff = float((f(z.double() + 1e-5 * a) - f(z.double() - 1e-5 * a)) / 2e-5)
    assert abs(diff - float((d.double() * a).sum())) <= 2 * HALF * float((d.double().abs() * a.abs()).sum())


# ------------------------------------------------------------------ together
def test_losses_of_a_moe_decoder_head():
    """One MoE feed-forward with its balance loss, and its output through a head that is trained on targets
    (linear cross-entropy) and on a teacher's list (distillation on the head's logits), as a training program
    strings the calls together; losses and gradients against 64-bit autograd of the whole."""
    T, H, E, k, Fe, V, S, K, tau = 256, 128, 8, 2, 64, 1000, 64, 8, 2.0
    g = gen(200)
    yn, x1 = randn(g, T, H).to(BF), randn(g, T, H).to(BF)
    Wr = (randn(g, E, H) / H ** 0.5).to(BF)
    We = torch.cat([randn(g, E, 2 * Fe * H) / H ** 0.5, randn(g, E, H * Fe) / Fe ** 0.5], 1).to(BF)
    W = (randn(g, V, H) * (2.0 / H ** 0.5)).to(BF)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    tgt[S - 1::S] = -1
    ids = torch.rand(T, V, generator=g, device="cuda").topk(K, 1).indices.to(torch.int32).contiguous()
    y = randn(g, T, K)
    n = int((tgt >= 0).sum())
    w_ce, w_kd = 0.5 / n, 0.5 * tau * tau / T
    e32 = lambda *s: torch.empty(*s, device="cuda")
    e16 = lambda *s: torch.empty(*s, dtype=BF, device="cuda")
    u8 = lambda b: torch.empty(b, dtype=torch.uint8, device="cuda")

    # the layer's output (its backward runs again below, once the output's gradient is known)
    out, dyn, dWr, dWe, gate = e16(T, H), e16(T, H), e16(E, H), torch.empty_like(We), e32(T, k)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    moe_sc = u8(ops.moe_scratch_bytes(T, H, E, k, Fe))
    moe = lambda dout: ops.moe_ffn(yn, x1, Wr, We, dout, k, Fe, out, dyn, dWr, dWe, idx, gate, moe_sc)
    moe(torch.zeros_like(out))
    # the head: targets without logits; the teacher on logits, in place; their gradients added by the products
    row_loss, dh, dW = e32(T), e16(T, H), e16(V, H)
    ops.linear_cross_entropy(out, W, tgt, w_ce, row_loss, dh, dW, u8(ops.linear_cross_entropy_scratch_bytes(T, H, V)))
    logits, row_kd = e16(T, V), e32(T)
    ops.gemm(out, W, T, V, H, D=logits)
    kept = logits.clone()
    ops.distill_topk(logits, None, y, ids, tau, 0.0, w_kd, None, row_kd, logits)
    dout, dW2 = e16(T, H), e16(V, H)
    ops.gemm(logits, W, T, H, V, b_mn=True, ldb=H, D=dout, R=dh)
    ops.gemm(logits, out, V, H, T, a_mn=True, lda=V, b_mn=True, ldb=H, D=dW2, R=dW)
    moe(dout)
    # the router's own losses
    zr, dzr = e32(T, E), e16(T, E)
    ops.gemm(yn, Wr, T, E, H, Dacc=zr, acc_mode=1)
    loss, counts, prob = e32(2), torch.empty(T // S, E, dtype=torch.int32, device="cuda"), e32(T // S, E)
    ops.router_balance(zr, idx, None, S, 0.01, 0.001, loss, counts, prob, dzr, u8(ops.router_balance_scratch_bytes(T, S, E)))
    dyn2, dWr2 = e16(T, H), e16(E, H)
    ops.gemm(dzr, Wr, T, H, E, b_mn=True, ldb=H, D=dyn2, R=dyn)
    ops.gemm(dzr, yn, E, H, T, a_mn=True, lda=E, b_mn=True, ldb=H, D=dWr2, R=dWr)
    torch.cuda.synchronize()

    # 64-bit autograd over the head and the router, from the layer's own BF16 output and selection
    o64, W64 = out.double().requires_grad_(), W.double().requires_grad_()
    yn64, Wr64 = yn.double().requires_grad_(), Wr.double().requires_grad_()
    z64 = o64 @ W64.t()
    has = tgt >= 0
    ce = torch.nn.functional.cross_entropy(z64[has], tgt[has].long(), reduction="sum")
    q = torch.softmax(y.double() / tau, 1)
    kd = (q * (q.log() - torch.log_softmax(z64 / tau, 1).gather(1, ids.long()))).sum()
    head = w_ce * ce + w_kd * kd
    zr64 = yn64 @ Wr64.t()
    f = torch.zeros(T // S, E, dtype=torch.float64, device="cuda")
    f.scatter_add_(1, idx.long().view(T // S, S * k), torch.ones(T // S, S * k, dtype=torch.float64, device="cuda"))
    assert torch.equal(counts.double(), f)
    f /= S * k
    P = torch.softmax(zr64, 1).view(T // S, S, E).mean(1)
    aux = 0.01 * E * (f * P).sum(1).mean() + 0.001 * torch.logsumexp(zr64, 1).square().mean()
    gh = torch.autograd.grad(head, (o64, W64))
    gr = torch.autograd.grad(aux, (yn64, Wr64))
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    # losses: FP32 for the targets; the teacher's see logits rounded to BF16, off by 2^-8 of up to about |z| / tau each
    ce, kd, aux0 = ce.detach(), kd.detach(), aux.detach()
    assert abs(float(row_loss.sum()) - float(ce)) <= 1e-5 * float(ce)
    assert abs(float(row_kd.sum()) - float(kd)) <= HALF * float(kept.abs().max()) / tau * T
    assert abs(float(loss.sum()) - float(aux0)) <= 1e-5 * float(aux0)
    # head gradients: logits, their gradient, the first of the two sums and the result are each rounded (2-norm: 2^-8
    # is the most any of them is off); the BF16 logits shift p by up to 2^-8 max|z| / tau
    tol = 5 * HALF + HALF * float(kept.abs().max()) / tau
    assert rel(dout, gh[0]) <= tol and rel(dW2, gh[1]) <= tol
    # router gradients: what the balance loss added to the layer's own, both rounded once more than it
    for full, own, want in ((dyn2, dyn, gr[0]), (dWr2, dWr, gr[1])):
        err = (full.double() - own.double() - want).norm()
        assert float(err) <= float(HALF * full.double().norm() + 2 * HALF * want.norm() + 1e-30)
