"""The loss operators without a GPU: refused calls, workspace sizes, and the
64-bit reference forms against differences of their own losses."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import host_memory_centric_gb300 as mt  # noqa: E402
from host_memory_centric_gb300 import ops  # noqa: E402
from tests import loss_reference as ref  # noqa: E402

P = 1 << 20  # an aligned address that no refused call may touch
ARG = -1


def lce(h=P, W=P, target=P, T=4, H=64, V=100, row_loss=P, dh=P, dW=P, scratch=P, nbytes=1 << 40):
    return mt.lib().mt_linear_cross_entropy(h, W, target, T, H, V, 1.0, row_loss, dh, dW, scratch, nbytes, None)


@pytest.mark.parametrize("bad", [dict(h=None), dict(W=None), dict(target=None), dict(row_loss=None), dict(scratch=None),
                                 dict(H=60), dict(H=0), dict(V=0), dict(V=(1 << 21) + 1), dict(T=-1), dict(h=P + 2),
                                 dict(W=P + 8), dict(dh=P + 2), dict(dW=P + 4), dict(scratch=P + 16), dict(nbytes=64)])
def test_linear_cross_entropy_refuses(bad):
    assert lce(**bad) == ARG


def test_linear_cross_entropy_scratch():
    size = mt.lib().mt_linear_cross_entropy_scratch_bytes
    assert size(-1, 64, 100, 1) == 0 and size(4, 60, 100, 1) == 0
    assert lce(nbytes=size(4, 64, 100, 1) - 1) == ARG
    # statistics alone need no exponentials; a long batch is cut into chunks, so the workspace stops growing
    assert size(4096, 64, 32000, 0) < size(4096, 64, 32000, 1) / 32
    V, H = 152064, 3584
    assert size(1 << 20, H, V, 1) < (4 << 30) + 4 * V * H  # exponentials of up to 3 GiB, the FP32 sum of dW
    assert size(0, 64, 100, 1) >= 0 and lce(T=0) == 0


def kd(logits=P, target=P, t_val=P, t_idx=P, rows=4, V=100, K=8, tau=1.0, row_ce=P, row_kd=P, dlogits=P):
    return mt.lib().mt_distill_topk(logits, target, t_val, t_idx, rows, V, K, tau, 1.0, 1.0, row_ce, row_kd, dlogits,
                                    None)


@pytest.mark.parametrize("bad", [dict(logits=None), dict(t_val=None), dict(t_idx=None), dict(row_kd=None),
                                 dict(target=None), dict(rows=-1), dict(V=0), dict(K=0), dict(K=1025), dict(tau=0.0),
                                 dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(logits=P + 2),
                                 dict(dlogits=P + 8)])
def test_distill_refuses(bad):
    assert kd(**bad) == ARG


def bal(logits=P, idx=P, valid=P, T=32, S=8, E=16, k=2, loss=P, counts=P, prob=P, dlogits=P, scratch=P,
        nbytes=1 << 40):
    return mt.lib().mt_router_balance(logits, idx, valid, T, S, E, k, 1.0, 1.0, loss, counts, prob, dlogits, scratch,
                                      nbytes, None)


@pytest.mark.parametrize("bad", [dict(logits=None), dict(idx=None), dict(loss=None), dict(counts=None),
                                 dict(prob=None), dict(scratch=None), dict(T=33), dict(S=0), dict(S=-8), dict(T=-8),
                                 dict(E=0), dict(E=513), dict(k=0), dict(k=17), dict(T=1 << 20, S=8),
                                 dict(T=1 << 30, S=1 << 30, k=2), dict(logits=P + 4), dict(dlogits=P + 2),
                                 dict(scratch=P + 64), dict(nbytes=16)])
def test_router_balance_refuses(bad):
    assert bal(**bad) == ARG


def test_no_rows_launch_nothing():
    assert lce(T=0) == 0 and kd(rows=0) == 0 and bal(T=0) == 0


def test_wrappers_refuse_what_the_library_would_misread():
    bf = torch.bfloat16
    h, W = torch.zeros(4, 64, dtype=bf), torch.zeros(100, 64, dtype=bf)
    tgt, loss = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    sc = torch.zeros(1 << 20, dtype=torch.uint8)
    for a in [(h, W, tgt, 1.0, loss, None, None, sc),  # not on a GPU
              (h.float(), W, tgt, 1.0, loss, None, None, sc), (h, W, tgt.long(), 1.0, loss, None, None, sc),
              (h.t().contiguous().t(), W, tgt, 1.0, loss, None, None, sc)]:
        with pytest.raises(mt.MtError):
            ops.linear_cross_entropy(*a)
    z, y, i = torch.zeros(4, 100, dtype=bf), torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(mt.MtError):
        ops.distill_topk(z[:, ::2], None, y, i, 1.0, 0.0, 1.0, None, loss, None)
    with pytest.raises(mt.MtError):
        ops.distill_topk(z, None, y, i[:, :4], 1.0, 0.0, 1.0, None, loss, None)
    with pytest.raises(mt.MtError):
        ops.router_balance(torch.zeros(30, 8), torch.zeros(30, 2, dtype=torch.int32), None, 8, 1.0, 0.0,
                           torch.zeros(2), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8), None, sc)


# ------------------------------------------------------------------ the reference forms themselves
def along(loss, x, d, step=1e-5):
    """Central difference of a scalar loss along d."""
    return float((loss(x + step * d) - loss(x - step * d)) / (2 * step))


def test_reference_linear_cross_entropy_gradients_match_differences():
    g = torch.Generator().manual_seed(1)
    h, W = torch.randn(6, 8, generator=g).double(), torch.randn(11, 8, generator=g).double()
    tgt = torch.tensor([0, 10, -1, 3, 11, 3], dtype=torch.int32)
    _, dh, dW, *_ = ref.linear_cross_entropy(h, W, tgt, 0.3)
    a, b = torch.randn(6, 8, generator=g).double(), torch.randn(11, 8, generator=g).double()
    assert abs(along(lambda x: 0.3 * ref.linear_cross_entropy(x, W, tgt, 0.3)[0].sum(), h, a) - float((dh * a).sum())) < 1e-8
    assert abs(along(lambda x: 0.3 * ref.linear_cross_entropy(h, x, tgt, 0.3)[0].sum(), W, b) - float((dW * b).sum())) < 1e-8
    assert float(dh[2].abs().max()) == 0.0 and float(dh[4].abs().max()) == 0.0


def test_reference_distill_gradient_matches_differences():
    g = torch.Generator().manual_seed(2)
    z = torch.randn(4, 13, generator=g).double()
    y = torch.randn(4, 3, generator=g)
    ids = torch.tensor([[0, 5, 5], [12, -1, 2], [-1, -1, 13], [1, 2, 3]], dtype=torch.int32)
    tgt = torch.tensor([5, -1, 4, 2], dtype=torch.int32)
    dz = ref.distill(z, tgt, y, ids, 1.7, 0.4, 0.9)[2]
    a = torch.randn(4, 13, generator=g).double()

    def total(x):
        ce, kd, *_ = ref.distill(x, tgt, y, ids, 1.7, 0.4, 0.9)
        return 0.4 * ce.sum() + 0.9 * kd.sum()

    assert abs(along(total, z, a) - float((dz * a).sum())) < 1e-8


def test_reference_router_balance_gradient_matches_differences():
    g = torch.Generator().manual_seed(3)
    z = torch.randn(12, 5, generator=g).double()
    idx = torch.randint(-1, 6, (12, 2), generator=g, dtype=torch.int32)
    valid = torch.tensor([1, 1, 0, 1, 0, 0, 0, 0, 1, 1, 1, 1], dtype=torch.uint8)
    d = ref.router_balance(z, idx, valid, 4, 0.7, 0.2)[3]
    a = torch.randn(12, 5, generator=g).double()
    # the counts do not depend on the logits, so the differences see f held constant, as the gradient does
    assert abs(along(lambda x: ref.router_balance(x, idx, valid, 4, 0.7, 0.2)[0].sum(), z, a) - float((d * a).sum())) < 1e-8
    assert float(d[4:8].abs().max()) == 0.0
