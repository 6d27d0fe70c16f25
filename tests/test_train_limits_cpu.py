"""Limits of the training operators (include/fc/train.h) that their documentation states,
without a GPU."""
import pytest

import bit_activation_compression_amd as fc
from test_train_cpu import NONE, P, _act, _linear, _weight_grad


def test_a_weight_gradient_is_never_null():
    """No tokens: zeros, or what was there; there is a dw in any case."""
    none = dict(T=0, dy=None, codes=None, s=None, z=None)
    assert _weight_grad(**none, acc=0, dw=None) == 1 and _weight_grad(**none, acc=1, dw=None) == 1
    assert _weight_grad(**none, acc=1) == 0


@pytest.mark.parametrize("kw", [dict(mc=P(4), ms=P(5), mz=P(6)), dict(dmul=P(8)), dict(dz=P(7)),
                                dict(codes=P(1), s=P(2), z=P(3), mc=P(4), ms=P(5), mz=P(6), dz=P(7), dmul=P(8))])
def test_a_second_factor_without_an_activation_is_forward_only(kw):
    assert _linear(act=0, a=None) == 1          # the forward layer takes it: a NULL operand is what it refuses
    assert _act(**dict(NONE, **kw)) == 10


def test_workspaces_of_split_sums():
    """The sizes that the tests of the products' workspaces count on."""
    need = fc.fc_linear_weight_grad_workspace_bytes(1, 1 << 16, 64, 64)
    assert need > 0 and need % (64 * 64 * 4) == 0
    kw = dict(R=1, T=1 << 16, K=64, H=64, group=8)
    assert _weight_grad(**kw, nbytes=need - 1) == 5
    assert _weight_grad(**kw, ws=None) == 1
    for other in (0, 1, 2, 3, 4):
        assert _weight_grad(**kw, ws=P(other), nbytes=need) == 9
