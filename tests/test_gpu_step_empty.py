"""Batches without rows through every entry point of the operators that close a
policy step, in each form of its arguments."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def none(cols, dtype=BF):
    return torch.empty(0, cols, dtype=dtype, device="cuda")


@pytest.mark.parametrize("d", [8, 13, 600])
@pytest.mark.parametrize("d_type", [BF, F32])
@pytest.mark.parametrize("act", [None, "relu", "gelu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_activation_gradient(lg, d, d_type, act, bias, given):
    db = torch.full((d,), 5.0, device="cuda") if bias else None
    dY = none(d) if given else None
    got = lg.linear_backward_act(none(d, d_type), None if act is None else none(d), act, dY=dY,
                                 d_bias=db)
    assert got.shape == (0, d) and got.dtype == BF and (dY is None or got is dY)
    assert db is None or not db.any()


@pytest.mark.parametrize("given", [False, True])
def test_the_others(lg, given):
    W = torch.ones(8, 16, dtype=BF, device="cuda")
    out = lg.linear(none(16), W, bias=torch.ones(8, device="cuda"), act="silu", residual=none(8),
                    out=none(8) if given else None, pre=none(8))
    assert out.shape == (0, 8)
    dX = lg.linear_backward_input(none(8), W, residual=none(16), out=none(16) if given else None)
    assert dX.shape == (0, 16)
    dW = torch.ones(8, 16, device="cuda") if given else None
    assert not lg.linear_backward_weight(none(8), none(16), dW=dW).any()
    u = torch.empty(0, device="cuda")
    t = lg.sample_tokens(none(100), u, tau=u, top_p=u, min_p=u,
                         top_k=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert all(x.shape == (0,) for x in t)
    b = lg.grad_norm_bind([none(4), torch.empty(0, device="cuda")],
                          out=[none(4, F32), None] if given else None)
    r = lg.grad_norm(b, max_norm=1.0, per_tensor=True)
    assert r.norm.item() == 0 and r.scale.item() == 1 and not r.norms.any()
    lg.grad_clip(b, r.scale)
