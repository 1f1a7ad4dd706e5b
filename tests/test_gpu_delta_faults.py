"""The gated delta rule's bounded device-side waits, without faulting the GPU.

A test hook keeps one kernel from making the copies of one 64-step chunk, so
the waits for them run out, after two seconds.  The launches finish, what
depends on the chunk is NaN, everything else has the bits of the undisturbed
call, and so has the next call.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, T, HV = 2, 150, 2   # three chunks, the last of 22 steps


@pytest.fixture
def m(cuda_dev):
    import rwkv_wkv_mixing_b200 as mod
    yield mod
    mod.gated_delta_set_fault_injection()


def draw(D):
    gen = torch.Generator(device="cuda").manual_seed(D)

    def r(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    unit = torch.nn.functional.normalize
    return dict(q=unit(r(B, T, 1, D), dim=-1).bfloat16(), k=unit(r(B, T, 1, D), dim=-1).bfloat16(),
                v=r(B, T, HV, D).bfloat16(), g=-0.1 * r(B, T, HV).abs(), beta=r(B, T, HV).sigmoid(),
                s=0.5 * r(B, HV, D, D), go=r(B, T, HV, D).bfloat16(), gs=0.5 * r(B, HV, D, D))


def forward(m, x, state):
    s_out = torch.zeros_like(x["s"]) if state else None
    o = m.gated_delta(x["q"], x["k"], x["v"], x["g"], x["beta"], s_in=x["s"], s_out=s_out)
    return o, s_out


def backward(m, x):
    return dict(zip(("q", "k", "v", "g", "beta", "s"),
                    m.gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["go"], s_in=x["s"],
                                           gs_out=x["gs"])))


@pytest.mark.parametrize("kernel, state, D", [(1, False, 64), (1, True, 128), (2, False, 128), (2, True, 64)])
def test_forward(m, kernel, state, D):
    x = draw(D)
    want = forward(m, x, state)
    m.gated_delta_set_fault_injection(kernel, 1)
    o, s_out = forward(m, x, state)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :64], want[0][:, :64])
    assert torch.isnan(o[:, 64:]).all()
    if state:
        assert torch.isnan(s_out).all()
    m.gated_delta_set_fault_injection()
    o, s_out = forward(m, x, state)
    assert torch.equal(o, want[0]) and (not state or torch.equal(s_out, want[1]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kernel", [1, 2, 3])
def test_backward(m, kernel, D):
    x = draw(D)
    want = backward(m, x)
    m.gated_delta_set_fault_injection(kernel, 1)
    got = backward(m, x)
    torch.cuda.synchronize()
    if kernel == 3:     # a chunk on its own
        for n in ("q", "k", "v", "g", "beta"):
            assert torch.isnan(got[n][:, 64:128]).all(), n
            got[n][:, 64:128] = want[n][:, 64:128]
            assert torch.equal(got[n], want[n]), n
        assert torch.equal(got["s"], want["s"])
    else:
        # forwards the states from chunk 1 on are missing, backwards their
        # gradients up to it.  (Without its preparation, the first step of the
        # chunk still has its state and its residual, and so its gq.)
        first = 65 if kernel == 1 else 64
        assert torch.equal(got["q"][:, :64], want["q"][:, :64])
        assert torch.isnan(got["q"][:, first:]).all()
        assert torch.isnan(got["v"][:, :128]).all()
        assert torch.equal(got["v"][:, 128:], want["v"][:, 128:])
        for n in ("k", "g", "beta", "s"):
            assert torch.isnan(got[n]).all(), n
    m.gated_delta_set_fault_injection()
    again = backward(m, x)
    assert all(torch.equal(again[n], want[n]) for n in want)


def test_hook_arguments(m):
    for bad in ((4, 0), (-1, 0), (1, -1)):
        with pytest.raises(m.WkvError, match="kernel must be"):
            m.gated_delta_set_fault_injection(*bad)
