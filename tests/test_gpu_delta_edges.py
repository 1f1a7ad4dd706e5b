"""The gated delta rule where its answers are easily a little or wholly off:
roundings of bf16 outputs, sizes of 0.

The oracle is the float64 step-by-step one; it is fed the rounded inputs.
"""
import numpy as np
import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m(cuda_dev):
    import rwkv_wkv_mixing_b200 as mod
    return mod


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def draw(B, T, HK, HV, DK, DV, dtype, seed):
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def dev(x, d=torch.float32):
        return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(d)

    def unit(*s):
        x = rng.normal(size=s)
        return x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-30)
    rate = np.exp(rng.uniform(-6, 0, size=(1, 1, HV)))
    return dict(q=dev(unit(B, T, HK, DK), dt), k=dev(unit(B, T, HK, DK), dt),
                v=dev(rng.normal(size=(B, T, HV, DV)), dt),
                g=dev(-rate * rng.exponential(1.0, size=(B, T, HV))),
                beta=dev(rng.uniform(size=(B, T, HV))),
                s_in=dev(0.5 * rng.normal(size=(B, HV, DK, DV))),
                go=dev(rng.normal(size=(B, T, HV, DV)), dt),
                gs_out=dev(0.5 * rng.normal(size=(B, HV, DK, DV))))


INPUTS = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("shape", [(2, 200, 2, 4, 64, 64), (1, 330, 1, 2, 128, 128), (1, 150, 1, 1, 96, 80),
                                   (2, 70, 1, 3, 40, 24), (1, 20, 1, 2, 64, 64), (1, 1500, 1, 1, 64, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_bf16_outputs_are_rounded_once(m, shape, with_state):
    """Half a step of bf16 at most, plus what the fp32 value before the
    rounding may be off by.  That value's operands have 16 bits or more, each
    rounding at most 2^-17 of an entry; six of them lie between the inputs and
    an output (S, P, the inverse, x, r, M), independent and uniform, so
    sqrt(6 / 3) 2^-17 of the terms' root sum of squares: 2^-16.5.  Six sigma of
    it, for terms of up to four times the output's root mean square: 2^-12."""
    x = draw(*shape, dtype="bf16", seed=sum(shape))
    s_out = torch.empty_like(x["s_in"]) if with_state else None
    o = m.gated_delta(*(x[n] for n in INPUTS), s_in=x["s_in"], s_out=s_out)
    want, _ = od.gated_delta(*(host(x[n]) for n in INPUTS), shape[4] ** -0.5, host(x["s_in"]))
    got = host(o)
    half = 2.0 ** -8 * 2.0 ** np.floor(np.log2(np.maximum(np.maximum(np.abs(want), np.abs(got)), 1e-30)))
    rms = np.sqrt((want ** 2).mean())
    over = (np.abs(got - want) - half) / rms
    assert over.max() <= 2.0 ** -12, f"{over.max():.2e} of the rms beyond the rounding, {np.mean(over > 2.0 ** -12):.1%}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 5, 1, 2, 0, 8), (2, 5, 1, 2, 8, 0), (2, 70, 2, 0, 8, 16), (1, 3, 2, 0, 0, 0)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sums_over_nothing_are_zero(m, shape, dtype):
    """Key or value heads without width, or no value heads: what is not empty
    of the outputs is a sum over nothing, not what its memory held."""
    x = draw(*shape, dtype=dtype, seed=3)
    nan = {n: torch.full_like(x[n], float("nan")) for n in ("q", "k", "v", "g", "beta")}
    o = nan["v"].clone()
    m.gated_delta(*(x[n] for n in INPUTS), s_in=x["s_in"], o=o, s_out=torch.empty_like(x["s_in"]))
    assert o.shape == x["v"].shape and (o == 0).all()
    del nan     # its blocks, full of NaN, are what the next outputs are handed
    grads = m.gated_delta_backward(*(x[n] for n in INPUTS), x["go"], s_in=x["s_in"], gs_out=x["gs_out"])
    for name, gr in zip(INPUTS + ("s_in",), grads):
        assert gr.shape == x[name].shape and (gr == 0).all(), name
