"""The gated delta rule where its answers are easily a little or wholly off:
roundings of bf16 outputs, sizes of 0, the ends of its buffers.

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


GUARD = 1024     # bytes around every buffer


class Guarded:
    """Buffers of exact sizes with guard bands, filled with 0xFF (NaN in every
    type): what a call leaves unwritten or reads before writing shows."""

    def __init__(self):
        self.bufs = []

    def __call__(self, nbytes):
        buf = torch.full((nbytes + 2 * GUARD,), 0xFF, dtype=torch.uint8, device="cuda")
        self.bufs.append(buf)
        return buf[GUARD:GUARD + nbytes]

    def like(self, t):
        return self(t.numel() * t.element_size()).view(t.dtype).view(t.shape)

    def check(self):
        for i, buf in enumerate(self.bufs):
            assert (buf[:GUARD] == 0xFF).all() and (buf[-GUARD:] == 0xFF).all(), f"buffer {i}"


TOL32, TOL16 = 2e-5, 1.5 * 2.0 ** -8     # as in test_gpu_delta.py


def assert_near(got, want, what):
    tol = TOL16 if got.dtype == torch.bfloat16 else TOL32
    got = host(got)
    assert np.isfinite(got).all(), what
    assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want) + 1e-30, what


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 1, 2, 64, 64), (2, 70, 1, 3, 64, 40), (1, 129, 1, 2, 128, 72), (2, 130, 2, 2, 72, 104),
                                   (1, 63, 1, 2, 33, 17), (1, 150, 1, 1, 8, 8), (1, 200, 1, 2, 24, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_outputs_and_scratch_stay_in_bounds(m, shape, dtype):
    """Every output and a scratch of the size asked for, through the C entry
    points: nothing around them changes, nothing in them is left out, and what
    the scratch held does not matter."""
    x = draw(*shape, dtype=dtype, seed=sum(shape))
    sizes, es = shape, x["q"].element_size()
    B, T, HK, HV, DK, DV = shape
    suffix, scale = ("" if dtype == "f32" else "_bf16"), DK ** -0.5
    p = {n: t.data_ptr() for n, t in x.items()}
    ins = [p[n] for n in INPUTS]
    stream = torch.cuda.current_stream().cuda_stream
    for with_state in (False, True):
        mem = Guarded()
        o, s_out = mem.like(x["v"]), mem.like(x["s_in"])
        n = m.lib.gated_delta_scratch(B, T, HV, DK, DV, es, with_state)
        st = getattr(m.lib, "gated_delta" + suffix)(*sizes, *ins, scale, o.data_ptr(), p["s_in"],
                                                    s_out.data_ptr() if with_state else None,
                                                    mem(n).data_ptr() if n else None, n, stream)
        assert st == m.WKV_OK, m.wkv_last_error()
        want, ws = od.gated_delta(*(host(x[i]) for i in INPUTS), scale, host(x["s_in"]))
        assert_near(o, want, "o")
        if with_state:
            assert_near(s_out, ws, "s_out")
        mem.check()
    mem = Guarded()
    outs = {n: mem.like(x[n]) for n in INPUTS + ("s_in",)}
    n = m.lib.gated_delta_backward_scratch(B, T, HV, DK, DV, es)
    st = getattr(m.lib, "gated_delta_backward" + suffix)(
        *sizes, *ins, scale, p["s_in"], p["go"], p["gs_out"], *(t.data_ptr() for t in outs.values()),
        mem(n).data_ptr(), n, stream)
    assert st == m.WKV_OK, m.wkv_last_error()
    want = od.gated_delta_backward(*(host(x[i]) for i in INPUTS), scale, host(x["go"]), host(x["s_in"]),
                                   host(x["gs_out"]))
    for (name, t), w in zip(outs.items(), want):
        assert_near(t, w, name)
    mem.check()


@pytest.mark.parametrize("shape", [(8, 33, 4, 32, 64, 72), (8, 56, 8, 32, 64, 64), (8, 57, 8, 32, 64, 64), (5, 32, 10, 30, 72, 104)],
                         ids=lambda s: "x".join(map(str, s)))
def test_more_heads_than_sms_around_the_chunked_lengths(m, shape):
    """Both sides of the lengths from which bf16 calls of many heads take the
    chunked kernels: wide states from 33 steps on, others from 57."""
    B, T, HK, HV, DK, DV = shape
    x = draw(*shape, dtype="bf16", seed=sum(shape))
    assert (m.lib.gated_delta_scratch(B, T, HV, DK, DV, 2, 1) > 0) == (T > (32 if DV > 64 else 56))
    s_out = torch.empty_like(x["s_in"])
    o = m.gated_delta(*(x[n] for n in INPUTS), s_in=x["s_in"], s_out=s_out)
    want, ws = od.gated_delta(*(host(x[n]) for n in INPUTS), DK ** -0.5, host(x["s_in"]))
    assert_near(o, want, "o")
    assert_near(s_out, ws, "s_out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 150, 2, 4, 64, 64), (2, 70, 1, 2, 128, 128), (2, 90, 1, 3, 40, 24)],
                         ids=lambda s: "x".join(map(str, s)))
def test_nan_in_a_gradient_stays_in_its_row_and_head(m, shape, dtype):
    """A NaN in one value head's v: the gradients of the other rows and of the
    other heads' own tensors have the bits they have without it; gq and gk sum
    over the value heads of a key head, the other key heads' stay too."""
    x = draw(*shape, dtype=dtype, seed=sum(shape))
    HK, HV = shape[2:4]
    run = lambda: m.gated_delta_backward(*(x[n] for n in INPUTS), x["go"], s_in=x["s_in"], gs_out=x["gs_out"])  # noqa: E731
    want = [t.clone() for t in run()]
    x["v"][0, 40, 1, 3] = float("nan")
    for name, got, w in zip(INPUTS + ("s_in",), run(), want):
        assert torch.equal(got[1], w[1]), name
        head = 1 // (HV // HK) if name in ("q", "k") else 1
        axis = 0 if name == "s_in" else 1     # of got[0]
        rest = [h for h in range(got[0].shape[axis]) if h != head]
        idx = torch.tensor(rest, dtype=torch.int64, device="cuda")
        assert torch.equal(got[0].index_select(axis, idx), w[0].index_select(axis, idx)), name
