"""The group norm with an activation at its edges: eps = 0 with token counts
that leave slots of a block empty, the ends of its buffers.

Tolerance against the float64 oracle, as the 2-norm of the difference over the
2-norm of the result: sums of D <= 128 terms and of N <= 129 tokens and the
activation's expf and division, each off by a few u = 2^-24, are below 100 u;
bf16 outputs add their rounding, 2^-8 of the value at most.
"""
import numpy as np
import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu

TOL32 = 100 * 2.0 ** -24
TOL16 = 2.0 ** -8 + TOL32


@pytest.fixture(scope="module")
def m(cuda_dev):
    import rwkv_wkv_mixing_b200 as mod
    return mod


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def draw(N, C, dtype, seed, gate):
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def dev(x, d=torch.float32):
        return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(d)
    return dict(x=dev(rng.normal(size=(N, C)) * 2 + 0.5, dt), weight=dev(rng.normal(size=C)),
                bias=dev(rng.normal(size=C)), gate=dev(rng.normal(size=(N, C)), dt) if gate else None,
                gy=dev(rng.normal(size=(N, C)), dt))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("N,G,D", [(1, 1, 64), (5, 12, 64), (33, 3, 40), (129, 12, 64), (2, 1, 7), (3, 2, 128)])
def test_no_eps(m, N, G, D, act, gate, dtype):
    """eps = 0 on groups that are not constant: token slots without a token
    have no spread either, and must not add to the sums over tokens."""
    x = draw(N, G * D, dtype, N + D, gate)
    kw = dict(weight=x["weight"], bias=x["bias"], gate=x["gate"], act=act, eps=0.0)
    wk = {**kw, **{n: host(x[n]) for n in ("weight", "bias", "gate")}}
    pairs = [("y", m.group_norm(x["x"], G, **kw), od.group_norm(host(x["x"]), G, **wk))]
    pairs += zip(("gx", "gweight", "gbias", "ggate"), m.group_norm_backward(x["x"], x["gy"], G, **kw),
                 od.group_norm_backward(host(x["x"]), host(x["gy"]), G, **wk))
    for name, got, want in pairs:
        if got is None:
            assert name == "ggate" and not gate
            continue
        tol = TOL16 if got.dtype == torch.bfloat16 else TOL32
        got = host(got)
        assert np.isfinite(got).all(), name
        assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want), name


GUARD = 1024     # bytes around every buffer


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,G,D", [(1, 1, 64), (5, 12, 64), (33, 3, 40), (700, 1, 7), (3, 2, 2049), (41, 5, 125), (9, 1, 512)])
def test_outputs_and_scratch_stay_in_bounds(m, N, G, D, dtype):
    """Every output and a scratch of the size asked for, through the C entry
    points, all filled with 0xFF (NaN) before: nothing around them changes,
    nothing in them is left out."""
    x = draw(N, G * D, dtype, N + D, True)
    bufs = []

    def mem(nbytes):
        bufs.append(torch.full((nbytes + 2 * GUARD,), 0xFF, dtype=torch.uint8, device="cuda"))
        return bufs[-1][GUARD:GUARD + nbytes]

    def like(t):
        return mem(t.numel() * t.element_size()).view(t.dtype).view(t.shape)
    suffix = "" if dtype == "f32" else "_bf16"
    stream = torch.cuda.current_stream().cuda_stream
    args = [N, G * D, G] + [x[n].data_ptr() for n in ("x", "weight", "bias", "gate")] + [1, 1e-5]
    y, gx, gw, gb, gg = (like(x[n]) for n in ("x", "x", "weight", "bias", "gate"))
    n = m.lib.group_norm_backward_scratch(N, G * D)
    scratch = mem(n)
    assert getattr(m.lib, "group_norm" + suffix)(*args, y.data_ptr(), stream) == m.WKV_OK, m.wkv_last_error()
    assert getattr(m.lib, "group_norm_backward" + suffix)(
        *args, x["gy"].data_ptr(), gx.data_ptr(), gw.data_ptr(), gb.data_ptr(), gg.data_ptr(), scratch.data_ptr(), n,
        stream) == m.WKV_OK, m.wkv_last_error()
    kw = dict(weight=host(x["weight"]), bias=host(x["bias"]), gate=host(x["gate"]), act="silu")
    want = [od.group_norm(host(x["x"]), G, **kw), *od.group_norm_backward(host(x["x"]), host(x["gy"]), G, **kw)]
    # sums of up to 4096 terms in trees, 700 tokens in at most 700 steps: as above
    for name, got, w in zip(("y", "gx", "gweight", "gbias", "ggate"), (y, gx, gw, gb, gg), want):
        tol = TOL16 if got.dtype == torch.bfloat16 else TOL32
        assert np.isfinite(host(got)).all(), name
        assert np.linalg.norm(host(got) - w) <= tol * np.linalg.norm(w), name
    for i, b in enumerate(bufs):
        assert (b[:GUARD] == 0xFF).all() and (b[-GUARD:] == 0xFF).all(), f"buffer {i}"
