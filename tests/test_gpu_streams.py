"""Calls on another stream than the current one: what they return is that
stream's memory, so that neither side overwrites what the other still uses.

Every buffer measures more than 1 MiB: torch's allocator then keeps one freed
block per buffer instead of parts of a shared one.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m(cuda_dev):
    import rwkv_wkv_mixing_b200 as mod
    return mod


B, T, C, H, D = 2, 1024, 512, 8, 64


def calls(m):
    gen = torch.Generator(device="cuda").manual_seed(1)

    def r(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    k, v, gy = r(B, T, C), r(B, T, C), r(B, T, C)
    w, u, mu = r(C).abs(), r(C), r(2, C).sigmoid()
    s = torch.zeros(B, 3, C, device="cuda")
    q, kk = (torch.nn.functional.normalize(r(B, T, H, D), dim=-1) for _ in range(2))
    vv, go = r(B, T, H, D), r(B, T, H, D)
    g, beta = -r(B, T, H).abs(), r(B, T, H).sigmoid()
    z = torch.complex(r(B, T, C), r(B, T, C))
    h = (q.bfloat16(), kk.bfloat16(), vv.bfloat16(), g, beta)
    hgo, hk, hv, a = go.bfloat16(), k.bfloat16(), v.bfloat16(), k.sigmoid()
    return {
        "wkv_forward": lambda st: [m.wkv_forward(w, u, k, v, stream=st)],
        "wkv_forward_bf16": lambda st: [m.wkv_forward_bf16(w, u, hk, hv, stream=st)],
        "wkv_forward_state": lambda st: [m.wkv_forward_state(w, u, k, v, s, stream=st)[0]],
        "wkv_forward_gated": lambda st: [m.wkv_forward_gated(w, u, k, v, gy, stream=st)],
        "token_shift": lambda st: [m.token_shift(k, mu, stream=st)],
        "diag_scan": lambda st: [m.diag_scan(a, v, stream=st)],
        "wkv_backward": lambda st: list(m.wkv_backward(w, u, k, v, gy, stream=st)[:2]),
        "lru_scan": lambda st: [m.lru_scan(w, u, z, stream=st)],
        "gated_delta": lambda st: [m.gated_delta(q, kk, vv, g, beta, stream=st)],
        "gated_delta_bf16": lambda st: [m.gated_delta(*h, stream=st)],
        "gated_delta_backward": lambda st: list(m.gated_delta_backward(q, kk, vv, g, beta, go, stream=st)[:3]),
        "gated_delta_backward_bf16": lambda st: list(m.gated_delta_backward(*h, hgo, stream=st)[:3]),
        "group_norm": lambda st: [m.group_norm(k, H, w, u, gate=v, act="silu", stream=st)],
        "group_norm_backward": lambda st: [x for x in m.group_norm_backward(k, gy, H, w, u, gate=v, act="silu",
                                                                           stream=st)[::3]],
    }


NAMES = ["wkv_forward", "wkv_forward_bf16", "wkv_forward_state", "wkv_forward_gated", "token_shift", "diag_scan",
         "wkv_backward", "lru_scan", "gated_delta", "gated_delta_bf16", "gated_delta_backward",
         "gated_delta_backward_bf16", "group_norm", "group_norm_backward"]


# The scans whose sequences span more than two tiles fold their carries in an
# order that differs from run to run: two runs are each within the tolerance of
# their parity tests of the exact result (relative to the largest value), so
# within twice that of one another.  The others repeat themselves exactly.
TOL = {"wkv_forward": 1e-5, "wkv_forward_bf16": 2e-2, "wkv_forward_state": 1e-5, "wkv_forward_gated": 1e-5,
       "diag_scan": 1e-5, "lru_scan": 1e-5, "wkv_backward": 1e-4}


@pytest.mark.parametrize("name", NAMES)
def test_results_belong_to_the_stream_of_the_call(m, name):
    call = calls(m)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks that the current stream just freed (work queued there may still
    # read them) are not what a call on another stream writes
    sizes = [(x.shape, x.dtype) for x in want]
    free = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
    freed = {x.data_ptr() for x in free}
    del free
    got = call(side)
    assert not freed & {x.data_ptr() for x in got}
    side.synchronize()
    for a, b in zip(got, want):
        if name in TOL:
            assert (a - b).abs().max() <= 2 * TOL[name] * b.abs().max()
        else:
            assert torch.equal(a, b)
    # a result dropped while the call is still queued stays that stream's
    # memory: the current stream's tensors keep what is written to them
    del got
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # some 10 ms
    got = call(side)
    del got
    mine = [torch.full(s, 7, dtype=d, device="cuda") for s, d in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in mine)
