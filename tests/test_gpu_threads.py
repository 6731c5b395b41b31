"""Host threads that call the library side by side, on the GPU: a call's launch
settings must not depend on what another thread is about to launch."""
import threading

import pytest
import torch

from mixture_experts_atomic_gb300 import binding as B

pytestmark = pytest.mark.gpu

from gpu_util import ensure_built  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
ROUNDS = 4000


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _calls_int4(L, d, h):
    s = B.make_shape(L, d, h, 4, 2, BF16, "silu")
    z = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    w = [z(B.moeblaze_int4_weight_bytes(4, d, h)), z(B.moeblaze_int4_scale_bytes(4, d, h, 128)), None, None,
         z(B.moeblaze_int4_weight_bytes(4, h, d)), z(B.moeblaze_int4_scale_bytes(4, h, d, 128))]
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(L, 1)
    ws = z(B.moeblaze_int4_workspace_bytes(s, 128))
    keep = [w, ids, ws, z(2 * L * d), z(8 * L), z(2 * L * d)]
    wt = B.Int4Weights(*[None if t is None else t.data_ptr() for t in w], 128)
    return keep, lambda st: B.moeblaze_int4_forward(s, keep[3].data_ptr(), ids.data_ptr(), keep[4].data_ptr(), wt,
                                                    keep[5].data_ptr(), ws.data_ptr(), ws.numel(), st)


def _calls_norm_bwd(L, d, dt):
    s = B.make_shape(L, d, 0, 1, 1, dt, "identity")
    m = [torch.zeros(L, d, dtype=dt, device="cuda") for _ in range(4)]
    v = [torch.zeros(L, device="cuda"), torch.ones(L, device="cuda"), torch.ones(d, device="cuda"),
         torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    ws = torch.zeros(B.moeblaze_layernorm_backward_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    a = [t.data_ptr() for t in (m[0], m[1], v[0], v[1], v[2], m[2], m[3], v[3], v[4], ws)]
    return (m, v, ws), lambda st: B.moeblaze_layernorm_backward(s, *a, ws.numel(), st)


def _calls_norm_fwd(L, d, dt):
    s = B.make_shape(L, d, 0, 1, 1, dt, "identity")
    m = [torch.zeros(L, d, dtype=dt, device="cuda") for _ in range(2)]
    v = [torch.ones(d, device="cuda"), torch.empty(L, device="cuda"), torch.empty(L, device="cuda")]
    x, y, w, mean, rstd = (t.data_ptr() for t in m + v)
    return (m, v), lambda st: B.moeblaze_layernorm_forward(s, x, None, w, None, 1e-5, None, y, mean, rstd, st)


def _calls_balance(L, E, K):
    s = B.make_shape(L, 1, 0, E, K, F32, "identity")
    t = [torch.zeros(L, E, device="cuda"), torch.zeros(L, K, dtype=torch.int32, device="cuda"),
         torch.empty(2, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(L, device="cuda"),
         torch.empty(B.moeblaze_balance_workspace_bytes(s), dtype=torch.uint8, device="cuda")]
    lg, ids, lo, c, lse, ws = (v.data_ptr() for v in t)
    return t, lambda st: B.moeblaze_balance_forward(s, lg, ids, None, lo, c, lse, ws, t[5].numel(), st)


def _calls_router(L, d):
    s = B.make_shape(L, d, 128, 8, 2, F32, "identity")
    t = [torch.zeros(L, d, device="cuda"), torch.zeros(d, 8, device="cuda"),
         torch.empty(L, 2, dtype=torch.int32, device="cuda"), torch.empty(L, 2, device="cuda")]
    x, Wr, ids, gates = (v.data_ptr() for v in t)
    return t, lambda st: B.moeblaze_router_forward(s, x, Wr, None, ids, gates, st)


def _calls_dispatch(L, E):
    s = B.make_shape(L, 128, 0, E, 8, F32, "identity")
    bufs = B.alloc_dispatch(s)
    ids = (torch.arange(8, dtype=torch.int32, device="cuda") + torch.zeros(L, 1, dtype=torch.int32, device="cuda")).contiguous()
    d = bufs.struct()
    return (bufs, ids), lambda st: B.moeblaze_dispatch_build(s, ids.data_ptr(), d, bufs.ws.data_ptr(), bufs.ws.numel(),
                                                             False, st)


@pytest.mark.parametrize("make,shapes", [
    (_calls_int4, [(8, 128, 256), (8, 1024, 256)]),
    (_calls_norm_bwd, [(64, 4200, BF16), (64, 5120, BF16)]),
    (_calls_norm_bwd, [(64, 520, F32), (64, 4992, F32)]),
    (_calls_norm_fwd, [(64, 513, BF16), (64, 8001, BF16)]),
    (_calls_balance, [(64, 384, 2), (64, 512, 2)]),
    (_calls_router, [(64, 1024), (64, 4096)]),
    (_calls_dispatch, [(64, 400), (64, 512)]),
], ids=["int4", "norm_backward_bf16", "norm_backward_f32", "norm_forward", "balance", "router", "dispatch"])
def test_threads_on_different_shapes(make, shapes):
    """Host threads that run one kernel on different shapes, each on its own stream: the shared memory that one call
    asks for is not taken from another."""
    jobs = [make(*shapes[i % 2]) for i in range(4)]
    bad = []
    start = threading.Barrier(len(jobs))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(ROUNDS):
            st = call(stream.cuda_stream)
            if st != B.OK:
                bad.append(st)
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(call,)) for _, call in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[:5])
