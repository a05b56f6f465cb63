"""The status word is shared by everything on a device. A recorded check of one call (a refused
update, a bad parent or page id: documented, the call carries on) is no reason for another call's
kernels to stop, and does not hide a wait that ran out.
"""

import ctypes

import pytest
import torch

import workloads
from io_aware_exact_04_gb300 import _lib, api
from test_serving_gpu import Cache, ints, normal, rows_like

pytestmark = pytest.mark.gpu

TIMEOUT, CHECK = 5, 6


def record_a_check(gpu):
    """An update that is refused (a source slot that there is not): info -1, -1, the word stays set."""
    kv = normal(2, 6, 1, 16, 64, dtype=torch.bfloat16, device=gpu)
    table, lens = ints([[0, 1], [2, -1]], gpu), ints([20, 16], gpu)
    info = api.cache_update(kv, table, lens, ints([0, 2], gpu), ints([20, 16], gpu))
    assert info.tolist() == [-1, -1]


@pytest.mark.parametrize("B,H,N,d,causal", [(1, 2, 32768, 64, True), (1, 2, 32768, 128, True), (2, 4, 8192, 64, False),
                                            (1, 8, 4096, 128, False)])
def test_a_recorded_check_stops_no_other_call(gpu, B, H, N, d, causal):
    """Long rows, whose waits outlast their first polls: the same results with the word set as with it clear."""
    x = workloads.draw(B, H, N, d, seed=d)
    q, k, v, do = (x[n].to(gpu) for n in ("q", "k", "v", "do"))

    def step():
        out = [torch.full_like(q, float("nan")) for _ in range(4)]
        o, lse = api.forward(q, k, v, causal=causal, out=out[0])
        dq, dk, dv = api.backward(q, k, v, o, do, lse, causal=causal, dq=out[1], dk=out[2], dv=out[3])
        torch.cuda.synchronize(gpu)
        return o, lse, dq, dk, dv

    api.device_status(gpu)
    want = step()
    assert api.device_status(gpu)[0] == 0
    record_a_check(gpu)
    for _ in range(3):
        got = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # the gradients sum N / 64 fp32 terms at most in an order that changes from run to run (each addition off by
        # half a step of a partial sum no larger than the terms' magnitudes together, taken as 64 of the largest
        # gradient), then round once: two roundings of neighbouring values lie a step apart at most
        for name, a, b in zip(("dq", "dk", "dv"), got[2:], want[2:]):
            a, b = a.float(), b.float()
            assert torch.isfinite(a).all(), name
            assert bool(((a - b).abs() <= 2 ** -7 * b.abs() + N * 2 ** -24 * float(b.abs().max())).all()), name
    code, detail = api.device_status(gpu)
    assert code == CHECK, detail


@pytest.mark.parametrize("d", [64, 128])
def test_a_recorded_check_stops_no_decoding(gpu, d):
    x = workloads.draw(4, 16, 1, d, seed=d, Nk=60000)
    q, k, v = (x[n].to(gpu) for n in ("q", "k", "v"))
    api.device_status(gpu)
    o, lse = api.forward_split(q, k, v, with_lse=True)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 0
    record_a_check(gpu)
    for _ in range(5):
        got, glse = api.forward_split(q, k, v, with_lse=True, out=torch.full_like(o, float("nan")))
        torch.cuda.synchronize(gpu)
        assert torch.equal(got, o) and torch.equal(glse, lse)
    assert api.device_status(gpu)[0] == CHECK


@pytest.mark.parametrize("d", [64, 128])
def test_a_timeout_replaces_a_recorded_check(gpu, monkeypatch, d):
    """In the build that leaves out a copy in every CTA: a bad page id, then the wait that runs out."""
    lib = _lib.load("libfa_withhold.so")
    monkeypatch.setattr(api, "_lib_fa", lambda: lib)
    api.device_status(gpu)
    c = Cache([4000], 1, 64, d, torch.bfloat16, gpu)
    table = c.table.clone()
    table[0, 0] = 1 << 20
    q, k, v = rows_like("plain", 1, 4, 1, d, torch.bfloat16, gpu)
    api.forward_tree(q, k, v, c.kv[0], c.kv[1], table, c.lens, ints([0, 1], gpu))
    torch.cuda.synchronize(gpu)
    code, detail = api.device_status(gpu)
    assert code == TIMEOUT and detail[0] == TIMEOUT and 60 <= detail[1] <= 72, detail
    assert api.device_status(gpu)[0] == 0


def test_a_wait_goes_on_beside_a_recorded_check(gpu):
    """A wait on a barrier that nothing arrives on runs for its whole limit (20 ms), then reports the timeout."""
    st = _lib.load("libfa_selftest.so")
    status = ints([CHECK, 46, 0, 0], gpu)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    rc = st.fa_selftest_wait_timeout(ctypes.c_void_p(status.data_ptr()), 20000,
                                     ctypes.c_void_p(torch.cuda.current_stream(gpu).cuda_stream))
    end.record()
    assert rc == 0
    torch.cuda.synchronize(gpu)
    assert status.tolist()[:2] == [TIMEOUT, 99]
    assert begin.elapsed_time(end) >= 19.0


@pytest.mark.parametrize("d", [64, 128])
def test_a_timeout_of_the_forward_replaces_a_recorded_check(gpu, monkeypatch, d):
    """As above, the check recorded by an earlier call, for the forward and the backward of equal heads."""
    lib = _lib.load("libfa_withhold.so")
    x = workloads.draw(1, 2, 512, d, seed=d)
    q, k, v, do = (x[n].to(gpu) for n in ("q", "k", "v", "do"))
    o, lse = api.forward(q, k, v)
    monkeypatch.setattr(api, "_lib_fa", lambda: lib)
    api.device_status(gpu)
    for call, sites in ((lambda: api.forward(q, k, v), range(1, 10)),
                        (lambda: api.backward(q, k, v, o, do, lse), range(20, 30))):
        api.tree_mask(ints([3], gpu), ints([0, 1], gpu), 1)  # no parent of its own index or above: recorded
        call()
        torch.cuda.synchronize(gpu)
        code, detail = api.device_status(gpu)
        assert code == TIMEOUT and detail[1] in sites, detail
        assert api.device_status(gpu)[0] == 0
    monkeypatch.undo()  # the context still works
    got, glse = api.forward(q, k, v)
    torch.cuda.synchronize(gpu)
    assert api.device_status(gpu)[0] == 0
    assert torch.equal(got, o) and torch.equal(glse, lse)


def test_the_detail_tells_checks_apart(gpu):
    """A serving call's bad offsets and a packed backward's sequence that is too long."""
    q = normal(300, 2, 64, dtype=torch.bfloat16, device=gpu)
    api.device_status(gpu)
    api.forward_prompt(q, q, q, ints([0, 200, 100], gpu))
    torch.cuda.synchronize(gpu)
    code, serving = api.device_status(gpu)
    assert code == CHECK
    x = q.transpose(0, 1).contiguous()  # [H, T, d]
    cu = ints([0, 300], gpu)
    o, lse = api.forward_varlen(x, x, x, cu, 300)
    api.backward_varlen(x, x, x, o, x, lse, cu, 200)
    torch.cuda.synchronize(gpu)
    code, packed = api.device_status(gpu)
    assert code == CHECK and packed[1] != serving[1], (packed, serving)
