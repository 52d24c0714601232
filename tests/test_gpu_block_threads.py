"""Block operators called by several host threads."""
import ctypes
import threading
import time

import pytest
import torch

from test_gpu_blocks import gen, norm_inputs, nss, randn, same_bits      # noqa: F401  (nss is a fixture)

pytestmark = pytest.mark.gpu


def _together(*work):
    """Runs the functions in threads of their own; re-raises what one of them raised."""
    start, errors = threading.Barrier(len(work)), []

    def run(f):
        try:
            start.wait()
            f()
        except BaseException as e:                           # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


def test_c_calls_of_one_kernel_at_two_sizes(nss):
    """Rows whose lengths give one kernel different amounts of shared memory, at the same time: every call is accepted."""
    from newton_schulz_stacked_gb300 import _binding as b
    lib = b.load()

    def norm_calls(cols):
        rows = 8
        x, y = torch.randn(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
        dy = torch.randn(rows, cols, device="cuda")
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        need = ctypes.c_size_t()
        b.check("mb_layer_norm_workspace_bytes", lib.mb_layer_norm_workspace_bytes(rows, cols, ctypes.byref(need)))
        ws, grads = torch.empty(need.value, device="cuda", dtype=torch.uint8), torch.empty(2, cols, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (dy.data_ptr(), cols, x.data_ptr(), cols, b.MB_F32, None, b.MB_F32, mean.data_ptr(), rstd.data_ptr(),
                y.data_ptr(), cols, grads[0].data_ptr(), grads[1].data_ptr(), rows, cols, ws.data_ptr(), need.value,
                stream.cuda_stream)

        def run():
            torch.cuda.set_device(0)
            for _ in range(3000):
                b.check("mb_layer_norm_backward", lib.mb_layer_norm_backward(*args))
            stream.synchronize()
            keep = (x, y, dy, mean, rstd, ws, grads)
            assert keep
        return run

    def router_calls(experts, k):
        logits = torch.randn(64, experts, device="cuda")
        index, gate = torch.empty(64, k, device="cuda", dtype=torch.int32), torch.empty(64, k, device="cuda")
        counts = torch.empty(experts, device="cuda", dtype=torch.int32)
        loss, used = torch.empty(1, device="cuda"), torch.empty(1, device="cuda", dtype=torch.int32)
        need = ctypes.c_size_t()
        b.check("mb_router_workspace_bytes", lib.mb_router_workspace_bytes(64, experts, ctypes.byref(need)))
        ws = torch.empty(max(need.value, 1), device="cuda", dtype=torch.uint8)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (logits.data_ptr(), experts, b.MB_F32, None, 64, experts, k, 0, index.data_ptr(), gate.data_ptr(),
                counts.data_ptr(), loss.data_ptr(), used.data_ptr(), ws.data_ptr(), need.value, stream.cuda_stream)

        def run():
            torch.cuda.set_device(0)
            for _ in range(3000):
                b.check("mb_router", lib.mb_router(*args))
            stream.synchronize()
            keep = (logits, index, gate, counts, loss, used, ws)
            assert keep
        return run

    _together(norm_calls(8192), norm_calls(4608), norm_calls(2568))
    _together(router_calls(1024, 8), router_calls(640, 8))
    _together(norm_calls(8177), norm_calls(6001))


def test_python_calls_side_by_side(nss):
    """Each thread on its own stream gets the bits that it gets alone."""
    x, w, b, dy = norm_inputs(1, 60, 4608, torch.bfloat16, torch.float32)
    x2, w2, b2, dy2 = norm_inputs(2, 60, 8192, torch.bfloat16, torch.float32)
    logits = randn(gen(3), 400, 256)
    _, mean, rstd = nss.mb_layer_norm(x, w, b)
    _, mean2, rstd2 = nss.mb_layer_norm(x2, w2, b2)
    calls = [lambda **s: nss.mb_layer_norm_backward(dy, x, mean, rstd, w, **s),
             lambda **s: nss.mb_layer_norm_backward(dy2, x2, mean2, rstd2, w2, **s),
             lambda **s: nss.mb_router(logits, 8, **s)]
    want = [c() for c in calls]
    torch.cuda.synchronize()

    def worker(call, ref):
        stream = torch.cuda.Stream()

        def run():
            for _ in range(200):
                got = call(stream=stream)
                stream.synchronize()
                for a, c in zip(got, ref):
                    same_bits(a, c, "beside other threads")
        return run

    _together(*(worker(c, r) for c, r in zip(calls, want)))


def test_other_threads_run_while_a_call_waits(nss):
    """A stream takes a limited number of launches; the call that finds it full waits, and only its own thread with it."""
    x, w, b, _ = norm_inputs(4, 4, 64, torch.float32, torch.float32)
    y, mean, rstd = nss.mb_layer_norm(x, w, b)
    torch.cuda.synchronize()
    stop, longest = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            longest[0] = max(longest[0], now - last)
            last = now

    ticker = threading.Thread(target=tick)
    ticker.start()
    time.sleep(0.05)
    longest[0], waited = 0.0, 0.0
    try:
        torch.cuda._sleep(2_000_000_000)                     # about a second of the GPU's clock, ahead of the calls
        for _ in range(20000):
            t = time.perf_counter()
            nss.mb_layer_norm(x, w, b, y=y, mean=mean, rstd=rstd)
            waited = max(waited, time.perf_counter() - t)
            if waited > 0.2:
                break
    finally:
        stop.set()
        ticker.join()
        torch.cuda.synchronize()
    assert waited > 0.2, "no call had to wait"
    assert longest[0] < 0.5 * waited, f"another thread stood still for {longest[0]:.3f} s of {waited:.3f}"
