"""The training operators under several host threads and streams."""
import threading

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _in_threads(*bodies):
    errors, start = [], threading.Barrier(len(bodies))

    def run(body):
        try:
            start.wait()
            body()
        except Exception as e:      # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_norms_of_two_widths_from_two_threads():
    """One kernel, two widths, two sizes of its shared memory."""
    def body(width, rows):
        f = torch.randn(rows, width, device="cuda").to(BF16)
        w = torch.ones(width, dtype=BF16, device="cuda")
        want = None

        def loop():
            nonlocal want
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(1500):
                    n = fadam.block_norm(f, f, w, post_weight=w)
                    g = fadam.block_norm_backward(None, f, f, n.h_out, n.rstd_post, n.rstd_pre, w,
                                                  post_weight=w)
                    want = want or (n, g)
                stream.synchronize()
            for a, b in zip((*want[0], *want[1]), (*n, *g)):
                assert a is None and b is None or torch.equal(a, b)
        return loop
    loops = body(2048, 1300), body(4096, 700)
    torch.cuda.synchronize()
    _in_threads(*loops)


def test_status_waits_for_every_stream():
    """What is still running on another stream may yet give up a wait."""
    fadam.ops_status()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)        # some 0.2 s
        done = side.record_event()
    assert fadam.ops_status() == 0
    assert done.query()
