"""The gated delta rule from several host threads at once, on streams of their own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.test_gpu_gdelta import backward, forward, inputs, tape_of  # noqa: E402


def test_threads_whose_calls_differ_in_size():
    """One kernel in blocks of different sizes: one team and two, four single warps and eight."""
    shapes = [(1, 64), (60, 64), (128, 64), (128, 128)]  # value heads, dv: the four forms
    data, want, wrong = [], [], []
    for n, (heads, dv) in enumerate(shapes):
        x = inputs("bf16", 130, 1, heads, 64, dv, seed=n)
        do = torch.randn(130, heads, dv, device="cuda").bfloat16()
        tape = tape_of(x, 1)
        o = forward(*x, 1, tape=tape)
        want.append([o, *backward(x, tape, do, 1).values()])
        data.append((x, do))
    torch.cuda.synchronize()
    start = threading.Barrier(len(shapes))

    def thread(n):
        x, do = data[n]
        try:
            start.wait()
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    tape = tape_of(x, 1)
                    got = [forward(*x, 1, tape=tape), *backward(x, tape, do, 1).values()]
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                    wrong.append((n, "other results"))
        except Exception as e:  # noqa: BLE001
            wrong.append((n, repr(e)))

    threads = [threading.Thread(target=thread, args=(n,)) for n in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
