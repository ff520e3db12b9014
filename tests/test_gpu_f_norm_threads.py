"""Layer norm called by several threads at once, in a process where each kernel is launched for the first time."""
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

CHILD = textwrap.dedent("""
    import threading

    import torch

    import nvfp4_block_scaled_13_b200 as nv

    # widths that one kernel instance takes with different sizes of its ring, the smallest and the largest among them
    FAMILIES = [(520, 1000, 1536, 2048), (2056, 4096, 6000, 8192), (8200, 12000, 16384), (10248, 12000, 16384), (2057, 4097, 6001, 8191),
                (521, 1001, 1537, 2047), (10243, 12001, 16383)]
    failed, answers = [], {}

    def work(x, dy, key, start):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            with torch.cuda.stream(stream):
                for _ in range(3):
                    r = nv.layer_norm_forward(x)
                    answers[key] = (r.y, *nv.layer_norm_backward(dy, x, None, r.mean, r.rstd))
            stream.synchronize()
        except Exception as e:
            failed.append(f"{key}: {e}")

    made = {}
    for widths in FAMILIES:
        for dtype in (torch.bfloat16, torch.float32):
            for cols in widths:
                x = torch.randn(40, cols, device="cuda").to(dtype)
                made[cols, dtype] = x, (x * 1e-3).roll(1, 0).contiguous()
    torch.cuda.synchronize()
    for widths in FAMILIES:
        for dtype in (torch.bfloat16, torch.float32):
            start = threading.Barrier(2 * len(widths))
            threads = [threading.Thread(target=work, args=(*made[cols, dtype], (cols, dtype, k), start)) for cols in widths for k in range(2)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
    assert not failed, failed
    for (cols, dtype, k), got in answers.items():
        x, dy = made[cols, dtype]
        r = nv.layer_norm_forward(x)
        want = (r.y, *nv.layer_norm_backward(dy, x, None, r.mean, r.rstd))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (cols, dtype)
    print("done")
""")


def test_threads_that_call_a_kernel_first_at_once(gpu):
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]
