"""Failing calls of the low-bit operators on several threads at once, without a GPU."""
import os
import subprocess
import threading

import pytest

from codebook_decode_gb300 import build, qtts

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_handles_message_is_one_of_those_that_were_left(tmp_path):
    build.build()
    exe = tmp_path / "threads"
    objs = [os.path.join(build.BUILD, n + ".o") for n in ("kv8_attention", "kv8_chunk")]
    subprocess.check_call([build.NVCC] + build._flags() + ["-Xcompiler", "-pthread",
                          os.path.join(HERE, "lowbit_threads_harness.cu")] + objs + ["-o", str(exe)])
    reads, torn = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert reads == 400000 and torn == 0


@pytest.mark.parametrize("calls", [
    [(lambda: qtts.qtts_w4_create(0, 64, 64), "N and K must be positive"),
     (lambda: qtts.qtts_w4_create(4, 64, 17), "group must be 32, 64 or 128")],
    [(lambda: qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 2, 96, 1e6, 16, 2, 64, 8)), "head_dim must be 64 or 128"),
     (lambda: qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 2, 64, 1e6, 16, 0, 64, 8)), "max_batch must be in 1..1024")]])
def test_a_refused_creation_tells_the_thread_that_asked(calls):
    build.build()
    wrong = []

    def run(call, text):
        for _ in range(20000):
            try:
                call()
            except qtts.QttsError as e:
                if text not in str(e):
                    wrong.append(str(e))

    threads = [threading.Thread(target=run, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, (len(wrong), wrong[0])
