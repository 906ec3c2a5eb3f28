"""The 8-bit cache's error word: read and cleared in one, while other threads and streams work."""
import threading
import time

import numpy as np
import pytest
import torch
from test_gpu_kv8 import Rig, bits, dev

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu


def test_an_error_after_a_status_call_is_there_for_the_next():
    """A thread keeps the default stream busy (0.2 ms at a time, never more than two in line). A call that another stream runs after
    qtts_kv8_status has returned reports an error; what that status call still had to clear must not take it along."""
    with Rig(2, 64) as r:
        k, w = bits(r.rows(2)[0]), r.nkv * r.d
        past = dev(np.array([64, 64], np.int32))  # past the block table
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        done = threading.Event()

        def busy():
            last = None
            while not done.is_set():
                torch.cuda._sleep(400000)
                now = torch.cuda.Event()
                now.record()
                while last and not last.query():
                    time.sleep(0)
                last = now

        t = threading.Thread(target=busy)
        t.start()
        try:
            seen = []
            for _ in range(300):
                qtts.qtts_kv8_append(r.c, 0, 2, 2, 1, None, past, r.bt, r.stride, k, w, k, w, side)
                side.synchronize()
                seen.append(r.status()[1])
        finally:
            done.set()
            t.join()
        torch.cuda.synchronize()
        assert seen == [qtts.QTTS_DEV_BAD_SESSION] * 300
        assert r.status() == (0, 0)
