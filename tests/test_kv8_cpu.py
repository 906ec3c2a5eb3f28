"""What the 8-bit cache and the 4-bit products refuse, without a GPU: the host
code's argument checks and the per-session check that the kernels run, in a
program built from their sources."""
import os
import subprocess

import pytest

from codebook_decode_gb300 import build, qtts

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def said(tmp_path_factory):
    build.build()
    exe = tmp_path_factory.mktemp("kv8") / "harness"
    objs = [os.path.join(build.BUILD, n + ".o") for n in ("kv8_attention", "kv8_chunk")]
    subprocess.check_call([build.NVCC] + build._flags() + [os.path.join(HERE, "kv8_host_harness.cu")] + objs +
                          ["-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    return {line.split(" ", 1)[0]: line.split(" ", 1)[1] for line in out.splitlines()}


def code(said, name):
    return int(said[name].split()[0])


@pytest.mark.parametrize("name", [
    "append_layer_low", "append_layer_high", "append_rows", "append_max_new", "append_stride", "append_one_each_rows",
    "append_one_each_max", "append_null_len", "append_null_table", "append_null_k", "append_null_v", "append_k_align",
    "append_k_narrow", "append_v_odd", "attend_null_q", "attend_null_out", "attend_q_narrow", "attend_out_align",
    "attend_null_work", "attend_work_align", "attend_scale_nan", "attend_scale_inf", "attend_too_much", "read_null_k",
    "read_v_align", "config_bytes"] + ["config_%d" % i for i in range(10)])
def test_bad_arguments_are_refused_with_a_message(said, name):
    assert code(said, name) == qtts.QTTS_E_INVALID
    assert len(said[name].split(" ", 1)[1]) > 8


def test_batches_outside_the_limit(said):
    assert code(said, "append_batch_0") == code(said, "append_batch_5") == qtts.QTTS_E_BATCH


def test_no_rows_are_nothing_to_do(said):
    assert code(said, "append_nothing") == qtts.QTTS_OK


def test_page_lists(said):
    assert code(said, "free_not_allocated") == code(said, "free_twice") == qtts.QTTS_E_POOL
    assert said["still_used"] == "1"  # a refused list frees nothing
    assert code(said, "alloc_too_many") == qtts.QTTS_E_POOL


def test_null_handles(said):
    assert said["null_handle"] == f"{qtts.QTTS_E_INVALID} {qtts.QTTS_E_INVALID} 0"


@pytest.mark.parametrize("name,rows,err", [
    ("session_fits", 3, 0), ("session_past_table", 0, 1), ("session_past_context", 0, 1), ("session_inactive", 0, 0),
    ("session_no_rows", 0, 0), ("session_rows_back", 0, 1), ("session_rows_past", 0, 1), ("session_rows_many", 0, 1),
    ("session_rows_negative", 0, 1), ("session_huge", 0, 1)])
def test_sessions_are_checked(said, name, rows, err):
    """rows the session takes part with, error word (QTTS_DEV_BAD_SESSION = 1)"""
    assert said[name] == f"{rows} {err}"


@pytest.mark.parametrize("N,K,group", [(0, 64, 64), (1, 0, 32), (1, 64, 16), (1, 96, 64), (1, 65, 32), (1 << 25, 64, 64),
                                       (4, 1 << 21, 128)])
def test_w4_shapes_are_refused_before_any_device_work(N, K, group):
    build.build()
    with pytest.raises(qtts.QttsError) as e:
        qtts.qtts_w4_create(N, K, group)
    assert e.value.code == qtts.QTTS_E_INVALID
