"""Row counts and bounds of any size in the 8-bit cache's calls, without a GPU."""
import os
import subprocess

import pytest

from codebook_decode_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def said(tmp_path_factory):
    build.build()
    exe = tmp_path_factory.mktemp("kv8") / "limits"
    objs = [os.path.join(build.BUILD, n + ".o") for n in ("kv8_attention", "kv8_chunk")]
    subprocess.check_call([build.NVCC] + build._flags() + [os.path.join(HERE, "kv8_limits_harness.cu")] + objs +
                          ["-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    return {line.split()[0]: int(line.split()[1]) for line in out.splitlines()}


@pytest.mark.parametrize("name,pages", [
    ("pages_of_1", 1), ("pages_of_17", 2), ("pages_by_rows", 3), ("pages_by_context", 3), ("pages_no_bounds", 16385),
    ("pages_near_the_end", 16385)])
def test_pages_that_a_sessions_rows_can_touch(said, name, pages):
    """n rows touch at most 1 + ceil((n - 1) / 16) pages."""
    assert said[name] == pages


@pytest.mark.parametrize("name,fits", [
    ("fits_8_columns", 1), ("fits_16_columns", 1), ("fits_16_columns_one_session", 1), ("fits_no_bounds", 1),
    ("fits_largest_prompt", 1), ("fits_too_many_pages", 0), ("fits_too_many_rows", 0)])
def test_attention_is_refused_only_for_what_its_sessions_can_have(said, name, fits):
    assert said[name] == fits
