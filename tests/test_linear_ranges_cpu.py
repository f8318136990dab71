"""Which tokens of a prompt cut along time each segment takes in and which it
zeroes, from the kernels' own index arithmetic compiled for the host."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def stop(tmp_path_factory):
    from linear_attention_recurrent_lq_b200 import build
    out = str(tmp_path_factory.mktemp("ranges") / "ranges.so")
    subprocess.run([os.environ.get("NVCC", "nvcc"), *build.NVCC_FLAGS, "-shared", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(build.HERE, "csrc"), "-o", out, os.path.join(ROOT, "tests", "linear_ranges.cu")], check=True)
    return ctypes.CDLL(out).host_lin_stop


@pytest.mark.parametrize("tokens,seg_len", [(4096, 64), (4096, 112), (777, 48), (256, 256), (1000, 16)])
def test_segments_write_each_output_once(stop, tokens, seg_len):
    for length in (0, 1, seg_len - 1, seg_len, seg_len + 1, tokens // 2, tokens - 1, tokens):
        taken, zeroed = [0] * tokens, [0] * tokens
        for begin in range(0, tokens, seg_len):
            end = min(tokens, begin + seg_len)
            t = stop(1, length, begin, end)
            assert begin <= t <= end
            for i in range(begin, t):
                taken[i] += 1
            for i in range(t, end):
                zeroed[i] += 1
        assert taken == [int(i < length) for i in range(tokens)]
        assert zeroed == [int(i >= length) for i in range(tokens)]


def test_a_segment_that_does_not_run_is_zeroed_whole(stop):
    for length in (0, 40, 100, 1000):
        assert stop(0, length, 64, 128) == 64
