"""Planning and release may write lengths and counts where they read them
(new_lens = context_lens, new_free = num_free): their kernels must not read these
through the read-only path, whose loads the compiler may move or repeat past the
writes. By the source, on the host; the results are in test_gpu_step_plan.py."""

import os
import re

import pytest

import paged_gqa_decode_reshape_gb300 as pg

SOURCE = os.path.join(os.path.dirname(os.path.abspath(pg.__file__)), "csrc", "step_plan.cu")


def kernels():
    """Kernels of the file: name and body up to the next one."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    parts = re.split(r"__global__ void __launch_bounds__\(\w+\) (\w+)\(", text)
    return dict(zip(parts[1::2], parts[2::2]))


@pytest.mark.parametrize("kernel", ["plan_kernel", "release_kernel"])
@pytest.mark.parametrize("name", ["ctx", "num_free"])
def test_what_may_be_written_in_place_is_not_read_as_read_only(kernel, name):
    body = kernels()[kernel]
    assert re.search(rf"\ba\.{name}\b", body)
    assert not re.findall(rf"__ld(?:g|cg|ca|cs|lu)\(\s*a\.{name}\b[^;]*", body)
    assert re.search(rf"load_once\(a\.{name}\b", body)


def test_what_a_kernel_writes_it_does_not_read_as_read_only():
    """Tables that planning writes, outputs, and the stack that release writes."""
    written = {"plan_kernel": ["bt", "new_lens", "new_free", "granted", "cu", "pos", "slots"],
               "plan_rows_kernel": ["pos", "slots"],
               "release_kernel": ["free_blocks", "new_lens", "new_free"]}
    for kernel, names in written.items():
        for name in names:
            assert not re.search(rf"__ldg\(\s*a\.{name}\b", kernels()[kernel]), (kernel, name)
