"""Kernels over the cache that are launched ahead of the end of the one before: a start ahead of that end orders no reads,
so each has to wait, whatever the call, before it looks at anything in memory."""
import os
import re

import pytest

from chunked_linear_attention_bounded_gb300.build import CSRC

FILES = ("bdla_cache.cu", "bdla_cache_shared.cu")
# what a call's pointers lead to
READ = re.compile(r"\b(a\.(list|n_list|q|tree|part_o|part_ml|o|lse)|c\.(pages|lens|k|v)|plan\.\w+|\*plan|table|walk\.begin)\b")


def _kernels():
    found = {}
    for name in FILES:
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in set(re.findall(r"launch_second\((\w+)", text)):
            start = re.search(r"__global__[^;{]*?\b%s\(" % kernel, text).start()
            found[kernel] = text[start:text.index("\n}\n", start)]
    return found


KERNELS = _kernels()


def test_all_are_found():
    assert set(KERNELS) == {"list_kernel", "cached_kernel", "combine_kernel", "shared_wide_kernel", "shared_join_kernel"}


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_the_wait_comes_before_every_read(kernel):
    lines = KERNELS[kernel].split("\n")
    lines = [x for x in lines if x.strip()]
    # a wait on every way through: at the function's own level, or of the form that is launched so (LIST)
    waits = [i for i, x in enumerate(lines) if re.fullmatch(r"    (attn::)?wait_for_previous\(\);\s*", x) or
             (re.fullmatch(r"        (attn::)?wait_for_previous\(\);\s*", x) and lines[i - 1].strip() == "if (LIST)")]
    assert waits, "no unconditional wait"
    body = lines.index("{") + 1
    before = "\n".join(lines[body:waits[0]])
    assert not READ.search(before), READ.search(before)
