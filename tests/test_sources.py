"""Rules of the kernel sources that no run can show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_group_wise_b200", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".cu")))


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _body(text, at):
    """The first braced block from `at` on."""
    i = text.index("{", text.index(")", text.index("(", at)))
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[at:j + 1]
    raise ValueError("unbalanced braces")


def _kernels(text):
    return [_body(text, m.start()) for m in re.finditer(r"__global__", text)]


@pytest.mark.parametrize("name", FILES)
def test_early_kernels_do_not_use_the_read_only_path(name):
    """A kernel that waits for the one before it (griddepcontrol.wait) may be resident while that one still writes its
    inputs, so it reads them by plain loads: no read-only load in the kernel or the helpers of its file, no
    restrict-qualified input."""
    text = _code(name)
    early = [k for k in _kernels(text) if re.search(r"\bpdl_wait\(\)", k)]
    if not early:
        return
    helpers = re.sub("|".join(re.escape(k) for k in _kernels(text)) or "$^", "", text, flags=re.S)
    for part in early + [helpers]:
        assert not re.search(r"__ldg\w*\s*\(|ld\.global(\.\w+)*\.nc", part)
    for k in early:
        assert not re.search(r"const\s[^,()]*\*\s*__restrict__", k[:k.index("{")])


@pytest.mark.parametrize("name", FILES)
def test_bounded_waits_begin_after_the_kernel_before(name):
    """A bounded wait for something that comes only once the kernel ahead has ended would count that kernel's time: in a
    kernel that waits for the one before it, that wait stands before the first bounded one."""
    for k in _kernels(_code(name)):
        early, bounded = re.search(r"\bpdl_wait\(\)", k), re.search(r"\b(mbar_wait\w*|kv4_wait)\(", k)
        if early and bounded:
            assert early.start() < bounded.start()
