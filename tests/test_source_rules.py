"""Rules of the kernels' memory model that no run can show, checked on the sources."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_quantized_moe_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    text = re.sub(r"//.*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    return re.sub(r"__(?:launch_bounds|align)__\s*\((?:[^()]|\([^()]*\))*\)", "", text)


def body(text, start):
    """The braces' contents that follow position `start`."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError("unbalanced braces")


def functions(name):
    """{name: body} of the device functions and kernels of a file."""
    text = source(name)
    found = re.finditer(r"(?:__global__|__device__)[^;{}=]*?\b(\w+)\s*\(", text)
    return {m.group(1): body(text, m.end()) for m in found}


def test_what_an_overlapped_kernel_writes_is_not_read_as_constant():
    """__ldg promises that the data stays as it is while the kernel lives; a kernel that is launched
    to overlap lives before grid_wait_previous(), while the one before it writes."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        for fn, code in functions(name).items():
            for after in code.split("grid_wait_previous();")[1:]:
                seen += 1
                assert "__ldg(" not in after, f"{name}: {fn}"
    assert seen >= 2


def test_logits_that_the_gradient_may_overwrite_are_not_read_as_constant():
    """moe_router_balance_backward's dlogits may be its logits: the kernel that writes them must not
    promise, by __ldg, that they stay as they are."""
    code = functions("balance.cu")
    assert "load4" in code["balance_grad_kernel"]
    assert "__ldg(" not in code["load4"]
    assert not re.search(r"__ldg\(\s*(?:logits|dlogits)", code["balance_grad_kernel"])


def test_tensor_memory_is_written_behind_a_fence():
    """A warp that waits on a barrier and then touches tensor memory that other threads' tcgen05
    operations used orders the two by tcgen05.fence::after_thread_sync (tc_fence_after)."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        for fn, code in functions(name).items():
            # a wait's condition, its way out, and what follows up to the first operation
            for m in re.finditer(r"(?:wait_uniform|wait_warp|mbar_wait_bounded\w*)\s*\(", code):
                rest = code[m.end():]
                op = re.search(r"\b(?:tmem_st_\w+|tmem_ld_\w+|mma_\w+|tc_mma\w*)\s*\(", rest)
                again = re.search(r"(?:wait_uniform|wait_warp|mbar_wait_bounded\w*)\s*\(", rest)
                if not op or (again and again.start() < op.start()) or rest[op.start():].startswith("mma_commit"):
                    continue
                seen += 1
                assert "tc_fence_after()" in rest[:op.start()], f"{name}: {fn}: {op.group(0)}"
    assert seen >= 4
