"""What the device sources keep to, read as text (nothing here needs a GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routing_grouped_expert_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")) +
                 glob.glob(os.path.join(ROOT, "include", "*.h")))


def asm_statements(src):
    """Every asm statement, its string literals joined."""
    for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", src, flags=re.S):
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))


def kernel_body(name, path):
    """The body of a __global__ function, comments taken out."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
    start = src.index("{", src.index(name + "("))
    depth = 0
    for i in range(start, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[start:i]
    raise AssertionError(f"{name}: no end")


def test_weight_gradients_read_nothing_before_it_is_handed_over():
    """The kernel starts while the one before it runs.  Starting early makes no
    writes visible: both of its ways to wait come before the first read of the
    plan, the masks and Z."""
    body = kernel_body("adapter_wgrad_kernel", "adapter.cu")
    first = min(body.index(what) for what in ("plan_of(", "a.masks", "load_2d(", "load_3d("))
    assert "if (a.call == 0) pdl_wait();" in body[:first]
    assert "take_over(a.status, a.call)" in body[:first]
    # and expand hands over after its own wait, in both of its forms
    for name in ("adapter_expand_split_kernel", "adapter_expand_kernel"):
        expand = kernel_body(name, "adapter.cu")
        at = expand.index("hand_over(a.status, a.call)")
        assert "pdl_wait();" in expand[:at] and "pdl_trigger();" not in expand[:at]


def test_every_copy_lands_in_one_cta():
    """The library serves several GPUs as well as one, so no tensor or bulk copy
    is sent to more than one CTA of a cluster: each CTA loads what it stages
    (a pair shares operands through its MMAs)."""
    seen = 0
    for path in SOURCES:
        for text in asm_statements(open(path).read()):
            if "cp.async.bulk" in text:
                seen += 1
                assert "multicast" not in text, (os.path.basename(path), text)
    assert seen >= 10


def test_no_bounded_wait_runs_while_an_earlier_launch_does():
    """A wait that depends on the launch before this one starts after that launch
    has ended: a low-rank product of more than a second is no time-out."""
    body = kernel_body("adapter_expand_kernel", "adapter.cu")
    epilogue = body[body.index("else if (warp >= 3)"):]
    assert "pdl_wait();" in epilogue[:epilogue.index("sh->acc_full")]
    guard = body[body.index("else if (warp == 2)"):body.index("else if (warp >= 3)")]
    assert "pdl_wait();" in guard[:guard.index("sh->loaded")]
    split = kernel_body("adapter_expand_split_kernel", "adapter.cu")
    split = split[:split.index("mbar_wait(&sh->loaded")]
    assert "pdl_wait();" in split[split.rindex("else {"):]
