"""Values that lanes pass each other with v_readlane, checked in the assembly that is compiled.

A lane's register is only written where the lane is active: a copy that the compiler makes
inside a loop that lanes leave at different turns lacks the values of those that have left.
So no kernel of rows by group may read another lane's register inside such a loop; what is
read there is passed on before it.  (Registers that v_writelane fills hold scalar registers
that were put aside: both instructions go by lane number, active or not.)
"""
import os
import re
import subprocess

import pytest

from two_sided_gptq_amd import build

SOURCE = os.path.join(build.CSRC, "groups.hip")


class Block:
    def __init__(self):
        self.code, self.next, self.before = [], [], []


def blocks_of(body):
    """A function's blocks, the first one its entry."""
    blocks, named = [Block()], {}
    for line in body.split("\n"):
        line = re.sub(r"\s+", " ", line.split(";")[0]).strip()
        label = re.match(r"(\.L\w+):", line)
        if label:
            if blocks[-1].code:
                blocks.append(Block())
            named[label.group(1)] = blocks[-1]
        elif line and not line.startswith((".", "_")):
            blocks[-1].code.append(line)
            if line.startswith(("s_branch", "s_cbranch", "s_endpgm")):
                blocks.append(Block())
    blocks = [b for b in blocks if b.code] + [b for b in named.values() if not b.code]
    for i, b in enumerate(blocks):
        last = b.code[-1] if b.code else ""
        if last.startswith(("s_branch", "s_cbranch")):
            b.next.append(named[last.split()[1]])
        if not last.startswith(("s_branch", "s_endpgm")) and i + 1 < len(blocks):
            b.next.append(blocks[i + 1])
        for n in b.next:
            n.before.append(b)
    return blocks


def reached(start, without):
    seen, todo = set(), [start]
    while todo:
        b = todo.pop()
        if b not in seen and b is not without:
            seen.add(b)
            todo += b.next
    return seen


def loops_of(blocks):
    """The natural loops, as sets of blocks."""
    loops = {}
    all_of = reached(blocks[0], None)
    for head in {n for b in all_of for n in b.next}:
        outside = reached(blocks[0], head)
        for latch in head.before:
            if latch not in all_of or latch in outside:
                continue  # not every way to it leads over the head
            loop, todo = loops.setdefault(head, {head}), [latch]
            while todo:
                b = todo.pop()
                if b not in loop:
                    loop.add(b)
                    todo += [p for p in b.before if p in all_of]
    return list(loops.values())


def reads_of_lanes(body):
    """(loops that lanes leave one by one, v_readlane in them)."""
    blocks = blocks_of(body)
    aside = {line.split()[1].rstrip(",") for b in blocks for line in b.code if line.startswith("v_writelane")}
    loops = loops_of(blocks)
    found, reads = [], []
    for b in blocks:
        if any(line.startswith("s_andn2_b64 exec, exec,") for line in b.code):
            around = [loop for loop in loops if b in loop]
            if around:
                found.append(min(around, key=len))
    for loop in found:
        reads += [line for b in loop for line in b.code
                  if line.startswith("v_readlane") and line.split()[2].rstrip(",") not in aside]
    return len(found), reads


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc is missing")
    out = str(tmp_path_factory.mktemp("assembly") / "groups.s")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    subprocess.run([build.hipcc(), *flags, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "--cuda-device-only", SOURCE, "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        return {m.group(1): m.group(2) for m in re.finditer(r"^(_ZN6bakron\w+):[^\n]*\n(.*?)^\.Lfunc_end", f.read(), re.S | re.M)}


def test_no_lane_is_read_where_others_may_have_left(kernels):
    gradients = [name for name in kernels if "combine_grad_kernel" in name]
    assert len(gradients) == 18
    bad = {}
    for name, body in kernels.items():
        count, reads = reads_of_lanes(body)
        assert count or name not in gradients  # the loop over columns was found
        if reads:
            bad[name] = reads
    assert not bad, "\n".join(f"{name}: {len(reads)}, {reads[0]}" for name, reads in bad.items())


def test_the_check_finds_one():
    loop = "s_mov_b64 s[0:1], 0\n.L1:\nv_readlane_b32 s4, v3, 1\nv_cmp_lt_u32_e32 vcc, v1, v2\ns_or_b64 s[0:1], vcc, s[0:1]\n" \
           "s_andn2_b64 exec, exec, s[0:1]\ns_cbranch_execnz .L1\ns_endpgm\n"
    assert reads_of_lanes(loop)[1] == ["v_readlane_b32 s4, v3, 1"]
    assert reads_of_lanes(loop.replace("v_readlane", "v_writelane_b32 v3, s4, 0\nv_readlane"))[1] == []
    before = "v_readlane_b32 s4, v3, 1\n" + loop.replace("v_readlane_b32 s4, v3, 1\n", "")
    assert reads_of_lanes(before) == (1, [])
