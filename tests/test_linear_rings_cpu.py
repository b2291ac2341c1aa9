"""What the play of the many-row product kernel's barrier protocol (tests/test_linear_protocol_cpu.py) leaves out of
csrc/linear_many.cu: the conversion groups' own way around the ring of copies, how it reads what its overlapped preparation writes, and
the registers that its roles share."""
import os
import re
import subprocess

import pytest

from slot_decode_window_gb300 import build
from tests.test_kv8_protocol_cpu import Bar, Machine
from tests.test_linear_protocol_cpu import SOURCE, constants


def play(tiles, stages, seed):
    """Rounded weights: copies and products go around the ring stage by stage, a conversion group by two, from its own first stage,
    with a phase that turns where its index does, as the kernel's `(st += 2) >= P::kStages` has it."""
    m, total = Machine(seed), sum(tiles)
    for i in range(stages):
        m.bars["full", i], m.bars["empty", i] = Bar(1), Bar(2)

    def copies():
        for use in range(total):
            if use >= stages:
                yield "wait", ("empty", use % stages), use // stages - 1
            m.mem["stage", use % stages] = None

            def landed(use=use):
                m.mem["stage", use % stages] = use
                m.arrive(("full", use % stages))
            yield "async", "copies", 1.0, landed

    def convert(group):
        st, turn = group, 0
        for use in range(group, total, 2):
            yield "wait", ("full", st), turn
            m.expect(("stage", st), use)
            yield "work", 1.0
            m.expect(("stage", st), use)
            yield "arrive", ("empty", st)
            st += 2
            if st >= stages:
                st, turn = group, turn + 1

    def products():
        for use in range(total):
            yield "wait", ("full", use % stages), use // stages
            yield "work", 1.0
            yield "arrive", ("empty", use % stages)

    m.run([copies(), convert(0), convert(1), products()])


def test_groups_that_keep_to_their_stages():
    assert "if ((st += 2) >= P::kStages) st = group, ph ^= 1;" in open(SOURCE).read()  # what is played here
    for tiles in ([1], [3, 1, 1, 4], [7, 9, 12], [33, 2, 18]):
        for seed in range(25):
            play(tiles, constants("bf16")["stages"], seed)


@pytest.mark.parametrize("stages", [3, 5, 7])
def test_an_odd_ring_is_found(stages):
    for seed in range(10):
        with pytest.raises(AssertionError):
            play([9, 12, 5], stages, seed)


def test_what_the_overlapped_preparation_writes_is_not_read_through_the_read_only_path():
    text = open(SOURCE).read()
    for helper in ("load4", "load16"):
        body = re.search(r"void %s\(.*?\n}\n|float4 %s\(.*?}\n" % (helper, helper), text, re.S)[0]
        assert "__ldg" not in body
    uses = [line for line in text.split("\n") if re.search(r"A\.undo_x \+ ", line)]
    assert len(uses) == 3 and all(re.search(r"load(4|16)\(A\.undo_x", line) for line in uses)


def test_registers_at_launch():
    """The roles' register shares are drawn from what a block is launched with: every variant has to be compiled with kRegs a thread
    (create refuses one that is not, as its waits for registers would never end)."""
    text = open(SOURCE).read()
    regs = int(re.search(r"kRegs = (\d+);", text)[1])
    cmd = [build.nvcc(), "-c", SOURCE, "-o", os.devnull, build.ARCH, "-O3", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
           "--expt-relaxed-constexpr", "-Xptxas", "-v"]
    out = subprocess.run(cmd, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    used = re.findall(r"entry function '\w*linear_many_kernel\w*'.*?Used (\d+) registers", out.stderr, re.S)
    assert len(used) == 2 * len(re.findall(r"setup<\w+, true>\(\)", text)) and set(used) == {str(regs)}
