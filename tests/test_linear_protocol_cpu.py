"""The barrier protocol of the many-row product kernel (csrc/linear_many.cu), played on the CPU with random delays.

As in tests/test_kv8_protocol_cpu.py, whose machine this is: every role waits, arrives, reads and writes in the kernel's
order, ring sizes and arrival counts are read from the source, and a wait that could pass on another phase than its own, a
stage of copies, a stage of weights or a set of accumulators that is not what its reader expects, at the start or at the
end of the reading, and a role that never ends are errors.
"""
import os
import re

import pytest

from tests.test_kv8_protocol_cpu import Bar, Machine

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "slot_decode_window_gb300", "csrc",
                      "linear_many.cu")


def constants(kind):
    """kind: f32, f16 or bf16."""
    text = open(SOURCE).read()
    sums = kind != "bf16"
    c = {n: int(v) for n, v in re.findall(r"(kConvert|kResults|kChunk) = (\d+)", text)}
    a, b = re.search(r"kStages = DT == kBF16 \? (\d) : (\d);", text).groups()
    c["stages"] = int(b if sums else a)
    a, b = re.search(r"kUnits = kSums \? (\d) : (\d);", text).groups()
    c["units"] = int(a if sums else b)
    a, b = re.search(r"kSets = DT == kF32 \? (\d) : (\d);", text).groups()
    c["sets"] = int(a if kind == "f32" else b)
    env = dict(c, sums=sums)
    c["count"] = {}
    for name, n in re.findall(r"mbar_init\(&?(\w+)(?:\[i\])?, ([^;]+?)\)(?=[,;])", text):
        n = re.sub(r"\(P::kSums \? (\w+) : ([\w /]+)\)", r"((\1) if sums else (\2))", n).replace("/", "//")
        c["count"][name] = eval(n, {}, env)
    return c


def play(tiles, kind, seed, change=None):
    """tiles: steps of each tile of a CTA (its sums' among them).  change: edits of the constants."""
    c = constants(kind)
    if change:
        change(c)
    m, sums, S = Machine(seed), kind != "bf16", c["stages"]
    sets, chunk_steps = c["sets"], c["kChunk"] if kind == "f32" else 1 << 30
    half_warps = c["kConvert"] // 2
    for name, n in dict(full=S, empty=S, a_full=c["units"], a_empty=c["units"], d_full=sets, d_empty=sets).items():
        for i in range(n):
            m.bars[name, i] = Bar(c["count"][name])
    total = sum(tiles)

    def copies():
        for use in range(total):
            st = use % S
            if use >= S:
                yield "wait", ("empty", st), use // S - 1
            m.mem["stage", st] = None  # being written

            def landed(use=use, st=st):
                m.mem["stage", st] = use
                m.arrive(("full", st))
            yield "async", "copies", 1.0, landed

    def convert(group, w):
        own = range(total) if sums else range(group, total, 2)
        for n, use in enumerate(own):
            st = use % S
            yield "wait", ("full", st), use // S
            m.expect(("stage", st), use)
            yield "work", 2.0
            m.expect(("stage", st), use)
            slot, turn = ((n & 1) * 2 + group, n // 2) if sums else (group, n)
            if turn >= 1:
                yield "wait", ("a_empty", slot), turn - 1
            m.mem["weights", slot, w] = None
            yield "work", 0.5
            m.mem["weights", slot, w] = use
            yield "arrive", ("a_full", slot)
            yield "arrive", ("empty", st)

    def products(half):
        use = chunk = 0
        for steps in tiles:
            for i in range(steps):
                at_set = chunk % sets
                if i % chunk_steps == 0:
                    if chunk >= sets:
                        yield "wait", ("d_empty", at_set), chunk // sets - 1
                    m.mem["sums", at_set, half] = None
                parts = c["units"] // 2
                for u in range(parts):
                    slot = (use & 1) * parts + u
                    yield "wait", ("a_full", slot), use // 2

                    def check(use=use, slot=slot):
                        m.expect(("stage", use % S), use)
                        for w in range(half_warps):  # half of the warps of a group write each half
                            if w // 4 == half:
                                m.expect(("weights", slot, w), use)
                    check()

                    def done(check=check, slot=slot):
                        check()
                        m.arrive(("a_empty", slot))
                    yield "async", "tensor", 1.0, done
                last = i == steps - 1 or i % chunk_steps == chunk_steps - 1

                def step_done(use=use, at_set=at_set, chunk=chunk, last=last):
                    m.arrive(("empty", use % S))
                    if last:
                        m.mem["sums", at_set, half] = chunk
                        m.arrive(("d_full", at_set))
                yield "async", "tensor", 0.01, step_done
                use += 1
                chunk += last

    def results():
        chunk = 0
        for steps in tiles:
            for _ in range(-(-steps // min(chunk_steps, steps))):
                at_set = chunk % sets
                yield "wait", ("d_full", at_set), chunk // sets
                for half in range(2):
                    m.expect(("sums", at_set, half), chunk)
                yield "work", 3.0
                for half in range(2):
                    m.expect(("sums", at_set, half), chunk)
                yield "arrive", ("d_empty", at_set)
                chunk += 1

    roles = [copies()] + [convert(g, w) for g in range(2) for w in range(half_warps)] + [products(h) for h in range(2)] + \
        [results() for _ in range(c["kResults"])]
    m.run(roles)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tiles", [[1], [2], [3, 1, 1, 4], [7, 9, 12], [1] * 9, [33, 2, 18]])
def test_protocol(kind, tiles):
    for seed in range(25):
        play(tiles, kind, seed)


def test_counts_are_read():
    c = constants("bf16")
    assert c["count"] == dict(full=1, empty=10, a_full=8, a_empty=2, d_full=2, d_empty=8, last=2) and c["stages"] == 6
    assert constants("f32")["count"]["empty"] == 18 and constants("f32")["units"] == 4


@pytest.mark.parametrize("kind,name", [("f32", "empty"), ("bf16", "empty"), ("f32", "a_full"), ("bf16", "a_full"), ("f16", "a_empty"),
                                       ("f32", "d_empty"), ("bf16", "d_empty"), ("f32", "d_full")])
def test_a_barrier_that_counts_one_too_few_is_found(kind, name):
    def change(c):
        c["count"][name] -= 1
    with pytest.raises(AssertionError):
        for seed in range(40):
            play([9, 12, 5], kind, seed, change)


def test_an_odd_number_of_stages_is_found_where_groups_keep_to_theirs():
    """(bf16) With an odd ring a group would skip phases of the stages that it waits on."""
    text = open(SOURCE).read()
    assert "kStages % 2 == 0" in text and "(st += 2) >= P::kStages" in text
