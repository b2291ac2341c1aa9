"""How the many-row product kernel (csrc/linear_many.cu) reads what its overlapped preparation writes."""
import re

from tests.test_linear_protocol_cpu import SOURCE


def test_what_the_overlapped_preparation_writes_is_not_read_through_the_read_only_path():
    text = open(SOURCE).read()
    for helper in ("load4", "load16"):
        body = re.search(r"void %s\(.*?\n}\n|float4 %s\(.*?}\n" % (helper, helper), text, re.S)[0]
        assert "__ldg" not in body
    uses = [line for line in text.split("\n") if re.search(r"A\.undo_x \+ ", line)]
    assert len(uses) == 3 and all(re.search(r"load(4|16)\(A\.undo_x", line) for line in uses)
