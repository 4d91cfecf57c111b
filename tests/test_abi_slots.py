"""CPU checks of inverse slot maps: the mark for a row without a slot."""
import os
import re
import struct

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_slot_is_one_byte_repeated_and_no_slot_number():
    # what a memset of bytes writes, negative, and not the -1 that a map's dummies hold
    b = pytest.importorskip("ball_tree_sparse_b200")
    assert struct.pack("<i", b.BT_NO_SLOT) == b"\x80" * 4
    assert b.BT_NO_SLOT < -1
    text = open(os.path.join(ROOT, "include", "bts.h")).read()
    assert int(re.search(r"#define\s+BT_NO_SLOT\s+\((-\d+)\)", text).group(1)) == b.BT_NO_SLOT
