"""csa_profile_next_call's events: every prof_begin of the sources is followed by one launch and its prof_end, before any
way out of the call (a hook left open would record its stop event in some later call)."""
import glob
import os
import re

from long_context_sparse_10_b200 import build


def test_every_hook_that_is_opened_is_closed_right_after_its_launch():
    seen = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        if os.path.basename(path) == "abi.cu":  # their definitions
            continue
        with open(path) as f:
            text = f.read()
        calls = [(m.start(), m.group(1)) for m in re.finditer(r"\b(prof_begin|prof_end)\(\w+\);", text)]
        assert len(calls) % 2 == 0, path
        for (a, begin), (b, end) in zip(calls[::2], calls[1::2]):
            assert (begin, end) == ("prof_begin", "prof_end"), f"{path}: {text[a:b][:200]}"
            assert "return" not in text[a:b], f"{path}: {text[a:b]}"
            seen += 1
    assert seen >= 8
