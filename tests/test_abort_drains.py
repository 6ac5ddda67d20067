"""Every producer waits for its last copies before it leaves, not only in a CTA that has aborted by
then: another warp's wait may run out later, and a CTA must not end under its own copies. Read from
the sources (tests/test_paged_tiles_protocol.py and tests/test_paged_ring_abort.py show why)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_37_b200", "csrc")


def _drains(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    return code, len(re.findall(r"mbar_drain\(", code))


def drains_behind_the_flag(code):
    """Drains with a test of the abort flag before them in the same statement or block."""
    return [m.start() for m in re.finditer(r"mbar_drain\(", code)
            if re.search(r"if \(\*abort_flag", code[:m.start()].rpartition("}")[2])]


def test_the_reading_sees_the_forms_that_were_once_there():
    for old in ("if (*abort_flag)\n for (int t = a; t < b; ++t)\n if (!IS_K || t != w) mbar_drain(&f[t], 0);",
                "if (*abort_flag && lane == 0) {\n for (int t = 0; t < k; ++t) mbar_drain(&f[t], 1);",
                "if (*abort_flag) {\n mbar_drain(q_full, 0u);\n for (;;) mbar_drain(&k, 0u); }"):
        assert drains_behind_the_flag("x; } " + old)


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and _drains(f)[1]))
def test_no_drain_is_behind_the_abort_flag(name):
    code, n = _drains(name)
    assert n and not drains_behind_the_flag(code)
