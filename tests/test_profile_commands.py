"""Every ncu command that the repository's files suggest leaves the GPU's clocks alone (CPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def texts():
    for top in ("", "examples", "gated_delta_rule_33_gb300", "oracle", "perf", "profiles", "tests"):
        for name in sorted(os.listdir(os.path.join(ROOT, top))):
            if name.endswith((".py", ".md", ".sh", ".cu", ".cuh")) and name != os.path.basename(__file__):
                yield os.path.join(top, name)


def test_ncu_commands_do_not_lock_the_clocks():
    found = 0
    for path in texts():
        for m in re.finditer(r"\bncu -[^\n]*(?:\n[^\n]*)?", open(os.path.join(ROOT, path)).read()):
            found += 1
            assert "--clock-control none" in m.group(0), (path, m.group(0))
    assert found > 0
