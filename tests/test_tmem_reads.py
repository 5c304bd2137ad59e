"""Values read out of tensor memory are there only after the wait for the reads.
To the compiler the two are instructions without a connection, so every wait names
the registers that it waits for: none may be used, or moved, ahead of it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_46_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


@pytest.mark.parametrize("name", SOURCES)
def test_every_wait_names_what_was_read(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    waits = re.findall(r"tmem_ld_wait\(([^)]*)\)", text)
    assert all(w.strip() for w in waits), f"{name}: a wait that names no registers"
    assert bool(waits) == bool(re.search(r"ptx::tmem_ld(8|16|32|_tiles4)\(", text))
