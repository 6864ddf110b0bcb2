"""Every macro that a HIP source or header of the package defines is used somewhere in them: a switch of
a tuning session does not stay behind."""
import glob
import os
import re

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_sharded_mixed_amd")
FILES = sorted(glob.glob(os.path.join(PKG, "*", "*.hip")) + glob.glob(os.path.join(PKG, "*", "*.h")))
TEXT = {f: open(f).read() for f in FILES}


@pytest.mark.parametrize("path", FILES, ids=lambda f: os.path.basename(f))
def test_macros_are_used(path):
    for name in re.findall(r"^\s*#\s*define\s+(\w+)", TEXT[path], flags=re.M):
        uses = sum(len(re.findall(rf"\b{name}\b", line)) for t in TEXT.values() for line in t.splitlines()
                   if not re.match(rf"\s*#\s*(define|ifndef|ifdef|undef)\s+{name}\b", line))
        assert uses > 0, f"{name} is defined in {os.path.basename(path)} and read by nothing"
