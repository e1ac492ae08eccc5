"""The documented examples, to be run as they stand."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def block(text):
    """The one Python example that has `text`."""
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S) if text in b]
    assert len(found) == 1, len(found)
    return found[0]
