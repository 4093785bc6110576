"""What the paged-cache calls promise beyond their results, as far as it shows
without a GPU: the sources, the argument checks, the binding."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_12_gb300", "csrc")


def _code(path):
    """A source file without its comments."""
    text = open(path, encoding="utf-8").read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)


def test_no_copy_or_commit_reaches_another_cta():
    # the library is loaded by every replica of a multi-GPU job, and a cache may be
    # any device pointer: a TMA copy goes to the CTA that issues it only
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        assert "multicast" not in _code(path), path
