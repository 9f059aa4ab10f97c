"""What the kernels' sources must not hold, whatever the compiler makes of it."""

import glob
import os
import re

from block_diffusion_masked_gb300 import build


def _sources():
    files = [f for e in ("cu", "cuh")
             for f in sorted(glob.glob(os.path.join(build.PKG, "csrc", f"*.{e}")))]
    assert len(files) > 15
    for f in files:
        with open(f, encoding="utf-8") as fh:
            yield os.path.basename(f), re.sub(r"//[^\n]*", "", fh.read())


def test_no_loads_of_the_read_only_path():
    """Kernels are launched while the kernel before them still runs, so that memory which it
    writes is not read-only for their time: neither loads of that path, nor pointers that
    let the compiler choose it."""
    for name, text in _sources():
        assert not re.search(r"__ldg\b|__ldca\b|ld\.global(\.\w+)*\.nc\b", text), name
        assert "__restrict__" not in text, name
