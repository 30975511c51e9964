"""The kernels' copies: every CTA copies what it reads itself, also where the
CTAs of a pair read the same page, since the library may be loaded by programs
that use several GPUs."""
import os
import re

from sequence_sharded_decode_gb300 import build


def test_no_kernel_issues_a_multicast_copy():
    found = []
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())   # adjacent string literals are one instruction
        found += [f"{name}: {m.group(0)[:80]}" for m in re.finditer(r"cp\.(async|reduce)[\w.:]*multicast[\w.:]*", text)]
        found += [f"{name}: {m.group(0)[:80]}" for m in re.finditer(r"multimem\.[\w.:]*", text)]
    assert not found
