"""Where the kernels allocate tensor memory, read from their sources.

A verify flagged GDN_VERIFY_OVERLAP takes 32 of an SM's 512 columns before it
waits for the kernel in front of it, and three such CTAs fit on an SM.  A kernel
that needs more than the other 416 columns must therefore hold them before it
lets the next kernel start: beside a CTA that allocates later, a flagged
verify's CTA and that one would each wait for the other.  (It is read, not run:
a run on a tree that breaks the rule could hang the GPU.)"""
import glob
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "speculative_decode_gated_gdn_gb300", "csrc")


def kernels():
    """(file, kernel's name, its body without comments, the file's text) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            open_at = text.index("{", m.end())
            depth, end = 0, open_at
            for end in range(open_at, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            name = re.findall(r"(\w+)\s*\(", text[m.end():open_at].replace("__launch_bounds__", ""))
            yield os.path.basename(path), name[-1] if name else "?", text[open_at:end], text


def columns(arg, text):
    name = arg.split("::")[-1].strip()
    return int(name) if name.isdigit() else int(re.search(r"\b%s = (\d+)" % name, text).group(1))


def test_large_allocations_come_before_the_trigger():
    seen = {}
    for path, name, body, text in kernels():
        m = re.search(r"tmem_alloc\(&[\w.]+,\s*([\w:]+)\)", body)
        if not m:
            continue
        cols = columns(m.group(1), text)
        seen[name] = cols
        trigger = body.find("pdl_trigger()")
        if cols > 512 - 3 * 32:
            sync = body.find("__syncthreads()", m.end())  # the allocating warp is through
            assert sync >= 0 and trigger > sync, f"{path}: {name} takes {cols} columns after it lets its dependents start"
    assert len(seen) >= 4 and min(seen.values()) == 32 and max(seen.values()) == 512, seen
