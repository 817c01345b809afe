"""Bounds of the table gradient's loads in the code the compiler makes, on the
CPU: rows are read without branches, columns outside a row at its end, so the
index of every load of a row's columns has to come out of a minimum.  The
kernels' sources hold the minimum; the optimizer has dropped it before, for
widths that leave few columns in their last 512, and a load past a row's end
changes no result and faults only where the memory ends."""
import os
import re
import subprocess

import pytest

from static_codebook_lossless_amd import build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def functions(ir):
    return {m.group(1): m.group(0) for m in re.finditer(r"^define [^\n]*?@(\w+)\(.*?^}", ir, re.S | re.M)}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("ir") / "embed.ll"
    subprocess.check_call([HIPCC] + build.HIPCC_FLAGS + ["-I", build.INCLUDE, "-I", build.CSRC, "-S", "-emit-llvm",
                                                         "--cuda-device-only", "-o", str(out),
                                                         os.path.join(build.CSRC, "embed.hip")],
                          stderr=subprocess.DEVNULL)
    return functions(out.read_text())


def unheld_loads(body):
    """Loads whose address is a row's start plus an index that is no minimum.

    A row's start is dy, the gradient or the partial sums plus a product
    (``row * distance``); everything else a kernel reads has its own bounds.
    """
    defs = dict(re.findall(r"^  (%[\w.]+) = ([^\n]*)", body, re.M))
    gep = re.compile(r"getelementptr (?:inbounds )?(?:nuw )?\S+, ptr addrspace\(1\) (%[\w.]+), i64 (%[\w.]+)")

    def leaves(v, seen=()):
        """The definitions a value is chosen from, through selections."""
        d = defs.get(v, "an argument")
        m = re.match(r"phi \S+ (.*)", d) or re.match(r"select i1 \S+, i64 (%[\w.]+), i64 (%[\w.]+)", d)
        if not m or v in seen:
            return [d]
        return [x for n in re.findall(r"%[\w.]+", " ".join(m.groups()) if d.startswith("select") else
                                      " ".join(re.findall(r"\[ (\S+),", m.group(1)))) for x in leaves(n, (*seen, v))]

    found, bad = 0, []
    for address in re.findall(r"= load [^,]*, ptr addrspace\(1\) (%[\w.]+),", body):
        m = gep.match(defs.get(address, ""))
        if not m:
            continue
        start = gep.match(defs.get(m.group(1), ""))
        if not start or not re.match(r"mul ", defs.get(start.group(2), "")):
            continue
        found += 1
        if not all("@llvm.umin.i64" in d for d in leaves(m.group(2))):
            bad.append((address, defs[address], leaves(m.group(2))))
    return found, bad


@pytest.mark.parametrize("kernel", ["sum_kernel", "join_kernel", "small_kernel"])
def test_every_load_of_columns_is_held_inside_its_row(kernels, kernel):
    bodies = {n: b for n, b in kernels.items() if kernel in n}
    assert len(bodies) >= 9
    for name, body in bodies.items():
        found, bad = unheld_loads(body)
        assert found >= 8, (name, found)  # 8 rows in flight, or the loop around them
        assert not bad, (name, len(bad), found, bad[0])
