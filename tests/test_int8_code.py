"""What the compiler makes of the 8-bit product kernels (no GPU needed): the properties of the
machine code that their sources count on and that no result shows."""
import os
import re
import subprocess

import pytest

from view_deformable_feature_amd import build as B


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The instructions of every kernel of i8.hip by its name."""
    out = str(tmp_path_factory.mktemp("code") / "i8.s")
    src = os.path.join(B.CSRC, "i8.hip")
    subprocess.run([B._hipcc(), *B.compile_flags(), "--offload-device-only", "-S", src, "-o", out],
                   check=True, capture_output=True)
    found, name = {}, None
    with open(out) as f:
        for line in f:
            m = re.match(r"(_ZN\w+):", line)
            if m:
                name = re.search(r"i8_[a-z]+_kernel", m.group(1)).group(0) + m.group(1)
                found[name] = []
            elif name and line.startswith("\t") and not line.startswith("\t."):
                found[name].append(line.strip())
    return found


def _products(kernels):
    names = [n for n in kernels if not n.startswith("i8_quantize")]
    assert {n.split("_kernel")[0] for n in names} == {"i8_rows", "i8_skinny", "i8_tile", "i8_big"}
    return names


def test_buffer_resources_are_scalar(kernels):
    """Row counts are whole numbers in scalar registers.  A resource built of a vector register
    would make each access a loop over its values, which reads them four at a time."""
    for name in _products(kernels):
        code = kernels[name]
        assert not any(i.startswith(("v_min_f64", "v_min_num_f64")) for i in code), name
        assert sum(i.startswith("v_readfirstlane") for i in code) < 8, name


def test_large_product_waits_for_its_fills(kernels):
    """Every barrier of the pipeline stands behind a wait for the fills of LDS and the reads from
    it, which the barrier itself does not wait for."""
    name, = (n for n in kernels if n.startswith("i8_big"))
    code = kernels[name]
    barriers = [k for k, i in enumerate(code) if i.startswith("s_barrier")]
    assert len(barriers) >= 3
    for k in barriers:
        waits = []
        for i in reversed(code[:k]):
            if not i.startswith("s_waitcnt"):
                break
            waits.append(i)
        assert any("vmcnt(0)" in i for i in waits), (name, code[k - 5:k + 1])
    # the two of the loop, between reads
    assert sum("vmcnt(0) lgkmcnt(0)" in code[k - 1] for k in barriers) >= 2
