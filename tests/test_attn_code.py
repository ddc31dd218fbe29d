"""What the compiler makes of the attention kernels (no GPU needed): the properties of the
machine code that their sources count on and that no result shows."""
import os
import re
import subprocess

import pytest

from view_deformable_feature_amd import build as B


@pytest.fixture(scope="module", params=["attn_forward", "attn_grad"])
def kernels(request, tmp_path_factory):
    """The instructions of every kernel by its name."""
    out = str(tmp_path_factory.mktemp("code") / "attn.s")
    src = os.path.join(B.CSRC, request.param + ".hip")
    subprocess.run([B._hipcc(), *B.compile_flags(), "--offload-device-only", "-S", src, "-o", out],
                   check=True, capture_output=True)
    code, name = {}, None
    with open(out) as f:
        for line in f:
            m = re.match(r"(_ZN\w+):", line)
            if m:
                name = re.search(r"attn_[a-z_]+_kernel", m.group(1)).group(0) + m.group(1)
                code[name] = []
            elif name and line.startswith("\t") and not line.startswith("\t."):
                code[name].append(line.strip())
    return code


def _fills(line):
    return line.startswith("buffer_load") and line.endswith(" lds")


def _product(line):
    return line.startswith("v_mfma")


def test_buffer_resources_are_scalar(kernels):
    """A resource that may differ between lanes would make each access a loop over its values, which
    goes back while lanes are left, in every fill of a tile.  What the source itself takes from the
    first lane stands by itself, three words to a tensor's tile in each copy of the loop's body."""
    for name, code in kernels.items():
        for k in (k for k, i in enumerate(code) if _fills(i)):
            assert not any(i.startswith("s_cbranch_execnz") for i in code[k:k + 6]), (name, code[k:k + 6])
        assert sum(i.startswith("v_readfirstlane") for i in code) < 32, name


def test_every_kernel_is_looked_at(kernels):
    """The names by which the tests pick their kernels are those of all that there are: three types by
    four sizes of a head, with and without a mask, and the small ones of each type."""
    count = {}
    for name in kernels:
        kind = re.match(r"attn_[a-z_]+_kernel", name).group(0)
        count[kind] = count.get(kind, 0) + 1
    assert count in ({"attn_forward_kernel": 24, "attn_few_kernel": 12, "attn_join_kernel": 3},
                     {"attn_grad_kernel": 24, "attn_delta_kernel": 3, "attn_grad_join_kernel": 3})


def test_barriers_wait_for_fills(kernels):
    """Between a fill of LDS and the next barrier stands a wait for all that is on its way, which
    the barrier itself is none for."""
    seen = 0
    for name, code in kernels.items():
        for k in (k for k, i in enumerate(code) if i.startswith("s_barrier")):
            for i in reversed(code[:k]):
                assert not _fills(i), (name, code[k - 12:k + 1])
                if i.startswith("s_waitcnt") and "vmcnt(0)" in i:
                    seen += 1
                    break
    assert seen > 24


def test_reads_of_tiles_wait_for_fills(kernels):
    """Between a fill and a read of a tile in the few-rows form, whose waves pass no barrier, a wait
    stands too: the loop's last fill is followed by one before its branch back."""
    few = {n: c for n, c in kernels.items() if n.startswith("attn_few_kernel")}
    for name, code in few.items():
        last = max(k for k, i in enumerate(code) if _fills(i))
        after = next(k for k in range(last, len(code))
                     if code[k].startswith("s_waitcnt") and "vmcnt(0)" in code[k])
        barrier = next(k for k in range(last, len(code)) if code[k].startswith("s_barrier"))
        assert after < barrier, name


def test_results_stay_in_registers(kernels):
    """The products' results stay where they are: the kernels of 16-bit types that two workgroups
    share a compute unit for move none of them between the two kinds of registers, and what goes
    through scratch memory is a few addresses and operands, and nothing in the forward."""
    found = 0
    for name, code in kernels.items():
        spills = sum(i.startswith("scratch_") for i in code)
        assert spills <= (48 if name.startswith("attn_grad_kernel") else 0), (name, spills)
        if name.startswith(("attn_forward_kernel", "attn_grad_kernel")) and "kernelIDF16" in name:
            assert not any("accvgpr" in i for i in code), name
            found += sum(_product(i) for i in code)
    assert found > 500


def test_no_packed_binary32(kernels):
    """The compiler was told to leave out packed binary32 instructions, and it does."""
    for name, code in kernels.items():
        assert not any(re.match(r"v_pk_(add|mul|fma)_f32", i) for i in code), name
