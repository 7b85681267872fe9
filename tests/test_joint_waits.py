"""Every kernel that multiplies by assembly (test_tile_waits says why these need a
check of their waits): the tiles and the three products of a backward pass in one
launch, all of them, and no other kernel does."""
import os
import re
import subprocess

import pytest

from test_tile_waits import OBJDUMP, code_objects, hazards

BY_ASSEMBLY = ("tile_kernel", "three_kernel")
# these multiply by the compiler's own instructions, which it waits for itself
BY_COMPILER = ("stream_kernel", "down_tiled_kernel")


def kind(name):
    """Which of the kernels above a (mangled) name is of; None of another."""
    found = [k for k in BY_ASSEMBLY + BY_COMPILER if k in name]
    assert len(found) <= 1, name
    return found[0] if found else None


def functions(text):
    """(name, instructions) of objdump's listing."""
    for body in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
        name, _, rest = body.partition(">:\n")
        yield name, [ln.strip() for ln in rest.splitlines()]


def check(text, counts):
    """Adds the kernels of a listing to counts, by their kind, and checks those that are by assembly."""
    for name, lines in functions(text):
        if not any(ln.startswith("v_mfma") for ln in lines):
            continue
        which = kind(name)
        assert which is not None, f"{name}: multiplies, and no check says how it waits"
        counts[which] = counts.get(which, 0) + 1
        if which in BY_ASSEMBLY:
            bad = hazards(lines)
            assert not bad, f"{name}: {len(bad)}, first {bad[0]}"


def test_a_product_without_its_wait_is_seen_in_both():
    mfma, read = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", "v_add_f32_e32 v20, v1, v21"
    for name in BY_ASSEMBLY:
        counts = {}
        check(f"0000 <_Z2{name}E>:\n{mfma}\ns_nop 15\ns_nop 15\n{read}\n", counts)
        assert counts == {name: 1}
        with pytest.raises(AssertionError):
            check(f"0000 <_Z2{name}E>:\n{mfma}\ns_nop 15\n{read}\n", {})
    with pytest.raises(AssertionError):
        check(f"0000 <_Z2other_kernelE>:\n{mfma}\n", {})


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")
def test_every_kernel_by_assembly_has_its_waits(tmp_path):
    counts = {}
    for i, code in enumerate(code_objects()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        check(subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", str(path)], capture_output=True, text=True, check=True).stdout,
              counts)
    print(counts)
    # two types, x cut or not, the weights' gradients cut or not; the tiles of two types and of 4 bits
    assert counts["three_kernel"] == 8 and counts["tile_kernel"] >= 121
