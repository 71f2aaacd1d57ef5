"""The order in which the compiled router publishes partial loads and parts of the
loss: a wavefront's stores have arrived before the barrier, or the count, that lets
another workgroup read them."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    """{function: instructions} of the router's kernels of the library built here."""
    import gradient_aggregation_amd as ga
    if not os.path.exists(ga.LIB_PATH):
        from gradient_aggregation_amd import build
        build.build()
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    at = tmp_path_factory.mktemp("objects")
    shutil.copy(ga.LIB_PATH, at / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=at, check=True, capture_output=True)
    found = {}
    for f in sorted(at.glob("lib.so.*gfx950*")):
        if b"k_load_end" not in f.read_bytes():
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], check=True, capture_output=True, text=True).stdout
        for block in re.split(r"\n(?=[0-9a-f]+ <)", text):
            name = re.match(r"[0-9a-f]+ <(\S+)>:", block)
            if name and re.search("k_load_end|k_routeI", name.group(1)):
                found[name.group(1)] = [x.split("//")[0].strip() for x in block.split("\n")[1:] if x.strip()]
    return found


def test_partial_loads_arrive_before_they_are_released(listing):
    # teams of up to 128 experts: 6 of binary32 logits, 5 of each 16-bit type
    released = {n: c for n, c in listing.items() if any(x.startswith("buffer_wbl2") for x in c)}
    assert len(released) == 6 + 2 * 5
    for name, code in released.items():
        for at in [i for i, x in enumerate(code) if x.startswith("buffer_wbl2")]:
            barrier = max(i for i in range(at) if code[i].startswith("s_barrier"))
            assert not any(x.startswith("global_store") for x in code[barrier:at]), name
            for x in reversed(code[:barrier]):
                if x.startswith("s_waitcnt") and "vmcnt(0)" in x:
                    break
                assert not re.match(r"global_store|s_c?branch", x), "%s: %s before the barrier, and no wait" % (name, x)


def test_parts_of_the_loss_arrive_before_their_count(listing):
    ends = {n: c for n, c in listing.items() if "k_load_end" in n}
    assert len(ends) == 2
    for name, code in ends.items():
        counts = [i for i, x in enumerate(code) if x.startswith("global_atomic_add")]
        assert len(counts) == 1, name
        store = max(i for i in range(counts[0]) if code[i].startswith("global_store_dwordx2"))
        assert "sc1" in code[store], name            # past this die's cache
        assert any(x.startswith("s_waitcnt") and "vmcnt(0)" in x for x in code[store:counts[0]]), name
        read = next(x for x in code[counts[0]:] if x.startswith("global_load_dwordx2"))
        assert "sc1" in read, name
