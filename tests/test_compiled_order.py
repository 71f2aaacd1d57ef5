"""What the compiled kernels do in which order, where a result depends on it.

A workgroup that publishes values which all of its wavefronts stored, and has one
thread release them to the other dies of the card, needs every wavefront's stores
to have arrived before that release: it writes back what is in the cache by then.
The barrier between the two waits for the wavefronts, not for their stores."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    """{function: instructions} of the layer-norm kernels of the library built here."""
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
        if b"k_ln_bwd" not in f.read_bytes():
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], check=True, capture_output=True, text=True).stdout
        for block in re.split(r"\n(?=[0-9a-f]+ <)", text):
            name = re.match(r"[0-9a-f]+ <(\S+)>:", block)
            if name and "k_ln_bwd" in name.group(1):
                found[name.group(1)] = [x.split("//")[0].strip() for x in block.split("\n")[1:] if x.strip()]
    return found


def test_stores_arrive_before_they_are_released(listing):
    # 5 type pairs, 9 teams of binary32 rows and 8 of 16-bit ones
    assert len(listing) == 9 + 4 * 8
    for name, code in listing.items():
        releases = [i for i, x in enumerate(code) if x.startswith("buffer_wbl2")]
        assert releases, name
        for at in releases:
            barrier = max(i for i in range(at) if code[i].startswith("s_barrier"))
            assert not any(x.startswith("global_store") for x in code[barrier:at]), name
            for x in reversed(code[:barrier]):
                if x.startswith("s_waitcnt") and "vmcnt(0)" in x:
                    break
                assert not re.match(r"global_store|s_c?branch", x), "%s: %s before the barrier, and no wait" % (name, x)
