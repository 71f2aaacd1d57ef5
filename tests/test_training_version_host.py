"""The version of the training-step operators' interface, and that a C program
finds them as the header declares them."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_says_the_header_s_version():
    import gradient_aggregation_amd as ga
    with open(os.path.join(ROOT, "include", "gradagg.h")) as f:
        header = int(re.search(r"#define GA_TRAINING_VERSION (\d+)", f.read()).group(1))
    assert ga.lib().ga_training_version() == header == 2


def test_c_layout_of_the_parameters(tmp_path):
    """Zeros choose rounding at random, and the new field lies where there was padding."""
    src = tmp_path / "layout.c"
    src.write_text("""
#include <stddef.h>
#include "gradagg.h"
_Static_assert(GA_TRAINING_VERSION >= 2, "m_rounding");
_Static_assert(sizeof(ga_adamw_params) == 32, "size");
_Static_assert(offsetof(ga_adamw_params, m_rounding) == 20, "in the padding");
_Static_assert(offsetof(ga_adamw_params, t) == 24, "t stays");
_Static_assert(GA_ROUND_RANDOM == 0 && GA_ROUND_NEAREST == 1, "roundings");
_Static_assert(sizeof(ga_clip) == 16 && sizeof(ga_adamw_state) == 32 && sizeof(ga_rows) == 16, "sizes");
""")
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-fsyntax-only", str(src)], check=True)
