"""The 256 x 256 kernel of the 8-bit floating point product writes its matrix instructions out, so the compiler does not
know when their results are there: no accumulator may be read or copied before the wait behind the last of them, and
none may be kept anywhere else inside the loop.  This looks at the assembly of the kernel built here."""
import os
import re
import subprocess

import pytest

from sparse_rank_adapter_amd import build


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="ROCm toolchain not found")
def test_no_accumulator_is_read_before_the_wait(tmp_path):
    out = str(tmp_path / "fp8_mm.s")
    flags = [f for f in build.CFLAGS if f != "-fPIC"]
    rc, log = build._run([build.HIPCC, *flags, "-S", "--offload-device-only", os.path.join(build.CSRC, "fp8_mm.hip"), "-o", out])
    assert rc == 0, log
    text = open(out).read()
    bodies = re.findall(r"^(_ZN\S*k_fp8_big\S*):.*?^\s*s_endpgm", text, re.S | re.M)
    assert len(bodies) == 4  # two kinds for each operand
    for m in re.finditer(r"^_ZN\S*k_fp8_big\S*:(.*?)^\s*s_endpgm", text, re.S | re.M):
        ops = [l.split(";")[0].split() for l in m.group(1).splitlines()]
        ops = [(o[0], o[1] if len(o) > 1 else "") for o in ops if o and not o[0].startswith((".", ";")) and not o[0].endswith(":")]
        assert sum(o == "v_mfma_scale_f32_16x16x128_f8f6f4" for o, _ in ops) == 256  # four steps of 64
        at = [i for i, (o, _) in enumerate(ops) if o.startswith("v_mfma")]
        # between the loop's first and last matrix instruction accumulators stay where they are, and nothing is spilled
        inside = [ops[i] for i in range(at[0], at[-1]) if ops[i][0].startswith(("v_accvgpr", "scratch_"))]
        assert inside == []
        pending = False
        nops = 0
        for o, arg in ops:
            if o.startswith("v_mfma"):
                pending, nops = True, 0
            elif o == "s_nop" and arg == "15":
                nops += 1
                pending = pending and nops < 2
            elif o.startswith("v_accvgpr_read") or o.startswith("v_accvgpr_mov"):
                assert not pending, "an accumulator is read before the wait"
