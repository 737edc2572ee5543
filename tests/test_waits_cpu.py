"""Waits that the hardware leaves to the program, read from the assembly of the
built library.  A vector memory instruction that takes its address from scalar
registers needs five wait states after the vector instruction that wrote them
(v_readfirstlane, say).  The compiler counts them in its own code but does not
look inside inline assembly, so each block has to bring its own."""
import os
import re
import shutil
import subprocess

import pytest

from routed_expert_execution_amd import build, moe

OBJDUMP = os.path.join(os.path.dirname(build.HIPCC), "..", "llvm", "bin", "llvm-objdump")
NEEDED = 5


def _scalars(operand):
    """Numbers of the scalar registers of one operand: s7 or s[6:7]."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def short_waits(lines):
    """(line number, states, instruction) of each vector memory instruction that
    reads a scalar register fewer than NEEDED wait states after a vector
    instruction wrote it, the code taken in its order in memory."""
    written, now, found = {}, 0, []  # scalar register -> wait states passed at its last vector write
    for i, line in enumerate(lines):
        text = line.split("//")[0].strip()
        if not text or text.endswith(":") or text.startswith("."):
            continue
        name, _, rest = text.partition(" ")
        ops = [o.strip().split(" ")[0] for o in rest.split(",")]
        if re.match(r"(global|flat|buffer|scratch)_", name):
            for s in set().union(*map(_scalars, ops)):
                if now - written.get(s, -NEEDED) < NEEDED:
                    found.append((i, now - written[s], text))
        now += int(ops[0], 0) + 1 if name == "s_nop" else 1
        if name.startswith("v_"):
            for o in ops[:2] if name.endswith(("_co_u32_e64", "_co_u32")) or "div_scale" in name else ops[:1]:
                written.update(dict.fromkeys(_scalars(o), now))
        elif name.startswith("s_") and name != "s_nop":
            for s in _scalars(ops[0]):
                written.pop(s, None)  # (a scalar write: no wait needed)
    return found


def test_the_reading_of_waits():
    near = ["v_readfirstlane_b32 s0, v1", "s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dwordx4 v2, s[0:1]"]
    assert [f[:2] for f in short_waits(near)] == [(3, 2)]
    assert not short_waits(near[:2] + ["s_nop 3"] + near[3:])
    assert [f[1] for f in short_waits(near[:2] + ["s_nop 2"] + near[3:])] == [4]
    assert not short_waits(near[:1] + ["s_add_u32 s0, s0, s8", "s_addc_u32 s1, s1, s9"] + near[1:])
    assert not short_waits(["v_readfirstlane_b32 s2, v1", "global_load_dword v2, v3, s[0:1]"])
    assert short_waits(["v_cmp_eq_u32_e64 s[4:5], v0, v1", "global_load_dword v2, v3, s[4:5] offset:16"])


def test_loads_wait_for_scalars_that_vector_instructions_write(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump beside hipcc")
    moe.library()  # (what is built)
    shutil.copy(build.LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    loads, bad = 0, []
    for f in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f], cwd=tmp_path, check=True, capture_output=True, text=True).stdout
        lines = text.splitlines()
        loads += sum("global_load_lds" in line for line in lines)
        bad += [(f, *b) for b in short_waits(lines)]
    assert objects and loads, "no device code read"
    assert not bad, (len(bad), bad[:8])


M0_KERNEL = r"""
#include "tile_gemm.h"
extern "C" __global__ void k(const char* p, char* q) {
    __shared__ __attribute__((aligned(16))) char lds[4096];
    typedef __attribute__((address_space(1))) const void G;
    typedef __attribute__((address_space(3))) void L;
    __builtin_amdgcn_global_load_lds((G*)(p + threadIdx.x * 16), (L*)lds, 16, 0, 0);
    moe::tile::load_lds16(moe::tile::lds_address(lds + 1024), threadIdx.x * 16, p + 4096);
    __builtin_amdgcn_global_load_lds((G*)(p + 8192 + threadIdx.x * 16), (L*)lds, 16, 0, 0);
    moe::tile::wait_loads_and_meet();
    q[threadIdx.x] = lds[threadIdx.x];
}
"""


def test_the_compiler_knows_that_a_load_into_lds_sets_m0(tmp_path):
    """Its own loads to one LDS address on both sides of the block: M0, their
    destination, is set for each of the three."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    (tmp_path / "m0.hip").write_text(M0_KERNEL)
    asm = subprocess.run([build.HIPCC, "-x", "hip", *build.FLAGS, "-I", build.CSRC, "--cuda-device-only", "-S", str(tmp_path / "m0.hip"),
                          "-o", "-"], check=True, capture_output=True, text=True).stdout
    steps = re.findall(r"s_\w+ (m0),|(global_load_lds)_dwordx4", asm)
    assert steps == [("m0", ""), ("", "global_load_lds")] * 3, asm
