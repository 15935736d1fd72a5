"""The wait states of the HBM-to-LDS loads that are written in assembly, which
the compiler does not add: in the helpers, and in the built library's code."""
import glob
import os
import re
import subprocess

import pytest

from newton_schulz_ns5_amd import _lib, build

LLVM = "/opt/rocm/llvm/bin/llvm-objdump"

SNIPPET = """
#include "device_util.h"
using namespace muon;
__global__ void fresh(const char* p, int n) {
  extern __shared__ char s[];
  lds_dma16_asm(rsrc_words(p + threadIdx.x / 64 * 4096, n), 0, threadIdx.x * 16, 0);
  __builtin_amdgcn_s_waitcnt(0);
}
__global__ void kept(const char* p, int n) {
  extern __shared__ char s[];
  const auto r = settled(rsrc_words(p + threadIdx.x / 64 * 4096, n));
  for (int i = 0; i < n; ++i) lds_dma16_asm(r, i * 1024, threadIdx.x * 16, i * 1024);
  __builtin_amdgcn_s_waitcnt(0);
}
"""


def compiled(tmp_path, text):
    src, out = tmp_path / "w.hip", tmp_path / "w.s"
    src.write_text(text)
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-w", "-S", "--offload-device-only", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    return r.returncode, out.read_text() if r.returncode == 0 else r.stderr


def body(asm, name):
    """Instructions of one function of a listing."""
    m = re.search(r"^\S*%s\S*:[^\n]*\n(.*?)s_endpgm" % name, asm, re.S | re.M)
    return [l.split(";")[0].strip() for l in m.group(1).splitlines() if re.match(r"\s+[a-z]", l) and not re.match(r"\s+\.", l)]


def test_a_fresh_descriptor_is_waited_for(tmp_path):
    rc, asm = compiled(tmp_path, SNIPPET)
    assert rc == 0, asm
    code = body(asm, "fresh")
    at = next(i for i, l in enumerate(code) if l.startswith("buffer_load_dwordx4"))
    assert any(l.startswith("v_readfirstlane") for l in code[:at])
    assert code[at - 1].split() == ["s_nop", "4"]
    # a descriptor kept from load to load: five once, after the last vector write of its words, one at the load
    code = body(asm, "kept")
    at = next(i for i, l in enumerate(code) if l.startswith("buffer_load_dwordx4"))
    assert code[at - 1].split() == ["s_nop", "0"]
    wait = max(i for i, l in enumerate(code[:at]) if l.split() == ["s_nop", "4"])
    assert not any(l.startswith(("v_readfirstlane", "v_readlane")) for l in code[wait:at])


def registers(word):
    """Scalar registers that an operand names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", word) or re.fullmatch(r"s(\d+)", word)
    if not m:
        return {"vcc"} if word.startswith("vcc") else set()
    return set(range(int(m.group(1)), int(m.group(m.lastindex)) + 1))


def hazards(code):
    """Loads of this listing that read a scalar register fewer than five wait
    states after a vector instruction wrote it, and LDS loads right after a
    write of M0."""
    found, loads = [], 0
    for i, (op, args) in enumerate(code):
        if not (op.startswith("buffer_load") and "lds" in args[-1].split()):
            continue
        loads += 1
        reads = registers(args[1]) | registers(args[2].split()[0])
        states, k = 0, i - 1
        while k >= 0 and states < 5:
            o, a = code[k]
            if o == "s_nop":
                states += int(a[0], 0) + 1
            else:
                if o.startswith("v_") and a and reads & registers(a[0]):
                    found.append((i, o, a))
                if states < 1 and a and a[0] == "m0":
                    found.append((i, o, a))
                states += 1
            k -= 1
    return loads, found


def test_the_scan_sees_a_hazard():
    load = ("buffer_load_dwordx4", ["v1", "s[4:7]", "s9 offen lds"])
    write, other = ("v_readfirstlane_b32", ["s6", "v0"]), ("s_add_i32", ["s1", "s2", "s3"])
    m0 = ("s_mov_b32", ["m0", "s30"])
    assert hazards([write, other, load])[1] and hazards([("v_readfirstlane_b32", ["s9", "v0"]), load])[1]
    assert hazards([m0, load])[1] and not hazards([m0, ("s_nop", ["0"]), load])[1]
    assert not hazards([write, ("s_nop", ["4"]), load])[1] and not hazards([write] + [other] * 5 + [load])[1]


def test_no_load_of_the_built_library_is_too_early(tmp_path):
    if not os.path.exists(_lib.LIB_PATH) or not os.path.exists(LLVM):
        pytest.skip("nothing is built, or there is no disassembler")
    link = tmp_path / "l.so"
    link.symlink_to(_lib.LIB_PATH)
    subprocess.run([LLVM, "--offloading", str(link)], check=True, capture_output=True, cwd=tmp_path)
    total = 0
    for obj in sorted(glob.glob(str(tmp_path / "*gfx950"))):
        text = subprocess.run([LLVM, "-d", "--no-show-raw-insn", obj], check=True, capture_output=True, text=True).stdout
        for part in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
            code = []
            for line in part.splitlines()[1:]:
                words = line.split("//")[0].strip().split(None, 1)
                if words:
                    code.append((words[0], [w.strip() for w in words[1].split(",")] if len(words) > 1 else []))
            loads, found = hazards(code)
            total += loads
            assert not found, (part.split(">")[0], found[:3])
    assert total > 100
