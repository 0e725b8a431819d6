"""Wait states that the hardware asks for around loads straight to LDS, in the built library's own device code. The
loads are asm statements, in and before which the compiler puts no waits of its own."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

SGPRS = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")
WRITES_SGPR = re.compile(r"v_(readfirstlane|readlane|cmp)")


def registers(text):
    out = set()
    for lo, hi, one in SGPRS.findall(text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def states(line):
    """Wait states that an instruction is worth to those after it."""
    return int(line.split()[1], 0) + 1 if line.startswith("s_nop") else 1


def faults(lines):
    """(loads to LDS, those that come too early) of a kernel's instructions: M0 needs one wait state after the scalar
    instruction that writes it, an address or buffer register five after a vector instruction that does."""
    loads, bad = 0, []
    for i, line in enumerate(lines):
        if not re.match(r"global_load_lds|(global|buffer)_load.*\blds\b", line):
            continue
        loads += 1
        wanted, passed = registers(line), 0
        for before in reversed(lines[max(0, i - 6):i]):
            if passed >= 5:
                break
            first = before.partition(" ")[2].partition(",")[0]
            if before.startswith("s_") and first == "m0" and passed < 1:
                bad.append((before, line))
            if WRITES_SGPR.match(before) and wanted & registers(first):
                bad.append((before, line))
            if before.startswith("s_"):  # its last writer: a scalar one, which needs no wait
                wanted -= registers(first)
            passed += states(before)
    return loads, bad


def test_the_rule_finds_what_comes_too_early():
    load, reg = "global_load_lds_dword v1, s[2:3] sc1", "v_readlane_b32 s3, v255, 39"
    assert faults(["s_mov_b32 m0, s4", "s_nop 0", load]) == (1, [])
    assert faults(["s_mov_b32 m0, s4", load])[1]
    assert faults(["s_mov_b32 m0, s4", "buffer_load_dwordx4 v31, s[16:19], 0 offen lds"])[1]
    assert faults([reg, "s_nop 2", "s_mov_b32 m0, s4", "s_nop 0", load]) == (1, [])
    assert faults([reg, "s_mov_b32 m0, s4", "s_nop 0", load])[1]
    assert faults([reg, "s_addc_u32 s3, s9, s3", "s_mov_b32 m0, s4", "s_nop 0", load]) == (1, [])


def kernels(tmp_path):
    """Instructions of each function of the library's device code."""
    lib = os.path.join(ROOT, "fp8_group_quant_amd", "libfp8q.so")
    assert os.path.exists(lib), "libfp8q.so is not built"
    (tmp_path / "lib.so").symlink_to(lib)  # what the bundle holds is written next to it
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    for part in sorted(tmp_path.glob("lib.so.*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(part)], check=True,
                              capture_output=True, text=True).stdout
        name, lines = None, []
        for line in text.splitlines():
            if m := re.match(r"(?:[0-9a-f]+ )?<(\S+)>:", line):
                if lines:
                    yield name, lines
                name, lines = m.group(1), []
            elif name and line.strip():
                lines.append(line.split("//")[0].strip())
        if lines:
            yield name, lines


def test_loads_to_lds_wait_for_their_registers(tmp_path):
    counts = {}
    for name, lines in kernels(tmp_path):
        loads, bad = faults(lines)
        assert not bad, (name, bad[:3])
        counts[name] = loads
    # both products' kernels were seen
    assert any(n and "gemm_dma_kernel" in k for k, n in counts.items())
    assert any(n and "gemm_mxfp4_kernel" in k for k, n in counts.items())
