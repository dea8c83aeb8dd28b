"""The wait states that the direct-to-LDS copies need, in the built libraries' gfx950 code, without a GPU.

The copies are inline assembly, which the compiler does not look into when it puts wait states between instructions, so
they are looked for here, over every path through a kernel:
  - a load that writes LDS takes its address there from m0: one wait state after a scalar instruction wrote it;
  - a load that takes scalar registers: five after a vector instruction wrote one of them.
"""
import re
import shutil
import subprocess
from pathlib import Path

import pytest

import gemm_w4a16_amd as w

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
LIBRARIES = [Path(w.library_path), Path(w.library_path).with_name("libw4a16_roof.so")]
pytestmark = pytest.mark.skipif(not Path(OBJDUMP).exists(), reason="no disassembler")

LINE = re.compile(r"^\t(\S+)(?:\s+(.*?))?\s*// ([0-9A-F]+):")
TARGET = re.compile(r"<[^>+]*(?:\+0x([0-9a-f]+))?>\s*$")
SGPRS = re.compile(r"\bs(?:(\d+)\b|\[(\d+):(\d+)\])")


def sgprs(operands):
    out = set()
    for one, lo, hi in SGPRS.findall(operands):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def functions(text):
    """(name, [(mnemonic, operands, index of a branch's target or None)]) of each function."""
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"\s*([0-9a-f]{16}) <(.+)>:", part)
        if not head:
            continue
        start, code, index = int(head[1], 16), [], {}
        for line in part.splitlines()[1:]:
            m = LINE.match(line)
            if not m:
                continue
            to = None
            if m[1].startswith(("s_branch", "s_cbranch")):
                t = TARGET.search(line)
                to = start + int(t[1] or "0", 16) if t else None
            index[int(m[3], 16)] = len(code)
            code.append((m[1], m[2] or "", to))
        yield head[2], [(m, o, index.get(to)) for m, o, to in code]


def faults(code):
    """(copies to LDS, [(what is read too early, the load)])"""
    before = [[] for _ in code]
    for i, (m, _, to) in enumerate(code):
        if i + 1 < len(code) and m not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before[i + 1].append(i)
        if to is not None:
            before[to].append(i)
    copies, found = 0, []
    for i, (m, o, _) in enumerate(code):
        to_lds = m.startswith(("global_load_lds", "buffer_load_lds")) or (m.startswith("buffer_load") and " lds" in o)
        if not to_lds:
            continue
        copies += 1
        reads, seen, paths = sgprs(o), {}, [(p, 0) for p in before[i]]
        while paths:
            p, waited = paths.pop()
            if waited >= 5 or seen.get(p, 5) <= waited:
                continue
            seen[p] = waited
            pm, po, _ = code[p]
            written = po.split(",")[:2] if "_co_" in pm or pm.startswith(("v_mad_u64", "v_mad_i64", "v_div_scale")) else po.split(",")[:1]
            if waited < 1 and pm.startswith("s_") and written[0].strip() == "m0" and not pm.startswith("s_cmp"):
                found.append(("m0", f"{m} {o}"))
            if pm.startswith("v_") and sgprs(" ".join(written)) & reads:
                found.append((f"{pm} {po}", f"{m} {o}"))
            waited += int(po.split()[0], 0) + 1 if pm == "s_nop" else 1
            paths += [(q, waited) for q in before[p]]
    return copies, found


def text_of(*lines):
    return "0000000000000100 <k>:\n" + "".join(f"\t{l} // {256 + 4 * i:012X}: 00000000{t}\n" for i, (l, t) in enumerate(lines))


def test_what_counts_as_a_fault():
    load = ("global_load_lds_dwordx4 v6, s[2:3]", "")
    def of(*lines):
        (_, code), = functions(text_of(*lines))
        return [f[0] for f in faults(code)[1]]
    assert of(("s_mov_b32 m0, s4", ""), load) == ["m0"]
    assert of(("s_add_u32 m0, s4, 0x400", ""), load) == ["m0"]
    assert of(("s_mov_b32 m0, s4", ""), ("s_nop 0", ""), load) == []
    assert of(("v_readfirstlane_b32 s3, v1", ""), ("s_mov_b32 m0, s4", ""), ("s_nop 0", ""), load) == ["v_readfirstlane_b32 s3, v1"]
    assert of(("v_readfirstlane_b32 s3, v1", ""), ("s_mov_b32 m0, s4", ""), ("s_nop 3", ""), load) == []
    assert of(("v_cmp_eq_u32_e64 s[4:5], s2, v1", ""), load) == []
    # ... along a loop's way back
    assert of(("s_nop 0", ""), load, ("s_mov_b32 m0, s4", ""), ("s_cbranch_scc1 65533", " <k+0x4>")) == []
    assert of(load, ("v_readlane_b32 s2, v1, 3", ""), ("s_cbranch_scc1 65533", " <k>")) == ["v_readlane_b32 s2, v1, 3"]


@pytest.mark.parametrize("library", LIBRARIES, ids=lambda p: p.name)
def test_copies_wait(library, tmp_path):
    if not library.exists():
        pytest.skip("not built")
    shutil.copy(library, tmp_path)  # (the code objects are written beside the file)
    subprocess.run([OBJDUMP, "--offloading", library.name], cwd=tmp_path, check=True, capture_output=True)
    copies, found = 0, []
    for obj in sorted(tmp_path.glob("*gfx950*")):
        if b"gfx950" not in obj.name.encode() or obj.stat().st_size == 0:
            continue
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", obj.name], cwd=tmp_path, check=True, capture_output=True, text=True).stdout
        if "load_lds" not in out:
            continue
        for name, code in functions(out):
            n, bad = faults(code)
            copies += n
            found += [(name, *f) for f in bad]
    assert copies > 50
    assert not found, f"{len(found)} of {copies} copies, the first: {found[:3]}"
