"""ISA checks on the adapter kernels that issue MFMAs from inline asm.

The compiler puts no wait states around asm, so the generated gfx950 assembly
of lora_few_kernel and lora_gemm_kernel has to have, in program order:

* no VALU write of an asm MFMA's register within 2 wait states before it;
* no read of an accumulator by another instruction before the MFMAs that wrote
  it have drained (an s_nop of 8 or more states since the last of them);
* in the loops that hold the MFMAs: no spills, no access to accumulators other
  than by MFMAs, and no loop over lanes around a copy (an operand that the
  compiler took for non-uniform).
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from post_weight_quantization_26_amd import build_lib
from test_asm_mfma_isa import _hipcc, _operands, _regs

KERNELS = {
    "lora_few.hip": [f"lora_few_kernelILb{f}ELi{mt}ELb{g}ELb{w}E"
                     for f in (0, 1) for mt in (2, 4) for g in (0, 1) for w in (0, 1)],
    "lora_few_back.hip": [f"lora_few_back_kernelILb{f}ELi{mt}ELi{g}ELb{w}E"
                          for f in (0, 1) for mt in (2, 4) for g in (1, 2, 4) for w in (0, 1)],
    "lora_gemm.hip": [f"lora_gemm_kernelILb{f}ELb{s}E" for f in (0, 1) for s in (0, 1)],
}


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc is not available")
    out = tmp_path_factory.mktemp("lora_isa")

    def compile_one(src):
        dst = str(out / (src + ".s"))
        res = subprocess.run([cc, *build_lib.COMMON, "--cuda-device-only", "-S",
                              os.path.join(build_lib.CSRC, src), "-o", dst],
                             capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        return src, open(dst).read()

    with cf.ThreadPoolExecutor(len(KERNELS)) as ex:
        return dict(ex.map(compile_one, KERNELS))


def body(asm, name):
    """Instructions as (text, from inline asm), labels as ("label:", False)."""
    m = re.search(r"^(_Z\S*" + name + r"\S*):[ \t]*(;.*)?$", asm, re.M)
    assert m, f"kernel {name} not found in the assembly"
    out, inside = [], False
    for line in asm[m.end():asm.index(".Lfunc_end", m.end())].split("\n"):
        s = line.strip()
        if s.startswith(";;#ASM"):
            inside = s.startswith(";;#ASMSTART")
        elif re.match(r"\.LBB\S+:", s):
            out.append((s.split(":")[0] + ":", False))
        elif s and not s.startswith((";", ".", "#")):
            out.append((s.split(";")[0].strip(), inside))
    return out


def states(s):
    m = re.match(r"s_nop (\d+)", s)
    return int(m.group(1)) + 1 if m else 0 if s.endswith(":") else 1


def written(s):
    if not s.startswith("v_") or s.startswith(("v_mfma", "v_readfirstlane", "v_readlane", "v_cmp")):
        return set()
    ops = _operands(s)
    return _regs(ops[0]) if ops else set()


@pytest.mark.parametrize("src,kernel", [(s, k) for s, ks in KERNELS.items() for k in ks])
def test_adapter_kernel_isa(assembly, src, kernel):
    ins = body(assembly[src], kernel)
    mfma = [i for i, (s, a) in enumerate(ins) if a and s.startswith("v_mfma_f32_16x16x32")]
    assert len(mfma) >= 64, f"{kernel}: {len(mfma)} MFMAs from asm"
    acc = set()
    for k in mfma:
        ops = [_regs(t.split()[0]) for t in _operands(ins[k][0])[:4]]
        assert all(r[0] == "a" for r in ops[0]), f"{kernel}: accumulator outside the AGPRs"
        acc |= ops[0]
        regs, n = set().union(*ops), 0
        for s, _ in reversed(ins[max(0, k - 8):k]):
            assert n >= 2 or not written(s) & regs, f"{kernel}: {s} right before {ins[k][0]}"
            n += states(s)
    drained = 99
    for i, (s, a) in enumerate(ins):
        if a and s.startswith("v_mfma"):
            drained = 0
            continue
        if not s.startswith("v_mfma") and drained < 8:
            read = set().union(set(), *(_regs(t.split()[0]) for t in _operands(s)[1:]))
            assert not read & acc, f"{kernel}: {s} reads an accumulator {drained} states after"
        m = re.match(r"s_nop (\d+)", s)
        drained = max(drained, int(m.group(1)) + 1) if m else drained
    # innermost loops around asm MFMAs
    label = {s[:-1]: i for i, (s, _) in enumerate(ins) if s.endswith(":")}
    loops = []
    for i, (s, _) in enumerate(ins):
        m = re.match(r"s_c?branch\S*\s+(\.LBB\S+)", s)
        if m and label.get(m.group(1), i) < i:
            loops.append((label[m.group(1)], i))
    inner = [(a, b) for a, b in loops if any(a < k < b for k in mfma) and
             not any(a <= c and d < b and any(c < k < d for k in mfma) for c, d in loops)]
    assert inner, f"{kernel}: no loop of MFMAs"
    for a, b in inner:
        # (lora_gemm's low-rank loop looks its adapters up and writes to LDS)
        low = any(s.startswith("ds_write") for s, _ in ins[a:b])
        for s, _ in ins[a:b]:
            assert not s.startswith(("scratch_", "v_accvgpr")), f"{kernel}: {s} in the main loop"
            assert low or not s.startswith("s_and_saveexec"), f"{kernel}: {s} in the main loop"
