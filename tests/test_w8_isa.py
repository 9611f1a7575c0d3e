"""ISA checks on the kernels of the 8-bit products, on the generated gfx950
assembly.

w8_gemm_kernel and w8_back_gemm_kernel issue their MFMAs from inline asm (the
256x256 main loop): the rules of the other kernels built on it hold for them.

w8_mid_kernel counts copies: a step's wait leaves exactly the copies of the step after it in flight. So the ones before the loop have to be
two whole steps of them and each step between two barriers one; nothing may be
spilled."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from post_weight_quantization_26_amd import build_lib
from test_asm_mfma_isa import _hipcc, _operands, _regs
from test_lora_isa import body, states, written

BIG = [("w8_gemm.hip", f"w8_gemm_kernelILb{f}ELb{g}ELi{a}ELb{c}E")
       for f in (0, 1) for g, a in ((0, 0), (1, 0), (1, 1)) for c in (0, 1)]
BIG += [("w8_back.hip", f"w8_back_gemm_kernelILb{f}ELb{c}E") for f in (0, 1) for c in (0, 1)]
TILES = [(128, 32), (128, 64), (128, 128), (256, 128)]
MID = [("w8_mid.hip", f"w8_mid_kernelILb{f}ELb{g}ELi{a}ELi{ra}ELi{tr}ELb{r}E", ra, tr)
       for f in (0, 1) for g, a in ((0, 0), (1, 0), (1, 1)) for ra, tr in TILES for r in (0, 1) if ra == 128 or not r]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc is not available")
    out = tmp_path_factory.mktemp("w8_isa")

    def compile_one(src):
        dst = str(out / (src + ".s"))
        res = subprocess.run([cc, *build_lib.COMMON, "--cuda-device-only", "-S",
                              os.path.join(build_lib.CSRC, src), "-o", dst],
                             capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        return src, open(dst).read()

    sources = sorted({x[0] for x in BIG + MID} | {"w8_few.hip", "w8_back_few.hip"})
    with cf.ThreadPoolExecutor(len(sources)) as ex:
        return dict(ex.map(compile_one, sources))


@pytest.mark.parametrize("src,kernel", BIG)
def test_big_kernel_isa(assembly, src, kernel):
    code = body(assembly[src], kernel)
    mfma = [i for i, (s, _) in enumerate(code) if s.startswith("v_mfma")]
    assert len(mfma) >= 3 * 128 and all(code[i][1] for i in mfma)
    assert not any(s.startswith("scratch_") for s, _ in code), "spills"
    assert not any(s.startswith("s_cbranch_exec") for s, _ in code[mfma[0]:mfma[-1]]), \
        "a loop over lanes among the matrix instructions"
    acc = set()
    for i in mfma:
        ops = _operands(code[i][0])
        acc |= _regs(ops[0])
        use = _regs(ops[1]) | _regs(ops[2])
        # an operand written by a vector instruction needs 2 wait states
        wait = 0
        for s, _ in reversed(code[max(0, i - 8):i]):
            if wait >= 2:
                break
            assert not written(s) & use, (kernel, s, code[i][0])
            wait += states(s)
    # accumulators: only MFMAs until a long nop behind the last one
    last = mfma[-1]
    nop = next(i for i in range(last, len(code)) if re.match(r"s_nop (15|[89]|1[0-4])", code[i][0]))
    for s, asm in code[mfma[0]:nop]:
        if s.startswith("v_mfma") or s.endswith(":"):
            continue
        for op in _operands(s):
            assert not _regs(op) & acc, (kernel, s)


def steps(code):
    """Loads issued in each stretch of code that a barrier begins or ends, with
    the wait before it: [(loads, vmcnt of the wait before the next barrier)]."""
    out, n, wait = [], 0, None
    for s, _ in code:
        if s.startswith("buffer_load"):
            n += 1
        elif s.startswith("s_waitcnt") and "vmcnt" in s:
            wait = int(re.search(r"vmcnt\((\d+)\)", s).group(1))
        elif s == "s_barrier":
            out.append((n, wait))
            n, wait = 0, None
    out.append((n, wait))
    return out


@pytest.mark.parametrize("src,kernel,ra,tr", MID)
def test_mid_kernel_loads(assembly, src, kernel, ra, tr):
    code = body(assembly[src], kernel)
    assert not any(s.startswith("scratch_") for s, _ in code), "spills"
    got = steps(code)
    per_step = (ra + tr) // 32
    # in the text: the loop's 3 steps, then up to 2 last ones, each behind a barrier
    assert len(got) == 1 + 3 + 2
    assert got[0] == (2 * per_step, per_step)
    for n, wait in got[1:-1]:
        assert (n, wait) == (per_step, per_step)
    assert got[-1][0] == per_step


FEW = [("w8_few.hip", f"w8_few_kernelILb{f}ELi{rb}ELb{g}ELi{a}E")
       for f in (0, 1) for rb, g, a in ((1, 0, 0), (2, 1, 0), (2, 1, 1))]
FEW += [("w8_back_few.hip", f"w8_back_few_kernelILb{f}ELi{tb}ELb{r}E")
        for f in (0, 1) for tb in (1, 2, 4) for r in (0, 1)]


@pytest.mark.parametrize("src,kernel", FEW)
def test_few_kernel_skips_by_branches(assembly, src, kernel):
    """Matrix instructions ignore the execution mask: nothing may be masked out
    up to the last of them, and nothing spilled."""
    code = body(assembly[src], kernel)
    last = max(i for i, (s, _) in enumerate(code) if s.startswith("v_mfma"))
    assert not any("saveexec" in s or s.startswith("v_cmpx") for s, _ in code[:last])
    assert not any(s.startswith("scratch_") for s, _ in code), "spills"
