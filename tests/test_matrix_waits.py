"""A vector instruction may touch what a matrix instruction writes only some instructions
later; nothing in the hardware waits. The compiler counts them, but has missed one where a
branch follows a product (tests on the GPU saw it as wrong sums). Here the assembly of the
kernels built from this source is walked along every path."""
import os
import re
import subprocess

import pytest

from speculative_decoding_verification_pipeline_amd import build

# wait states until a vector instruction reads or overwrites the result: 7 behind 4 passes,
# 11 behind 8, one less where the operands are binary32
NEED = {"v_mfma_f32_16x16x32_bf16": 7, "v_mfma_f32_16x16x32_f16": 7, "v_mfma_f32_32x32x16_bf16": 11,
        "v_mfma_f32_16x16x4_f32": 10}


def registers(text):
    out = set()
    for kind, a, b in re.findall(r"\b([av])\[(\d+):(\d+)\]", text):
        out |= {(kind, i) for i in range(int(a), int(b) + 1)}
    return out | {(kind, int(a)) for kind, a in re.findall(r"(?<![\w\[])([av])(\d+)\b", text)}


def functions(asm):
    """Name by name the instructions, as (operation, operands), and where labels stand."""
    out, name = {}, None
    for line in asm.splitlines():
        line = line.split(";")[0].rstrip()
        if m := re.match(r"^(_Z\w+):", line):
            name = m.group(1)
            out[name] = ([], {})
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and (m := re.match(r"^(\.LBB\w+):", line)):
            out[name][1][m.group(1)] = len(out[name][0])
        elif name and line.startswith("\t") and not line.startswith("\t."):
            op, _, rest = line.strip().partition(" ")
            out[name][0].append((op, rest))
    return out


def early(code, labels):
    """Pairs of a matrix instruction and one that touches its result too early."""
    bad = []
    for i, (op, rest) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        need, dst = NEED[op], registers(rest.split(",")[0])
        seen, todo = {}, [(i + 1, 0)]
        while todo:
            j, waited = todo.pop()
            if j >= len(code) or waited >= need or seen.get(j, need) <= waited:
                continue
            seen[j] = waited
            op2, rest2 = code[j]
            if op2 == "s_endpgm":
                continue
            if op2 == "s_nop":
                todo.append((j + 1, waited + int(rest2) + 1))
                continue
            if op2.startswith(("s_branch", "s_cbranch")):
                todo.append((labels[rest2.strip()], waited + 1))
                if op2 == "s_branch":
                    continue
            elif op2.startswith("v_mfma"):
                operands = re.findall(r"[av]\[\d+:\d+\]|[av]\d+|-?[\d.]+", rest2)
                if registers(" ".join(operands[1:3])) & dst:
                    bad.append((code[i], code[j], waited))
                    continue
                if registers(operands[0]) == dst:  # sums go on: a result of its own
                    continue
            elif op2.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")):
                if registers(rest2) & dst:
                    bad.append((code[i], code[j], waited))
                    continue
            todo.append((j + 1, waited + 1))
    return bad


def test_the_walk_sees_a_missing_wait():
    asm = "_Zf:\n\tv_mfma_f32_16x16x32_f16 a[0:3], v[4:7], v[8:11], 0\n{}\ts_cbranch_vccnz .LBB0_2\n" \
          "\tv_mov_b32_e32 v1, 0\n.LBB0_2:\n\tv_accvgpr_read_b32 v2, a3\n\ts_endpgm\n.Lfunc_end0:\n"
    for nops, count in (("", 1), ("\ts_nop 4\n", 1), ("\ts_nop 5\n", 0)):
        (code, labels), = functions(asm.format(nops)).values()
        assert bool(early(code, labels)) == bool(count)


@pytest.mark.parametrize("source", ["ss_attend.hip", "ss_lmhead.hip", "ss_lmhead_quant.hip"])
def test_results_of_products_are_waited_for(source, tmp_path):
    out = tmp_path / "k.s"
    subprocess.run([build.hipcc(), *build.CFLAGS, "-I", build.INCLUDE, "-x", "hip", "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, source), "-o", str(out)], check=True, capture_output=True)
    kernels = {n: f for n, f in functions(out.read_text()).items() if any(o.startswith("v_mfma") for o, _ in f[0])}
    assert kernels
    for name, (code, labels) in kernels.items():
        assert not early(code, labels), name
