"""A VALU result has to be two wait states old before a matrix instruction reads
it.  The compiler keeps that distance for the MFMAs it issues itself but does not
see into the inline asm that issues those of gemm_bf16.hip.  This CPU test compiles
that file for gfx950, keeps the assembly, and checks on every control-flow path of
every kernel instance that no register a VALU instruction writes is read by an MFMA
before that."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_isa_hazards import HIPCC, SRC, _blocks, _cost, _kernels

WAIT_STATES = 2


def _regs(op):
    m = re.match(r"([va])\[(\d+):(\d+)\]$", op.strip())
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"([va])(\d+)$", op.strip())
    return {(m[1], int(m[2]))} if m else set()


def _operands(t):
    return t.split(None, 1)[1].split(",") if " " in t else []


def _valu_writes(t):
    if not t.startswith("v_") or t.startswith("v_mfma") or t.startswith("v_cmp"):
        return set()
    return _regs(_operands(t)[0])


def _early_reads(lines):
    blocks, preds = _blocks([t.split(";")[0].strip() for t in lines])
    found = []

    def back(k, end, use, ws, seen):
        ins = blocks[k][1]
        for j in range(end - 1, -1, -1):
            if _valu_writes(ins[j]) & use:
                return ins[j], ws
            ws += _cost(ins[j])
            if ws >= WAIT_STATES:
                return None
        for p in preds[k]:
            if (p, ws) not in seen:
                seen.add((p, ws))
                r = back(p, len(blocks[p][1]), use, ws, seen)
                if r:
                    return r
        return None

    for k, (_, ins) in enumerate(blocks):
        for j, t in enumerate(ins):
            if t.startswith("v_mfma"):
                r = back(k, j, set().union(*map(_regs, _operands(t)[1:])), 0, set())
                if r:
                    found.append((t, r))
    return found


def test_checker_finds_a_planted_read():
    lines = ["v_cvt_pk_bf16_f32 v7, v9, v8",
             "s_cbranch_scc1 .LBB0_2",
             ".LBB0_2:",
             "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"]
    assert len(_early_reads(lines)) == 1
    assert _early_reads(lines[:1] + ["s_nop 0"] + lines[1:]) == []
    assert _early_reads(["v_accvgpr_write_b32 a2, v9"] + lines[3:])
    assert _early_reads(["v_mov_b32 v8, v7"] + lines[3:]) == []


@pytest.mark.skipif(shutil.which(HIPCC) is None and not os.path.exists(HIPCC),
                    reason="hipcc not installed")
def test_gemm_operands_are_old_enough(tmp_path):
    out = tmp_path / "g.s"
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
                        "-ffp-contract=off", "-fno-fast-math", "-Xclang", "-target-feature",
                        "-Xclang", "-packed-fp32-ops", "-S", "--cuda-device-only", SRC, "-o",
                        str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = _kernels(out.read_text())
    # 3 tile shapes x (r == 16 or not) x (reduction tail or not) x (mask or not)
    assert len(kernels) == 24, sorted(kernels)
    for name, lines in kernels.items():
        assert any(t.startswith("v_mfma") for t in lines), name
        early = _early_reads(lines)
        assert not early, (name, early[:3])
