"""The generated code behind matrix instructions: their results take some passes to reach the registers, and the
hardware does not hold back an instruction that touches these before. The compiler counts the wait states along the
code as it lies, and not always along a branch that is taken; here every path of the built library's code is walked.
No GPU needed."""
import functools
import os
import re
import subprocess

import pytest

import gated_delta_rule_chunk_amd as kda
from tests.test_mla_wait_states import LLVM, _code_objects

# Cycles / 4 of a matrix instruction on gfx950
PASSES = {"32x32x16_bf16": 8, "16x16x32_bf16": 4, "16x16x16_bf16": 4, "32x32x2_f32": 16, "16x16x4_f32": 8,
          "16x16x128_f8f6f4": 8}


def _shape(name):
    return re.match(r"v_mfma_(?:scale_)?f32_(\w+?)(?:_e64)?$", name).group(1)


def wait_states(name):
    """Between a matrix instruction and another one's use of its result: passes + 2 for float32 operands, + 4 for
    narrower ones (CDNA3 and CDNA4 instruction set documents, manually inserted wait states; CDNA4 has one more for
    the narrow ones of 4 passes and more)."""
    shape = _shape(name)
    return PASSES[shape] + (2 if shape.endswith("_f32") else 4)


@functools.lru_cache(None)
def _registers(text):
    out = set()
    for m in re.finditer(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        lo = int(m.group(2) or m.group(4))
        out |= {(m.group(1), i) for i in range(lo, int(m.group(3) or lo) + 1)}
    return frozenset(out)


def _early(code, i):
    """Uses of the i-th instruction's result before it is there: [(index, wait states)]. code: (mnemonic, operands,
    registers that must be there, index of a branch's target)."""
    name, _, dst, _ = code[i]
    need, found = wait_states(name), []
    paths, seen = [(i + 1, 0)], {}
    while paths:
        j, states = paths.pop()
        while j < len(code) and states < need and seen.get(j, need) > states:
            seen[j] = states
            what, ops, regs, target = code[j]
            if regs & dst:
                # (a matrix instruction that adds to the result is ordered by the hardware)
                found.append((j, states))
                break
            if what == name:
                states = max(states, PASSES[_shape(name)])       # a SIMD's matrix unit takes one after the other
            states += int(ops[0], 0) + 1 if what == "s_nop" else 1
            if what == "s_endpgm":
                break
            if what == "s_branch":
                j = target
                continue
            if target is not None:
                paths.append((target, states))
            j += 1
    return found


def _parse(text):
    """{function: its instructions} of a disassembly"""
    out, now = {}, None
    for line in text.splitlines():
        head = re.match(r"([0-9a-f]+) <(.+)>:$", line)
        if head:
            base, now = int(head.group(1), 16), []
            out[head.group(2)] = now
        elif now is not None and "//" in line:
            body, _, comment = line.partition("//")
            name, _, rest = body.strip().partition(" ")
            to = re.search(r"<.+\+0x([0-9a-f]+)>", comment)
            now.append((int(re.match(r"\s*([0-9A-Fa-f]+):", comment).group(1), 16) - base, name,
                        [x.strip() for x in rest.split(",")], int(to.group(1), 16) if to else None))
    for fn, lines in out.items():
        at = {a: i for i, (a, *_) in enumerate(lines)}
        code = []
        for _, name, ops, to in lines:
            regs = frozenset()
            if name.startswith("v_mfma"):
                regs = _registers(ops[0])                # (what is looked for; a use is of the first two operands)
            elif name.startswith(("v_", "ds_", "global_", "buffer_", "scratch_", "flat_")):
                regs = _registers(",".join(ops))
            code.append((name, ops, regs, at[to] if name.startswith(("s_branch", "s_cbranch")) else None))
        out[fn] = code
    return out


def _check(code):
    """Matrix results of a function that are used too early"""
    uses = [(n, o, _registers(",".join(o[1:3])) if n.startswith("v_mfma") else r, t) for n, o, r, t in code]
    bad = []
    for i, (name, _, regs, _) in enumerate(code):
        if name.startswith("v_mfma"):
            uses[i], kept = code[i], uses[i]
            bad += [(i, name, code[j][0], states) for j, states in _early(uses, i)]
            uses[i] = kept
    return bad


def test_the_walk_finds_an_early_read():
    """The walk itself, on a few lines: the first path is too short by one, the second long enough."""
    def lines(n):
        return "\n".join(["0000000000001000 <f>:", "\tv_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], v[24:27], v[0:15] // 000000001000:",
                          "\ts_cbranch_vccnz 5 // 000000001008: <f+0x20>", "\ts_nop 15 // 00000000100C:",
                          "\tv_mov_b32_e32 v30, v0 // 000000001010:", "\ts_endpgm // 000000001014:",
                          f"\ts_nop {n} // 000000001020:", "\tv_max_f32_e32 v31, v15, v15 // 000000001024:",
                          "\ts_endpgm // 000000001028:"])
    assert [b[2:] for b in _check(_parse(lines(9))["f"])] == [("v_max_f32_e32", 11)]
    assert not _check(_parse(lines(10))["f"])


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_chunk_amd import _build
        _build.build()
    d = tmp_path_factory.mktemp("matrix")
    fat, out = d / "fat.bin", {}
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", f".hip_fatbin={fat}", kda.LIB_PATH,
                    os.devnull], check=True)
    for i, part in enumerate(_code_objects(fat.read_bytes())):
        obj = d / f"{i}.o"
        obj.write_bytes(part)
        out.update(_parse(subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", str(obj)],
                                         capture_output=True, text=True, check=True).stdout))
    return out


def test_results_are_there_when_they_are_used(functions):
    with_matrix = {fn for fn, code in functions.items() if any(n.startswith("v_mfma") for n, *_ in code)}
    for part in ("mla_fwd_kernel", "mla_dq_kernel", "mla_dkv_kernel", "mla_step_kernel", "mla_mx_step", "mla_weigh"):
        assert any(part in fn for fn in with_matrix), part
    bad = {fn: x for fn in with_matrix if (x := _check(functions[fn]))}
    assert not bad, "\n".join(f"{fn}: {x[:3]}" for fn, x in bad.items())
