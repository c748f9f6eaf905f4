"""The generated code of the loads from global memory into LDS: the wait states
that the CDNA4 instruction set leaves to software. The compiler inserts them for
its own instructions, but not inside inline assembly, so the built library's
code is read. No GPU needed."""
import os
import re
import struct
import subprocess

import pytest

import gated_delta_rule_chunk_amd as kda

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(fat):
    """The gfx950 code objects of a .hip_fatbin section (one bundle a source file)."""
    at = fat.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", fat, at + 24)
        p = at + 32
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", fat, p)
            triple = fat[p + 24:p + 24 + length].decode()
            p += 24 + length
            if "gfx950" in triple:
                yield fat[at + offset:at + offset + size]
        at = fat.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{function: its instructions, each as (mnemonic, operands)}"""
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_chunk_amd import _build
        _build.build()
    d = tmp_path_factory.mktemp("code")
    fat = d / "fat.bin"
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", f".hip_fatbin={fat}", kda.LIB_PATH,
                    os.devnull], check=True)
    out = {}
    for i, code in enumerate(_code_objects(fat.read_bytes())):
        obj = d / f"{i}.o"
        obj.write_bytes(code)
        text = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", "--no-leading-addr",
                               str(obj)], capture_output=True, text=True, check=True).stdout
        now = None
        for line in text.splitlines():
            head = re.match(r"(?:[0-9a-f]+ )?<(.+)>:$", line)
            if head:
                now = out.setdefault(head.group(1), [])
            elif now is not None and line.strip():
                name, _, rest = line.split("//")[0].strip().partition(" ")
                now.append((name, [x.strip() for x in rest.split(",")] if rest else []))
    return out


def _sgprs(operand):
    """Scalar registers of an operand (vcc as -1)."""
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m.group(1))} if m else {-1} if operand == "vcc" else set()


def _vector_writes(name, ops):
    """Scalar registers that a vector instruction writes."""
    if not name.startswith("v_") or not ops:
        return set()
    return _sgprs(ops[0]) | (_sgprs(ops[1]) if len(ops) > 1 and ("_co_" in name or "div_scale" in name) else set())


def _scalar_writes(name, ops):
    """Scalar registers that a scalar instruction writes."""
    if not name.startswith("s_") or not ops or name.startswith(("s_cmp", "s_bitcmp", "s_nop", "s_waitcnt")):
        return set()
    return _sgprs(ops[0])


def _back(code, i):
    """Instructions before the i-th, nearest first, each with the wait states between the two."""
    states = 0
    for name, ops in reversed(code[max(0, i - 8):i]):
        yield states, name, ops
        states += int(ops[0], 0) + 1 if name == "s_nop" else 1


def _loads(kernels):
    for fn, code in kernels.items():
        for i, (name, ops) in enumerate(code):
            if "_load_lds_" in name or (name.startswith("buffer_load") and ops and ops[-1].endswith(" lds")):
                yield fn, code, i, ops


def test_the_library_loads_into_lds(kernels):
    """What the other tests look at is there, in every kernel that stages tiles."""
    have = {fn for fn, *_ in _loads(kernels)}
    for part in ("mla_fwd_kernel", "mla_dq_kernel", "mla_dkv_kernel", "mla_step_kernel"):
        names = {fn for fn in kernels if part in fn and not fn.endswith(".kd")}
        assert names and names <= have, part


def test_scalar_base_written_by_a_vector_instruction(kernels):
    """Five wait states between a vector instruction's write of a scalar register and a load that takes its
    address from it: with fewer the load may read the register's old value. (None where a scalar instruction has
    written it since: the hardware orders those.)"""
    bad = {}
    for fn, code, i, ops in _loads(kernels):
        base = set().union(*(_sgprs(x.split()[0]) for x in ops if x))
        for states, name, o in _back(code, i):
            if states < 5 and _vector_writes(name, o) & base:
                bad[fn] = bad.get(fn, 0) + 1
                break
            base -= _scalar_writes(name, o)
    assert not bad, bad


def test_m0_written_before_the_load(kernels):
    """One wait state between a write of m0 and a load into LDS, which takes its place there from m0."""
    bad = {}
    for fn, code, i, _ in _loads(kernels):
        states, name, o = next(_back(code, i))
        if o and o[0] == "m0":
            bad[fn] = bad.get(fn, 0) + 1
    assert not bad, bad


def test_m0_has_no_other_use(kernels):
    """The loads of the latent-attention kernels change m0, which the compiler does not know."""
    for fn in {fn for fn, *_ in _loads(kernels) if "mla" in fn}:
        for i, (name, ops) in enumerate(kernels[fn]):
            if "m0" in ops:
                assert (name, ops[0]) == ("s_mov_b32", "m0"), (fn, name, ops)
                assert any("_load_lds_" in x for x, _ in kernels[fn][i + 2:i + 5]), fn


def test_no_lane_is_left_out(kernels):
    """A load issued under a changed exec mask is followed by its restoration, which nothing comes between."""
    for fn, code, i, _ in _loads(kernels):
        if any(o and o[0] in ("exec_lo", "exec_hi") for s, _, o in _back(code, i) if s < 3):
            assert code[i + 1] == ("s_mov_b64", ["exec", "-1"]), fn
