"""The feed-forward's widest shapes write their matrix instructions out by hand, so the compiler does not know when their
results may be read: on the library's own gfx950 code, that no main loop touches an accumulation register with anything
but a matrix instruction, that everything behind one waits first, and that no operand is written right before one."""
import glob
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def disassemble(directory):
    """{kernel: [(address, instruction)]} of the built library."""
    lib = os.path.join(directory, "lib.so")
    os.symlink(os.path.join(ROOT, "combine_ep_layout_amd", "libep_layout.so"), lib)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=directory)
    kernels = {}
    for code in glob.glob(lib + "*gfx950*"):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", code], check=True, capture_output=True, text=True).stdout
        name = None
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
            body = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+)", line)
            if head:
                name = head.group(1)
                kernels[name] = []
            elif body and name:
                kernels[name].append((int(body.group(2), 16), body.group(1)))
    return kernels


@pytest.fixture(scope="module")
def wide(tmp_path_factory):
    kernels = disassemble(str(tmp_path_factory.mktemp("isa")))
    found = {k: v for k, v in kernels.items() if re.search(r"ffn_gemm_kernel.*ShapeILi\dELi256ELi256E", k)}
    assert len(found) == 5                          # one for each product
    return found


def touches_accumulators(instruction):
    return re.search(r"\ba(\d|\[)|accvgpr", instruction) is not None


def loops(code):
    """Innermost loops with a matrix instruction: the instructions from a backward branch's target to the branch."""
    at = {a: i for i, (a, _) in enumerate(code)}
    spans = []
    for i, (a, text) in enumerate(code):
        m = re.match(r"s_c?branch\S* (\d+)", text)
        if m:
            offset = int(m.group(1))
            if offset >= 0x8000:
                start = at[a + 4 + 4 * (offset - 0x10000)]
                if any("v_mfma" in t for _, t in code[start:i]):
                    spans.append((start, i))
    return [s for s in spans if not any(o != s and s[0] <= o[0] and o[1] <= s[1] for o in spans)]


def test_the_reader_of_the_code_sees_what_it_looks_for():
    assert touches_accumulators("v_accvgpr_read_b32 v1, a2") and touches_accumulators("global_store_dwordx4 v[0:1], a[4:7], off")
    assert not touches_accumulators("v_add_u32_e32 v1, s2, v3") and not touches_accumulators("s_waitcnt vmcnt(0)")
    code = [(0, "s_nop 0"), (4, "v_mfma_f32 a[0:3], v0, v1, a[0:3]"), (12, "s_cbranch_scc1 65533"), (16, "s_cbranch_scc0 65531")]
    assert loops(code) == [(1, 2)]


def test_main_loops_leave_the_accumulators_alone(wide):
    for name, code in wide.items():
        inner = loops(code)
        assert len(inner) == (1 if "Li4ELi256" in name else 3), (name, len(inner))     # full, 128 and 64 rows high
        for a, z in inner:
            other = [t for _, t in code[a:z] if touches_accumulators(t) and "v_mfma" not in t]
            assert not other, (name, other[:3])


def states_to_first_read(code, last):
    """Fewest states on any way from behind the instruction `last` to one that names an accumulation register and is no
    matrix instruction, at most 18 (a barrier, a wait or a branch counts as one state, an s_nop n as n + 1)."""
    at = {a: i for i, (a, _) in enumerate(code)}
    fewest, best, todo = 18, {}, [(last + 1, 0)]
    while todo:
        i, states = todo.pop()
        if i >= len(code) or states >= fewest or best.get(i, 99) <= states:
            continue
        best[i] = states
        a, t = code[i]
        if touches_accumulators(t):
            if "v_mfma" not in t:
                fewest = states
            continue
        nop, jump = re.match(r"s_nop (\d+)", t), re.match(r"s_(c?)branch\S* (\d+)", t)
        states += int(nop.group(1)) + 1 if nop else 1
        if jump:
            offset = int(jump.group(2))
            todo.append((at[a + 4 + 4 * (offset - 0x10000 if offset >= 0x8000 else offset)], states))
        if not (jump and not jump.group(1)) and not t.startswith("s_endpgm"):
            todo.append((i + 1, states))
    return fewest


def test_the_walk_behind_a_loop():
    code = [(0, "v_mfma a[0:3]"), (4, "s_cbranch_scc1 2"), (8, "s_nop 7"), (12, "v_accvgpr_read_b32 v0, a0"),
            (16, "s_branch 65534"), (20, "s_endpgm")]
    assert states_to_first_read(code, 0) == 2               # the jump over the wait: branch, branch, read
    assert states_to_first_read(code[:1] + [(4, "s_nop 7")] + code[2:], 0) == 16
    assert states_to_first_read([(0, "v_mfma a[0:3]"), (4, "s_nop 15"), (8, "s_nop 3"), (12, "v_accvgpr_read_b32 v0, a0")], 0) == 18


def test_results_are_read_after_their_wait(wide):
    """Behind the last matrix instruction of a loop, 18 states pass before anything else names an accumulation register:
    what the kernels write out, not what the scalar instructions of the loop's end happen to take."""
    for name, code in wide.items():
        for a, z in loops(code):
            last = max(i for i in range(a, z) if "v_mfma" in code[i][1])
            assert states_to_first_read(code, last) >= 18, (name, code[a][0], states_to_first_read(code, last))


def test_operands_are_not_written_right_before_their_use(wide):
    """Two states lie between a vector instruction and a matrix instruction: the one written with it."""
    for name, code in wide.items():
        for i, (_, t) in enumerate(code):
            if "v_mfma" in t:
                assert code[i - 1][1] == "s_nop 1", (name, code[i - 1], t)
