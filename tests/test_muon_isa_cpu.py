"""The widest tiles of the orthogonalisation write their matrix instructions out by hand, as the feed-forward's do: the
same rules, on the library's own gfx950 code."""
import re

import pytest

from test_ffn_isa_cpu import disassemble, loops, states_to_first_read, touches_accumulators


@pytest.fixture(scope="module")
def wide(tmp_path_factory):
    kernels = disassemble(str(tmp_path_factory.mktemp("isa")))
    found = {k: v for k, v in kernels.items() if re.search(r"muon_gemm_kernel.*ShapeILi\dELi256ELi256E", k)}
    assert len(found) == 5                          # one for each product
    return found


def test_main_loops_leave_the_accumulators_alone(wide):
    for name, code in wide.items():
        inner = loops(code)
        assert len(inner) == 1, (name, len(inner))
        for a, z in inner:
            assert all("v_mfma_f32_16x16x32_f16" in t for _, t in code[a:z] if "v_mfma" in t)
            other = [t for _, t in code[a:z] if touches_accumulators(t) and "v_mfma" not in t]
            assert not other, (name, other[:3])


def test_results_are_read_after_their_wait(wide):
    for name, code in wide.items():
        for a, z in loops(code):
            last = max(i for i in range(a, z) if "v_mfma" in code[i][1])
            assert states_to_first_read(code, last) >= 18, (name, states_to_first_read(code, last))


def test_operands_are_not_written_right_before_their_use(wide):
    for name, code in wide.items():
        for i, (_, t) in enumerate(code):
            if "v_mfma" in t:
                assert code[i - 1][1] == "s_nop 1", (name, code[i - 1], t)
