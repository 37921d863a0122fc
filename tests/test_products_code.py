"""What the compiler has to leave alone in the products by tiles, in the code
that it makes of them here.

The large tiles name their 256 accumulators in inline assembly, where the
compiler does not know of a matrix instruction's latency: between the first and the
last of them it may not move one, nor read or write one.  And a load
straight into LDS takes its window from scalar registers: where the compiler took
it to differ from lane to lane, it would build a loop around every load."""
import os
import re
import subprocess

import pytest

from lossless_weight_compression_bf16_amd import build as W


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    try:
        hipcc = W.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("code") / "products.s"
    flags = [f for f in W.flags() if f not in ("-shared", "-fPIC", "-Wall")]
    subprocess.run([hipcc, *flags, "-w", "-S", "--cuda-device-only", os.path.join(W.CSRC, "ops", "wc_products.hip"), "-o", str(out)],
                   check=True, stderr=subprocess.DEVNULL)
    text = out.read_text()
    found = {}
    for m in re.finditer(r"^(_ZN2wc3ops\w+):", text, re.M):
        found[m.group(1)] = text[m.start():text.index(".Lfunc_end", m.start())]
    assert found
    return found


def _large(kernels):
    return {n: c for n, c in kernels.items() if "ELi256ELi256" in n and "v_mfma" in c}


def test_accumulators_stay_where_they_are(kernels):
    large = _large(kernels)
    assert len(large) >= 8
    for name, code in large.items():
        at = [m.start() for m in re.finditer("v_mfma", code)]
        between = code[at[0]:at[-1]]
        assert "v_accvgpr" not in between, name
        assert "scratch_" not in between, name


def test_results_are_waited_for(kernels):
    """18 wait states at least from a matrix instruction of 8 passes to a reading of its result."""
    for name, code in _large(kernels).items():
        lines = [x.strip() for x in code.splitlines()]
        for i, line in enumerate(lines):
            if not line.startswith("v_accvgpr_read"):
                continue
            waits = 0
            for back in reversed(lines[:i]):
                if back.startswith("v_mfma") or waits >= 18:
                    break
                if back.startswith("s_nop"):
                    waits += int(back.split()[1], 0) + 1
                elif re.match(r"[sv]_|ds_|buffer_|global_", back):
                    waits += 1
            assert waits >= 18, (name, i)


def test_no_loop_around_a_load(kernels):
    """A loop over the values that lanes have of a window reads its first lane and goes back while lanes are left."""
    tiles = {n: c for n, c in kernels.items() if re.search(r"buffer_load_dwordx4 .*\blds\b", c)}
    assert len(tiles) >= 20
    for name, code in tiles.items():
        for m in re.finditer(r"^(\.LBB\w+):", code, re.M):
            end = re.search(r"s_cbranch_execnz " + re.escape(m.group(1)) + r"\b", code[m.start():])
            assert not end or " lds" not in code[m.start():m.start() + end.start()], name


def test_nothing_is_spilled_in_the_tiles(kernels):
    for name, code in kernels.items():
        if re.search(r"buffer_load_dwordx4 .*\blds\b", code):
            assert "scratch_store" not in code, name
