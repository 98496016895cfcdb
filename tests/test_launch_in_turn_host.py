"""Kernels that start while the kernel before them still runs: what their sources must not do.  No GPU is needed."""
import re

import pytest

from selective_state_space_prefill_gb300 import build


def _code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)


def _in_turn():
    """The sources that launch such kernels, and the headers that they include."""
    files = [p for p in build.CSRC.glob("*.cu") if "launch_in_turn(" in _code(p)]
    names = {n for p in files for n in re.findall(r'#include "([^"]+)"', p.read_text())}
    return sorted(files + [build.CSRC / n for n in names if (build.CSRC / n).exists()])


def test_the_sources_are_found():
    assert {"norm.cu", "spec.cu", "w4.cu", "w4_tiles.cu", "common.cuh", "w4.cuh"} <= {p.name for p in _in_turn()}


@pytest.mark.parametrize("path", _in_turn(), ids=lambda p: p.name)
def test_no_load_is_non_coherent(path):
    """A non-coherent load is defined only for memory that nothing writes while the kernel runs; the kernel before
    may be writing it, and the wait for that kernel does not order such a load."""
    found = re.findall(r"__ldg\b|\.global\.nc\b|__restrict__|__ldlu\b|\btex[123]D", _code(path))
    assert not found, found


@pytest.mark.parametrize("path", [p for p in _in_turn() if p.suffix == ".cu"], ids=lambda p: p.name)
def test_every_kernel_launched_so_waits_for_the_one_before(path):
    """What a launch names has after_previous() in its body, ahead of next_may_start()."""
    code = _code(path)
    bodies = re.findall(r"__global__[^;{]*?\b(k_\w+)\([^{]*\{(.*?)\n\}\n", code, flags=re.S)
    assert bodies
    for name, body in bodies:
        if name in ("k_w4_quantize", "k_expire_wait"):   # launched the usual way
            assert "after_previous" not in body and "next_may_start" not in body
            continue
        assert body.count("after_previous()") == 1, name
        if "next_may_start()" in body:
            assert body.index("after_previous()") < body.index("next_may_start()"), name


def test_tensor_copies_come_behind_their_fence():
    """A thread's tensor copies of what the kernel before wrote are ordered behind the wait by a proxy fence."""
    for path in _in_turn():
        code = _code(path)
        if path.suffix != ".cu" or "tma_load_2d(" not in code:
            continue
        for part in re.split(r"\} else if \(warp", code[code.index("after_previous()"):]):
            at = part.find("tma_load_2d(")
            assert at < 0 or 0 <= part.find("before_copies()") < at, path.name


def test_who_exchanges_words_stays_as_long_as_they_may_come():
    """Every kernel that makes an Exchange gives a warp up as a whole and ends by leave(), with no way out before it;
    a warp that gave up sends nothing to CTAs that may have left."""
    seen = 0
    for path in _in_turn():
        if path.suffix != ".cu":
            continue
        for name, body in re.findall(r"__global__[^;{]*?\b(k_\w+)\([^{]*\{(.*?)\n\}\n", _code(path), flags=re.S):
            if "Exchange<" in body:
                seen += 1
                assert body.rstrip().endswith("all.leave();"), name
                assert not re.search(r"^    (if [^\n]*)?return;", body, flags=re.M), name
                assert body.rfind(".settle()") >= body.rfind(".word("), name
    assert seen >= 4
    code = _code(build.CSRC / "exchange.cuh")
    send = code[code.index("void send("):code.index("uint32_t word(")]
    assert "!dead" in send
    row = _code(build.CSRC / "spec.cu")
    assert row.count(".word(") == 4 and "all.settle();" in row[row.index("row_wide("):row.index("struct Raw")]


def test_a_cta_does_not_end_before_its_copies():
    """A warp that issues tensor copies into shared memory counts them and waits for the last ones by a wait of its own,
    whatever waits expired before; the one that issues products has a commit for them then."""
    code = _code(build.CSRC / "w4_tiles.cu")
    parts = [p for p in re.split(r"\} else (?:if \(warp|\{)", code[code.index("k_w4_tiles("):])]
    copies = [p for p in parts if "tma_load_2d(" in p]
    assert len(copies) == 2
    for p in copies:
        assert "++issued" in p and p.index("Waiter last{status}") > p.index("tma_load_2d(") and "i < issued; ++i) last(" in p
    products = [p for p in parts if "mma_from_tmem(" in p[:3000] and "mma_commit(&d_full" in p]
    assert len(products) == 1 and "mma_commit(done)" in products[0] and "last(done, 0)" in products[0]
