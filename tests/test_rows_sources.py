"""What no run can show about the row products' kernels: rules that their
sources have to keep."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_scale_search_b200", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def calls(text, name):
    """The argument texts of every call of `name`."""
    for m in re.finditer(re.escape(name) + r"\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def test_what_a_running_grid_writes_is_not_read_as_read_only_data():
    """The few-token kernel starts while k_few_prep still runs (programmatic
    launch).  The tokens, their sums and their powers of two, and pointers made
    from them, may not go through the read-only path, which may be moved over
    the wait for that grid, and are not touched before it."""
    text = code("rows_few.cuh")
    made = {"x_few", "x_sums", "row_x"}
    for _ in range(3):   # pointers assigned from them, and from those
        for m in re.finditer(r"(\w+)(?:\[\w+\])*\s*=([^=;]*);", text):
            if "few_prepared" not in m[2] and "__ldg" not in m[2] and any(re.search(rf"\b{n}\b", m[2]) for n in made):
                made.add(m[1])
    assert {"xp", "sp"} <= made
    for arg in [a for f in ("__ldg", "__ldcs", "__ldcg") for a in calls(text, f)]:
        assert not any(re.search(rf"\b{n}\b", arg) for n in made), arg
    before = text[text.index("k_rows_few(const"):text.index("grid_wait();", text.index("k_rows_few(const"))]
    assert not any(re.search(rf"\b{n}\b", before) for n in made)


def test_a_counter_of_one_translation_unit_is_read_by_its_own_function():
    """rows_core.cuh is compiled once per format, each with a counter of
    given-up waits of its own (a static variable).  A host function in it that
    reads the counter must be static too: of one with external linkage the
    linker may keep a single copy, which reads one format's counter for all."""
    text = code("rows_core.cuh")
    own = re.findall(r"^static (?:__device__ |std::atomic<\w+> )\w*\s*(\w+)\s*[={]", text, flags=re.M)
    assert "g_rw_timeouts" in own
    found = 0
    # functions at the file's left margin, up to the closing brace there
    for m in re.finditer(r"^(?!template|namespace|struct|constexpr|enum)([^\n;{]*\([^;{]*\))\s*\{\n(.*?)^\}", text, flags=re.S | re.M):
        if re.search("__device__|__global__", m[1]) or "template" in text[:m.start()].splitlines()[-1] or not any(re.search(rf"\b{n}\b", m[2]) for n in own):
            continue
        found += 1
        assert m[1].startswith("static "), m[1]
    assert found
