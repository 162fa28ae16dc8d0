"""The search for a work item's sequence (find_sequence in common.hpp), run on the CPU:
tests/c/item_search.cpp compiles that function and what it uses for a wave of 64 lanes
that take turns."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COMMON = os.path.join(ROOT, "bit_tensor_activation_amd", "csrc", "common.hpp")


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    text = open(COMMON).read()
    args = text[text.index("struct KvArgs {"):]
    args = args[:args.index("};") + 2]
    rest = text[text.index("constexpr int kBlockTokens"):text.rindex("}  // namespace btq")]
    assert "find_sequence" in rest and "cut_range" in rest
    d = tmp_path_factory.mktemp("search")
    (d / "search.inc").write_text(args + "\n" + rest)
    exe = str(d / "search")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-I", str(d),
                    os.path.join(ROOT, "tests", "c", "item_search.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)

    def run(what):
        r = subprocess.run([exe, what], capture_output=True, text=True, timeout=100)
        assert r.returncode == 0 and r.stdout.strip() == "all ok", r.stdout + r.stderr
    return run


def test_items_stay_inside_the_batch_whatever_the_starts_hold(search):
    search("unordered")


def test_every_row_of_ascending_starts_has_one_item(search):
    # starts before 0 and past T among them, which are cut to the batch
    search("sorted")
