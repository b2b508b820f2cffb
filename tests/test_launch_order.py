"""Kernels that may start before the one in front of them has finished touch no
global memory before they wait for it.  Read from the sources: a race has no
result that a run could be trusted to show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_05_b200", "csrc")

# what reads or writes global memory in this library's kernels
ACCESS = re.compile(r"map\.len\(|map\.row<|tma_load_2d\(&?s?|__ldg\(|cp_async16|bulk_load\(\w+ ?\+|load_tile\(i|"
                    r"row_setup\(|p\.idx\[|qrow|part_lse \+|part_o \+|prefetch_l2\(|\.load\(q0")


def _bodies():
    """(file, kernel, text of its body) of every kernel in the sources."""
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        s = re.sub(r"//[^\n]*", "", open(f).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^{;]*?\)\)?\s+)?(\w+)\s*\(", s):
            start = s.index("{", m.end())
            depth, i = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(s[i], 0)
                i += 1
            yield os.path.basename(f), m.group(1), s[start:i]


def _dependents():
    names = set()
    for f in glob.glob(os.path.join(CSRC, "*.cu")):
        s = open(f).read()
        for m in re.finditer(r"launch_pdl\((\w+)|cudaLaunchKernelEx\(&cfg, (\w+)", s):
            n = m.group(1) or m.group(2)
            if n == "kern":                            # a choice of instantiations
                n = re.search(r"auto kern = [^;]*?(\w+_kernel)<", s[:m.start()]).group(1)
            names.add(n)
    return names - {"kernel"}


KERNELS = {k: (f, b) for f, k, b in _bodies()}


def test_the_reader_finds_the_kernels():
    assert {"attn8_kernel", "cache_write_kernel", "norm_rope_kernel", "sparse_attn_decode_kernel",
            "attn_combine_f16_kernel", "topk_seg_collect_final_kernel"} <= _dependents() <= set(KERNELS)


@pytest.mark.parametrize("name", sorted(_dependents()))
def test_dependents_wait_first(name):
    body = KERNELS[name][1]
    wait = body.find("pdl_wait();")
    assert wait >= 0
    early = [m.group(0) for m in ACCESS.finditer(body[:wait])]
    # a lambda that loads is defined, not called, above the wait
    early = [e for e in early if not (e.startswith("bulk_load") and "auto load_tile" in body[:wait])]
    assert not early, early
    # a wait that is left out needs a reason that the launcher knows
    line = body[:wait].rsplit("\n", 1)[1].strip()
    assert line in ("", "sm100::", "if (!p.after_selection)"), line


def test_only_the_path_leaves_the_wait_out():
    s = open(os.path.join(CSRC, "dsa_api.cu")).read()
    calls = re.findall(r"return run_attn\(c, s,[^;]*?(true|false)\);", s)
    assert calls == ["false", "false", "true"]
    forward = s[s.index("dsa_status dsa_forward("):]
    assert "true);" in forward[:forward.index("\n}\n")]
    # what comes before it there: a launch of the indexer or of the fill kernel that waits for everything
    assert "indexer" in open(os.path.join(CSRC, "indexer.cu")).read() and "launch_pdl" not in \
        open(os.path.join(CSRC, "indexer.cu")).read()
    topk = open(os.path.join(CSRC, "topk.cu")).read()
    assert "topk_fill_kernel<<<" in topk and "topk_row_kernel<<<" in topk
