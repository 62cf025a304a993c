"""The norms around a block may write over the rows that they read (h and y over x
and r, dx and dr over dy, dh, x and h), so that these are not read through loads
that want memory to be read-only for the whole kernel.  No run shows the
difference by itself: the kernels' text is looked at."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "transformer_reduce_gb300", "csrc")


def test_read_only_loads_take_gates_gammas_and_betas_alone():
    with open(os.path.join(CSRC, "block_norm.cuh"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    helper = text.index("void bn_pairs(")
    end = text.index("\n}\n", helper)
    body, rest = text[helper:end], text[:helper] + text[end:]
    assert "ld_cached16" in body and "load1_cached" in body
    assert "ld_cached16" not in rest
    vectors = r"(f|a)\.(gate|gamma_post|beta_post|gamma_pre|beta_pre)\b|gate,"
    for use in re.findall(r"bn_pairs<T, AL>\(\s*(.*)", rest) + \
            re.findall(r"load1_cached\(\s*(.*)", rest):
        assert re.match(vectors, use), use
    # statistics are read-only too; nothing else is read that way
    for use in re.findall(r"__ldg\(\s*(.*)", rest):
        assert use.startswith("a.stats_in"), use
