"""The order of the delta-rule scan's tensor-core products, read from the kernel's source.

Products that accumulate onto the same columns are issued one after another without a wait between them.  The
architecture keeps them in order where accumulator and shape are the same, so every product has to name an accumulator of
the table, each of which has one first column and one width, and no two may share a column.
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(__file__), "..", "bounded_memory_attention_b200", "csrc", "rma_gdn_prefill.cu")


def test_products_take_disjoint_accumulators_of_one_shape():
    src = open(SOURCE).read()
    assert src.count("ptx::mma_ts1") == 1, "a product beside product<>() may have any accumulator and shape"
    names = [n for n in re.search(r"enum \{ (kAccD[^}]*)\}", src)[1].replace(" ", "").split(",") if n != "kAccumulators"]
    columns = dict(re.findall(r"(kTm[SWXU]) = (\d+)", src))
    table = re.search(r"kAcc\[kAccumulators\] = \{(.*)\};", src)[1]
    spans = [(int(columns.get(c, c)), int(w)) for c, w in re.findall(r"\{(\w+), (\d+)\}", table)]
    assert len(spans) == len(names)
    used = sorted(x for c, w in spans for x in range(c, c + w))
    assert len(used) == len(set(used)) and used[-1] < 512
    assert set(re.findall(r" product<(\w+)", src)) == set(names)
