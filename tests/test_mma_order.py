"""Products over one place of tensor memory wait for one another, read from
the sources (no GPU).

Products that accumulate in different places have no order between them, also
where one thread issues both: a product that writes where another one reads its
operand has to be issued behind a wait for that one's completion."""
import os
import re

from tree_speculative_decoding_attn_gb300 import _build


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())


def test_scores_over_the_weights_wait_for_the_values_product():
    """Prompt attention: S(j + 1) lies over P(j), which P(j) V(j) reads."""
    text = source("prompt.cu")
    issued, over = text.index("mma_commit(&bars->pv[i])"), text.index("scores(j + 1);")
    assert issued < over
    assert re.search(r"\bwait\([^;]*bars->pv\[i\]", text[issued:over]), "scores are issued over P without a wait for its product"
