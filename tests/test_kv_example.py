"""The example of a drafted-tree server gives the tokens that one-at-a-time decoding gives."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_drafted_trees_give_the_plain_tokens(full_table):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_tree_step as ex
    import workloads
    import byte_level_bpe_gb300 as tk
    tokenizer = tk.Tokenizer(full_table, workloads.SPECIALS)
    prompts = ["Shard the request over four ranks.", "1, 2, 3,", "", "中文 text, mixed", "x" * 700]
    prompts = [p or "a" for p in prompts]
    model = ex.Model(100277, 512)
    batch, first = ex.prefill(model, tokenizer, prompts, 64, 512)
    state = batch.lengths.clone(), batch.cursor.clone(), batch.table.clone()
    done, kept = ex.generate_drafted(batch, first, 6)
    assert kept > 0 and all(len(d) >= 6 for d in done)
    batch.lengths, batch.cursor, batch.table = state
    plain = ex.generate_plainly(batch, first, max(len(d) for d in done))
    model.workspace.status()
    for d, p in zip(done, plain):
        assert d == p[:len(d)]
    tokenizer.close()
