"""Draft verification with starts that do not ascend: a range that runs backwards takes no part, and
every other sequence is that of its own range."""
import pytest
import torch

import attention_harness as ah
import selective_state_update_ssu_amd as ssu
from test_gpu_layer import Draw

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROWS, WINDOW = 9, 4
STARTS = [[0, 5, 3, 3], [0, 5, 3, 8], [5, 0, 4, 9], [0, 3, 2, 7], [7, 9, 0, 5], [4, 4, 0, 2], [0, 5, 1, 6, 2, 7],
          [3, 5, 0, 5, 9], [-1, 3, 5, 9], [0, 3, 8, 12], [0, 9, 3, 5], [2, 0, 1, 0, 2, 4, 3, 9]]


def case(seed, cu, vocab, io, scores, draft):
    d, B = Draw(seed), len(cu) - 1
    score = d.normal(ROWS, vocab) * 2
    probs = torch.softmax(d.normal(B, WINDOW, vocab) * 2, -1)
    drafts = torch.multinomial(probs.view(-1, vocab), 1, generator=d.g).view(B, WINDOW).to(torch.int32)
    for b in range(0, B, 2):  # some drafts that the target likes
        for i in range(WINDOW):
            drafts[b, i] = int(score[min(max(cu[b], 0) + i, ROWS - 1)].argmax())
    t = d.uniform(0.5, 1.5, B)
    t[1::3] = 0.0
    return dict(target=(score if scores else torch.softmax(score, -1)).to(io), drafts=drafts,
                uniforms=d.uniform(0, 1, B, WINDOW + 1), probs=probs.to(io) if draft else None,
                temperature=t if scores else None)


@pytest.mark.parametrize("cu", STARTS)
@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("vocab,io", [(5, F32), (1000, F16), (20001, BF16)])
def test_other_sequences_of_a_table_with_a_bad_range(cu, scores, draft, vocab, io):
    c = case(vocab, cu, vocab, io, scores, draft)
    tokens, counts, slack = ah.verify(c["target"], c["drafts"], c["uniforms"], cu, c["probs"], c["temperature"])
    # (As far from its border as test_gpu_batch.check asks, so that the expected numbers are certain.)
    assert not scores or min(slack) > 2.0 ** -35
    assert 0 < sum(n > 0 for n in counts)
    n = ssu.batch.verify_workspace_bytes(ROWS, len(cu) - 1, vocab, scores)
    workspace = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # numbers of no meaning
    got, accepted = ssu.verify_drafts(
        c["target"].to(DEV), c["drafts"].to(DEV), c["uniforms"].to(DEV),
        torch.tensor(cu, dtype=torch.int32, device=DEV), workspace=workspace,
        draft_probs=c["probs"].to(DEV) if draft else None,
        temperature=c["temperature"].to(DEV) if scores else None)
    assert accepted.tolist() == counts
    assert got.tolist() == tokens
