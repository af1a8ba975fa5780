"""The example's bookkeeping of rejected candidates (examples/decode_layers.py), against the plan's definition: no page
is lost or held twice, however many candidates each step rejects.  Needs no GPU."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("page,requests,k", [(16, 3, 4), (16, 1, 20), (64, 5, 7), (32, 2, 70)])
def test_no_page_is_lost_when_candidates_are_rejected(page, requests, k):
    import decode_layers as ex

    rng = np.random.default_rng(page + k)
    width, pages = 12, 12 * requests
    free = torch.from_numpy(rng.permutation(pages)).to(torch.int32)
    table = torch.full((requests, width), -1, dtype=torch.int32)
    lens = torch.zeros((requests,), dtype=torch.int32)
    opened = 0
    while int(lens.max()) + 1 + k <= width * page:
        new = rng.integers(0, k + 2, requests)
        t, seq, _, slots, used = ref.plan(lens.tolist(), new, free.tolist(), table.tolist(), int(new.sum()), page)
        assert min(slots, default=0) >= 0 and len(set(slots)) == len(slots)
        table, free = torch.from_numpy(t).to(torch.int32), free[used:]
        kept = torch.from_numpy(lens.numpy() + np.minimum(new, rng.integers(1, k + 2, requests))).to(torch.int32)
        back = ex.give_back(table, torch.tensor(seq, dtype=torch.int32), kept, page)
        opened += back.numel()
        free, lens = torch.cat([back, free]), kept
        held = table[table >= 0].tolist()
        assert sorted(held + free.tolist()) == list(range(pages))
        assert (table >= 0).sum(1).tolist() == [-(-int(n) // page) for n in lens]
    assert opened > 0       # (some rejected candidates had opened a page)
