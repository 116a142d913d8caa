"""GPU: qsa_tree_attention where its parts meet: hand-over between the CTAs of a pair under load, rows far below
their maximum, workspaces of other sizes, tables that break the contract, on each of its paths."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa
from tests.drafts_testutil import make_batch, reference, run_tree

pytestmark = pytest.mark.gpu
SCALE = 1 / 16


def test_many_calls_give_the_same_bits():
    # long runs of tiles on every pair, beside calls on another stream that change what the SMs do meanwhile
    pool, seqs = make_batch([(5000, 30), (300, 25), (7100, 44), (2600, 9)], seed=41)
    params = (2048, 131072, SCALE)
    first = run_tree(pool, seqs, params=params, with_ids=False)[1]
    ref, _, bound = reference(pool, seqs, *params)
    assert (np.abs(first.double().cpu().numpy() - ref) <= bound).all()
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    tree = torch.from_numpy(pool["tree"].view(np.int32)).cuda()
    n_tok, table = pool["q"].shape[0], torch.from_numpy(seqs).cuda()
    ws = torch.empty(qsa.qsa_tree_attention_workspace_bytes(4, n_tok, 7144, params), dtype=torch.uint8, device="cuda")
    outs = torch.full((60, *first.shape), float("nan"), dtype=torch.float16, device="cuda")
    side, noise = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(side):
            noise = noise @ noise * 1e-2
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], pool["kq"].shape[0], table, 4, n_tok,
                               tree, 7144, None, outs[i], ws, params=params)
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    assert all(torch.equal(o, first) for o in outs)
