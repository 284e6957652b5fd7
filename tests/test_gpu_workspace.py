"""One workspace through calls of different batch sizes."""
import numpy as np
import pytest
import torch

from tests.helpers import pointers_from_parents
from tests.test_gpu_q8 import DEV, Att, _ops, bounds, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 64])
def test_attention_of_few_before_accept_of_many(n):
    """The attention's partial results must not lie where the accept of a larger batch counts its arrivals."""
    import oracle
    ops = _ops()
    a = Att(1, n, 8, 2, 128, 16, [3001], seed=1)
    args = list(a.device())
    b, m, S, V = 600, 4, 2, 517
    size = max(ops.spec_workspace_size(ops.OP_VERIFY_ATTENTION_Q8, 1, n, 1, 1, 8, 2, args[16]), ops.spec_workspace_size(ops.OP_VERIFY_GREEDY, b, m, 1, V))
    ws = args[-1] = ops.Workspace(size)
    gen = torch.Generator().manual_seed(2)
    nt, ns = (np.tile(x, b) for x in pointers_from_parents([-1, 0, 0, 1]))
    drafts = torch.randint(0, V, (b * m,), generator=gen, dtype=torch.int32)
    logits = torch.randn(b * m, V, generator=gen)
    for i in range(0, b * m, m):
        if i % 3:
            logits[i, drafts[i + 1]] = 9.0
    want = oracle.verify_greedy(b, m, S, logits.numpy(), drafts.numpy(), np.arange(b * m, dtype=np.int32), nt, ns)
    tree = [i32(x.tolist()) for x in (np.arange(b * m), nt, ns)]
    dev_logits, dev_drafts = logits.to(DEV), drafts.to(DEV)
    for _ in range(3):
        got = [torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((b * m,), (b, S + 1), (b,), (b, S + 1), (b,))]
        a.out.fill_(3.0)
        ops.spec_verify_attention_q8(*args)
        ops.spec_verify_greedy(b, m, S, dev_logits, dev_drafts, *tree, *got, ws)
        assert ws.last_error() == 0
        a.check()
        for x, k in zip(got, ("predict", "accept_index", "accept_lens", "accepted_tokens", "next_root")):
            assert np.array_equal(x.cpu().numpy(), want[k].reshape(x.shape)), k
