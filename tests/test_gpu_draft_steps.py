"""The step calls together, as the example runs them: pages, append, attention, gate, routing,
the FFN and the verification of drafts, prompts first and then steps, eager and captured."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests.test_gpu_route import plain as plain_route
from tests.test_gpu_verify import plain as plain_verify

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("draft_steps", os.path.join(ROOT, "examples", "draft_steps.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("prompts,drafts", [([70, 1, 33], 3), ([5], 1), ([64, 16, 17, 130, 2], 7)])
def test_steps_hang_together(lib, example, graph, prompts, drafts):
    steps, length, state = 6, list(prompts), {"turn": 0, "probs": None}

    def watch(s):
        """After each step: rows, pages, routing and verification against plain ones."""
        first = state["probs"] is None
        turn = state["turn"]
        new = prompts if first else [drafts + 1] * len(prompts)
        before = [0] * len(prompts) if first else state["keep"]
        cu = np.concatenate([[0], np.cumsum(new)])
        after = s.lengths[1 - turn].tolist()
        assert s.seen["cu"].tolist() == cu.tolist()
        assert after == [k + n for k, n in zip(before, new)]
        assert s.seen["seqs"].tolist() == [b for b, n in enumerate(new) for _ in range(n)]
        assert s.seen["positions"].tolist() == [before[b] + i for b, n in enumerate(new) for i in range(n)]
        held = [row[: -(-n // s.page)] for row, n in zip(s.table.tolist(), after)]
        free = s.free.tolist()[: s.counts[1 - turn].item()]
        assert sorted(sum(held, []) + free) == list(range(s.free.numel()))         # every page once
        logits, ids, weights = s.routed
        for t in range(0, logits.shape[0], 7):
            want, w = plain_route(logits[t].double().cpu().numpy(), s.top_k, s.bias.double().cpu().numpy(), 4, 2, 1.0, renorm=True)
            assert ids[t].tolist() == want.tolist()
            assert np.abs(weights[t].double().cpu().numpy() - w).max() <= 24 * 2.0 ** -24
        p = s.seen["probs"].double().cpu().numpy()
        # the step's own tokens and drafts are those made at the end of the step before it
        tokens = s.seen["tokens"].tolist() if first else state["tokens"]
        q = None if first else state["q"]
        u = s.u[state["step"] if not first else 0].double().tolist()
        rows = len(prompts) * (drafts + 1)
        accepted, emitted = s.accepted.tolist(), s.emitted.tolist()
        for b, n in enumerate(new):
            d = 0 if first else drafts
            a, t, bad = plain_verify(p, q, tokens, (int(cu[b]), int(cu[b + 1])), d, [0.0] * len(tokens) if first else u[:rows], u[rows + b])
            assert not bad and accepted[b] == a
            start = int(cu[b + 1]) - 1 - d
            assert emitted[b] == tokens[start + 1: start + 1 + a] + [t] + [-1] * (drafts - a)
            length[b] += 0 if first else a + 1
        assert s.keep.tolist() == length
        state.update(turn=1 - turn, probs=p, keep=list(length), tokens=s.tokens.tolist(), q=s.draft_probs.double().cpu().numpy(),
                     step=s.step_no.item())

    server, history = example.run(prompts, steps, drafts, graph=graph, watch=watch)
    assert lib.moe_read_device_status(server.err) == (lib.MOE_OK, 0)
    assert len(history) == steps + 1
    taken = sum(sum(a) for a, _ in history[1:])
    assert 0 < taken < steps * drafts * len(prompts)          # some are taken and some are not


def test_captured_steps_are_the_eager_ones(example):
    a, b = example.run([40, 7], 4, graph=False), example.run([40, 7], 4, graph=True)
    assert a[1] == b[1]
    assert torch.equal(a[0].table, b[0].table) and torch.equal(a[0].keep, b[0].keep)
