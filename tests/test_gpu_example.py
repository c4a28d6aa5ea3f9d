"""The example that runs append, attention, verify and distillation together:
the drafter learns the target's rows, so its loss falls and more of its drafts
are accepted, and no call reports anything."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples",
                    "speculative_round.py")


def load():
    spec = importlib.util.spec_from_file_location("speculative_round", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_drafter_learns_while_it_drafts():
    accepted, losses, status = load().main(rounds=80, verbose=False)
    assert status == 0
    assert sum(losses[-10:]) < 0.8 * sum(losses[:10])
    assert sum(accepted[-10:]) > 1.5 * sum(accepted[:10])


def test_chunks_give_the_logits_of_the_whole_text():
    """The target's logits of a text are the same whether it goes through the
    cache at once, token by token, or in chunks after rejected ones."""
    m = load()
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, V = 40, 500
    t = m.Target(V, 8, 2, 64, 1, n + 8, 16, gen)
    text = torch.randint(V, (n,), generator=gen, device="cuda")
    other = torch.randint(V, (n,), generator=gen, device="cuda")

    def run(tokens, length):
        i32 = dict(dtype=torch.int32, device="cuda")
        k = len(tokens)
        return t.logits(tokens, torch.tensor([0, k], **i32),
                        torch.tensor([length], **i32), k, None)

    whole = run(text, n)
    single = torch.cat([run(text[i:i + 1], i + 1) for i in range(n)])
    parts, at = [], 0
    for k in (7, 1, 16, 3, 13):
        run(other[at:at + k + 2], at + k + 2)  # rejected: overwritten next
        parts.append(run(text[at:at + k], at + k))
        at += k
    # bf16 activations: the same keys, summed in another order
    tol = 2.0 ** -6 * whole.abs().max()
    assert at == n
    assert bool(((single - whole).abs() <= tol).all())
    assert bool(((torch.cat(parts) - whole).abs() <= tol).all())
