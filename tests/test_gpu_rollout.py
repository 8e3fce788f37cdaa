"""Drawing, learning and clipping together: rollouts from drafts, their log
probabilities, a policy step with clipped gradients."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import verify_oracle as VO  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from examples import tied_lm
    return tied_lm


def models(E, vocab=600):
    m = E.TiedLM(vocab=vocab, dim=64, hidden=128, seed=1)
    d = E.TiedLM(vocab=vocab, dim=32, hidden=64, seed=2)
    teacher = E.bigram_teacher(vocab, 8)
    for s in range(12):
        for x in (m, d):
            E.distill_step(x, E.teacher_batches(teacher, vocab, 512, x.nd, s))
    return m, d


@pytest.mark.parametrize("k", [0, 3])
def test_rollouts_are_the_definition_on_the_models_logits(E, k, monkeypatch):
    m, d = models(E)
    n, vocab = 40, m.vocab
    last = torch.randint(vocab, (n,), generator=torch.Generator().manual_seed(3)).int().cuda()
    calls = []
    real = E.Z.zero3_verify_draft

    def spy(*a):
        calls.append(a)
        return real(*a)

    monkeypatch.setattr(E.Z, "zero3_verify_draft", spy)
    seen = {}
    for name, model in (("target", m), ("draft", d)):
        def forward(tokens, train=True, model=model, name=name):
            out = type(model).forward(model, tokens, train)
            seen.setdefault(name, []).append(out[0].clone())
            return out
        model.forward = forward
    g = torch.Generator("cuda").manual_seed(5)
    counts, tokens, lps = E.speculate(m, d, last, k, g, temperature=0.5)
    assert len(calls) == k + 1
    # the same random numbers, in the order in which they are drawn
    g = torch.Generator("cuda").manual_seed(5)
    for _ in range(k):
        torch.empty(n, vocab, device="cuda").exponential_(generator=g)
    u = torch.rand(n, k, device="cuda", generator=g)
    e = torch.empty(n, vocab, device="cuda").exponential_(generator=g)
    x = seen["target"][0].view(n, k + 1, vocab).double().cpu().numpy()
    y = torch.stack(seen["draft"], 1).double().cpu().numpy() if k else None
    ids = np.zeros((n, 0), int)
    if k:  # what the draft drew
        g2 = torch.Generator("cuda").manual_seed(5)
        ids = np.stack([VO.verify(y[:, j:j + 1], None, np.zeros((n, 0)), np.zeros((n, 0)),
                                  torch.empty(n, vocab, device="cuda").exponential_(generator=g2).double()
                                  .cpu().numpy(), 2.0)[1][:, 0] for j in range(k)], 1)
    want = VO.verify(x, y, ids, u.double().cpu().numpy(), e.double().cpu().numpy(), 2.0, 2.0)
    np.testing.assert_array_equal(counts.cpu().numpy(), want[0])
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[1])
    assert np.all(np.abs(lps.cpu().numpy() - want[2]) <= 1.3e-5 + 2.0 ** -21 * np.abs(want[2]))


def test_a_clipped_policy_step_on_rollouts(E):
    """The rollout's log probabilities are the policy's own; the clipped step is the
    unclipped one on gradients that have been scaled down."""
    m, d = models(E)
    n, k, vocab = 64, 3, m.vocab
    g = torch.Generator("cuda").manual_seed(6)
    batches = []
    for r in range(m.nd):
        last = torch.randint(vocab, (n,), generator=torch.Generator().manual_seed(r)).int().cuda()
        counts, tokens, lps = E.speculate(m, d, last, k, g)
        inputs, targets, adv = E.rollout_batch(last, tokens, torch.ones_like(lps))
        batches.append((inputs, targets, adv))
        logits, _ = m.forward(inputs, train=False)
        m.release()
        lp = torch.empty(n * (k + 1), device="cuda")
        E.Z.zero3_token_logprobs(logits.data_ptr(), E.Z.BF16, n * (k + 1), vocab, vocab,
                                 targets.data_ptr(), E.Z.I32, 1.0, 0, lp.data_ptr(), stream=m.stream)
        live = targets >= 0
        assert torch.equal(live.view(n, k + 1).sum(1), counts + 1)
        assert torch.all((lp - lps.view(-1))[live].abs() <= 2.6e-5 + 2.0 ** -20 * lp[live].abs())
    before = [x.clone() for x in m.master]
    E.policy_step(m, batches, max_norm=1e-2)
    inv = np.float32(1.0 / m.nd)
    total = sum(x.float() for x in m.grads) * float(inv)
    norm = float(total.double().norm())
    assert abs(float(m.norm) - norm) <= 9 * 2.0 ** -24 * norm + 2.0 ** -23 * norm
    assert norm > 1e-2  # clipped
    assert all(not torch.equal(a, b) for a, b in zip(before, m.master))
    assert all(torch.isfinite(x).all() for x in m.master)


def test_unclipped_steps_are_the_plain_ones(E):
    a, _ = models(E)
    b, _ = models(E)
    assert all(torch.equal(x, y) for x, y in zip(a.master, b.master))
    a.step()
    b.step(max_norm=float("inf"))
    assert all(torch.equal(x, y) for x, y in zip(a.master, b.master))
    assert torch.equal(a.full, b.full)
