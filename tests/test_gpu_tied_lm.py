"""The example that trains a tied language model with the vocabulary operators
around the sharded step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from examples import tied_lm
    return tied_lm


def test_tied_gradient_holds_head_and_lookup(E):
    """The table's slice of G_q is the head's product with the lookup's gradient
    added on top in binary32 and rounded once: bit for bit what the operator
    gives on a binary32 copy of the product."""
    from zero_sharded_optimizer_shard_gb300 import zero3 as Z
    vocab, dim, n = 1000, 64, 700
    m = E.TiedLM(vocab=vocab, dim=dim, hidden=128)
    tokens = torch.randint(vocab // 8, (n,), generator=torch.Generator().manual_seed(3)).cuda()
    logits, saved = m.forward(tokens)
    d = (torch.softmax(logits.float(), 1) - torch.nn.functional.one_hot(tokens, vocab)).bfloat16()
    m.backward(1, d, saved)
    _, (x, w1, w2), h, wte = saved
    assert not m.grads[0].any()
    o, (a, b) = m.views[0]
    head = m.grads[0][o:o + a * b].view(a, b)
    torch.matmul(d.t(), h.detach(), out=head)
    want = head.float()
    Z.zero3_embedding_backward(x.grad.data_ptr(), Z.BF16, dim, tokens.data_ptr(), Z.I64, n, m.scale, 1,
                               want.data_ptr(), Z.F32, vocab, dim, dim, m.workspace.data_ptr(),
                               m.workspace.numel(), m.stream)
    got = m.grads[1][o:o + a * b].view(a, b)
    assert torch.equal(got, want.bfloat16())
    assert not torch.equal(got, head)
    assert torch.equal(got[vocab // 8:], head[vocab // 8:])  # tokens that do not occur
    for t, p in ((1, w1), (2, w2)):
        o, (a, b) = m.views[t]
        assert torch.equal(m.grads[1][o:o + a * b].view(a, b), p.grad)


@pytest.mark.parametrize("hardest", [None, 1.0])
def test_distillation_learns_the_teacher(E, hardest):
    vocab = 512
    m = E.TiedLM(vocab=vocab, dim=64, hidden=128)
    teacher = E.bigram_teacher(vocab, 8)
    losses = [float(E.distill_step(m, E.teacher_batches(teacher, vocab, 1024, m.nd, s), hardest=hardest))
              for s in range(40)]
    assert all(np.isfinite(losses))
    assert losses[-1] < 0.5 * losses[0]


def test_policy_raises_rewarded_tokens(E):
    vocab, n = 512, 600
    m = E.TiedLM(vocab=vocab, dim=64, hidden=128)
    g = torch.Generator().manual_seed(4)
    batch = []
    for _ in range(m.nd):
        tokens = torch.randint(vocab, (n,), generator=g)
        targets = (tokens * 7 + 1) % vocab
        targets[:5] = -1
        batch.append((tokens.cuda(), targets.cuda(), torch.ones(n, device="cuda")))
    lps = [float(E.policy_step(m, batch)[0]) for _ in range(20)]
    assert lps[-1] > lps[0] + 0.5


def test_decoding_takes_the_best_token(E):
    vocab = 512
    m = E.TiedLM(vocab=vocab, dim=64, hidden=128)
    first = torch.tensor([3, 500, 77], dtype=torch.int32, device="cuda")
    ids, lps = E.decode(m, first, 4, k=5)
    tokens = first
    for s in range(4):
        logits, _ = m.forward(tokens, train=False)
        m.release()
        # the lowest index among equal logits, in descending order
        order = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :5]
        assert torch.equal(ids[s].long(), order)
        assert torch.all(lps[s][:, :-1] >= lps[s][:, 1:])
        tokens = ids[s, :, 0].contiguous()
