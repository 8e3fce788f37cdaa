"""A small tied language model trained under ZeRO-3 with the vocabulary
operators: distillation from a teacher's top logits, a policy step on log
probabilities and entropy, and decoding.

The model is wte [vocab, dim] (embedding and output head), w1 [dim, hidden] and
w2 [hidden, dim]: h = x + gelu(x w1) w2, logits = h wte^T.  Its parameters live
as the ranks' shards; every pass gathers the submodules (zero3_fetch_submodules),
and every rank's gradients go into its flat bf16 buffer, which zero3_step
reduces.  The tied table's gradient has two parts there: the head's product
writes the slice, and zero3_embedding_backward adds the lookup's on top.

    python examples/tied_lm.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from zero_sharded_optimizer_shard_gb300 import zero3 as Z  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class TiedLM:
    """The sharded model and its N_d ranks' buffers, on the current device and
    stream."""

    def __init__(self, vocab=8192, dim=256, hidden=512, n_ranks=2, lr=5e-3, seed=0, device="cuda"):
        self.vocab, self.dim, self.hidden, self.nd, self.dev = vocab, dim, hidden, n_ranks, device
        shapes = [(vocab, dim), (dim, hidden), (hidden, dim)]
        numels = [a * b for a, b in shapes]
        self.plan = Z.Plan(numels, [0, 1, 1], n_ranks, threshold=0)
        self.hp = Z.hparams(lr=lr, weight_decay=0.0)
        self.t = 0
        info = self.plan.info
        g = torch.Generator().manual_seed(seed)
        flat = torch.zeros(info.psi_pad)
        self.views = []  # (offset, shape) in a flat buffer
        for t, shape in enumerate(shapes):
            o = self.plan.tensor(t).offset
            flat[o:o + numels[t]] = 0.02 * torch.randn(numels[t], generator=g)
            self.views.append((o, shape))
        S = info.shard_len
        self.master = [flat[r * S:(r + 1) * S].to(device) for r in range(n_ranks)]
        self.m = [torch.zeros(S, device=device) for _ in range(n_ranks)]
        self.v = [torch.zeros(S, device=device) for _ in range(n_ranks)]
        self.sparam = [torch.empty(S, dtype=BF, device=device) for _ in range(n_ranks)]
        self.full = torch.empty(info.psi_pad, dtype=BF, device=device)
        self.grads = [torch.zeros(info.psi_pad, dtype=BF, device=device) for _ in range(n_ranks)]
        self.gathered = [torch.empty(self.plan.submodule(k)[1], dtype=BF, device=device) for k in (0, 1)]
        self.scale = dim ** 0.5
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)
        Z.zero3_cast_params(self.plan, self._ptrs(self.master), self._ptrs(self.sparam),
                            self.full.data_ptr(), None, 0, info.psi_pad, self.stream)

    @property
    def stream(self):
        return torch.cuda.current_stream().cuda_stream

    @staticmethod
    def _ptrs(ts):
        return [t.data_ptr() for t in ts]

    def gather(self):
        """All parameters: wte, w1, w2."""
        Z.zero3_fetch_submodules(self.plan, [0, 1], self._ptrs(self.sparam), None,
                                 self._ptrs(self.gathered), self.stream)
        n1 = self.dim * self.hidden
        rest = self.gathered[1]
        return (self.gathered[0].view(self.vocab, self.dim), rest[:n1].view(self.dim, self.hidden),
                rest[n1:].view(self.hidden, self.dim))

    def release(self):
        for k in (0, 1):
            Z.zero3_release_submodule(self.plan, k)

    def forward(self, tokens, train=True):
        """Logits [n, vocab] of int32 or int64 tokens [n], and what backward() needs."""
        wte, w1, w2 = self.gather()
        n = tokens.numel()
        x = torch.empty(n, self.dim, dtype=BF, device=self.dev)
        Z.zero3_embedding_forward(wte.data_ptr(), Z.BF16, self.vocab, self.dim, self.dim,
                                  tokens.data_ptr(), id_type(tokens), n, self.scale, x.data_ptr(),
                                  Z.BF16, self.dim, self.stream)
        with torch.set_grad_enabled(train):
            leaves = [x, w1.detach(), w2.detach()]
            if train:
                for a in leaves:
                    a.requires_grad_()
            h = x + torch.nn.functional.gelu(x @ leaves[1]) @ leaves[2]
        logits = h.detach() @ wte.t()
        return logits, (tokens, leaves, h, wte)

    def backward(self, rank, dlogits, saved):
        """Rank `rank`'s gradients from those of its logits."""
        tokens, (x, w1, w2), h, wte = saved
        h.backward(dlogits @ wte)
        g = [self.grads[rank][o:o + a * b].view(a, b) for o, (a, b) in self.views]
        torch.matmul(dlogits.t(), h.detach(), out=g[0])
        g[1].copy_(w1.grad)
        g[2].copy_(w2.grad)
        n = tokens.numel()
        need = Z.zero3_embedding_workspace(n, self.vocab, self.dim)
        if self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.dev)
        Z.zero3_embedding_backward(x.grad.data_ptr(), Z.BF16, self.dim, tokens.data_ptr(),
                                   id_type(tokens), n, self.scale, 1, g[0].data_ptr(), Z.BF16,
                                   self.vocab, self.dim, self.dim, self.workspace.data_ptr(),
                                   self.workspace.numel(), self.stream)
        self.release()

    def step(self):
        self.t += 1
        Z.zero3_step(self.plan, self.hp, self.t, self._ptrs(self.grads), 0, self._ptrs(self.master),
                     self._ptrs(self.m), self._ptrs(self.v), self._ptrs(self.sparam),
                     self.full.data_ptr(), None, 0, self.plan.info.psi_pad, self.stream)


def id_type(tokens):
    return Z.I64 if tokens.dtype == torch.int64 else Z.I32


def distill_step(model, batches, temperature=1.0, hardest=None):
    """One optimizer step on the ranks' batches (tokens [n], teacher_ids [n, k]
    int32, teacher_logits [n, k] float32); returns the mean loss of all tokens.

    hardest = None: the mean loss; it and the gradient come from one call, the
    gradient in the logits' place.  Otherwise only the tokens whose loss exceeds
    `hardest` times the batch's mean are learned from, which is known after the
    losses: they first, then the gradient."""
    total = 0.0
    for rank, (tokens, ids, teacher) in enumerate(batches):
        logits, saved = model.forward(tokens)
        n, k = ids.shape
        args = (logits.data_ptr(), Z.BF16, n, model.vocab, model.vocab, teacher.data_ptr(), Z.F32,
                ids.data_ptr(), id_type(ids), k, k, 1.0 / temperature)
        loss = torch.empty(n, dtype=F32, device=model.dev)
        if hardest is None:
            w = torch.full((n,), 1.0 / n, dtype=F32, device=model.dev)
            Z.zero3_distill_loss(*args, w.data_ptr(), loss.data_ptr(), 0, logits.data_ptr(),
                                 model.vocab, model.stream)
        else:
            lse = torch.empty(n, dtype=F32, device=model.dev)
            Z.zero3_distill_loss(*args, 0, loss.data_ptr(), lse.data_ptr(), 0, 0, model.stream)
            hard = (loss > hardest * loss.mean()).to(F32)
            dloss = hard / hard.sum().clamp(min=1.0)
            Z.zero3_distill_backward(*args, lse.data_ptr(), dloss.data_ptr(), logits.data_ptr(),
                                     model.vocab, model.stream)
        model.backward(rank, logits, saved)
        total = total + loss.mean()
    model.step()
    return total / len(batches)


def policy_step(model, batches, entropy_bonus=0.01):
    """One optimizer step that raises advantage * log p(target) + entropy_bonus *
    entropy on the ranks' batches (tokens [n], targets [n], advantage [n] float32;
    a target outside the vocabulary is padding); returns the mean log
    probability and entropy."""
    lp = ent = 0.0
    for rank, (tokens, targets, advantage) in enumerate(batches):
        logits, saved = model.forward(tokens)
        n = tokens.numel()
        logprob, lse, entropy = torch.empty(3, n, dtype=F32, device=model.dev)
        row = (logits.data_ptr(), Z.BF16, n, model.vocab, model.vocab, targets.data_ptr(),
               id_type(targets), 1.0)
        Z.zero3_token_logprobs(*row, 0, logprob.data_ptr(), lse.data_ptr(), entropy.data_ptr(),
                               stream=model.stream)
        dlogprob = -advantage / n
        dentropy = torch.full((n,), -entropy_bonus / n, dtype=F32, device=model.dev)
        Z.zero3_token_logprobs_backward(*row, lse.data_ptr(), entropy.data_ptr(), dlogprob.data_ptr(),
                                        dentropy.data_ptr(), logits.data_ptr(), model.vocab,
                                        model.stream)
        model.backward(rank, logits, saved)
        lp, ent = lp + logprob.mean(), ent + entropy.mean()
    model.step()
    return lp / len(batches), ent / len(batches)


@torch.no_grad()
def decode(model, first, steps, k=5):
    """The most probable continuation of tokens [n] int32: ids [steps, n, k] and
    log probabilities [steps, n, k] of the k best tokens; the best one is the
    next input."""
    n = first.numel()
    ids = torch.empty(steps, n, k, dtype=torch.int32, device=model.dev)
    lps = torch.empty(steps, n, k, dtype=F32, device=model.dev)
    logprob = torch.empty(n, dtype=F32, device=model.dev)
    tokens = first
    for s in range(steps):
        logits, _ = model.forward(tokens, train=False)
        Z.zero3_token_logprobs(logits.data_ptr(), Z.BF16, n, model.vocab, model.vocab,
                               tokens.data_ptr(), Z.I32, 1.0, k, logprob.data_ptr(), 0, 0,
                               ids[s].data_ptr(), lps[s].data_ptr(), model.stream)
        model.release()
        tokens = ids[s, :, 0].contiguous()
    return ids, lps


def bigram_teacher(vocab, k, seed=1, device="cuda"):
    """A teacher that knows k successors of every token: ids [vocab, k] int32 and
    logits [vocab, k], falling by 0.5."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.randint(vocab, (vocab, 1), generator=g) + torch.arange(k) * (vocab // k)) % vocab
    logits = (-0.5 * torch.arange(k, dtype=F32)).expand(vocab, k).contiguous()
    return ids.to(torch.int32).to(device), logits.to(device)


def teacher_batches(teacher, vocab, n, n_ranks, seed, device="cuda"):
    ids, logits = teacher
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(n_ranks):
        tokens = torch.randint(vocab, (n,), generator=g).to(torch.int32).to(device)
        out.append((tokens, ids[tokens.long()].contiguous(), logits[tokens.long()].contiguous()))
    return out


def main():
    vocab, k, n = 4096, 8, 2048
    model = TiedLM(vocab=vocab)
    teacher = bigram_teacher(vocab, k)
    for s in range(60):
        loss = distill_step(model, teacher_batches(teacher, vocab, n, model.nd, s),
                            hardest=1.0 if s % 4 == 3 else None)
        if s % 10 == 0 or s == 59:
            print(f"distillation step {s}: loss {float(loss):.4f}")
    batch = []
    for tokens, ids, _ in teacher_batches(teacher, vocab, n, model.nd, 1000):
        batch.append((tokens, ids[:, 1].contiguous(), torch.ones(n, device=model.dev)))
    for s in range(10):
        lp, ent = policy_step(model, batch)
    print(f"policy steps: mean log probability {float(lp):.4f}, entropy {float(ent):.4f}")
    ids, lps = decode(model, batch[0][0][:4].contiguous(), 6)
    print("decoded:", ids[:, :, 0].t().tolist())


if __name__ == "__main__":
    main()
