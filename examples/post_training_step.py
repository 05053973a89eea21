"""Post-training steps on one packed batch, from raw token rows to updated weights.

Raw rows are packed into documents (``pack_docs``), labels and the loss mask are
made in the zigzag layout of cp context-parallel ranks (``roll_labels_zigzag``),
and a small bigram model gives logits for every position.  Three losses then
train it, one after the other, each from the logits and their gradient that
the library returns:

* the clipped policy loss, mean over documents, one advantage per document, a
  KL term against the model before training;
* the preference loss over pairs of documents;
* distillation from the eight best logits of a teacher.

    python examples/post_training_step.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import context_packed_sequence_gb300 as thd  # noqa: E402

VOCAB, EOD, CP = 1000, 999, 2


def batch(device, seed=0):
    """(tokens, labels, loss_mask, cu_seqlens_padded) of 6 raw rows of 64 tokens, all in the zigzag layout."""
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, EOD, (6, 64), generator=g, dtype=torch.int32)
    raw[:, 20] = EOD            # two documents a row
    raw[::2, 45] = EOD          # three in every other
    tok, cu_v, cu = thd.pack_docs(raw.to(device), EOD, 2 * CP)
    labels, masks, _ = thd.roll_labels_zigzag(tok, cu_v, cu, CP, 0)
    here = thd.partition_indices(cu, tok.numel(), CP).reshape(-1).long()
    return tok[here].long(), labels[0], masks[0], cu


class Bigram(torch.nn.Module):
    """Logits of the next token from the present one."""

    def __init__(self, device, seed):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        self.table = torch.nn.Parameter((torch.randn(VOCAB, VOCAB, generator=g) * 0.5).to(device))

    def forward(self, tokens):
        return self.table[tokens].bfloat16()


def train(model, tokens, loss_and_gradient, steps, lr):
    """Plain gradient descent; returns the loss before every step."""
    losses = []
    for _ in range(steps):
        logits = model(tokens)
        loss, dlogits = loss_and_gradient(logits.detach())
        losses.append(loss)
        model.table.grad = None
        logits.backward(dlogits)
        with torch.no_grad():
            model.table -= lr * model.table.grad
    return [v.item() for v in losses]


def main(device="cuda", steps=12):
    tokens, labels, mask, cu = batch(device)
    docs = cu.numel() - 1
    status = thd.new_status(device)
    model = Bigram(device, 1)
    weights, doc_ids = thd.loss_weights(mask, cu, CP, thd.DOC_MEAN, status=status)
    ref, _ = thd.token_logprobs(model(tokens).detach(), labels, mask, status=status)
    out = {}

    advantages = torch.linspace(1.0, -1.0, docs, device=device)

    def policy(logits):
        r = thd.policy_loss(logits, labels, weights, ref, advantages, ref_logprobs=ref, doc_ids=doc_ids, clip_high=0.28,
                            kl_coef=0.05, status=status)
        return r.loss, r.dlogits
    out["policy"] = train(model, tokens, policy, steps, lr=100.0)

    chosen = torch.arange(0, docs // 2, device=device, dtype=torch.int32)
    rejected = torch.arange(docs - docs // 2, docs, device=device, dtype=torch.int32)

    def preference(logits):
        lp, lse = thd.token_logprobs(logits, labels, mask, status=status)
        r = thd.preference_loss(lp, mask, cu, chosen, rejected, ref_logprobs=ref, cp=CP, beta=0.1, status=status)
        return r.loss, thd.token_logprobs_backward(logits, labels, lse, r.dlogprobs, status=status)
    out["preference"] = train(model, tokens, preference, steps, lr=10.0)

    scores, ids = torch.topk(Bigram(device, 2)(tokens).float().detach(), 8, dim=1)
    ids, scores = ids.to(torch.int32).contiguous(), scores.contiguous()

    def distill(logits):
        r = thd.distill_topk_loss(logits, ids, scores, weights, temperature=2.0, status=status)
        return r.loss, r.dlogits
    out["distillation"] = train(model, tokens, distill, steps, lr=300.0)

    thd.check_status(status, "post_training_step")
    return out


if __name__ == "__main__":
    for name, losses in main().items():
        print(f"{name:13s} " + " ".join(f"{v:8.4f}" for v in losses))
