"""Cases of the packed-sequence loss operators: label log-probabilities, the clipped policy loss, the preference loss and
the distillation loss over a teacher's top logits, forward and backward.

Every case is a microbatch of packed documents as ``pack_docs`` and ``roll_labels`` leave it: T rows of logits over a
vocabulary of V, int32 labels, a uint8 loss mask (prompts and padding are off) and the padded document boundaries, in the
contiguous layout (cp = 1) or the zigzag layout of cp ranks.  With ``own`` false ``run`` computes an operator from
elementary torch operations in 32 bits; with ``own`` true it calls this package.  ``exact`` differentiates the losses'
definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LARGEST = 8192 * 151936 * 2     # bytes of logits of the largest listed case
TINY = -1e30


def listed():
    return [
        # scoring a long packed batch under the old or the reference policy (vocabulary of the packing pipeline workload)
        dict(name="score_8192x151936_bf16", kind="score", T=8192, V=151936, dtype="bf16", cp=1, docs=9, prompt=0.0, tau=1.0),
        # one token of one sequence: the latency of a call
        dict(name="score_1x151936_bf16", kind="score", T=1, V=151936, dtype="bf16", cp=1, docs=1, prompt=0.0, tau=1.0),
        # a training step through log-probabilities with a caller's own loss on top; vocabulary and length odd, fp16
        dict(name="logprob_step_2049x50257_f16", kind="logprob_step", T=2049, V=50257, dtype="f16", cp=1, docs=5, prompt=0.25, tau=0.7),
        # one reinforcement learning microbatch in the zigzag layout, mean over documents, a third of it prompts
        dict(name="policy_8192x151936_bf16", kind="policy", T=8192, V=151936, dtype="bf16", cp=8, docs=12, prompt=0.3, tau=1.0, reduction="doc", kl=0.05),
        # the same in fp32 logits with an odd vocabulary and length and one advantage per token, no KL term
        dict(name="policy_1531x50257_f32", kind="policy", T=1531, V=50257, dtype="f32", cp=1, docs=7, prompt=0.4, tau=0.9, reduction="token", kl=0.0),
        # the tiny configuration's rows and vocabulary: launches and latency only
        dict(name="policy_24x1000_bf16", kind="policy", T=24, V=1000, dtype="bf16", cp=2, docs=3, prompt=0.25, tau=1.0, reduction="doc", kl=0.1),
        # chosen and rejected answers packed side by side, zigzag layout
        dict(name="preference_4096x151936_bf16", kind="preference", T=4096, V=151936, dtype="bf16", cp=4, docs=16, prompt=0.4, tau=1.0, beta=0.1, smooth=0.0, mean=False),
        # a short fp32 batch with ragged sizes, length-normalised, with label smoothing
        dict(name="preference_611x32003_f32", kind="preference", T=611, V=32003, dtype="f32", cp=1, docs=6, prompt=0.2, tau=1.0, beta=2.0, smooth=0.1, mean=True),
        # distilling a long batch from a teacher's 64 best logits
        dict(name="distill_4096x151936_bf16", kind="distill", T=4096, V=151936, dtype="bf16", cp=1, docs=6, prompt=0.2, tau=2.0, K=64, absent=0.0, normalize=True),
        # a teacher that kept up to 20 log-probabilities of each token: odd sizes, entries missing
        dict(name="distill_777x50257_f16", kind="distill", T=777, V=50257, dtype="f16", cp=1, docs=3, prompt=0.1, tau=1.0, K=20, absent=0.2, normalize=False),
        # the tiny configuration again
        dict(name="distill_24x1000_f32", kind="distill", T=24, V=1000, dtype="f32", cp=2, docs=3, prompt=0.0, tau=1.5, K=8, absent=0.0, normalize=True),
    ]


def draw(rng):
    kind = rng.choice(["score", "logprob_step", "policy", "preference", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    V = int(round(math.exp(rng.uniform(math.log(1000), math.log(151936)))))
    if rng.random() < 0.5:
        V = V // 128 * 128
    most = min(8192, LARGEST // (V * DTYPES[dtype].itemsize))
    T = int(round(math.exp(rng.uniform(0.0, math.log(most)))))
    cp = rng.choice([1, 1, 2, 4, 8]) if kind in ("policy", "preference") else 1
    if cp > 1:
        T = max(2 * cp, T // (2 * cp) * (2 * cp))
    T = max(T, 4 * cp) if kind == "preference" else T
    unit = 2 * cp if cp > 1 else 1
    docs = rng.randint(min(2, T // unit) if kind == "preference" else 1, min(24, T // unit))
    case = dict(kind=kind, T=T, V=V, dtype=dtype, cp=cp, docs=docs, prompt=rng.choice([0.0, 0.2, 0.5]), tau=rng.choice([0.6, 1.0, 1.3]))
    if kind == "policy":
        case.update(reduction=rng.choice(["doc", "token"]), kl=rng.choice([0.0, 0.01, 0.2]))
    if kind == "preference":
        case.update(beta=rng.choice([0.05, 0.1, 1.0]), smooth=rng.choice([0.0, 0.1]), mean=rng.random() < 0.5)
    if kind == "distill":
        case.update(K=rng.choice([1, 5, 20, 50, 64, 100, 128]), absent=rng.choice([0.0, 0.3]), normalize=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(rng, T, docs, unit):
    """`docs` document lengths, multiples of `unit`, that add up to T."""
    n = T // unit
    cuts = torch.sort(torch.randperm(n - 1, generator=rng)[:docs - 1]).values + 1 if docs > 1 else torch.empty(0, dtype=torch.int64)
    edges = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([n])])
    return [int(v) * unit for v in edges.diff()]


def _zigzag_rows(lengths, cp):
    """The global row at each position of the zigzag layout of cp ranks."""
    rows = []
    for r in range(cp):
        start = 0
        for L in lengths:
            c = L // (2 * cp)
            rows.append(torch.arange(start + r * c, start + (r + 1) * c))
            rows.append(torch.arange(start + (2 * cp - 1 - r) * c, start + (2 * cp - r) * c))
            start += L
    return torch.cat(rows)


def _active(case):
    return max(1, round(case["T"] * (1 - case["prompt"])))


def prepare(case, seed):
    T, V, cp = case["T"], case["V"], case["cp"]
    host = torch.Generator().manual_seed(seed)
    gpu = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    lengths = _lengths(host, T, case["docs"], 2 * cp if cp > 1 else 1)
    cu = torch.tensor([0] + lengths).cumsum(0)
    # prompts: the first share of every document has no loss; so has the last row (no next token) of the longer ones
    mask = torch.ones(T, dtype=torch.uint8)
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        mask[a:a + int((b - a) * case["prompt"])] = 0
        if b - a > 4:
            mask[b - 1] = 0
    if cp > 1:
        mask = mask[_zigzag_rows(lengths, cp)]
    s = dict(case=case, cu=cu.to(torch.int32).cuda(), mask=mask.cuda())
    labels = torch.randint(0, V, (T,), generator=gpu, device="cuda")
    # logits of a trained model: a broad background and a label that stands out of it by a varying amount
    logits = torch.empty(T, V, dtype=dt, device="cuda")
    lift = torch.randn(T, generator=gpu, device="cuda") * 3 + math.log(V) + 1.5
    logp = torch.empty(T, device="cuda")
    top_ids = top = None
    if case["kind"] == "distill":
        K = case["K"]
        top_ids = torch.empty(T, K, dtype=torch.int64, device="cuda")
        top = torch.empty(T, K, device="cuda")
    step = max(1, (1 << 28) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        z = torch.randn(b - a, V, generator=gpu, device="cuda") * 2
        rows = torch.arange(b - a, device="cuda")
        z[rows, labels[a:b]] += lift[a:b]
        logits[a:b] = z.to(dt)
        z = logits[a:b].float() / case["tau"]
        logp[a:b] = z[rows, labels[a:b]] - torch.logsumexp(z, 1)
        if top is not None:
            # a teacher near the student: its logits are the student's with noise, its best K kept, best first
            t = logits[a:b].float() + torch.randn(b - a, V, generator=gpu, device="cuda")
            best = torch.topk(t, K, dim=1)
            top_ids[a:b] = best.indices
            top[a:b] = best.values if case["normalize"] else best.values / case["tau"] - torch.logsumexp(t / case["tau"], 1, keepdim=True)
        del z
    s.update(logits=logits, labels=labels.to(torch.int32))
    noise = lambda scale: torch.randn(T, generator=gpu, device="cuda") * scale  # noqa: E731
    if case["kind"] == "logprob_step":
        s["dlogprobs"] = noise(1.0) / T * s["mask"]
    if case["kind"] == "policy":
        drift = noise(0.15)
        # the definition jumps where a ratio meets a clip bound: no ratio within 1e-3 of one
        for edge in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
            near = (drift - edge).abs() < 1e-3
            drift = torch.where(near, edge + torch.where(drift < edge, -1e-3, 1e-3), drift)
        s["old"] = logp - drift
        s["ref"] = logp + noise(0.3)
        s["advantages"] = torch.randn(case["docs"] if case["reduction"] == "doc" else T, generator=gpu, device="cuda")
    if case["kind"] == "preference":
        s["ref"] = logp + noise(0.3)
        order = torch.randperm(case["docs"], generator=host)
        pairs = max(1, case["docs"] // 2)
        s["chosen"] = order[:pairs].to(torch.int32).cuda()
        s["rejected"] = order[-pairs:].to(torch.int32).cuda()
    if case["kind"] == "distill":
        gone = torch.rand(T, case["K"], generator=gpu, device="cuda") < case["absent"]
        gone[:, 0] = False
        s["teacher_ids"] = torch.where(gone, -1, top_ids).to(torch.int32)
        s["teacher_scores"] = top
    return s


CLIP = (0.2, 0.28)


def work(case):
    T, V = case["T"], case["V"]
    e = DTYPES[case["dtype"]].itemsize
    rows = _active(case)
    read, written = rows * V * e + 5 * T, 8 * T
    per = 5            # scale, subtract, exponential, sum, maximum
    if case["kind"] != "score":
        written += T * V * e
        per = 9        # and scale, subtract, exponential, multiply
    if case["kind"] == "distill":
        read += rows * case["K"] * 8
    return {"bytes": read + written, "flops": rows * V * per}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return RUN[s["case"]["kind"]][1 if own else 0](s)


def _plain_rows(s):
    """(z, lse, lp): scaled logits in 32 bits, their log-sum-exp and the labels' log-probabilities."""
    z = s["logits"].float() / s["case"]["tau"]
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + (z - top).exp().sum(1).log()
    lp = z.gather(1, s["labels"].long()[:, None])[:, 0] - lse
    return z, lse, lp


def _plain_dlogits(s, z, lse, g):
    """g_t (1[v = label] - p_v) / tau, rounded once."""
    d = (z - lse[:, None]).exp() * (-g / s["case"]["tau"])[:, None]
    at = s["labels"].long()[:, None]
    d.scatter_(1, at, d.gather(1, at) + (g / s["case"]["tau"])[:, None])
    return d.to(s["logits"].dtype)


def _plain_doc_ids(s):
    """Document of each row: local slot j of every rank lies in the document whose share [cu[i]/cp, cu[i+1]/cp) holds it."""
    cp, T = s["case"]["cp"], s["case"]["T"]
    slots = torch.arange(T // cp, device="cuda", dtype=torch.int32)
    docs = torch.searchsorted(s["cu"] // cp, slots, right=True) - 1
    return docs.repeat(cp)


def _plain_weights(s, reduction):
    on = s["mask"].float()
    docs = _plain_doc_ids(s)
    if reduction == "token":
        return on / on.sum().clamp(min=1), docs
    n = torch.zeros(s["cu"].numel() - 1, device="cuda").index_add_(0, docs, on)
    return on / (n.clamp(min=1) * (n > 0).sum().clamp(min=1))[docs], docs


def _plain_score(s):
    on = s["mask"] != 0
    z, lse, lp = _plain_rows(s)
    return {"logprobs": torch.where(on, lp, 0.0), "lse": torch.where(on, lse, 0.0)}


def _own_score(s):
    import context_packed_sequence_gb300 as thd
    lp, lse = thd.token_logprobs(s["logits"], s["labels"], s["mask"], temperature=s["case"]["tau"])
    return {"logprobs": lp, "lse": lse}


def _plain_logprob_step(s):
    on = s["mask"] != 0
    z, lse, lp = _plain_rows(s)
    return {"logprobs": torch.where(on, lp, 0.0), "lse": torch.where(on, lse, 0.0), "dlogits": _plain_dlogits(s, z, lse, s["dlogprobs"])}


def _own_logprob_step(s):
    import context_packed_sequence_gb300 as thd
    tau = s["case"]["tau"]
    lp, lse = thd.token_logprobs(s["logits"], s["labels"], s["mask"], temperature=tau)
    dlogits = thd.token_logprobs_backward(s["logits"], s["labels"], lse, s["dlogprobs"], temperature=tau)
    return {"logprobs": lp, "lse": lse, "dlogits": dlogits}


def _plain_policy(s):
    c = s["case"]
    w, docs = _plain_weights(s, c["reduction"])
    adv = s["advantages"][docs] if c["reduction"] == "doc" else s["advantages"]
    on = w != 0
    z, lse, lp = _plain_rows(s)
    r = (lp - s["old"]).exp()
    cut = r.clamp(1 - CLIP[0], 1 + CLIP[1])
    used = r * adv <= cut * adv
    d = s["ref"] - lp
    kl = d.exp() - d - 1
    loss = torch.where(on, w * (c["kl"] * kl - torch.where(used, r * adv, cut * adv)), 0.0).sum()
    g = torch.where(on, w * (c["kl"] * (1 - d.exp()) - torch.where(used, r * adv, 0.0)), 0.0)
    return {"loss": loss, "kl": torch.where(on, w * kl, 0.0).sum(), "clip_fraction": torch.where(on & ~used, w, 0.0).sum(),
            "logprobs": torch.where(on, lp, 0.0), "dlogits": _plain_dlogits(s, z, lse, g)}


def _own_policy(s):
    import context_packed_sequence_gb300 as thd
    c = s["case"]
    by_doc = c["reduction"] == "doc"
    w, docs = thd.loss_weights(s["mask"], s["cu"], c["cp"], thd.DOC_MEAN if by_doc else thd.TOKEN_MEAN)
    out = thd.policy_loss(s["logits"], s["labels"], w, s["old"], s["advantages"], ref_logprobs=s["ref"], doc_ids=docs if by_doc else None,
                          clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=c["kl"], temperature=c["tau"])
    return {"loss": out.loss, "kl": out.kl, "clip_fraction": out.clip_fraction, "logprobs": out.logprobs, "dlogits": out.dlogits}


def _plain_preference(s):
    c = s["case"]
    on = s["mask"] != 0
    docs = _plain_doc_ids(s)
    z, lse, lp = _plain_rows(s)
    lp = torch.where(on, lp, 0.0)
    add = lambda v: torch.zeros(s["cu"].numel() - 1, device="cuda").index_add_(0, docs, v)  # noqa: E731
    n = add(on.float())
    per = 1 / n.clamp(min=1) if c["mean"] else torch.ones_like(n)
    sums, gain = add(lp) * per, add(torch.where(on, lp - s["ref"], 0.0)) * per
    i, j = s["chosen"].long(), s["rejected"].long()
    h = c["beta"] * (gain[i] - gain[j])
    softplus = lambda x: x.clamp(min=0) + (1 + (-x.abs()).exp()).log()  # noqa: E731
    loss = ((1 - c["smooth"]) * softplus(-h) + c["smooth"] * softplus(h)).mean()
    dh = (c["smooth"] / (1 + (-h).exp()) - (1 - c["smooth"]) / (1 + h.exp())) * c["beta"] / h.numel()
    ds = torch.zeros_like(n).index_add_(0, i, dh).index_add_(0, j, -dh)
    g = torch.where(on, (ds * per)[docs], 0.0)
    return {"loss": loss, "margins": h, "doc_logprobs": sums, "logprobs": lp, "dlogprobs": g, "dlogits": _plain_dlogits(s, z, lse, g)}


def _own_preference(s):
    import context_packed_sequence_gb300 as thd
    c = s["case"]
    lp, lse = thd.token_logprobs(s["logits"], s["labels"], s["mask"], temperature=c["tau"])
    out = thd.preference_loss(lp, s["mask"], s["cu"], s["chosen"], s["rejected"], ref_logprobs=s["ref"], cp=c["cp"], beta=c["beta"],
                              label_smoothing=c["smooth"], length_normalized=c["mean"])
    dlogits = thd.token_logprobs_backward(s["logits"], s["labels"], lse, out.dlogprobs, temperature=c["tau"])
    return {"loss": out.loss, "margins": out.margins, "doc_logprobs": out.doc_logprobs, "logprobs": lp, "dlogprobs": out.dlogprobs, "dlogits": dlogits}


def _plain_distill(s):
    c = s["case"]
    tau = c["tau"]
    w, _ = _plain_weights(s, "token")
    on = w != 0
    z, lse, _ = _plain_rows(s)
    here = s["teacher_ids"] >= 0
    ids = s["teacher_ids"].long().clamp(min=0)
    t = torch.where(here, s["teacher_scores"] / tau if c["normalize"] else s["teacher_scores"], TINY)
    if c["normalize"]:
        top = t.amax(1, keepdim=True)
        t = t - top - (t - top).exp().sum(1, keepdim=True).log()
    q = torch.where(here, t.exp(), 0.0)
    each = tau * tau * torch.where(here, q * (t - (z.gather(1, ids) - lse[:, None])), 0.0).sum(1)
    losses = torch.where(on, each, 0.0)
    d = (z - lse[:, None]).exp() * q.sum(1, keepdim=True)
    d.scatter_add_(1, ids, -q)
    d = torch.where(on[:, None], d * (w * tau)[:, None], 0.0)
    return {"loss": (w * losses).sum(), "token_losses": losses, "dlogits": d.to(s["logits"].dtype)}


def _own_distill(s):
    import context_packed_sequence_gb300 as thd
    c = s["case"]
    w, _ = thd.loss_weights(s["mask"], s["cu"], c["cp"], thd.TOKEN_MEAN)
    out = thd.distill_topk_loss(s["logits"], s["teacher_ids"], s["teacher_scores"], w, temperature=c["tau"], normalize=c["normalize"])
    return {"loss": out.loss, "token_losses": out.token_losses, "dlogits": out.dlogits}


RUN = {"score": (_plain_score, _own_score), "logprob_step": (_plain_logprob_step, _own_logprob_step), "policy": (_plain_policy, _own_policy),
       "preference": (_plain_preference, _own_preference), "distill": (_plain_distill, _own_distill)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    T, V, tau, cp = case["T"], case["V"], case["tau"], case["cp"]
    kind = case["kind"]
    on = s["mask"].cpu().bool()
    cu = s["cu"].cpu().tolist()
    # the document of each row, by walking every rank's share of every document
    doc = torch.empty(T, dtype=torch.int64)
    at = 0
    for _ in range(cp):
        for i in range(len(cu) - 1):
            n = (cu[i + 1] - cu[i]) // cp
            doc[at:at + n] = i
            at += n
    members = [torch.nonzero(on & (doc == i))[:, 0].cuda() for i in range(len(cu) - 1)]
    w = torch.zeros(T, dtype=torch.float64)
    if case.get("reduction") == "doc":
        live = [m for m in members if len(m)]
        for m in live:
            w[m.cpu()] = 1.0 / (len(m) * len(live))
    elif on.any():
        w[on] = 1.0 / int(on.sum())
    w, keep = w.cuda(), on.cuda()
    labels = s["labels"].long()
    step = max(1, (1 << 27) // V)

    def rows(a, b):
        return (s["logits"][a:b].double() / tau).requires_grad_()

    out_lp, out_lse = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    dlogits = None if kind == "score" else torch.zeros(T, V, dtype=torch.float64, device="cuda")

    def logprobs():
        for a in range(0, T, step):
            b = min(T, a + step)
            with torch.no_grad():
                z = s["logits"][a:b].double() / tau
                out_lse[a:b] = torch.logsumexp(z, 1)
                out_lp[a:b] = z.gather(1, labels[a:b, None])[:, 0] - out_lse[a:b]
        out_lp[~keep] = 0
        out_lse[~keep] = 0

    def pull(loss_of):
        """Sums the rows' losses and keeps their gradients, a block of rows at a time; loss_of(lp, z, a, b) is a scalar."""
        total = 0.0
        for a in range(0, T, step):
            b = min(T, a + step)
            z = rows(a, b)
            logp = torch.log_softmax(z, 1)
            loss = loss_of(logp.gather(1, labels[a:b, None])[:, 0], logp, a, b)
            if loss.requires_grad:
                dlogits[a:b] = torch.autograd.grad(loss, z)[0] / tau
            total = total + float(loss.detach())
        dlogits[~keep] = 0
        return torch.tensor(total, dtype=torch.float64)

    if kind == "score":
        logprobs()
        return {"logprobs": out_lp, "lse": out_lse}
    if kind == "logprob_step":
        logprobs()
        pull(lambda lp, logp, a, b: (lp * s["dlogprobs"][a:b].double()).sum())
        return {"logprobs": out_lp, "lse": out_lse, "dlogits": dlogits}
    if kind == "policy":
        adv = s["advantages"].double()
        adv = adv[doc.cuda()] if case["reduction"] == "doc" else adv
        seen = {"kl": 0.0, "clip": 0.0}

        def policy(lp, logp, a, b):
            k = keep[a:b]
            lp, wt, A = lp[k], w[a:b][k], adv[a:b][k]
            ratio = torch.exp(lp - s["old"][a:b][k].double())
            bounded = torch.clamp(ratio, 1 - CLIP[0], 1 + CLIP[1])
            gap = s["ref"][a:b][k].double() - lp
            kl = torch.expm1(gap) - gap
            seen["kl"] += float((wt * kl).sum().detach())
            seen["clip"] += float((wt * (ratio * A > bounded * A)).sum().detach())
            return (wt * (case["kl"] * kl - torch.minimum(ratio * A, bounded * A))).sum()

        logprobs()
        loss = pull(policy)
        return {"loss": loss, "kl": torch.tensor(seen["kl"], dtype=torch.float64), "clip_fraction": torch.tensor(seen["clip"], dtype=torch.float64),
                "logprobs": out_lp, "dlogits": dlogits}
    if kind == "preference":
        logprobs()
        leaf = out_lp.clone().requires_grad_()
        mean = case["mean"]
        score = lambda v, m: v[m].mean() if mean and len(m) else v[m].sum()  # noqa: E731
        sums = torch.stack([score(leaf, m) for m in members])
        ref = torch.stack([score(s["ref"].double(), m) for m in members])
        gain = sums - ref
        h = case["beta"] * (gain[s["chosen"].long()] - gain[s["rejected"].long()])
        ls = torch.nn.functional.logsigmoid
        loss = -((1 - case["smooth"]) * ls(h) + case["smooth"] * ls(-h)).mean()
        g = torch.autograd.grad(loss, leaf)[0]
        pull(lambda lp, logp, a, b: (lp * g[a:b]).sum())
        return {"loss": loss.detach(), "margins": h.detach(), "doc_logprobs": sums.detach(), "logprobs": out_lp, "dlogprobs": g, "dlogits": dlogits}
    if kind == "distill":
        losses = torch.zeros(T, dtype=torch.float64, device="cuda")

        def distill(lp, logp, a, b):
            ids = s["teacher_ids"][a:b].long()
            t = s["teacher_scores"][a:b].double()
            if case["normalize"]:
                t = torch.log_softmax(torch.where(ids >= 0, t / tau, -math.inf), 1)
            q = torch.where(ids >= 0, t.exp(), 0.0)
            gap = torch.where(ids >= 0, t, 0.0) - logp.gather(1, ids.clamp(min=0))
            each = torch.where(keep[a:b], tau * tau * (q * gap).sum(1), 0.0)
            losses[a:b] = each.detach()
            return (w[a:b] * each).sum()

        loss = pull(distill)
        return {"loss": loss, "token_losses": losses, "dlogits": dlogits}
    return None
