"""Losses of a packed batch (label log-probabilities, clipped policy loss,
preference loss, distillation from a teacher's top logits): the GPU against the
64-bit oracle, the oracle's gradients against central differences, and every
refusal.

Tolerances.  A row's sum of exponentials is held in 32 bits: its terms carry
the exponential's 2^-22 and the rounding of an exponent of at most 2^5 (2^-19),
both weighted by the term's share of the sum, and adding n terms rounds n
times at random signs; together well below 2e-6 of the sum, which is the
absolute error of the log-sum-exp.  A scalar is then rounded to 32 bits.  So
log-probabilities: 3e-6 + 2.4e-7 |x|.  Sums over n such rows: n times that,
times the weights.  A gradient g (1[v = y] - p_v) has the relative error of
the exponential and of the sum (8e-6 of g p_v), the error of g itself, and one
rounding to the type of the logits: half an ulp, 2^-9 (bf16), 2^-12 (f16; 2^-25
absolute below its normal range), doubled because the values before rounding
may differ.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import losses as O
import context_packed_sequence_gb300 as thd
from context_packed_sequence_gb300 import _lib as L

gpu = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.4e-7}
FLOOR = {BF16: 1e-30, F16: 2.0 ** -24, F32: 1e-30}


def lp_tol(x):
    return 3e-6 + 2.4e-7 * np.abs(np.where(np.isfinite(x), x, 0))


def same(got, want, tol):
    """|got - want| <= tol where want is finite, equal elsewhere."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (got[~fine], want[~fine])
    off = np.abs(got - want) - np.broadcast_to(tol, want.shape)
    bad = np.where(fine, off, -1.0) > 0
    assert not bad.any(), (int(bad.sum()), got[bad][:5], want[bad][:5])


def same_gradient(got, want, dtype, row_error):
    """row_error [T]: error of the row's coefficient g, and 8e-6 |g| for p."""
    want = np.asarray(want)
    tol = np.abs(want) * (ROUND[dtype] + 8e-6) + np.asarray(row_error)[:, None] + FLOOR[dtype]
    same(got.double().cpu().numpy(), want, tol)


def make_logits(seed, T, V, dtype, stride=None, offset=0, spread=3.0):
    """[T, V] logits on the GPU, a view of a wider buffer when stride or offset ask for one; and the same in numpy."""
    g = np.random.default_rng(seed)
    stride = V if stride is None else stride
    buf = torch.full((offset + T * stride + 64,), float("nan"), dtype=dtype, device="cuda")
    z = buf[offset:offset + T * stride].view(T, stride)[:, :V] if T else buf[:0].view(0, V)
    vals = torch.from_numpy((g.standard_normal((T, V)) * spread).astype(np.float32)).to("cuda").to(dtype)
    if T:
        z.copy_(vals)
    return z, vals.double().cpu().numpy()


def dev(x, dtype):
    return torch.as_tensor(np.asarray(x), device="cuda").to(dtype).contiguous()


SHAPES = [  # T, V, row stride (None: V), offset of the first element
    (1, 1, None, 0), (3, 2, None, 0), (5, 7, None, 0), (4, 33, 40, 0), (7, 1000, None, 0), (2, 1000, None, 3),
    (3, 4097, None, 0), (3, 4096, 4099, 1), (2, 32003, None, 0), (2, 50257, 50304, 0), (1, 151936, None, 0),
    (3, 151936, None, 5),
]
TYPES = [BF16, F16, F32]


# ---------------------------------------------------------------------------
# the oracle itself
# ---------------------------------------------------------------------------

def _differences(f, z, h=1e-5):
    d = np.zeros_like(z)
    for i in np.ndindex(*z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        d[i] = (f(up) - f(down)) / (2 * h)
    return d


def test_oracle_gradients_are_the_losses_differences():
    """Central differences: error h^2 f''' / 6 ~ 1e-10 and rounding 1e-16 / h ~ 1e-11 per unit of the loss."""
    g = np.random.default_rng(0)
    T, V = 6, 9
    z = g.standard_normal((T, V)) * 2
    y = g.integers(0, V, T)
    w = np.array([0.5, 0.0, 0.25, 1.0, 0.125, 0.5])
    old = O.token_logprobs(z, y, tau=0.7)[0] + g.standard_normal(T) * 0.1
    ref = old + g.standard_normal(T) * 0.3
    A = g.standard_normal(T)
    pol = lambda x: O.policy_loss(x, y, w, old, A, ref=ref, kl_coef=0.3, tau=0.7)  # noqa: E731
    assert np.allclose(pol(z)["dlogits"], _differences(lambda x: pol(x)["loss"], z), atol=1e-8)
    ids = g.integers(-1, V, (T, 4))
    sc = g.standard_normal((T, 4))
    for norm in (True, False):
        dis = lambda x: O.distill_topk_loss(x, ids, sc - (0 if norm else 3), w, tau=1.7, normalize=norm)  # noqa: E731
        assert np.allclose(dis(z)["dlogits"], _differences(lambda x: dis(x)["loss"], z), atol=1e-8)
    cu, mask = [0, 2, 2, 4, 6], [1, 1, 0, 1, 1, 1]
    for kw in (dict(), dict(label_smoothing=0.2, margin=0.5, length_normalized=True)):
        pref = lambda lp: O.preference_loss(lp, mask, cu, [0, 3, 2], [2, 0, 1], ref=ref, beta=0.8, **kw)  # noqa: E731
        lp = O.token_logprobs(z, y)[0]
        assert np.allclose(pref(lp)["dlogprobs"], _differences(lambda x: pref(x)["loss"], lp), atol=1e-8)
        gp = pref(lp)["dlogprobs"]
        through = lambda x: pref(O.token_logprobs(x, y)[0])["loss"]  # noqa: E731
        assert np.allclose(O.token_logprobs_backward(z, y, gp), _differences(through, z), atol=1e-8)


def test_oracle_weights():
    w, docs = O.loss_weights([1, 1, 0, 1], [0, 2, 2, 4], 1, O.DOC_MEAN)
    assert docs.tolist() == [0, 0, 2, 2] and w.tolist() == [0.25, 0.25, 0.0, 0.5]
    w, docs = O.loss_weights([1, 0, 1, 1, 0, 0, 1, 1], [0, 4, 8], 2, O.TOKEN_MEAN)
    assert docs.tolist() == [0, 0, 1, 1] * 2 and w.tolist() == [0.2, 0, 0.2, 0.2, 0, 0, 0.2, 0.2]
    assert O.loss_weights([0, 0], [0, 2], 1, O.DOC_MEAN)[0].tolist() == [0, 0]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_host_checks_return_before_any_launch():
    """Bad arguments come back as THD_ERR_INVALID_ARG from the C entries; nothing is enqueued (there is no GPU here)."""
    lib = L.load()
    fake = 1 << 20

    def z(**kw):
        a = dict(data=fake, rows=4, row_stride=8, vocab=8, dtype=L.DTYPE_BF16, temperature=1.0, reserved=0)
        a.update(kw)
        return ctypes.byref(L.ThdLogits(*a.values()))

    def grad(**kw):
        a = dict(dlogits=fake * 2, row_stride=8, scale=1.0, reserved=0)
        a.update(kw)
        return ctypes.byref(L.ThdGradient(*a.values()))

    bad_z = [dict(data=None), dict(data=fake + 1), dict(rows=-1), dict(rows=1 << 31), dict(row_stride=7), dict(vocab=0),
             dict(dtype=3), dict(dtype=-1), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
             dict(temperature=1e5), dict(row_stride=1 << 62)]
    bad_g = [dict(dlogits=None), dict(dlogits=fake * 2 + 1), dict(row_stride=7), dict(scale=float("inf")),
             dict(scale=float("nan")), dict(dlogits=fake + 16), dict(dlogits=fake, row_stride=16)]
    INV = L.ERR_INVALID_ARG
    score = lambda zz, y=fake, lp=fake, lse=fake: lib.thd_token_logprobs(zz, y, None, lp, lse, None, None)  # noqa: E731
    back = lambda zz, g, y=fake, lse=fake, dl=fake: lib.thd_token_logprobs_backward(zz, y, lse, dl, g, None, None)  # noqa: E731
    for kw in bad_z:
        assert score(z(**kw)) == INV, kw
        assert back(z(**kw), grad()) == INV, kw
    assert score(None) == INV and score(z(), y=None) == INV and score(z(), lp=None) == INV and score(z(), lse=None) == INV
    for kw in bad_g:
        assert back(z(), grad(**kw)) == INV, kw
    assert back(z(), None) == INV and back(z(), grad(), y=None) == INV and back(z(), grad(), lse=None) == INV
    assert back(z(), grad(), dl=None) == INV

    def pol(**kw):
        a = dict(old_logprobs=fake, ref_logprobs=None, advantages=fake, doc_ids=None, num_docs=0, clip_low=0.2,
                 clip_high=0.2, kl_coef=0.0)
        a.update(kw)
        return ctypes.byref(L.ThdPolicy(*a.values()))

    def policy(zz, p, g=None, y=fake, w=fake, lp=fake, sums=fake, ws=fake, n=48):
        return lib.thd_policy_loss(zz, y, w, p, g, lp, sums, ws, n, None, None)

    assert lib.thd_policy_loss_workspace_bytes(4) == 48 and lib.thd_policy_loss_workspace_bytes(-1) == 0
    for kw in bad_z:
        assert policy(z(**kw), pol()) == INV, kw
    for kw in bad_g:
        assert policy(z(), pol(), grad(**kw)) == INV, kw
    for kw in (dict(old_logprobs=None), dict(advantages=None), dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-1.0),
               dict(clip_high=float("inf")), dict(clip_low=float("nan")), dict(kl_coef=float("nan")),
               dict(doc_ids=fake, num_docs=-1)):
        assert policy(z(), pol(**kw)) == INV, kw
    for kw in (dict(y=None), dict(w=None), dict(lp=None), dict(sums=None), dict(ws=None), dict(n=47), dict(ws=fake + 2)):
        assert policy(z(), pol(), **kw) == INV, kw
    assert policy(z(), None) == INV

    def teacher(**kw):
        a = dict(ids=fake, scores=fake, count=4, dtype=L.DTYPE_F32, normalize=1, reserved=0)
        a.update(kw)
        return ctypes.byref(L.ThdTeacher(*a.values()))

    def distill(zz, te, g=None, w=fake, tl=fake, loss=fake):
        return lib.thd_distill_topk_loss(zz, te, w, g, tl, loss, None, None)

    for kw in bad_z:
        assert distill(z(**kw), teacher()) == INV, kw
    for kw in bad_g:
        assert distill(z(), teacher(), grad(**kw)) == INV, kw
    for kw in (dict(ids=None), dict(scores=None), dict(scores=fake + 2), dict(count=0), dict(count=1025), dict(dtype=7)):
        assert distill(z(), teacher(**kw)) == INV, kw
    assert distill(z(), None) == INV and distill(z(), teacher(), w=None) == INV
    assert distill(z(), teacher(), tl=None) == INV and distill(z(), teacher(), loss=None) == INV

    def weights(mask=fake, cu=fake, n=2, T=2052, cp=2, red=0, w=fake, docs=None, ws=fake, nb=8):
        return lib.thd_loss_weights(mask, cu, n, T, cp, red, w, docs, ws, nb, None, None)

    size = lib.thd_loss_weights_workspace_bytes
    assert size(2, 2048) == 0 and size(2, 2049) == 8 and size(2048, 8) == 0 and size(2049, 8) == 4 * 2049 and size(-1, 8) == 0
    for kw in (dict(mask=None), dict(cu=None), dict(n=-1), dict(T=-1), dict(T=1 << 31), dict(T=6), dict(cp=0), dict(cp=65),
               dict(red=3), dict(red=-1), dict(w=None), dict(ws=None), dict(nb=7), dict(ws=fake + 1)):
        assert weights(**kw) == INV, kw

    def pref(lp=fake, mask=fake, cu=fake, n=2, T=8, cp=2, c=fake, r=fake, P=1, beta=0.1, eps=0.0, margin=0.0, loss=fake,
             margins=fake, dlp=fake, g=fake, ws=fake, nb=16, params=True):
        p = ctypes.byref(L.ThdPreference(None, beta, eps, margin, 0)) if params else None
        return lib.thd_preference_loss(lp, mask, cu, n, T, cp, c, r, P, p, loss, margins, dlp, g, ws, nb, None, None)

    assert lib.thd_preference_loss_workspace_bytes(2) == 16
    for kw in (dict(lp=None), dict(mask=None), dict(cu=None), dict(n=-1), dict(T=6), dict(cp=65), dict(c=None), dict(r=None),
               dict(P=-1), dict(beta=float("inf")), dict(eps=-0.1), dict(eps=1.1), dict(eps=float("nan")),
               dict(margin=float("nan")), dict(loss=None), dict(margins=None), dict(dlp=None), dict(g=None), dict(ws=None),
               dict(nb=15), dict(params=False)):
        assert pref(**kw) == INV, kw


def test_structs_match_the_header(tmp_path):
    """ctypes mirrors against sizeof and offsetof from the C compiler."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    mirrors = {"thd_logits_t": L.ThdLogits, "thd_gradient_t": L.ThdGradient, "thd_policy_t": L.ThdPolicy,
               "thd_preference_t": L.ThdPreference, "thd_teacher_t": L.ThdTeacher}
    lines = []
    for c, m in mirrors.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in m._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include "thd.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    r = subprocess.run([cc, "-std=c11", str(src), "-o", str(tmp_path / "s"), "-I", os.path.join(root, "include"),
                        "-I", os.path.join(cuda, "include")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    want = []
    for m in mirrors.values():
        want.append(ctypes.sizeof(m))
        want += [getattr(m, f).offset for f, _ in m._fields_]
    assert got == want


def test_python_layer_refuses_cpu_tensors():
    z, y = torch.zeros(2, 4), torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(2)
    with pytest.raises(TypeError):
        thd.token_logprobs(z, y)
    with pytest.raises(TypeError):
        thd.policy_loss(z, y, f, f, f)
    with pytest.raises(TypeError):
        thd.distill_topk_loss(z, y, f, f)
    with pytest.raises(TypeError):
        thd.loss_weights(torch.zeros(2, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        thd.preference_loss(f, y, y, y, y)


@gpu
def test_python_layer_refuses_shapes_and_types():
    z = torch.zeros(4, 8, device="cuda", dtype=BF16)
    y = torch.zeros(4, device="cuda", dtype=torch.int32)
    f = torch.zeros(4, device="cuda")
    for bad in (z.double(), z.int()):
        with pytest.raises(TypeError):
            thd.token_logprobs(bad, y)
    for bad in (z[0], z.t(), z[:, ::2], z[:, :0], z.as_strided((4, 8), (4, 1)), z.unsqueeze(0)):
        with pytest.raises(ValueError):
            thd.token_logprobs(bad, y)
    with pytest.raises(TypeError):
        thd.token_logprobs(z, y.long())
    with pytest.raises(ValueError):
        thd.token_logprobs(z, y[:3])
    with pytest.raises(TypeError):
        thd.token_logprobs(z, y, loss_mask=torch.ones(4, device="cuda", dtype=torch.bool))
    with pytest.raises(thd.ThdError) as e:
        thd.token_logprobs(z, y, temperature=0.0)
    assert e.value.kind == "invalid_arg"
    with pytest.raises(ValueError):
        thd.token_logprobs_backward(z, y, f, f, out=torch.zeros(4, 9, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        thd.token_logprobs_backward(z, y, f, f, out=torch.zeros(4, 8, device="cuda"))
    big = torch.zeros(8, 8, device="cuda", dtype=BF16)
    with pytest.raises(thd.ThdError):  # partly overlapping
        thd.token_logprobs_backward(big[:4], y, f, f, out=big[2:6])
    with pytest.raises(ValueError):
        thd.policy_loss(z, y, f, f, f[:3])
    with pytest.raises(TypeError):
        thd.policy_loss(z, y, f, f, f, doc_ids=f)
    with pytest.raises(thd.ThdError):
        thd.policy_loss(z, y, f, f, f, clip_low=-1.0)
    ids = torch.zeros(4, 3, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        thd.distill_topk_loss(z, ids, torch.zeros(4, 2, device="cuda"), f)
    with pytest.raises(TypeError):
        thd.distill_topk_loss(z, ids, ids, f)
    with pytest.raises(thd.ThdError):
        thd.distill_topk_loss(z, torch.zeros(4, 1025, device="cuda", dtype=torch.int32), torch.zeros(4, 1025, device="cuda"), f)
    m = torch.ones(8, device="cuda", dtype=torch.uint8)
    cu = torch.tensor([0, 8], device="cuda", dtype=torch.int32)
    with pytest.raises(thd.ThdError):
        thd.loss_weights(m, cu, cp=3)
    with pytest.raises(thd.ThdError):
        thd.loss_weights(m, cu, reduction=5)
    with pytest.raises(ValueError):
        thd.preference_loss(torch.zeros(8, device="cuda"), m, cu, y, y[:2])


# ---------------------------------------------------------------------------
# weights and documents
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("lengths,cp", [([1], 1), ([3, 0, 5, 1], 1), ([0, 0, 7], 1), ([4, 8, 0, 12], 2), ([16, 48, 16], 8),
                                        ([12, 24], 3), ([1000, 37, 2051], 1), ([128 * 40, 64], 4), ([2] * 700, 1), ([1] * 2049, 1),
                                        ([2000, 48], 1), ([2000, 49], 1), ([8 * 2000, 0, 8 * 301], 4)])
@pytest.mark.parametrize("reduction", [thd.TOKEN_MEAN, thd.DOC_MEAN, thd.TOKEN_SUM])
def test_loss_weights(lengths, cp, reduction):
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T = cu[-1]
    for seed, share in ((0, 0.6), (1, 0.0), (2, 1.0)):
        mask = (np.random.default_rng(seed).random(T) < share).astype(np.uint8)
        st = thd.new_status()
        w, docs = thd.loss_weights(dev(mask, torch.uint8), dev(cu, torch.int32), cp, reduction, status=st)
        thd.check_status(st)
        want_w, want_docs = O.loss_weights(mask, cu, cp, reduction)
        assert docs.tolist() == want_docs.tolist()
        same(w.cpu().numpy(), want_w, 2.4e-7 * want_w)   # two roundings


@gpu
def test_boundary_errors_reach_the_status_word():
    m = torch.ones(8, device="cuda", dtype=torch.uint8)
    f = torch.zeros(8, device="cuda")
    pair = torch.zeros(1, device="cuda", dtype=torch.int32)
    for cu, cp, kind in (([4, 8], 2, "cu_nonzero_start"), ([0, 8, 4, 8], 2, "cu_non_monotone"), ([0, 6, 8], 2, "len_not_divisible"),
                         ([0, 4], 2, "total_mismatch"), ([0, 16], 1, "total_mismatch"), ([0, -3, 8], 1, "cu_non_monotone")):
        c = dev(cu, torch.int32)
        st = thd.new_status()
        thd.loss_weights(m, c, cp, status=st)
        assert L.STATUS_NAMES[thd.status_read(st)] == kind
        st = thd.new_status()
        thd.preference_loss(f, m, c, pair, pair, cp=cp, status=st)
        assert L.STATUS_NAMES[thd.status_read(st)] == kind
    st = thd.new_status()
    thd.loss_weights(m, dev([0, 5, 8], torch.int32), 1, status=st)   # any length goes in the contiguous layout
    thd.check_status(st)


# ---------------------------------------------------------------------------
# log-probabilities
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,stride,offset", SHAPES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_token_logprobs_forward_and_backward(T, V, stride, offset, dtype, tau):
    z, zn = make_logits(T * 1000 + V, T, V, dtype, stride, offset)
    g = np.random.default_rng(V)
    y = g.integers(0, V, T)
    mask = np.ones(T, dtype=np.uint8)
    if T > 2:
        mask[1] = 0
        z[1] = float("nan")     # what a masked row holds is not read
    st = thd.new_status()
    lp, lse = thd.token_logprobs(z, dev(y, torch.int32), dev(mask, torch.uint8), temperature=tau, status=st)
    want_lp, want_lse = O.token_logprobs(zn, y, mask, tau)
    same(lp.cpu().numpy(), want_lp, lp_tol(want_lp))
    same(lse.cpu().numpy(), want_lse, lp_tol(want_lse))
    up = g.standard_normal(T) * mask
    d = thd.token_logprobs_backward(z, dev(y, torch.int32), lse, dev(up, F32), temperature=tau, grad_scale=2.0, status=st)
    thd.check_status(st)
    up32 = dev(up, F32).double().cpu().numpy() * 2
    want = O.token_logprobs_backward(zn, y, up32, tau)
    # the saved lse is itself rounded: 2.4e-7 |lse| of p
    same_gradient(d, want, dtype, np.abs(up32) / tau * (8e-6 + 2.4e-7 * np.abs(want_lse)))


@gpu
def test_no_mask_and_no_status():
    z, zn = make_logits(5, 4, 300, F32)
    y = np.array([0, 299, 7, 150])
    lp, lse = thd.token_logprobs(z, dev(y, torch.int32))
    want_lp, want_lse = O.token_logprobs(zn, y)
    same(lp.cpu().numpy(), want_lp, lp_tol(want_lp))
    same(lse.cpu().numpy(), want_lse, lp_tol(want_lse))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [5, 1000, 70001])
def test_infinities_and_lowest_values(dtype, V):
    """Rows of: one finite logit; the type's lowest value everywhere; nothing above -inf; half of the vocabulary at
    -inf; the label at -inf; +inf; NaN."""
    low = torch.finfo(dtype).min
    z, zn = make_logits(V, 7, V, dtype)
    y = np.array([V // 2, 1, 2, V - 1, 3, 0, 0])
    zn = zn.copy()
    zn[0] = -np.inf
    zn[0, V // 2] = 2.0
    zn[1] = low
    zn[2] = -np.inf
    zn[3, : V // 2] = -np.inf
    zn[4, 3] = -np.inf
    zn[5, V - 1] = np.inf
    zn[6, V - 2] = np.nan
    z.copy_(torch.from_numpy(zn).to(dtype).cuda())
    lp, lse = (t.cpu().numpy() for t in thd.token_logprobs(z, dev(y, torch.int32)))
    with np.errstate(all="ignore"):
        want_lp, want_lse = O.token_logprobs(zn[:5], y[:5])
    same(lp[:5], want_lp, lp_tol(want_lp))
    same(lse[:5], want_lse, 3e-6 + 2.4e-7 * np.abs(np.where(np.isfinite(want_lse), want_lse, 0)))
    assert lp[2] == -np.inf and lse[2] == -np.inf and lp[4] == -np.inf
    assert lse[5] == np.inf and lp[5] == -np.inf and np.isnan(lp[6]) and np.isnan(lse[6])
    up = np.array([1.0, -2.0, 3.0, 0.5])
    d = thd.token_logprobs_backward(z[:4], dev(y[:4], torch.int32), dev(lse[:4], F32), dev(up, F32))
    want = O.token_logprobs_backward(zn[:4], y[:4], up)
    # lse of row 1 is the lowest value itself (rounded like one), so p there is known only as far as exp(lse - z)
    assert not torch.isnan(d).any() and (d[2] == 0).all()
    rows = [0, 2, 3]
    same_gradient(d[rows], want[rows], dtype, np.abs(up[rows]) * 1e-5)


# ---------------------------------------------------------------------------
# policy loss
# ---------------------------------------------------------------------------

def _policy_case(seed, zn, y, tau, T, docs=None):
    g = np.random.default_rng(seed)
    lp = O.token_logprobs(zn, y, tau=tau)[0]
    drift = g.standard_normal(T) * 0.3
    for edge in (np.log(0.8), np.log(1.28)):    # not within 1e-3 of where the loss jumps
        drift = np.where(np.abs(drift - edge) < 1e-3, edge + 2e-3, drift)
    old = (lp - drift).astype(np.float32)
    ref = (lp + g.standard_normal(T) * 0.3).astype(np.float32)
    n = T if docs is None else int(docs.max()) + 1
    A = g.standard_normal(n).astype(np.float32)
    return old, ref, A


def _check_policy(out, want, w, dtype, A_of_row, kl, tau, scale=1.0):
    w = np.abs(np.asarray(w, dtype=np.float64))
    same(out.logprobs.cpu().numpy(), want["logprobs"], lp_tol(want["logprobs"]))
    # d loss / d lp is at most r |A| + kl exp(d) <= 8 |A| + 8 here
    slope = 8 * np.abs(A_of_row) + 8 * abs(kl)
    err = 5e-6 * slope + 5e-7 * (1 + slope)
    same(out.loss.item(), want["loss"], (w * err).sum())
    same(out.kl.item(), want["kl"], (w * 8 * 5e-6).sum() + 1e-9)
    same(out.clip_fraction.item(), want["clip_fraction"], 1e-6 * w.sum())
    if out.dlogits is not None:
        same_gradient(out.dlogits, want["dlogits"] * scale, dtype, scale * w * slope * 1.6e-5 / tau)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,stride,offset", SHAPES)
def test_policy_loss(T, V, stride, offset, dtype):
    tau = 0.8
    z, zn = make_logits(T * 77 + V, T, V, dtype, stride, offset)
    g = np.random.default_rng(V + 1)
    y = g.integers(0, V, T)
    w = np.abs(g.standard_normal(T)).astype(np.float32)
    if T > 2:
        w[2] = 0
        z[2] = float("nan")
    old, ref, A = _policy_case(V, zn, y, tau, T)
    for kl in (0.0, 0.2):
        st = thd.new_status()
        out = thd.policy_loss(z, dev(y, torch.int32), dev(w, F32), dev(old, F32), dev(A, F32),
                              ref_logprobs=dev(ref, F32) if kl else None, clip_low=0.2, clip_high=0.28, kl_coef=kl,
                              temperature=tau, status=st)
        thd.check_status(st)
        want = O.policy_loss(zn, y, w, old, A, ref=ref if kl else None, clip_low=0.2, clip_high=0.28, kl_coef=kl, tau=tau)
        _check_policy(out, want, w, dtype, A, kl, tau)
        alone = thd.policy_loss(z, dev(y, torch.int32), dev(w, F32), dev(old, F32), dev(A, F32),
                                ref_logprobs=dev(ref, F32) if kl else None, clip_low=0.2, clip_high=0.28, kl_coef=kl,
                                temperature=tau, need_dlogits=False)
        assert alone.dlogits is None and alone.loss.item() == out.loss.item() and torch.equal(alone.logprobs, out.logprobs)


@gpu
@pytest.mark.parametrize("cp", [1, 2, 4])
def test_policy_loss_over_documents(cp):
    """One advantage per document, mean over documents, rows in the layout of cp ranks."""
    lengths = [16, 0, 32, 8]
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T, V = cu[-1], 509
    z, zn = make_logits(cp, T, V, BF16)
    g = np.random.default_rng(cp)
    y = g.integers(0, V, T)
    mask = (g.random(T) < 0.7).astype(np.uint8)
    w, docs = thd.loss_weights(dev(mask, torch.uint8), dev(cu, torch.int32), cp, thd.DOC_MEAN)
    want_w, want_docs = O.loss_weights(mask, cu, cp, O.DOC_MEAN)
    old, ref, A = _policy_case(cp, zn, y, 1.0, T, want_docs)
    out = thd.policy_loss(z, dev(y, torch.int32), w, dev(old, F32), dev(A, F32), ref_logprobs=dev(ref, F32), doc_ids=docs,
                          clip_low=0.2, clip_high=0.28, kl_coef=0.1, grad_scale=64.0)
    want = O.policy_loss(zn, y, want_w, old, A, ref=ref, docs=want_docs, clip_low=0.2, clip_high=0.28, kl_coef=0.1)
    _check_policy(out, want, want_w, BF16, A[want_docs], 0.1, 1.0, scale=64.0)


@gpu
def test_policy_gradient_is_the_losses_difference():
    """(loss(z + h u) - loss(z - h u)) / 2h against sum(dlogits u): the difference's own error is h^2 f''' / 6 (1e-4 h^2
    scale 1 here, h = 1e-2: below 1e-3) plus 2e-6 / h of rounding (2e-4)."""
    T, V = 8, 257
    z, zn = make_logits(3, T, V, F32, spread=1.0)
    g = np.random.default_rng(3)
    y, u = g.integers(0, V, T), torch.from_numpy(g.standard_normal((T, V)).astype(np.float32)).cuda()
    old, ref, A = _policy_case(3, zn, y, 1.0, T)
    w = dev(np.full(T, 1.0 / T), F32)
    f = lambda x, **kw: thd.policy_loss(x, dev(y, torch.int32), w, dev(old, F32), dev(A, F32), ref_logprobs=dev(ref, F32),  # noqa: E731
                                        clip_low=0.9, clip_high=5.0, kl_coef=0.3, **kw)
    h = 1e-2
    diff = (f(z + h * u, need_dlogits=False).loss.double() - f(z - h * u, need_dlogits=False).loss.double()) / (2 * h)
    along = (f(z).dlogits.double() * u.double()).sum()
    assert abs(diff.item() - along.item()) < 2e-3


# ---------------------------------------------------------------------------
# preference loss
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("lengths,cp", [([1, 1], 1), ([5, 0, 9, 3], 1), ([8, 16, 0, 24], 2), ([2000, 513, 1], 1), ([16, 64, 32], 8)])
@pytest.mark.parametrize("eps,margin,mean,with_ref", [(0.0, 0.0, False, True), (0.1, 0.5, True, True), (0.0, 1.0, True, False)])
def test_preference_loss(lengths, cp, eps, margin, mean, with_ref):
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T, N = cu[-1], len(lengths)
    g = np.random.default_rng(T + cp)
    lp = -np.abs(g.standard_normal(T) * 3).astype(np.float32)
    ref = (lp + g.standard_normal(T) * 0.2).astype(np.float32)
    mask = (g.random(T) < 0.8).astype(np.uint8)
    hidden = lp.copy()
    hidden[mask == 0] = np.nan      # masked rows are not read
    for pairs in ([(0, 1)], [(0, N - 1), (N - 1, 0), (1, 0), (0, 0)], [], [(int(a), int(b)) for a, b in g.integers(0, N, (700, 2))]):
        c, r = [p[0] for p in pairs], [p[1] for p in pairs]
        st = thd.new_status()
        out = thd.preference_loss(dev(hidden, F32), dev(mask, torch.uint8), dev(cu, torch.int32), dev(c, torch.int32), dev(r, torch.int32),
                                  ref_logprobs=dev(ref, F32) if with_ref else None, cp=cp, beta=0.3, label_smoothing=eps,
                                  margin=margin, length_normalized=mean, status=st)
        thd.check_status(st)
        want = O.preference_loss(lp, mask, cu, c, r, ref=ref if with_ref else None, cp=cp, beta=np.float32(0.3),
                                 label_smoothing=eps, margin=margin, length_normalized=mean)
        # sums are pairs of floats: a rounding or three of the result
        size = np.abs(want["doc_logprobs"])
        same(out.doc_logprobs.cpu().numpy(), want["doc_logprobs"], 2.4e-7 * size)
        err = 0.3 * 2 * 2.4e-7 * (np.abs(want["margins"]).max(initial=0) / 0.3 + (0 if with_ref else size.max())) + 1e-7
        same(out.margins.cpu().numpy(), want["margins"], err)
        same(out.loss.item(), want["loss"], err + 5e-7 * (1 + want["loss"]))
        same(out.dlogprobs.cpu().numpy(), want["dlogprobs"], 0.3 * 2 * (err + 1e-6))


@gpu
def test_preference_pairs_out_of_range_are_reported_and_add_nothing():
    cu, mask = [0, 3, 6], np.ones(6, dtype=np.uint8)
    lp = -np.arange(1.0, 7.0)
    for c, r in (([0, 2], [1, 0]), ([0, 1], [1, -1])):
        st = thd.new_status()
        out = thd.preference_loss(dev(lp, F32), dev(mask, torch.uint8), dev(cu, torch.int32), dev(c, torch.int32), dev(r, torch.int32))
        assert out.margins[1].item() == 0
        thd.preference_loss(dev(lp, F32), dev(mask, torch.uint8), dev(cu, torch.int32), dev(c, torch.int32), dev(r, torch.int32), status=st)
        assert L.STATUS_NAMES[thd.status_read(st)] == "index_range"
    extreme = np.array([-1e4, -2.0, -3.0, 0.0, 0.0, -np.inf])
    for c, r in (([0], [1]), ([1], [0])):
        out = thd.preference_loss(dev(extreme, F32), dev(mask, torch.uint8), dev(cu, torch.int32), dev(c, torch.int32), dev(r, torch.int32), beta=1.0)
        assert out.loss.item() == (np.inf if c == [1] else 0.0)
        assert torch.equal(out.dlogprobs, dev([0.0] * 6 if c == [0] else [1 / 1.0] * 3 + [-1.0] * 3, F32))


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,stride,offset", SHAPES)
@pytest.mark.parametrize("K,normalize", [(1, True), (5, True), (33, False), (700, True)])
def test_distill(T, V, stride, offset, dtype, K, normalize):
    tau = 1.5
    z, zn = make_logits(T * 13 + V, T, V, dtype, stride, offset)
    g = np.random.default_rng(V + K)
    ids = g.integers(0, V, (T, K))               # repeats among them
    ids[g.random((T, K)) < 0.2] = -1
    scores = (g.standard_normal((T, K)) * 2 - (0 if normalize else 4)).astype(np.float32)
    scores[g.random((T, K)) < 0.05] = -np.inf
    w = np.abs(g.standard_normal(T)).astype(np.float32)
    if T > 2:
        w[1] = 0
        z[1] = float("nan")
        ids[2] = -1                               # a row without entries
        scores[0] = -np.inf
        scores[0, 0], ids[0, 0] = 0.25, V - 1
    sdt = [F32, BF16, F16][K % 3]
    st_scores = torch.from_numpy(scores).cuda().to(sdt)
    st = thd.new_status()
    out = thd.distill_topk_loss(z, dev(ids, torch.int32), st_scores, dev(w, F32), temperature=tau, normalize=normalize, status=st)
    thd.check_status(st)
    sn = st_scores.double().cpu().numpy()
    want = O.distill_topk_loss(zn, ids, sn, w, tau, normalize)
    with np.errstate(all="ignore"):
        mass = np.array([1.0 if normalize else np.exp(sn[t][(ids[t] >= 0)]).sum() for t in range(T)])
    big = tau * tau * (1 + mass) * 40             # log-probabilities up to 40 in size here
    same(out.token_losses.cpu().numpy(), want["token_losses"], big * 1e-6 + 5e-6)
    same(out.loss.item(), want["loss"], (w * (big * 1e-6 + 5e-6)).sum())
    same_gradient(out.dlogits, want["dlogits"], dtype, w * tau * (mass + 1) * 1.6e-5)
    alone = thd.distill_topk_loss(z, dev(ids, torch.int32), st_scores, dev(w, F32), temperature=tau, normalize=normalize, need_dlogits=False)
    assert alone.dlogits is None and alone.loss.item() == out.loss.item()


@gpu
@pytest.mark.parametrize("K", [2, 31, 64, 257, 1024])
@pytest.mark.parametrize("V", [4096, 50257])
def test_distill_repeated_ids_are_one_entry_of_the_gradient(K, V):
    """Rows whose ids all differ, one id given twice (at either end, beside each other), one id given K times, and ids of which
    many fall on one another's places whatever they are hashed with (0, 1, 2, ...); tolerances as in test_distill."""
    g = np.random.default_rng(K + V)
    T, tau = 6, 0.75
    z, zn = make_logits(K, T, V, F32)
    ids = np.stack([g.permutation(V)[:K] for _ in range(T)])
    ids[1, -1] = ids[1, 0]
    ids[2, K // 2] = ids[2, K // 2 - 1]
    ids[3] = V - 1
    ids[4] = np.arange(K)
    ids[5] = np.arange(K)[::-1] * (V // K)
    ids[5, ::3] = -1
    scores = (g.standard_normal((T, K)) * 2).astype(np.float32)
    w = np.abs(g.standard_normal(T)).astype(np.float32)
    out = thd.distill_topk_loss(z, dev(ids, torch.int32), dev(scores, F32), dev(w, F32), temperature=tau)
    want = O.distill_topk_loss(zn, ids, scores.astype(np.float64), w, tau, True)
    same(out.token_losses.cpu().numpy(), want["token_losses"], tau * tau * 2 * 40 * 1e-6 + 5e-6)
    same_gradient(out.dlogits, want["dlogits"], F32, w * tau * 2 * 1.6e-5)


@gpu
@pytest.mark.parametrize("T,V,dtype", [(700, 151936, BF16), (300, 50257, F16), (900, 4096, F32)])
def test_the_loss_alone_is_the_loss_with_a_gradient(T, V, dtype):
    """Over many rows, some without loss: the same bits with and without the gradient, and the logits stay."""
    z, _ = make_logits(T, T, V, dtype)
    g = np.random.default_rng(V)
    f = lambda a: dev(a, F32)  # noqa: E731
    w = g.random(T) * (g.random(T) < 0.7)
    y, old, A = dev(g.integers(0, V, T), torch.int32), f(g.standard_normal(T) - 8), f(g.standard_normal(T))
    ids, sc = dev(g.integers(0, V, (T, 40)), torch.int32), f(g.standard_normal((T, 40)))
    keep = z.clone()
    for call in (lambda **kw: thd.policy_loss(z, y, f(w), old, A, **kw)[:4],
                 lambda **kw: thd.distill_topk_loss(z, ids, sc, f(w), **kw)[:2]):
        for a, b in zip(call(), call(need_dlogits=False)):
            assert torch.equal(a, b)
    assert torch.equal(z, keep)


@gpu
@pytest.mark.parametrize("T,V,dtype", [(500, 151936, BF16), (700, 50257, F16), (400, 32003, F32), (2000, 1000, BF16)])
def test_gradients_of_many_rows_in_place(T, V, dtype):
    """Rows shared by several blocks, the next ones fetched while a gradient replaces the logits: the bits of a gradient
    elsewhere.  Labels at the ends and within every block's part."""
    z, _ = make_logits(T + 1, T, V, dtype)
    y = (torch.arange(T, device="cuda") * 7919 % V).to(torch.int32)
    y[::5], y[1::5] = 0, V - 1
    g = np.random.default_rng(V)
    f = lambda a: dev(a, F32)  # noqa: E731
    w, old, A = f(g.random(T) * (g.random(T) < 0.8)), f(g.standard_normal(T) - 8), f(g.standard_normal(T))
    ids, sc = dev(g.integers(0, V, (T, 20)), torch.int32), f(g.standard_normal((T, 20)))
    lse = thd.token_logprobs(z, y)[1]
    for call in (lambda x, **kw: thd.token_logprobs_backward(x, y, lse, w, **kw),
                 lambda x, **kw: thd.policy_loss(x, y, w, old, A, **kw).dlogits,
                 lambda x, **kw: thd.distill_topk_loss(x, ids, sc, w, **kw).dlogits):
        want, over = call(z), z.clone()
        assert torch.equal(call(over, out=over), want)


@gpu
def test_distill_gradient_is_the_losses_difference():
    """As for the policy loss: a directional difference within 2e-3."""
    T, V, K = 6, 300, 12
    z, _ = make_logits(9, T, V, F32, spread=1.0)
    g = np.random.default_rng(9)
    u = torch.from_numpy(g.standard_normal((T, V)).astype(np.float32)).cuda()
    ids, sc = dev(g.integers(0, V, (T, K)), torch.int32), dev(g.standard_normal((T, K)), F32)
    w = dev(np.full(T, 1.0 / T), F32)
    f = lambda x, **kw: thd.distill_topk_loss(x, ids, sc, w, temperature=1.3, **kw)  # noqa: E731
    h = 1e-2
    diff = (f(z + h * u, need_dlogits=False).loss.double() - f(z - h * u, need_dlogits=False).loss.double()) / (2 * h)
    assert abs(diff.item() - (f(z).dlogits.double() * u.double()).sum().item()) < 2e-3


# ---------------------------------------------------------------------------
# what all of them share
# ---------------------------------------------------------------------------

def _steps(z, y, out=None, status=None, stream=None):
    """The three calls that write a gradient, as functions of the logits; rows 1 and 4 without loss."""
    T = z.shape[0]
    g = np.random.default_rng(T)
    w = np.full(T, 0.5)
    w[1::3] = 0
    f = lambda a: dev(a, F32)  # noqa: E731
    old, A = f(-np.ones(T) * 5), f(g.standard_normal(T))
    ids = dev(g.integers(0, z.shape[1], (T, 6)), torch.int32)
    sc = f(g.standard_normal((T, 6)))
    lse = thd.token_logprobs(z, y)[1]
    w = f(w)
    torch.cuda.synchronize()
    kw = dict(out=out, status=status, stream=stream)
    return [lambda x: thd.token_logprobs_backward(x, y, lse, w, **kw),
            lambda x: thd.policy_loss(x, y, w, old, A, **kw).dlogits,
            lambda x: thd.distill_topk_loss(x, ids, sc, w, **kw).dlogits]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(5, 999), (4, 40000), (2, 151936), (2, 1000003)])
def test_in_place_and_strided_gradients_equal_the_plain_ones(T, V, dtype):
    """The gradient over the logits themselves, into a wider matrix and into one of another alignment: the same bits, and
    nothing outside the rows is written."""
    z, _ = make_logits(V, T, V, dtype)
    y = torch.arange(T, device="cuda", dtype=torch.int32)
    for i, step in enumerate(_steps(z, y)):
        want = step(z)
        for pad, off in ((8, 0), (5, 3)):
            wide = torch.full((T * (V + pad) + off,), 7.0, device="cuda", dtype=dtype)
            view = wide[off:].view(T, V + pad)[:, :V]
            _steps(z, y, out=view)[i](z)
            assert torch.equal(view, want)
            assert (wide[off:].view(T, V + pad)[:, V:] == 7).all() and (wide[:off] == 7).all()
        over = z.clone()
        got = _steps(over, y, out=over)[i](over)
        assert got.data_ptr() == over.data_ptr() and torch.equal(over, want)


@gpu
def test_bad_labels_and_ids_are_reported_and_their_rows_take_no_part():
    z, zn = make_logits(1, 4, 50, BF16)
    f = lambda *a: torch.tensor(a, device="cuda")  # noqa: E731
    w = f(1.0, 1.0, 0.0, 1.0)
    for bad in (50, -1, 1 << 30, -(1 << 31)):
        y = torch.tensor([3, bad, bad, 5], device="cuda", dtype=torch.int32)   # row 2 has no loss: not looked at
        ok = torch.tensor([3, 0, 0, 5], device="cuda", dtype=torch.int32)
        lp, lse = thd.token_logprobs(z, y, (w != 0).to(torch.uint8))
        want, _ = thd.token_logprobs(z, ok)
        assert lp[1].item() == 0 and lse[1].item() == 0 and lp[2].item() == 0
        assert torch.equal(lp[[0, 3]], want[[0, 3]])
        d = thd.token_logprobs_backward(z, y, lse, w)
        assert (d[1:3] == 0).all() and (d[0] != 0).any()
        out = thd.policy_loss(z, y, w, lp, f(1.0, 1.0, 1.0, 1.0))
        assert (out.dlogits[1:3] == 0).all() and abs(out.loss.item() + 2) < 1e-5
        for call in (lambda s: thd.token_logprobs(z, y, (w != 0).to(torch.uint8), status=s),
                     lambda s: thd.token_logprobs_backward(z, y, lse, w, status=s),
                     lambda s: thd.policy_loss(z, y, w, lp, w, status=s)):
            st = thd.new_status()
            call(st)
            assert L.STATUS_NAMES[thd.status_read(st)] == "index_range"
    docs = torch.tensor([0, 2, 9, 1], device="cuda", dtype=torch.int32)
    ok = torch.zeros(4, device="cuda", dtype=torch.int32)
    st = thd.new_status()
    out = thd.policy_loss(z, ok, w, thd.token_logprobs(z, ok)[0], f(1.0, 1.0), doc_ids=docs)
    assert (out.dlogits[1:3] == 0).all() and abs(out.loss.item() + 2) < 1e-5
    thd.policy_loss(z, ok, w, w, f(1.0, 1.0), doc_ids=docs, status=st)
    assert L.STATUS_NAMES[thd.status_read(st)] == "index_range"
    ids = torch.tensor([[1, 50], [-5, 2], [99, 99], [0, 3]], device="cuda", dtype=torch.int32)
    sc = torch.zeros(4, 2, device="cuda")
    st = thd.new_status()
    got = thd.distill_topk_loss(z, ids, sc, w)
    want = O.distill_topk_loss(zn, ids.cpu().numpy(), sc.cpu().numpy(), w.cpu().numpy())
    same(got.token_losses.cpu().numpy(), want["token_losses"], 1e-5)
    thd.distill_topk_loss(z, ids, sc, w, status=st)
    assert L.STATUS_NAMES[thd.status_read(st)] == "index_range"


@gpu
def test_a_set_status_word_stops_every_call():
    z, _ = make_logits(2, 6, 100, F32)
    y = torch.zeros(6, device="cuda", dtype=torch.int32)
    st = torch.full((1,), L.ERR_TOTAL_MISMATCH, device="cuda", dtype=torch.int32)
    keep = torch.full((6, 100), 9.0, device="cuda")
    for step in _steps(z, y, out=keep, status=st):
        step(z)
        assert (keep == 9).all()
    assert thd.status_read(st) == L.ERR_TOTAL_MISMATCH


@gpu
def test_no_rows_at_all():
    z = torch.zeros(0, 10, device="cuda", dtype=BF16)
    y, f = torch.zeros(0, device="cuda", dtype=torch.int32), torch.zeros(0, device="cuda")
    m, cu = torch.zeros(0, device="cuda", dtype=torch.uint8), torch.zeros(1, device="cuda", dtype=torch.int32)
    assert thd.token_logprobs(z, y)[0].shape == (0,)
    assert thd.token_logprobs_backward(z, y, f, f).shape == (0, 10)
    assert thd.policy_loss(z, y, f, f, f).loss.item() == 0
    assert thd.distill_topk_loss(z, torch.zeros(0, 3, device="cuda", dtype=torch.int32), torch.zeros(0, 3, device="cuda"), f).loss.item() == 0
    w, docs = thd.loss_weights(m, cu)
    assert w.numel() == 0 and docs.numel() == 0
    assert thd.preference_loss(f, m, cu, y, y).loss.item() == 0


@gpu
@pytest.mark.parametrize("T,V", [(300, 5003), (700, 70001), (9, 151936)])
def test_repeated_runs_give_the_same_bits_on_another_stream_and_in_a_graph(T, V):
    z, _ = make_logits(4, T, V, BF16)
    y = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    want = [s(z) for s in _steps(z, y)]
    side = torch.cuda.Stream()
    steps = _steps(z, y, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [s(z) for s in steps]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.empty_like(z)
    steps = _steps(z, y, out=out)
    for step, w in zip(steps, want):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(z)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


@gpu
def test_rows_past_two_to_the_31_elements():
    """Offsets of more than 2^31 elements: the last rows of a matrix of 2.15 G logits, the others without loss."""
    V = 151936
    T = (1 << 31) // V + 4
    z = torch.zeros(T, V, device="cuda", dtype=BF16)
    tail, tail_n = make_logits(8, 2, V, BF16)
    z[-2:] = tail
    y = torch.full((T,), V - 1, device="cuda", dtype=torch.int32)
    w = torch.zeros(T, device="cuda")
    w[-2:] = 0.5
    want_lp, want_lse = O.token_logprobs(tail_n, [V - 1] * 2)
    lp, lse = thd.token_logprobs(z, y, (w != 0).to(torch.uint8))
    same(lp[-2:].cpu().numpy(), want_lp, lp_tol(want_lp))
    assert (lp[:-2] == 0).all()
    A = torch.ones(T, device="cuda")
    out = thd.policy_loss(z, y, w, lp, A)
    yn = [V - 1] * 2
    same_gradient(out.dlogits[-2:], O.token_logprobs_backward(tail_n, yn, [-0.5] * 2), BF16, np.full(2, 0.5 * 2e-5))
    assert not out.dlogits[:-2].any()
    assert abs(out.loss.item() + 1) < 1e-5
    d = thd.token_logprobs_backward(z, y, lse, w, out=out.dlogits)
    same_gradient(d[-2:], O.token_logprobs_backward(tail_n, yn, [0.5] * 2), BF16, np.full(2, 0.5 * 2e-5))
    assert not d[:-2].any()


@gpu
@pytest.mark.parametrize("cp", [1, 2])
def test_one_training_step_from_raw_rows(cp):
    """pack_docs -> labels -> weights -> policy loss, and -> preference loss, rows in the layout of cp ranks: every row's
    label and document are the oracle's."""
    E = 98
    raw = [[1, 2, 3, E, 4, 5, 6, 7], [8, 9, E, 10, 11, 12, 13, E], [14, 15, 16, 17, 18, 19, 20, 21]]
    tok, cu_v, cu = thd.pack_docs(torch.tensor(raw, dtype=torch.int32, device="cuda"), E, 2 * cp)
    roll = thd.roll_labels(tok, cu_v, cu, 0) if cp == 1 else thd.roll_labels_zigzag(tok, cu_v, cu, cp, 0)
    y, mask = roll[0][0], roll[1][0]
    T, V, N = tok.numel(), 99, cu.numel() - 1
    z, zn = make_logits(11, T, V, BF16)
    st = thd.new_status()
    w, docs = thd.loss_weights(mask, cu, cp, thd.DOC_MEAN, status=st)
    want_w, want_docs = O.loss_weights(mask.tolist(), cu.tolist(), cp, O.DOC_MEAN)
    old, ref, A = _policy_case(1, zn, y.cpu().numpy(), 1.0, T, want_docs)
    out = thd.policy_loss(z, y, w, dev(old, F32), dev(A, F32), ref_logprobs=dev(ref, F32), doc_ids=docs, clip_low=0.2,
                          clip_high=0.28, kl_coef=0.1, status=st)
    want = O.policy_loss(zn, y.cpu().numpy(), want_w, old, A, ref=ref, docs=want_docs, clip_low=0.2, clip_high=0.28, kl_coef=0.1)
    _check_policy(out, want, want_w, BF16, A[want_docs], 0.1, 1.0)
    lp, lse = thd.token_logprobs(z, y, mask, status=st)
    c, r = [0, 1], [N - 1, 2]
    pref = thd.preference_loss(lp, mask, cu, dev(c, torch.int32), dev(r, torch.int32), ref_logprobs=dev(ref, F32), cp=cp, status=st)
    d = thd.token_logprobs_backward(z, y, lse, pref.dlogprobs, status=st)
    thd.check_status(st)
    lpn = lp.double().cpu().numpy()
    wp = O.preference_loss(lpn, mask.tolist(), cu.tolist(), c, r, ref=ref, cp=cp, beta=np.float32(0.1))
    same(pref.loss.item(), wp["loss"], 2e-6)
    same(pref.dlogprobs.cpu().numpy(), wp["dlogprobs"], 1e-6)
    same_gradient(d, O.token_logprobs_backward(zn, y.cpu().numpy(), wp["dlogprobs"]), BF16, np.full(T, 3e-6))


@gpu
def test_the_example_trains():
    """examples/post_training_step.py: every loss falls, and what it runs on leaves no error."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "post_training_step.py")
    spec = importlib.util.spec_from_file_location("post_training_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses = module.main(steps=8)
    assert sorted(losses) == ["distillation", "policy", "preference"]
    for name, values in losses.items():
        assert np.isfinite(values).all() and values[-1] < values[0], (name, values)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(1200, 151936), (400, 40001), (3000, 12289)])
def test_many_rows_at_once(T, V, dtype):
    """Enough rows that every cluster takes several, with runs of rows without loss between them: each loss against torch
    in 64 bits on a sample of the rows."""
    if dtype == F32 and V == 151936:
        T = 500
    z = torch.randn(T, V, device="cuda", dtype=torch.float32, generator=torch.Generator("cuda").manual_seed(V)).mul_(2).to(dtype)
    g = np.random.default_rng(V)
    y = torch.from_numpy(g.integers(0, V, T)).cuda().to(torch.int32)
    w = np.full(T, 1.0 / T)
    for a in range(0, T, 37):
        w[a:a + int(g.integers(0, 20))] = 0
    w = dev(w, F32)
    on = (w != 0).to(torch.uint8)
    st = thd.new_status()
    lp, lse = thd.token_logprobs(z, y, on, status=st)
    ids = torch.from_numpy(g.integers(0, V, (T, 16))).cuda().to(torch.int32)
    sc = dev(g.standard_normal((T, 16)), F32)
    A = dev(g.standard_normal(T), F32)
    pol = thd.policy_loss(z, y, w, lp - 0.1, A, ref_logprobs=lp + 0.2, clip_low=0.5, clip_high=0.5, kl_coef=0.1, status=st)
    dis = thd.distill_topk_loss(z, ids, sc, w, status=st)
    back = thd.token_logprobs_backward(z, y, lse, w, status=st)
    thd.check_status(st)
    pick = np.unique(np.concatenate([[0, T - 1], g.integers(0, T, 24)]))
    zn, yn, wn = z[pick].double().cpu().numpy(), y.cpu().numpy()[pick], w.double().cpu().numpy()[pick]
    want_lp, want_lse = O.token_logprobs(zn, yn, wn != 0)
    lpn = lp.double().cpu().numpy()[pick]
    same(lpn, want_lp, lp_tol(want_lp))
    same(lse.cpu().numpy()[pick], want_lse, lp_tol(want_lse))
    An = A.cpu().numpy()[pick]
    want = O.policy_loss(zn, yn, wn, lpn - 0.1, An, ref=lpn + 0.2, clip_low=0.5, clip_high=0.5, kl_coef=0.1)
    same_gradient(pol.dlogits[pick], want["dlogits"], dtype, wn * (8 * np.abs(An) + 1) * 1.6e-5)
    want = O.distill_topk_loss(zn, ids.cpu().numpy()[pick], sc.double().cpu().numpy()[pick], wn)
    same(dis.token_losses.cpu().numpy()[pick], want["token_losses"], 80 * 1e-6 + 5e-6)
    same_gradient(dis.dlogits[pick], want["dlogits"], dtype, wn * 2 * 1.6e-5)
    want = O.token_logprobs_backward(zn, yn, wn)
    same_gradient(back[pick], want, dtype, wn * (8e-6 + 2.4e-7 * np.abs(want_lse)))
    idle = w == 0
    for d in (pol.dlogits, dis.dlogits, back):
        assert not d[idle].any()
    assert not lp[idle].any() and not lse[idle].any() and not dis.token_losses[idle].any()


def test_oracle_is_exported():
    assert oracle.losses is O
